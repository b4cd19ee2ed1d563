"""Thin binding of the gated linear recurrence in libstepq.so
(include/stepq_block.h): ragged prompts, their gradients, and single tokens.

As in the other bindings, tensors become raw pointers, status codes become
exceptions, tensor arguments are checked against the sizes the call implies
before the library sees their pointers, and there is no fallback.
"""
from __future__ import annotations

import ctypes

from . import stepq as _s
from .linear import _refuse, check_current, check_dense, dense, dtype_code, leading, stream_of
from .stepq import STEPQ_ERR_UNSUPPORTED, StepqError

EXPORTED = ("stepq_scan_workspace_bytes", "stepq_scan_saved_bytes", "stepq_scan_forward", "stepq_scan_backward",
            "stepq_scan_step")
MAX_STRIDE = 1 << 24      # elements from token to token


class stepq_scan_desc(ctypes.Structure):
    _fields_ = [("width", ctypes.c_int32), ("dtype", ctypes.c_int32), ("rate", ctypes.c_float)]


_lib = None


def address(t):
    """What the library takes for a tensor that has been checked, or for None."""
    return None if t is None else t.data_ptr()


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = _s.lib()
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        for f in (L.stepq_scan_workspace_bytes, L.stepq_scan_saved_bytes):
            f.restype = sz
            f.argtypes = [P, i32, i64]
        L.stepq_scan_forward.restype = ctypes.c_int
        L.stepq_scan_forward.argtypes = [P, i32, i64, P, P, i64, P, i64, P, i64, P, P, i32, P, P, P, i64, P, sz, P, sz, P]
        L.stepq_scan_backward.restype = ctypes.c_int
        L.stepq_scan_backward.argtypes = [P, i32, i64, P, P, i64, P, i64, P, i64, P, P, sz, P, i64, P, i32, P, P, P, i64,
                                          P, i64, P, i64, P, P, sz, P]
        L.stepq_scan_step.restype = ctypes.c_int
        L.stepq_scan_step.argtypes = [P, i32, P, i32, P, i64, P, i64, P, i64, P, P, P, i64, P]
        _lib = L
    return _lib


class GatedRecurrence:
    """h_t = a_t h_{t-1} + sqrt(1 - a_t^2) s(gate_x_t) x_t with the retention
    a_t = exp(-rate s(gate_a_t) softplus(decay)), for `width` channels; dtype is that of
    x, the gates, y and their gradients."""

    def __init__(self, width: int, dtype=None, rate: float = 8.0):
        import torch
        self.width, self.rate = int(width), float(rate)
        self.dtype = torch.float32 if dtype is None else dtype
        self._f32, self._i32, self._u8, self._tensor = torch.float32, torch.int32, torch.uint8, torch.Tensor
        self.desc = stepq_scan_desc(self.width, dtype_code(self.dtype), self.rate)
        self._desc = ctypes.addressof(self.desc)
        # an empty call runs the library's own checks of the description
        null = ctypes.c_void_p()
        _s._check(lib().stepq_scan_step(self._desc, 0, null, 1, null, 0, null, 0, null, 0, null, null, null, 0, null),
                  "GatedRecurrence")

    def _bytes(self, function, batch: int, total_tokens: int) -> int:
        n = int(function(self._desc, int(batch), int(total_tokens)))
        if n == 0 and batch != 0:
            raise StepqError(STEPQ_ERR_UNSUPPORTED, "GatedRecurrence", f"{batch} requests of {total_tokens} tokens")
        return n

    def workspace(self, batch: int, total_tokens: int, device="cuda"):
        """A workspace for calls of up to `batch` requests of up to `total_tokens` tokens together."""
        import torch
        return torch.empty(max(16, self._bytes(lib().stepq_scan_workspace_bytes, batch, total_tokens)), dtype=torch.uint8,
                           device=device)

    def saved(self, batch: int, total_tokens: int, device="cuda"):
        """What a forward pass of exactly these sizes saves for its backward pass."""
        import torch
        return torch.empty(max(16, self._bytes(lib().stepq_scan_saved_bytes, batch, total_tokens)), dtype=torch.uint8,
                           device=device)

    def states(self, num_slots: int, device="cuda"):
        """Zeroed states [num_slots, width]."""
        import torch
        return torch.zeros(num_slots, self.width, dtype=torch.float32, device=device)

    def _rows(self, where: str, name: str, t, tokens: int, index: int) -> int:
        """Checks a [tokens, width] tensor whose tokens may be strided; returns that stride."""
        if not isinstance(t, self._tensor) or t.get_device() != index or index < 0 or t.dtype is not self.dtype:
            _refuse(where, f"{name} must be a {self.dtype} tensor on cuda:{max(index, 0)}")
        if t.shape != (tokens, self.width):
            _refuse(where, f"{name} must have shape {[tokens, self.width]} (got {list(t.shape)})")
        n, e = t.stride()
        if tokens <= 1:      # the only token's stride says nothing
            n = self.width
        if (e != 1 and self.width > 1) or n < self.width:
            _refuse(where, f"{name}'s channels must lie side by side and its tokens must not overlap (strides {list(t.stride())})")
        if n > MAX_STRIDE:
            _refuse(where, f"{name}'s tokens may lie at most {MAX_STRIDE} elements apart (got {n})")
        return n

    def _place(self, index: int):
        import torch
        return torch.device("cuda", index) if index >= 0 else None

    def _slots(self, where, slot_ids, state, resume, batch, index):
        if (slot_ids is None) != (state is None):
            _refuse(where, "slot_ids and states belong together")
        if state is not None:
            if not dense(slot_ids, self._i32, (batch,), index):
                check_dense(where, "slot_ids", slot_ids, (batch,), self._i32, self._place(index))
            if not dense(state, self._f32, (leading(where, "state", state), self.width), index):
                check_dense(where, "state", state, (None, self.width), self._f32, self._place(index))
            if state.shape[0] < 1:
                _refuse(where, "there are no states")
        elif resume is not None:
            _refuse(where, "requests without a state cannot resume from one")

    def _common(self, where, cu_seqlens, rows, decay, slot_ids, state, resume, workspace):
        """Checks what the two passes over prompts have in common; (batch, tokens, device index, strides)."""
        batch, tokens = leading(where, "cu_seqlens", cu_seqlens) - 1, leading(where, "x", rows[0][1])
        if not _s._checks:
            return batch, tokens, decay.get_device(), [t.stride(0) if tokens > 1 else self.width for _, t in rows]
        index = decay.get_device() if isinstance(decay, self._tensor) else -1
        if index < 0 or not dense(decay, self._f32, (self.width,), index):
            check_dense(where, "decay", decay, (self.width,), self._f32, self._place(index))
        if batch < 0 or not dense(cu_seqlens, self._i32, (batch + 1,), index):
            check_dense(where, "cu_seqlens", cu_seqlens, (None,), self._i32, self._place(index))
            _refuse(where, "cu_seqlens must have an entry more than there are requests")
        strides = [self._rows(where, name, t, tokens, index) for name, t in rows]
        self._slots(where, slot_ids, state, resume, batch, index)
        if resume is not None and not dense(resume, self._u8, (batch,), index):
            check_dense(where, "resume", resume, (batch,), self._u8, self._place(index))
        if workspace is not None:
            self._buffer(where, "workspace", workspace, index)
        check_current(where, index)
        return batch, tokens, index, strides

    def _workspace(self, where, workspace, batch, tokens, stream, device):
        if workspace is None and batch > 0:
            if stream is not None:
                _refuse(where, "a call on another stream needs a workspace of its own")
            workspace = self.workspace(batch, tokens, device)
        return workspace

    def _buffer(self, where, name, t, index):
        if not (isinstance(t, self._tensor) and t.dtype is self._u8 and t.get_device() == index and t.dim() == 1 and
                t.is_contiguous()):
            check_dense(where, name, t, (None,), self._u8, self._place(index))

    def prefill(self, cu_seqlens, x, gate_a, gate_x, decay, slot_ids, state, y, resume=None, saved=None, workspace=None,
                stream=None) -> None:
        """stepq_scan_forward: prompts of ragged lengths; request b's tokens are rows
        cu_seqlens[b] .. cu_seqlens[b+1]-1.  Writes y and the slots of state (slot_ids and
        state may both be None).  `saved` (see saved()) is what backward() reads.  The
        workspace may be kept between calls (see workspace()); without one, it is taken
        from torch's allocator, on the current stream."""
        where = "stepq_scan_forward"
        batch, tokens, i, (xs, as_, gs, ys) = self._common(
            where, cu_seqlens, (("x", x), ("gate_a", gate_a), ("gate_x", gate_x), ("y", y)), decay, slot_ids, state, resume,
            workspace)
        if saved is not None and _s._checks:
            self._buffer(where, "saved", saved, i)
        if batch == 0:
            return
        workspace = self._workspace(where, workspace, batch, tokens, stream, decay.device)
        if tokens == 0:          # empty tensors have no address; every request is empty
            x = gate_a = gate_x = y = decay
            xs = as_ = gs = ys = self.width
        p = address
        _s._check(lib().stepq_scan_forward(self._desc, batch, tokens, p(cu_seqlens), p(x), xs, p(gate_a), as_, p(gate_x), gs,
                                           p(decay), p(slot_ids), 0 if state is None else state.shape[0], p(resume), p(state),
                                           p(y), ys, p(saved), 0 if saved is None else saved.numel(), p(workspace),
                                           workspace.numel(), stream_of(stream, i)), where)

    def backward(self, cu_seqlens, x, gate_a, gate_x, decay, saved, dy, dx, dgate_a, dgate_x, ddecay, slot_ids=None,
                 dstate=None, resume=None, workspace=None, stream=None) -> None:
        """stepq_scan_backward: from dy, and from the gradients of the states that requests end
        with in the slots of dstate, those of x, the gates and decay, and in the slots of dstate
        those of the states that requests start from."""
        where = "stepq_scan_backward"
        rows = (("x", x), ("gate_a", gate_a), ("gate_x", gate_x), ("dy", dy), ("dx", dx), ("dgate_a", dgate_a),
                ("dgate_x", dgate_x))
        batch, tokens, i, strides = self._common(where, cu_seqlens, rows, decay, slot_ids, dstate, resume, workspace)
        if _s._checks:
            self._buffer(where, "saved", saved, i)
            if not dense(ddecay, self._f32, (self.width,), i):
                check_dense(where, "ddecay", ddecay, (self.width,), self._f32, decay.device)
        workspace = self._workspace(where, workspace, batch, tokens, stream, decay.device)
        p = address
        ptrs = [p(t) for _, t in rows]
        if tokens == 0:
            ptrs, strides = [p(decay)] * 7, [self.width] * 7
        (xp, ap, gp, dyp, dxp, dap, dgp), (xs, as_, gs, dys, dxs, das, dgs) = ptrs, strides
        _s._check(lib().stepq_scan_backward(self._desc, batch, tokens, p(cu_seqlens), xp, xs, ap, as_, gp, gs, p(decay),
                                            p(saved), saved.numel(), dyp, dys, p(slot_ids),
                                            0 if dstate is None else dstate.shape[0], p(resume), p(dstate), dxp, dxs, dap, das,
                                            dgp, dgs, p(ddecay), p(workspace), 0 if workspace is None else workspace.numel(),
                                            stream_of(stream, i)), where)

    def step(self, slot_ids, x, gate_a, gate_x, decay, state, y, stream=None) -> None:
        """stepq_scan_step: one token of every request, updating the slots of state."""
        where = "stepq_scan_step"
        batch = leading(where, "slot_ids", slot_ids)
        if _s._checks:
            i = decay.get_device() if isinstance(decay, self._tensor) else -1
            if i < 0 or not dense(decay, self._f32, (self.width,), i):
                check_dense(where, "decay", decay, (self.width,), self._f32, self._place(i))
            strides = (self._rows(where, "x", x, batch, i), self._rows(where, "gate_a", gate_a, batch, i),
                       self._rows(where, "gate_x", gate_x, batch, i), self._rows(where, "y", y, batch, i))
            if state is None or slot_ids is None:
                _refuse(where, "a step needs states")
            self._slots(where, slot_ids, state, None, batch, i)
            check_current(where, i)
        else:
            strides = [t.stride(0) if batch > 1 else self.width for t in (x, gate_a, gate_x, y)]
        p = address
        xs, as_, gs, ys = strides
        _s._check(lib().stepq_scan_step(self._desc, batch, p(slot_ids), state.shape[0], p(x), xs, p(gate_a), as_, p(gate_x),
                                        gs, p(decay), p(state), p(y), ys, stream_of(stream, decay.get_device())), where)

"""Thin binding of the linear-attention entry points of libstepq.so
(include/stepq_seq.h): ragged prompts in the chunked form, single tokens in the
recurrent form, for the additive and the delta rule with one decay per head.

As in the binding of the packed step, tensors become raw pointers, status codes
become exceptions, tensor arguments are checked against the sizes the call
implies before the library sees their pointers, and there is no fallback.
"""
from __future__ import annotations

import ctypes

from . import stepq as _s
from .stepq import STEPQ_ERR_INVALID_ARG, StepqError

STEPQ_F32 = 0
STEPQ_BF16 = 1
STEPQ_F16 = 2
RULE_ADDITIVE = 0
RULE_DELTA = 1

EXPORTED = ("stepq_linear_workspace_bytes", "stepq_linear_prefill_bytes", "stepq_linear_prefill", "stepq_linear_step")

_RULES = {"additive": RULE_ADDITIVE, "delta": RULE_DELTA}


class stepq_linear_desc(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("num_qk_heads", ctypes.c_int32), ("d", ctypes.c_int32),
                ("rule", ctypes.c_int32), ("dtype", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = _s.lib()
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.stepq_linear_workspace_bytes.restype = sz
        L.stepq_linear_workspace_bytes.argtypes = [P, i32, i64]
        L.stepq_linear_prefill_bytes.restype = sz
        L.stepq_linear_prefill_bytes.argtypes = [P, i32, i64]
        L.stepq_linear_prefill.restype = ctypes.c_int
        L.stepq_linear_prefill.argtypes = [P, i32, i64, P, P, i64, P, i64, P, i64, P, P, P, i32, P, P, P, i64, P,
                                           sz, P]
        L.stepq_linear_step.restype = ctypes.c_int
        L.stepq_linear_step.argtypes = [P, i32, P, i32, P, i64, P, i64, P, i64, P, P, P, P, i64, P]
        _lib = L
    return _lib


def dtype_code(dtype) -> int:
    """The library's code of a torch dtype; StepqError for one it does not take."""
    import torch
    codes = {torch.float32: STEPQ_F32, torch.bfloat16: STEPQ_BF16, torch.float16: STEPQ_F16}
    if dtype not in codes:
        raise StepqError(STEPQ_ERR_INVALID_ARG, "dtype", f"{dtype} is not float32, bfloat16 or float16")
    return codes[dtype]


def current_stream(device_index: int) -> int:
    """The handle of torch's current stream on this device, without building a stream object."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device_index) if raw is not None else torch.cuda.current_stream(device_index).cuda_stream


def stream_of(stream, device_index: int) -> int:
    return current_stream(device_index) if stream is None else _s._stream(stream)


def dense(t, dtype, shape, device_index: int) -> bool:
    """Whether t is a contiguous tensor of this dtype and shape on this GPU (what
    check_dense explains when it is not)."""
    try:
        return t.dtype is dtype and t.shape == shape and t.get_device() == device_index and t.is_contiguous()
    except AttributeError:
        return False


def _refuse(where: str, detail: str):
    raise StepqError(STEPQ_ERR_INVALID_ARG, where, detail)


_current_device = None      # torch's, without what it does around the call


def check_current(where: str, device_index: int) -> None:
    """The library launches on the current device: the call's tensors have to lie there."""
    global _current_device
    if _current_device is None:
        import torch
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    if _current_device() != device_index:
        _refuse(where, f"the tensors are on cuda:{device_index}, which is not the current device")


def leading(where: str, name: str, t) -> int:
    """The leading size of a tensor, before anything else is known of it."""
    try:
        return t.shape[0]
    except (AttributeError, IndexError, TypeError):
        _refuse(where, f"{name} must be a torch tensor with its rows first")


def check_dense(where: str, name: str, t, shape: tuple, dtype, device) -> None:
    """A contiguous device tensor of this dtype and shape (None in a shape: any size)."""
    import torch
    if not isinstance(t, torch.Tensor):
        _refuse(where, f"{name} must be a torch tensor")
    if not t.is_cuda:
        _refuse(where, f"{name} must be a device tensor (got {t.device})")
    if t.device != device:
        _refuse(where, f"{name} is on {t.device}, the call's tensors are on {device}")
    if t.dtype != dtype:
        _refuse(where, f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        _refuse(where, f"{name} must have shape {list(shape)} (got {list(t.shape)})")
    if not t.is_contiguous():
        _refuse(where, f"{name} must be contiguous")


class LinearAttention:
    """Linear attention with one decay per head: head counts, head size, rule
    ("additive" or "delta") and element type of q, k, v and o."""

    def __init__(self, num_heads: int, d: int, num_qk_heads: int | None = None, rule: str = "delta", dtype=None):
        import torch
        if rule not in _RULES:
            _refuse("LinearAttention", f"unknown rule {rule!r}; known: {sorted(_RULES)}")
        self.H, self.D = int(num_heads), int(d)
        self.Hk = self.H if num_qk_heads is None else int(num_qk_heads)
        self.rule, self.dtype = rule, torch.float32 if dtype is None else dtype
        self.desc = stepq_linear_desc(self.H, self.Hk, self.D, _RULES[rule], dtype_code(self.dtype))
        self._desc = ctypes.addressof(self.desc)
        # an empty call runs the library's own checks of the description
        null = ctypes.c_void_p()
        _s._check(lib().stepq_linear_step(self._desc, 0, null, 1, null, 0, null, 0, null, 0, null, null, null, null, 0,
                                          null), "LinearAttention")
        self._qk_row, self._v_row = self.Hk * self.D, self.H * self.D
        self._state = (self.H, self.D, self.D)

    def workspace_bytes(self, batch: int, total_tokens: int) -> int:
        return int(lib().stepq_linear_workspace_bytes(self._desc, int(batch), int(total_tokens)))

    def workspace(self, batch: int, total_tokens: int, device="cuda"):
        """A workspace for calls of up to `batch` requests of up to `total_tokens` tokens together."""
        import torch
        return torch.empty(max(16, self.workspace_bytes(batch, total_tokens)), dtype=torch.uint8, device=device)

    def states(self, num_slots: int, device="cuda"):
        """Zeroed states [num_slots, H, D, D], row = key channel, column = value channel."""
        import torch
        return torch.zeros(num_slots, self.H, self.D, self.D, dtype=torch.float32, device=device)

    def _strided(self, where: str, name: str, t, tokens: int, heads: int, device) -> int:
        """Checks a [tokens, heads, D] tensor whose tokens may be strided; returns that stride."""
        import torch
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device or t.dtype != self.dtype:
            _refuse(where, f"{name} must be a {self.dtype} tensor on {device}")
        if t.shape != (tokens, heads, self.D):
            _refuse(where, f"{name} must have shape {[tokens, heads, self.D]} (got {list(t.shape)})")
        n, m, e = t.stride()
        if e != 1 or (m != self.D and heads > 1):
            _refuse(where, f"{name}'s heads must lie side by side within a token (strides {list(t.stride())})")
        if tokens <= 1:      # the only token's stride says nothing
            n = heads * self.D
        if n < heads * self.D or n * t.element_size() % 16 or t.data_ptr() % 16:
            _refuse(where, f"{name}'s tokens must not overlap and must lie on 16-byte boundaries (stride {n})")
        return n

    def _common(self, where, q, k, v, beta, gate, slot_ids, state, o, batch, tokens):
        """Checks what prompts and tokens have in common; returns the strides of q, k, v and o."""
        import torch
        f32 = torch.float32
        i = state.get_device() if isinstance(state, torch.Tensor) else -1
        dev = state.device if i >= 0 else None
        per_head = (tokens, self.H)
        if not (i >= 0 and state.dtype is f32 and state.shape[1:] == self._state and state.is_contiguous()):
            check_dense(where, "state", state, (None,) + self._state, f32, dev)
        if not dense(slot_ids, torch.int32, (batch,), i):
            check_dense(where, "slot_ids", slot_ids, (batch,), torch.int32, dev)
        if not dense(gate, f32, per_head, i):
            check_dense(where, "gate", gate, per_head, f32, dev)
        if (beta is None) != (self.rule == "additive"):
            _refuse(where, "beta belongs to the delta rule alone")
        if beta is not None and not dense(beta, f32, per_head, i):
            check_dense(where, "beta", beta, per_head, f32, dev)
        qk, vo = (tokens, self.Hk, self.D), (tokens, self.H, self.D)
        return (self._qk_row if dense(q, self.dtype, qk, i) else self._strided(where, "q", q, tokens, self.Hk, dev),
                self._qk_row if dense(k, self.dtype, qk, i) else self._strided(where, "k", k, tokens, self.Hk, dev),
                self._v_row if dense(v, self.dtype, vo, i) else self._strided(where, "v", v, tokens, self.H, dev),
                self._v_row if dense(o, self.dtype, vo, i) else self._strided(where, "o", o, tokens, self.H, dev))

    def _strides(self, *tensors):
        return tuple(t.stride(0) if t.shape[0] > 1 else t.shape[1] * self.D for t in tensors)

    def prefill(self, cu_seqlens, q, k, v, beta, gate, slot_ids, state, o, resume=None, workspace=None,
                stream=None) -> None:
        """stepq_linear_prefill: prompts of ragged lengths; request b's tokens are rows
        cu_seqlens[b] .. cu_seqlens[b+1]-1.  Writes o and the slots of state.  The
        workspace may be kept between calls (see workspace()); without one, what this
        call needs, if anything, is taken from torch's allocator, on the current stream."""
        import torch
        where = "stepq_linear_prefill"
        batch, tokens = leading(where, "slot_ids", slot_ids), leading(where, "v", v)
        if _s._checks:
            qs, ks, vs, os_ = self._common(where, q, k, v, beta, gate, slot_ids, state, o, batch, tokens)
            i = state.get_device()
            check_current(where, i)
            if not dense(cu_seqlens, torch.int32, (batch + 1,), i):
                check_dense(where, "cu_seqlens", cu_seqlens, (batch + 1,), torch.int32, state.device)
            if resume is not None and not dense(resume, torch.uint8, (batch,), i):
                check_dense(where, "resume", resume, (batch,), torch.uint8, state.device)
            if workspace is not None and not (isinstance(workspace, torch.Tensor) and workspace.dtype is torch.uint8 and
                                              workspace.get_device() == i and workspace.dim() == 1 and
                                              workspace.is_contiguous()):
                check_dense(where, "workspace", workspace, (None,), torch.uint8, state.device)
        else:
            qs, ks, vs, os_ = self._strides(q, k, v, o)
        if batch == 0:
            return
        if workspace is None:
            need = lib().stepq_linear_prefill_bytes(self._desc, batch, tokens)
            if need > 0:
                if stream is not None:
                    _refuse(where, "a call on another stream needs a workspace of its own")
                workspace = torch.empty(need, dtype=torch.uint8, device=state.device)
        if tokens == 0:          # empty tensors have no address; every request is empty
            q = k = v = o = gate = state
            beta = None if self.rule == "additive" else state
            qs = ks = self._qk_row
            vs = os_ = self._v_row
        p = _s._ptr
        _s._check(lib().stepq_linear_prefill(self._desc, batch, tokens, p(cu_seqlens), p(q), qs, p(k), ks, p(v), vs,
                                             p(beta), p(gate), p(slot_ids), state.shape[0], p(resume), p(state), p(o),
                                             os_, p(workspace), 0 if workspace is None else workspace.numel(),
                                             stream_of(stream, state.get_device())), where)

    def step(self, slot_ids, q, k, v, beta, gate, state, o, stream=None) -> None:
        """stepq_linear_step: one token of every request, updating the slots of state."""
        where = "stepq_linear_step"
        batch = leading(where, "slot_ids", slot_ids)
        if _s._checks:
            qs, ks, vs, os_ = self._common(where, q, k, v, beta, gate, slot_ids, state, o, batch, batch)
            check_current(where, state.get_device())
        else:
            qs, ks, vs, os_ = self._strides(q, k, v, o)
        p = _s._ptr
        _s._check(lib().stepq_linear_step(self._desc, batch, p(slot_ids), state.shape[0], p(q), qs, p(k), ks, p(v), vs,
                                          p(beta), p(gate), p(state), p(o), os_, stream_of(stream, state.get_device())),
                  where)

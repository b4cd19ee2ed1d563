"""Thin binding of the norms around a block in libstepq.so (include/stepq_block.h):
the norm behind a block, its gate, its residual scale, the residual sum and the norm before
the next block in one pass, and their gradients.

As in the other bindings, tensors become raw pointers, status codes become
exceptions, tensor arguments are checked against the sizes the call implies
before the library sees their pointers, and there is no fallback.
"""
from __future__ import annotations

import ctypes

from . import stepq as _s
from .linear import _refuse, check_current, check_dense, dense, dtype_code, leading, stream_of
from .recurrence import address
from .stepq import STEPQ_ERR_UNSUPPORTED, StepqError

EXPORTED = ("stepq_norm_forward", "stepq_norm_workspace_bytes", "stepq_norm_backward")

_ACTIVATIONS = {"silu": 0, "sigmoid": 1}


class stepq_norm_desc(ctypes.Structure):
    _fields_ = [("width", ctypes.c_int32), ("heads", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("post", ctypes.c_int32), ("pre", ctypes.c_int32), ("eps", ctypes.c_float)]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = _s.lib()
        P, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        L.stepq_norm_workspace_bytes.restype = sz
        L.stepq_norm_workspace_bytes.argtypes = [P, i64]
        L.stepq_norm_forward.restype = ctypes.c_int
        L.stepq_norm_forward.argtypes = [P, i64, P, i64, P, i64, P, i64, P, P, P, P, i64, P, i64, P]
        L.stepq_norm_backward.restype = ctypes.c_int
        L.stepq_norm_backward.argtypes = [P, i64, P, i64, P, i64, P, i64, P, P, P, P, i64, P, i64, P, i64, P, i64, P, i64, P, P,
                                          P, P, sz, P]
        _lib = L
    return _lib


class BlockNorm:
    """For rows of `width` values, `heads` of them side by side in a token:
    n = rms_norm(block) post_weight, t = residual + scale n act(gate), y = rms_norm(t) pre_weight,
    with `post` and `pre` saying which of the norms there are and "silu" or "sigmoid" as
    activation.  Gate, residual, weights and scale are left out by not passing them."""

    def __init__(self, width: int, heads: int = 1, dtype=None, activation: str = "silu", post: bool = True, pre: bool = True,
                 eps: float = 1e-6):
        import torch
        if activation not in _ACTIVATIONS:
            _refuse("BlockNorm", f"unknown activation {activation!r}; known: {sorted(_ACTIVATIONS)}")
        self.width, self.heads, self.post, self.pre = int(width), int(heads), bool(post), bool(pre)
        self.dtype = torch.float32 if dtype is None else dtype
        self._f32, self._tensor = torch.float32, torch.Tensor
        self.desc = stepq_norm_desc(self.width, self.heads, dtype_code(self.dtype), _ACTIVATIONS[activation], int(self.post),
                                    int(self.pre), float(eps))
        self._desc = ctypes.addressof(self.desc)
        # an empty call runs the library's own checks of the description
        null = ctypes.c_void_p()
        _s._check(lib().stepq_norm_forward(self._desc, 0, null, 0, null, 0, null, 0, null, null, null, null, 0, null, 0, null),
                  "BlockNorm")
        self._row = self.heads * self.width

    def workspace(self, tokens: int, device="cuda"):
        """A workspace for backward passes of up to `tokens` tokens."""
        import torch
        n = int(lib().stepq_norm_workspace_bytes(self._desc, int(tokens)))
        if n == 0 and tokens != 0:
            raise StepqError(STEPQ_ERR_UNSUPPORTED, "BlockNorm", f"{tokens} tokens")
        return torch.empty(max(16, n), dtype=torch.uint8, device=device)

    def _rows(self, where: str, name: str, t, tokens: int, index: int) -> int:
        """The stride of a [tokens, heads * width] tensor whose tokens may be strided; 0 for None."""
        if t is None:
            return 0
        if not _s._checks:
            return t.stride(0) if tokens > 1 else self._row
        if not isinstance(t, self._tensor) or t.get_device() != index or t.dtype is not self.dtype:
            _refuse(where, f"{name} must be a {self.dtype} tensor on cuda:{max(index, 0)}")
        if t.shape != (tokens, self._row):
            _refuse(where, f"{name} must have shape {[tokens, self._row]} (got {list(t.shape)})")
        n, e = t.stride()
        if tokens <= 1:      # the only token's stride says nothing
            n = self._row
        if (e != 1 and self._row > 1) or n < self._row:
            _refuse(where, f"{name}'s values must lie side by side and its tokens must not overlap (strides {list(t.stride())})")
        return n

    def _device(self, where: str, block) -> int:
        if not isinstance(block, self._tensor) or not block.is_cuda:
            _refuse(where, "block must be a device tensor")
        return block.get_device()

    def _weights(self, where: str, index: int, weights) -> None:
        for name, w in weights:
            if w is not None and not dense(w, self._f32, (self.width,), index):
                import torch
                check_dense(where, name, w, (self.width,), self._f32, torch.device("cuda", index))

    def forward(self, block, out, normed=None, gate=None, residual=None, post_weight=None, scale=None, pre_weight=None,
                stream=None) -> None:
        """stepq_norm_forward: writes t to out and, where there is a norm before the next block,
        y to normed (out may then be None).  out and normed may be the buffers of inputs."""
        where = "stepq_norm_forward"
        tokens = leading(where, "block", block)
        i = self._device(where, block)
        rows = self._rows
        bs, os_, ns = rows(where, "block", block, tokens, i), rows(where, "out", out, tokens, i), rows(where, "normed", normed, tokens, i)
        gs, rs = rows(where, "gate", gate, tokens, i), rows(where, "residual", residual, tokens, i)
        if _s._checks:
            self._weights(where, i, (("post_weight", post_weight), ("scale", scale), ("pre_weight", pre_weight)))
            if (normed is not None) != self.pre or (out is None and not self.pre):
                _refuse(where, "normed belongs to a norm before the next block, and out is needed where there is none")
            check_current(where, i)
        if tokens == 0:
            return
        p = address
        _s._check(lib().stepq_norm_forward(self._desc, tokens, p(block), bs, p(gate), gs, p(residual), rs, p(post_weight),
                                           p(scale), p(pre_weight), p(out), os_, p(normed), ns, stream_of(stream, i)), where)

    def backward(self, block, out, d_out, d_block, d_normed=None, gate=None, d_gate=None, d_residual=None, post_weight=None,
                 d_post_weight=None, scale=None, d_scale=None, pre_weight=None, d_pre_weight=None, workspace=None,
                 stream=None) -> None:
        """stepq_norm_backward: from the gradients d_out of t (None: there is none) and d_normed of y,
        those of block, gate and residual, and of the weights that are asked for.  out is what
        forward() wrote; it is read only where there is a norm before the next block."""
        import torch
        where = "stepq_norm_backward"
        tokens = leading(where, "block", block)
        i = self._device(where, block)
        named = (("block", block), ("gate", gate), ("out", out if self.pre else None), ("d_out", d_out), ("d_normed", d_normed),
                 ("d_block", d_block), ("d_gate", d_gate), ("d_residual", d_residual))
        bs, gs, os_, dos, dns, dbs, dgs, drs = (self._rows(where, name, t, tokens, i) for name, t in named)
        if _s._checks:
            self._weights(where, i, (("post_weight", post_weight), ("scale", scale), ("pre_weight", pre_weight),
                                     ("d_post_weight", d_post_weight), ("d_scale", d_scale), ("d_pre_weight", d_pre_weight)))
            if workspace is not None and not (isinstance(workspace, torch.Tensor) and workspace.dtype is torch.uint8 and
                                              workspace.get_device() == i and workspace.dim() == 1 and
                                              workspace.is_contiguous()):
                check_dense(where, "workspace", workspace, (None,), torch.uint8, block.device)
            check_current(where, i)
        if workspace is None and not (d_post_weight is None and d_scale is None and d_pre_weight is None):
            if stream is not None:
                _refuse(where, "a call on another stream needs a workspace of its own")
            workspace = self.workspace(tokens, block.device)
        p = address
        ptrs = [p(t) for _, t in named]
        (bp, gp, op, dop, dnp, dbp, dgp, drp) = ptrs
        _s._check(lib().stepq_norm_backward(self._desc, tokens, bp, bs, gp, gs, op, os_, p(post_weight), p(scale), p(pre_weight),
                                            dop, dos, dnp, dns, dbp, dbs, dgp, dgs, drp, drs, p(d_post_weight), p(d_scale),
                                            p(d_pre_weight), p(workspace), 0 if workspace is None else workspace.numel(),
                                            stream_of(stream, i)), where)

"""Thin binding of the verification of drafted tokens in libstepq.so
(include/stepq_block.h): which of a request's drafts a target model accepts, and the token
after them, from given random numbers.

As in the other bindings, tensors become raw pointers, status codes become
exceptions, tensor arguments are checked before the library sees their
pointers, and there is no fallback.
"""
from __future__ import annotations

import ctypes

from . import stepq as _s
from .linear import check_current, check_dense, dense, dtype_code, stream_of
from .recurrence import address
from .stepq import STEPQ_ERR_INVALID_ARG, STEPQ_ERR_UNSUPPORTED, StepqError

EXPORTED = ("stepq_verify_workspace_bytes", "stepq_verify_drafts")

_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = _s.lib()
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.stepq_verify_workspace_bytes.restype = sz
        L.stepq_verify_workspace_bytes.argtypes = [i32, i32, i32]
        L.stepq_verify_drafts.restype = ctypes.c_int
        L.stepq_verify_drafts.argtypes = [i32, i32, i32, P, i32, i64, P, i64, P, P, P, P, P, P, P, sz, P]
        _lib = L
    return _lib


class DraftVerify:
    """Verification for `batch` requests of up to `drafts` drafted tokens over `vocab` tokens (drafts = 0
    draws tokens): keeps the workspace and the buffers of the result, which the next call
    overwrites.  Calls of one object on different streams therefore have to be ordered by
    the caller, as two calls on one workspace do."""

    def __init__(self, batch: int, drafts: int, vocab: int, dtype=None, device="cuda"):
        import torch
        self.batch, self.drafts, self.vocab = int(batch), int(drafts), int(vocab)
        self.dtype = torch.float32 if dtype is None else dtype
        self._code = dtype_code(self.dtype)
        self._f32, self._i32, self._tensor = torch.float32, torch.int32, torch.Tensor
        null = ctypes.c_void_p()       # an empty call runs the library's own checks of the sizes
        _s._check(lib().stepq_verify_drafts(0, self.drafts, self.vocab, null, self._code, self.vocab, null, 0, null, null, null,
                                            null, null, null, null, 0, null), "DraftVerify")
        if self.batch < 1:
            raise StepqError(STEPQ_ERR_INVALID_ARG, "DraftVerify", "batch must be at least 1")
        need = lib().stepq_verify_workspace_bytes(self.batch, self.drafts, self.vocab)
        if need == 0:
            raise StepqError(STEPQ_ERR_UNSUPPORTED, "DraftVerify", "too many rows")
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)
        self.device = self.workspace.device
        self._index = self.workspace.get_device()
        self.accepted = torch.empty(self.batch, dtype=torch.int32, device=device)
        self.tokens = torch.empty(self.batch, self.drafts + 1, dtype=torch.int32, device=device)

    def _logits(self, where: str, name: str, t, rows: int) -> int:
        """The stride of [rows, vocab] logits whose rows may be strided."""
        if _s._checks:
            if not isinstance(t, self._tensor) or t.get_device() != self._index or t.dtype is not self.dtype:
                raise StepqError(STEPQ_ERR_INVALID_ARG, where, f"{name} must be a {self.dtype} tensor on {self.device}")
            if t.shape != (rows, self.vocab) or (self.vocab > 1 and t.stride(1) != 1):
                raise StepqError(STEPQ_ERR_INVALID_ARG, where, f"{name} must be [{rows}, {self.vocab}] with rows in one piece "
                                 f"(got {list(t.shape)}, strides {list(t.stride())})")
        return t.stride(0) if rows > 1 else self.vocab      # the only row's stride says nothing

    def __call__(self, logits, draft_tokens, uniforms, draft_logits=None, num_drafts=None, temperature=None, stream=None):
        """stepq_verify_drafts of logits [batch * (drafts + 1), vocab] (rows may be strided), draft_tokens
        [batch, drafts] and uniforms [batch, drafts + 1]; draft_logits [batch * drafts, vocab] (None: the
        draft was certain of its tokens), num_drafts [batch] (None: all) and temperature [batch]
        (None: 1).  Returns (accepted [batch], tokens [batch, drafts + 1]).  draft_tokens may be None
        where drafts is 0."""
        where, b, k, i = "stepq_verify_drafts", self.batch, self.drafts, self._index
        stride = self._logits(where, "logits", logits, b * (k + 1))
        draft_stride = 0 if draft_logits is None or k == 0 else self._logits(where, "draft_logits", draft_logits, b * k)
        if _s._checks:
            if (k > 0 or draft_tokens is not None) and not dense(draft_tokens, self._i32, (b, k), i) or i < 0:
                check_dense(where, "draft_tokens", draft_tokens, (b, k), self._i32, self.device)
            if not dense(uniforms, self._f32, (b, k + 1), i):
                check_dense(where, "uniforms", uniforms, (b, k + 1), self._f32, self.device)
            if num_drafts is not None and not dense(num_drafts, self._i32, (b,), i):
                check_dense(where, "num_drafts", num_drafts, (b,), self._i32, self.device)
            if temperature is not None and not dense(temperature, self._f32, (b,), i):
                check_dense(where, "temperature", temperature, (b,), self._f32, self.device)
            check_current(where, i)
        p = address
        _s._check(lib().stepq_verify_drafts(b, k, self.vocab, p(logits), self._code, stride,
                                            p(draft_logits) if k else None, draft_stride, p(draft_tokens) if k else None,
                                            p(num_drafts), p(temperature), p(uniforms), p(self.accepted), p(self.tokens),
                                            p(self.workspace), self.workspace.numel(), stream_of(stream, i)), where)
        return self.accepted, self.tokens

"""Thin binding of beam selection and state reordering in libstepq.so
(include/stepq_seq.h): the best continuations of every request over its beams
and the vocabulary, and the states' slots brought in line with them.

As in the binding of the packed step, tensors become raw pointers, status codes
become exceptions, tensor arguments are checked before the library sees their
pointers, and there is no fallback.
"""
from __future__ import annotations

import ctypes

from . import stepq as _s
from .linear import check_current, check_dense, dense, dtype_code, leading, stream_of
from .stepq import STEPQ_ERR_INVALID_ARG, STEPQ_ERR_UNSUPPORTED, StepqError

EXPORTED = ("stepq_beam_workspace_bytes", "stepq_beam_select", "stepq_beam_reorder")
MAX_REGIONS = 128


class stepq_region(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("slot_bytes", ctypes.c_size_t)]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = _s.lib()
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.stepq_beam_workspace_bytes.restype = sz
        L.stepq_beam_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.stepq_beam_select.restype = ctypes.c_int
        L.stepq_beam_select.argtypes = [i32, i32, i32, i32, P, i32, i64, P, P, i32, P, P, P, P, sz, P]
        L.stepq_beam_reorder.restype = ctypes.c_int
        L.stepq_beam_reorder.argtypes = [i32, i32, P, P, i32, P, i32, P, P]
        _lib = L
    return _lib


class BeamSelect:
    """Selection for `batch` requests of `beams` beams over `vocab` tokens, no more
    and no fewer: keeps the workspace and the buffers of the result, which the next
    call overwrites.  Calls of one object on different streams therefore have to be
    ordered by the caller, as two calls on one workspace do."""

    def __init__(self, batch: int, beams: int, vocab: int, num_out: int | None = None, dtype=None, eos_token: int = 0,
                 device="cuda"):
        import torch
        self.batch, self.beams, self.vocab = int(batch), int(beams), int(vocab)
        self.num_out = self.beams if num_out is None else int(num_out)
        self.dtype, self.eos_token = torch.float32 if dtype is None else dtype, int(eos_token)
        self._code = dtype_code(self.dtype)
        null = ctypes.c_void_p()       # an empty call runs the library's own checks of the sizes
        _s._check(lib().stepq_beam_select(0, self.beams, self.vocab, self.num_out, null, self._code, self.vocab, null, null,
                                          0, null, null, null, null, 0, null), "BeamSelect")
        if self.batch < 1:
            raise StepqError(STEPQ_ERR_INVALID_ARG, "BeamSelect", "batch must be at least 1")
        need = lib().stepq_beam_workspace_bytes(self.batch, self.beams, self.vocab, self.num_out)
        if need == 0:
            raise StepqError(STEPQ_ERR_UNSUPPORTED, "BeamSelect", "too many rows")
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)
        self.device = self.workspace.device
        self._index = self.workspace.get_device()
        self.tokens = torch.empty(self.batch, self.num_out, dtype=torch.int32, device=device)
        self.parents = torch.empty_like(self.tokens)
        self.scores = torch.empty(self.batch, self.num_out, dtype=torch.float32, device=device)

    def __call__(self, logits, scores, finished=None, stream=None):
        """stepq_beam_select of logits [batch * beams, vocab] (rows may be strided)
        and scores [batch * beams]: (tokens, parents, scores), each
        [batch, num_out], in order."""
        where = "stepq_beam_select"
        rows = self.batch * self.beams
        if _s._checks:
            import torch
            i = self._index
            if not isinstance(logits, torch.Tensor) or logits.get_device() != i or logits.dtype is not self.dtype:
                raise StepqError(STEPQ_ERR_INVALID_ARG, where, f"logits must be a {self.dtype} tensor on {self.device}")
            if logits.shape != (rows, self.vocab) or (self.vocab > 1 and logits.stride(1) != 1):
                raise StepqError(STEPQ_ERR_INVALID_ARG, where, f"logits must be [{rows}, {self.vocab}] with rows in one "
                                 f"piece (got {list(logits.shape)}, strides {list(logits.stride())})")
            if not dense(scores, torch.float32, (rows,), i) or i < 0:
                check_dense(where, "scores", scores, (rows,), torch.float32, self.device)
            if finished is not None and not dense(finished, torch.uint8, (rows,), i):
                check_dense(where, "finished", finished, (rows,), torch.uint8, self.device)
            check_current(where, i)
        stride = logits.stride(0) if rows > 1 else self.vocab      # the only row's stride says nothing
        p = _s._ptr
        _s._check(lib().stepq_beam_select(self.batch, self.beams, self.vocab, self.num_out, p(logits), self._code, stride,
                                          p(scores), p(finished), self.eos_token, p(self.tokens), p(self.parents),
                                          p(self.scores), p(self.workspace), self.workspace.numel(),
                                          stream_of(stream, self._index)), where)
        return self.tokens, self.parents, self.scores


def reorder(beams: int, slot_ids, parents, buffers, new_slot_ids, num_slots: int | None = None, stream=None) -> None:
    """stepq_beam_reorder of the slots of `buffers`, contiguous device tensors
    that hold num_slots slots each (a packed pool, its scales, the states of a
    layer, ...; num_slots is the first buffer's leading size where it is not
    given).  slot_ids, parents and new_slot_ids: int32 [batch * beams]."""
    where = "stepq_beam_reorder"
    n = leading(where, "slot_ids", slot_ids)
    if num_slots is None:
        if not buffers:
            raise StepqError(STEPQ_ERR_INVALID_ARG, where, "num_slots is needed where there are no buffers")
        num_slots = leading(where, "a buffer", buffers[0])
    if len(buffers) > MAX_REGIONS:
        raise StepqError(STEPQ_ERR_UNSUPPORTED, where, f"more than {MAX_REGIONS} buffers")
    if num_slots < 1 or beams < 1:
        raise StepqError(STEPQ_ERR_INVALID_ARG, where, "beams and num_slots must be at least 1")
    if _s._checks:
        import torch
        if not isinstance(slot_ids, torch.Tensor):
            check_dense(where, "slot_ids", slot_ids, (n,), torch.int32, None)
        dev, i = slot_ids.device, slot_ids.get_device()
        for name, t in (("slot_ids", slot_ids), ("parents", parents), ("new_slot_ids", new_slot_ids)):
            if i < 0 or not dense(t, torch.int32, (n,), i):
                check_dense(where, name, t, (n,), torch.int32, dev)
        if n % beams:
            raise StepqError(STEPQ_ERR_INVALID_ARG, where, f"{n} slots are no whole number of requests of {beams} beams")
        for t in buffers:
            if not isinstance(t, torch.Tensor) or t.get_device() != i or not t.is_contiguous() or t.nbytes % num_slots:
                raise StepqError(STEPQ_ERR_INVALID_ARG, where,
                                 f"a buffer must be a contiguous tensor on {dev} of {num_slots} equal slots")
        check_current(where, i)
    regions = (stepq_region * len(buffers))(*((t.data_ptr(), t.nbytes // num_slots) for t in buffers))
    p = _s._ptr
    _s._check(lib().stepq_beam_reorder(n // beams, int(beams), p(slot_ids), p(parents), int(num_slots), regions, len(buffers),
                                       p(new_slot_ids), stream_of(stream, slot_ids.get_device())), where)

"""What the bindings of prompts, tokens and beams refuse before the library sees a
pointer: things that are no tensors, and tensors of a device that is not current."""
import types

import numpy as np
import pytest

from quantized_recurrent_state_packed_amd import beam as B
from quantized_recurrent_state_packed_amd import build_lib
from quantized_recurrent_state_packed_amd import linear as LN
from quantized_recurrent_state_packed_amd import stepq as S


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not S.LIB_PATH.exists():
        build_lib.build()


def linear_arguments(torch, device):
    x = torch.zeros(5, 2, 16, device=device)
    f = torch.zeros(5, 2, device=device)
    return dict(q=x, k=x, v=x, beta=f, gate=f, slot_ids=torch.arange(5, dtype=torch.int32, device=device),
                state=torch.zeros(5, 2, 16, 16, device=device), o=torch.zeros_like(x))


@pytest.mark.parametrize("name", ["slot_ids", "q", "k", "v", "beta", "gate", "state", "o"])
@pytest.mark.parametrize("value", [None, 3, [1, 2], np.zeros((5, 2, 16), np.float32), "0-dim"], ids=str)
def test_linear_attention_refuses_what_is_no_tensor(name, value):
    import torch
    att = LN.LinearAttention(2, 16)
    a = linear_arguments(torch, "cpu")
    a[name] = torch.tensor(1) if isinstance(value, str) else value
    with pytest.raises(S.StepqError) as e:
        att.step(**a)
    assert e.value.status == S.STEPQ_ERR_INVALID_ARG
    for more in (dict(), dict(workspace=3), dict(resume=[1])):
        with pytest.raises(S.StepqError) as e:
            att.prefill(torch.tensor([0, 1, 2, 3, 4, 5], dtype=torch.int32), **a, **more)
        assert e.value.status == S.STEPQ_ERR_INVALID_ARG


@pytest.mark.parametrize("value", [None, 3, [1, 2], np.zeros(4, np.int32), "0-dim"], ids=str)
def test_beams_refuse_what_is_no_tensor(value):
    import torch
    bad = torch.tensor(1) if isinstance(value, str) else value
    ids = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros(4, 16)
    for args in ((bad, ids, [pool], ids.clone()), (ids, bad, [pool], ids.clone()), (ids, ids, [bad], ids.clone()),
                 (ids, ids, [pool], bad)):
        with pytest.raises(S.StepqError) as e:
            B.reorder(2, *args)
        assert e.value.status == S.STEPQ_ERR_INVALID_ARG
    sel = B.BeamSelect(1, 2, 10, device="cpu")
    for args in ((bad, torch.zeros(2)), (torch.zeros(2, 10), bad)):
        with pytest.raises(S.StepqError) as e:
            sel(*args)
        assert e.value.status == S.STEPQ_ERR_INVALID_ARG


@pytest.mark.gpu
def test_workspace_and_resume_that_are_no_tensors():
    import torch
    att = LN.LinearAttention(2, 16)
    a = linear_arguments(torch, "cuda")
    cu = torch.tensor([0, 1, 2, 3, 4, 5], dtype=torch.int32, device="cuda")
    for more in (dict(workspace=3), dict(workspace=np.zeros(1 << 20, np.uint8)), dict(resume=[1] * 5)):
        with pytest.raises(S.StepqError) as e:
            att.prefill(cu, **a, **more)
        assert e.value.status == S.STEPQ_ERR_INVALID_ARG
    att.prefill(cu, **a)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_tensors_of_a_device_that_is_not_current_are_refused(monkeypatch):
    """The library launches on the current device, so another device's tensors (and its
    default stream, whose handle is the same 0) must not reach it."""
    import torch
    att = LN.LinearAttention(2, 16)
    a = linear_arguments(torch, "cuda")
    cu = torch.tensor([0, 1, 2, 3, 4, 5], dtype=torch.int32, device="cuda")
    ids = torch.arange(4, dtype=torch.int32, device="cuda")
    pool, new = torch.zeros(4, 16, device="cuda"), torch.empty_like(ids)
    sel = B.BeamSelect(1, 2, 10)
    x, s = torch.zeros(2, 10, device="cuda"), torch.zeros(2, device="cuda")
    calls = (lambda: att.step(**a), lambda: att.prefill(cu, **a), lambda: B.reorder(2, ids, ids % 2, [pool], new),
             lambda: sel(x, s))
    for call in calls:
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(LN, "_current_device", lambda: 1)
    for call in calls:
        with pytest.raises(S.StepqError, match="current") as e:
            call()
        assert e.value.status == S.STEPQ_ERR_INVALID_ARG

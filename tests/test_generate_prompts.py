"""Prompts that the beam generator refuses: each has to be a non-empty list of
tokens of the vocabulary, one for every request.  On the CPU; nothing is launched."""
import types

import pytest

from quantized_recurrent_state_packed_amd import build_lib
from quantized_recurrent_state_packed_amd import generate as G
from quantized_recurrent_state_packed_amd import stepq as S


@pytest.fixture(scope="module")
def generator():
    import torch
    if not S.LIB_PATH.exists():
        build_lib.build()
    model = G.RandomModel(vocab=61, width=24, layers=2, heads=3, d=16, device="cpu")
    layout = types.SimpleNamespace(handle=0, alloc=lambda n, device: (torch.zeros(n, 16), torch.zeros(n, 16)))
    return G.BeamGenerator(model, 3, 2, layout, device="cpu")


@pytest.mark.parametrize("prompts,why", [
    ([[1, 2], [], [3]], "request 1's prompt is empty"), ([[], [1], [2]], "request 0's prompt is empty"),
    ([[1], [2], []], "request 2's prompt is empty"), ([[], [], []], "request 0's prompt is empty"),
    ([[1], [2]], "2 prompts for a batch of 3"), ([[1], [2], [3], [4]], "4 prompts for a batch of 3"),
    ([[1], [61], [2]], "request 1's prompt has tokens outside of the vocabulary of 61"),
    ([[1], [5], [2, -1]], "request 2's prompt has tokens outside of the vocabulary of 61"),
])
def test_prompts_that_are_refused(generator, prompts, why):
    with pytest.raises(S.StepqError, match=why) as e:
        generator.prefill(prompts)
    assert e.value.status == S.STEPQ_ERR_INVALID_ARG
    with pytest.raises(S.StepqError, match=why):
        generator.run(prompts, 1)

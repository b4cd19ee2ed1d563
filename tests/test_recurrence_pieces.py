"""The gated linear recurrence on sizes whose forward pass takes pieces of 128 tokens: requests of several pieces and runs
of pieces, more than one block of columns, every type, rows in pairs and one channel a lane.

A forward pass of few workgroups takes pieces of 64 tokens, in eight waves, as the backward pass always does; states then go from
run to run of 64 of them.  Those of 128 tokens have four waves, and runs of 16.  Which one a case takes is checked by the rule
of the library's source, against which the sizes here were chosen."""
import re

import numpy as np
import pytest

from test_recurrence import Case, RATE
from test_seq_host import CSRC
from quantized_recurrent_state_packed_amd import recurrence as RC

RULE = (CSRC / "scan_internal.hpp").read_text()
LONG = [127, 128, 129, 0, 2047, 2048, 2049, 4097]       # 1, 1, 2, 0, 16, 16, 17 and 33 pieces


def constant(name):
    return int(re.search(rf"\b{name} = (\d+)", RULE).group(1))


def large(tokens, batch, width):
    """Whether the forward pass takes pieces of 128 tokens."""
    piece = constant("kScanTokens") * constant("kScanWaves")
    assert piece == 128
    return (tokens // piece + batch) * -(-width // 128) >= constant("kFewGroups")


def large_case(*args, **kw):
    c = Case(*args, **kw)
    assert large(c.T, c.batch, c.width)
    return c


def test_the_rule_stands_where_it_is_read():
    assert "scan_pieces(total_tokens, batch, kScanPiece) * ((d.width + 127) / 128) < kFewGroups ? kFewPiece : kScanPiece" in RULE
    assert large(10829, 8, 130) and not large(1500, 1, 203)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("width,pad", [(130, 0), (130, 1), (203, 0)])
def test_requests_of_several_pieces(width, pad, dtype):
    large_case(LONG, width, dtype, seed=width + pad, pad=pad).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_many_blocks_of_columns(dtype):
    large_case([129, 0, 2049, 128, 400], 1408, dtype).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_unknown_slots_of_requests_of_several_pieces(dtype):
    large_case(LONG, 130, dtype, seed=1, bad=((4, -1), (5, 1 << 30), (2, 10))).check()


@pytest.mark.gpu
@pytest.mark.parametrize("resume,slots", [(False, True), (False, False)])
def test_requests_of_several_pieces_that_start_from_zero(resume, slots):
    large_case(LONG, 130, "bf16", seed=2, resume=resume, slots=slots).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nothing_saved(dtype):
    large_case(LONG, 203, dtype, seed=3).check(gradients=False)


@pytest.mark.gpu
def test_a_value_that_is_not_finite_spoils_its_own_request_and_channel_alone():
    """At the 2500th token of a request of 4097, in its 20th piece: what is behind it, in its channel."""
    import torch
    c, d = (large_case(LONG, 203, "f32", seed=4) for _ in range(2))
    start, end = int(c.cu_host[7]), int(c.cu_host[8])
    c.x[start + 2500, 150] = float("nan")
    for k in (c, d):
        ws, saved = k.buffers()
        k.forward(saved, workspace=ws)
        k.backward(saved, workspace=ws)
    torch.cuda.synchronize()
    inside = slice(int(c.cu_host[0]), end)
    rest = torch.ones_like(c.y, dtype=torch.bool)
    rest[start:end, 150] = False
    for n in ("y", "dx", "dga", "dgx"):
        assert torch.equal(getattr(c, n)[inside][rest[inside]], getattr(d, n)[inside][rest[inside]]), n
    assert torch.isnan(c.y[start + 2500:end, 150]).all()
    assert torch.equal(c.y[start:start + 2500, 150], d.y[start:start + 2500, 150])


@pytest.mark.gpu
@pytest.mark.parametrize("width", [203, 256])
def test_same_bits_again_on_another_stream_and_in_a_graph(width):
    """Two calls at once on two streams, each with its own workspace, and replays of a captured one."""
    import torch

    def case():
        return large_case([3000, 0, 2049, 64, 5000], width, "bf16", seed=9)

    first = case()
    ws, saved = first.buffers()
    first.forward(saved, workspace=ws)
    first.backward(saved, workspace=ws)
    cases = [(case(), torch.cuda.Stream()) for _ in range(2)]
    buffers = [c.buffers() for c, _ in cases]
    torch.cuda.synchronize()
    for (c, stream), (ws, saved) in zip(cases, buffers):
        c.forward(saved, workspace=ws, stream=stream)
        c.backward(saved, workspace=ws, stream=stream)
    torch.cuda.synchronize()

    def same(c):
        for n in ("y", "dx", "dga", "dgx"):
            a, b = (getattr(k, n)[c.cu_host[0]:c.cu_host[-1]] for k in (c, first))
            assert torch.equal(a, b), n
        for n in ("ddecay", "state", "dstate"):
            assert torch.equal(getattr(c, n), getattr(first, n)), n

    for c, _ in cases:
        same(c)
    c = case()
    state0, dstate0 = c.state.clone(), c.dstate.clone()
    ws, saved = c.buffers()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward(saved, workspace=ws)
        c.backward(saved, workspace=ws)
    for _ in range(3):
        c.state.copy_(state0), c.dstate.copy_(dstate0), c.y.zero_(), c.ddecay.fill_(5.0)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        same(c)


@pytest.mark.gpu
def test_rows_past_32_bits():
    """A request of 140 tokens 2^25 bytes apart and more, among 199 empty ones."""
    import torch
    rows, width, stride, batch = 140, 64, 1 << 24, 200
    assert large(rows, batch, width)
    rec = RC.GatedRecurrence(width, torch.bfloat16, RATE)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, ga, gx = (torch.randn(rows, width, generator=g, device="cuda").bfloat16() for _ in range(3))
    flat = torch.zeros((rows - 1) * stride + width, dtype=torch.bfloat16, device="cuda")
    assert flat.numel() * 2 > 1 << 32
    far = flat.as_strided((rows, width), (stride, 1))
    far.copy_(x)
    cu = torch.from_numpy(np.r_[np.zeros(77), np.full(batch + 1 - 77, rows)].astype(np.int32)).cuda()
    decay, y, z = torch.full((width,), -3.0, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    rec.prefill(cu, x, ga, gx, decay, None, None, y)
    rec.prefill(cu, far, ga, gx, decay, None, None, z)
    rec.prefill(cu, x, ga, gx, decay, None, None, far)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and torch.equal(far, y)

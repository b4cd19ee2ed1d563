"""The variants of the prefill of 16-bit inputs: each is reached by some call, none
is built that no call reaches, and each gives the recurrence's result, on both
sides of every number of (request, head) pairs where another one takes over."""
import re
import subprocess

import numpy as np
import pytest

from quantized_recurrent_state_packed_amd import build_lib
from quantized_recurrent_state_packed_amd import stepq as S
from test_linear import OUT_TOL, Run, far
from test_linear_precision import STATE
from test_seq_host import run


def test_the_library_holds_the_variants_that_calls_reach_and_no_others(tmp_path):
    reached = set(run(tmp_path, "linear_host.cpp", "linear_api.cpp").splitlines())
    if not S.LIB_PATH.exists():
        build_lib.build()
    names = subprocess.run(["nm", str(S.LIB_PATH)], capture_output=True, text=True, check=True).stdout
    parts = {"DF16b": 1, "DF16_": 2}
    built = {f"walk {d} {parts[t]} {delta} {tiles} {waves} {one} {p}" for d, t, delta, tiles, waves, one, p in re.findall(
        r"k_linear16_walkILi(\d+)E(DF16b|DF16_)Lb([01])ELi(\d+)ELi(\d+)ELb([01])ELi(\d+)E", names)}
    built |= {f"chunks {d} {parts[t]} {delta}" for d, t, delta in re.findall(
        r"k_linear16_chunksILi(\d+)E(DF16b|DF16_)Lb([01])E", names)}
    assert built and built == reached


def recurrence64(r, resume):
    """o and the requests' states by the recurrence in binary64 on the GPU, all requests' tokens in step."""
    import torch
    n = torch.tensor(r.lengths, device="cuda")
    first = torch.from_numpy(r.cu[:-1].astype(np.int64)).cuda()
    rep = r.H // r.q.shape[1]
    m = torch.from_numpy(r.before[r.slots]).cuda().double()
    m *= torch.tensor(resume, device="cuda", dtype=torch.float64)[:, None, None, None]
    o = torch.zeros(r.v.shape, device="cuda", dtype=torch.float64)
    for t in range(max(r.lengths)):
        live = (n > t).nonzero()[:, 0]
        at = first[live] + t
        k, q = (x[at].double().repeat_interleave(rep, 1) for x in (r.k, r.q))
        mt = m[live] * r.gate[at].double()[:, :, None, None]
        u = r.v[at].double()
        if r.beta is not None:
            u = r.beta[at].double()[..., None] * (u - (mt * k[..., None]).sum(-2))
        mt += k[..., None] * u[:, :, None, :]
        o[at] = (mt * q[..., None]).sum(-2)
        m[live] = mt
    return o, m


def check(r, resume):
    ro, rm = recurrence64(r, resume)
    r.prefill(resume)
    slots = r.slots.tolist()
    state = r.state.double().cpu().numpy()
    o, ro, rm = r.o.double().cpu().numpy(), ro.cpu().numpy(), rm.cpu().numpy()
    for b, slot in enumerate(slots):
        at = slice(r.cu[b], r.cu[b + 1])
        assert far(state[slot], rm[b]) <= STATE, b
        for h in range(r.H):
            if r.lengths[b]:
                assert far(o[at][:, h], ro[at][:, h]) <= OUT_TOL[r.dtype], (b, h)
    rest = [s for s in range(r.num_slots) if s not in set(slots)]
    assert np.array_equal(r.state.cpu().numpy()[rest], r.before[rest])
    assert bool((r.untouched == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("rule", ["delta", "additive"])
@pytest.mark.parametrize("dtype,D,heads,batch", [
    ("bf16", 128, 16, 2), ("bf16", 128, 32, 2), ("bf16", 128, 13, 5), ("bf16", 128, 32, 3), ("bf16", 128, 64, 2),
    ("bf16", 128, 43, 3), ("bf16", 128, 50, 4),
    ("f16", 128, 16, 2), ("f16", 128, 11, 3), ("f16", 128, 32, 2), ("f16", 128, 13, 5), ("f16", 128, 32, 3), ("f16", 128, 64, 2),
    ("f16", 128, 43, 3), ("f16", 128, 50, 4),
    ("bf16", 64, 40, 1), ("bf16", 64, 43, 3), ("f16", 64, 43, 3), ("f16", 64, 50, 5),
    ("f16", 32, 64, 4), ("f16", 32, 43, 6), ("bf16", 32, 64, 6), ("bf16", 32, 77, 5), ("bf16", 32, 64, 13), ("f16", 32, 64, 11),
    ("bf16", 16, 64, 13), ("f16", 16, 43, 3)])
def test_numbers_of_pairs(dtype, D, heads, batch, rule):
    g = np.random.default_rng(heads * batch)
    lengths = [int(x) for x in g.choice([70, 129, 200, 33, 1, 64], size=batch)]
    lengths[0] = 200
    r = Run(dtype, heads, heads if heads % 2 else heads // 2, D, rule, lengths, seed=batch, fused=heads == 32)
    check(r, [b % 2 for b in range(batch)])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,heads,lengths", [(128, 96, [2900]), (64, 128, [2300]), (128, 40, [3000, 10, 5001]), (64, 60, [4001, 0, 700])],
                         ids=str)
def test_segments_of_more_than_four_chunks(dtype, D, heads, lengths):
    r = Run(dtype, heads, heads // 2, D, "additive", lengths, seed=heads)
    check(r, [1] + [0] * (len(lengths) - 1))


@pytest.mark.gpu
@pytest.mark.parametrize("rule", ["delta", "additive"])
def test_calls_in_one_launch_take_no_workspace(rule):
    """As many pairs as fill the chip: no memory is taken, on another stream either,
    and the result is the one with a workspace, bit for bit."""
    import torch
    r = Run("bf16", 24, 12, 128, rule, [130, 70, 64, 1, 0, 200, 90, 33], seed=3)
    assert prefill_bytes(r.att, 8, int(r.cu[-1])) == 0
    r.prefill()
    want = [r.o.clone(), r.state.clone()]
    cu, slots = torch.from_numpy(r.cu).cuda(), torch.from_numpy(r.slots).cuda()
    side = torch.cuda.Stream()
    r.o.fill_(7.0)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    r.att.prefill(cu, r.q, r.k, r.v, r.beta, r.gate, slots, r.state, r.o, stream=side)
    assert torch.cuda.max_memory_allocated() == before
    torch.cuda.synchronize()
    assert torch.equal(r.o, want[0]) and torch.equal(r.state, want[1])
    few = Run("bf16", 2, 1, 128, "delta", [130], seed=3)
    with pytest.raises(S.StepqError):
        few.att.prefill(torch.from_numpy(few.cu).cuda(), few.q, few.k, few.v, few.beta, few.gate,
                        torch.from_numpy(few.slots).cuda(), few.state, few.o, stream=side)


def prefill_bytes(att, batch, tokens):
    from quantized_recurrent_state_packed_amd import linear
    return linear.lib().stepq_linear_prefill_bytes(att._desc, batch, tokens)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,heads,rule,tokens", [
    ("bf16", 128, 2, "delta", 140), ("f16", 128, 2, "delta", 140), ("bf16", 64, 2, "delta", 140), ("f16", 64, 2, "additive", 140),
    ("bf16", 128, 2, "additive", 600), ("bf16", 32, 2, "delta", 140), ("f32", 128, 2, "delta", 140), ("f32", 64, 2, "additive", 140)])
def test_token_offsets_past_32_bits(dtype, D, heads, rule, tokens):
    """Tokens as far apart as is accepted, 2^24 elements: offsets of 2^32 bytes and more
    within q, k, v and o, and 2^31 bytes within a chunk.  Prompts, then a step of all rows."""
    import torch
    r = Run(dtype, heads, 1, D, rule, [tokens], seed=40)
    wide = torch.empty(tokens, 1 << 24, dtype=r.q.dtype, device="cuda")
    places = {}
    for at, (name, x) in zip((0, 1 << 12, 1 << 20, (1 << 24) - (1 << 12)), (("q", r.q), ("k", r.k), ("v", r.v), ("o", r.o))):
        places[name] = wide[:, at:at + x.shape[1] * D].unflatten(1, x.shape[1:])
        places[name].copy_(x)
    assert places["o"].stride(0) == 1 << 24 and (tokens - 1) * wide.stride(0) * wide.element_size() > 2 ** 32
    r.q, r.k, r.v, r.o = (places[n] for n in "qkvo")
    ro, rm = recurrence64(r, [1])
    r.prefill([1])
    factor = {"f32": 1e-5}.get(dtype, STATE)
    assert far(r.state[int(r.slots[0])].cpu().numpy(), rm[0].cpu().numpy()) <= factor
    assert far(r.o.double().cpu().numpy(), ro.cpu().numpy()) <= OUT_TOL[dtype]
    del ro, rm
    n = torch.arange(tokens, dtype=torch.int32, device="cuda")
    state = torch.randn(tokens, heads, D, D, device="cuda")
    before = state.double()
    r.att.step(n, r.q, r.k, r.v, r.beta, r.gate, state, r.o)
    torch.cuda.synchronize()
    k, q = (x.double().repeat_interleave(heads, 1) for x in (r.k, r.q))
    m = before * r.gate.double()[..., None, None]
    u = r.v.double()
    if r.beta is not None:
        u = r.beta.double()[..., None] * (u - (m * k[..., None]).sum(-2))
    m += k[..., None] * u[:, :, None, :]
    assert far(state.cpu().numpy(), m.cpu().numpy()) <= 1e-5
    assert far(r.o.double().cpu().numpy(), (m * q[..., None]).sum(-2).cpu().numpy()) <= OUT_TOL[dtype]

"""Linear attention over prompts and single tokens against the recurrence in
binary64 (tests/linear_ref.py), its refusals, and its ABI.

Tolerances, as relative 2-norms of every (request, head)'s outputs and state:
 * states and binary32 outputs of binary32 inputs: the arithmetic is binary32; a
   value passes at most four products of depth <= 192, each within about
   sqrt(192) * 2^-24 in the 2-norm of values without cancellation: 3.3e-6, and
   cancellation in v - M^T k costs a factor of up to 3: 1e-5;
 * states of 16-bit inputs: an operand may be held as two bfloat16 parts, which
   leaves about 2^-17 of its size (2^-16 at the bottom of a binade), in at most
   three chained products: 2.3e-5;
 * binary16 outputs: one rounding, at most 2^-11, on top: 5e-4;
 * bfloat16 outputs: one rounding of the result and one of each of three
   operands of the readout, each uniform within 2^-9: sqrt(4 / 3) * 2^-9 =
   2.3e-3 in the 2-norm, doubled for short vectors: 4.5e-3;
 * keys that all but coincide make (I + B)^-1 as large as the chunk is long in
   the worst case, damped by the retention: four times the above.
"""
import ctypes
import re
from pathlib import Path

import numpy as np
import pytest

from linear_ref import inputs, recurrence
from quantized_recurrent_state_packed_amd import build_lib
from quantized_recurrent_state_packed_amd import linear as LN
from quantized_recurrent_state_packed_amd import stepq as S

HEADER = Path(__file__).resolve().parents[1] / "include" / "stepq_seq.h"
STATE_TOL = {"f32": 1e-5, "f16": 2.3e-5, "bf16": 2.3e-5}
OUT_TOL = {"f32": 1e-5, "f16": 5e-4, "bf16": 4.5e-3}


@pytest.fixture(scope="module")
def lib():
    if not S.LIB_PATH.exists():
        build_lib.build()
    return LN.lib()


def torch_dtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


# ------------------------------------------------------------------ ABI, CPU

def test_header_and_library_agree_on_the_linear_entry_points(lib):
    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    names = set(re.findall(r"\b(stepq_linear_[a-z_]+)\s*\(", text))
    assert names == set(LN.EXPORTED)
    for n in names:
        assert hasattr(lib, n)


def desc(H=4, Hk=2, d=32, rule=LN.RULE_DELTA, dtype=LN.STEPQ_F32):
    return LN.stepq_linear_desc(H, Hk, d, rule, dtype)


@pytest.mark.parametrize("change,status", [
    (dict(H=0), S.STEPQ_ERR_INVALID_ARG), (dict(Hk=0), S.STEPQ_ERR_INVALID_ARG), (dict(Hk=3), S.STEPQ_ERR_INVALID_ARG),
    (dict(rule=2), S.STEPQ_ERR_INVALID_ARG), (dict(rule=-1), S.STEPQ_ERR_INVALID_ARG),
    (dict(dtype=3), S.STEPQ_ERR_INVALID_ARG), (dict(d=0), S.STEPQ_ERR_INVALID_ARG),
    (dict(d=48), S.STEPQ_ERR_UNSUPPORTED), (dict(d=256), S.STEPQ_ERR_UNSUPPORTED),
    (dict(H=1 << 17, Hk=1), S.STEPQ_ERR_UNSUPPORTED),
])
def test_descriptions_that_are_refused(lib, change, status):
    d = desc(**change)
    assert lib.stepq_linear_workspace_bytes(ctypes.addressof(d), 1, 64) == 0
    for call in (prefill_status, step_status):
        assert call(lib, d) == status


# Addresses that are never dereferenced: every call below is refused before a launch.
GOOD = 4096


def prefill_status(lib, d, batch=1, tokens=64, cu=GOOD, q=GOOD, qs=64, k=GOOD, ks=64, v=GOOD, vs=128, beta=GOOD,
                   gate=GOOD, slots=GOOD, num_slots=1, resume=None, state=GOOD, o=GOOD, os_=128, ws=GOOD, nbytes=None):
    d_ = None if d is None else ctypes.addressof(d)
    n = 0 if nbytes is None else nbytes
    return lib.stepq_linear_prefill(d_, batch, tokens, cu, q, qs, k, ks, v, vs, beta, gate, slots, num_slots, resume,
                                    state, o, os_, ws, n, None)


def step_status(lib, d, batch=1, slots=GOOD, num_slots=1, q=GOOD, qs=64, k=GOOD, ks=64, v=GOOD, vs=128, beta=GOOD,
                gate=GOOD, state=GOOD, o=None, os_=128):
    d_ = None if d is None else ctypes.addressof(d)
    return lib.stepq_linear_step(d_, batch, slots, num_slots, q, qs, k, ks, v, vs, beta, gate, state, o, os_, None)


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(tokens=-1), dict(num_slots=0), dict(cu=None), dict(cu=GOOD + 2), dict(slots=None),
    dict(slots=GOOD + 2), dict(q=None), dict(k=None), dict(v=None), dict(gate=None), dict(state=None), dict(o=None),
    dict(beta=None), dict(q=GOOD + 8), dict(v=GOOD + 4), dict(o=GOOD + 2), dict(state=GOOD + 8), dict(qs=60), dict(ks=66),
    dict(vs=64), dict(os_=127), dict(ws=None), dict(ws=GOOD + 8, nbytes=1 << 30), dict(nbytes=0),
    dict(nbytes=4 * 2 * (2 * 64 * 64 + 128) * 4 - 1),
])
def test_prefill_arguments_that_are_refused(lib, bad):
    assert prefill_status(lib, desc(), **bad) == S.STEPQ_ERR_INVALID_ARG


def test_prefill_sizes_beyond_the_grid_are_refused(lib):
    assert prefill_status(lib, desc(), tokens=1 << 31, nbytes=1 << 60) == S.STEPQ_ERR_UNSUPPORTED
    assert prefill_status(lib, desc(H=1 << 16, Hk=1), tokens=(1 << 31) - 1, nbytes=1 << 60) == S.STEPQ_ERR_UNSUPPORTED
    assert prefill_status(lib, desc(H=1 << 16, Hk=1, d=128), batch=1 << 13, tokens=0) == S.STEPQ_ERR_UNSUPPORTED
    assert prefill_status(lib, desc(), tokens=1 << 28, nbytes=1 << 60) == S.STEPQ_ERR_UNSUPPORTED
    assert step_status(lib, desc(H=1 << 10, Hk=1), batch=1 << 13, vs=1 << 15, os_=1 << 15) == S.STEPQ_ERR_UNSUPPORTED
    assert prefill_status(lib, desc(), qs=(1 << 24) + 64, nbytes=1 << 60) == S.STEPQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(num_slots=0), dict(slots=None), dict(q=None), dict(o=None), dict(beta=None), dict(qs=60),
    dict(vs=64), dict(state=GOOD + 4), dict(gate=GOOD + 2),
])
def test_step_arguments_that_are_refused(lib, bad):
    assert step_status(lib, desc(), **bad) == S.STEPQ_ERR_INVALID_ARG


def test_beta_with_the_additive_rule_and_null_descriptions_are_refused(lib):
    add = desc(rule=LN.RULE_ADDITIVE)
    assert prefill_status(lib, add) == S.STEPQ_ERR_INVALID_ARG
    assert step_status(lib, add, o=GOOD) == S.STEPQ_ERR_INVALID_ARG
    assert prefill_status(lib, None) == S.STEPQ_ERR_INVALID_ARG
    assert step_status(lib, None) == S.STEPQ_ERR_INVALID_ARG
    assert lib.stepq_linear_workspace_bytes(None, 1, 1) == 0


def test_empty_batches_are_accepted_without_a_launch(lib):
    assert prefill_status(lib, desc(), batch=0, cu=None, q=None, ws=None) == S.STEPQ_OK
    assert step_status(lib, desc(), batch=0, slots=None) == S.STEPQ_OK


def test_workspace_grows_with_tokens_and_requests(lib):
    d = desc()
    size = lambda b, t: lib.stepq_linear_workspace_bytes(ctypes.addressof(d), b, t)  # noqa: E731
    assert size(0, 0) == 0 and 0 < size(1, 0) == size(1, 63) < size(1, 64) == size(2, 0)
    assert size(-1, 64) == 0 and size(1, -1) == 0 and size(1, 1 << 31) == 0


@pytest.mark.parametrize("g", range(6))
def test_chunk_index_ranges_do_not_overlap(g):
    """Request b's chunks start at cu[b] // 64 + b: the ranges are disjoint, within
    the workspace, and a search for the last b with cu[b] // 64 + b <= index finds
    each chunk's request, for lengths around the chunk's size, zeros among them."""
    r = np.random.default_rng(g)
    n = r.choice([0, 0, 1, 63, 64, 65, 127, 128, 129, 300], size=int(r.integers(1, 40)))
    cu = np.r_[0, np.cumsum(n)]
    owner = {}
    for b in range(n.size):
        for c in range(-(-int(n[b]) // 64)):
            w = int(cu[b]) // 64 + b + c
            assert w not in owner and w < int(cu[-1]) // 64 + n.size
            owner[w] = (b, c)
    first = cu[:-1] // 64 + np.arange(n.size)
    assert np.all(np.diff(first) > 0)
    for w, (b, _) in owner.items():
        assert int(np.searchsorted(first, w, side="right")) - 1 == b


def test_binding_refuses_bad_tensors_before_the_library(lib):
    import torch
    with pytest.raises(S.StepqError, match="unknown rule"):
        LN.LinearAttention(4, 32, rule="gated")
    with pytest.raises(S.StepqError, match="not float32"):
        LN.LinearAttention(4, 32, dtype=torch.float64)
    with pytest.raises(S.StepqError) as e:
        LN.LinearAttention(4, 48)
    assert e.value.status == S.STEPQ_ERR_UNSUPPORTED
    with pytest.raises(S.StepqError) as e:
        LN.LinearAttention(4, 32, num_qk_heads=3)
    assert e.value.status == S.STEPQ_ERR_INVALID_ARG
    att = LN.LinearAttention(2, 16)
    x, f = torch.zeros(5, 2, 16), torch.zeros(5, 2)
    with pytest.raises(S.StepqError, match="device tensor"):
        att.step(torch.zeros(5, dtype=torch.int32), x, x, x, f, f, torch.zeros(5, 2, 16, 16), x)


# ---------------------------------------------------------------------- GPU

def far(x, y):
    """Relative 2-norm of x - y (absolute where y is zero)."""
    d, n = np.linalg.norm(np.asarray(x, np.float64) - y), np.linalg.norm(y)
    return float(d / n) if n else float(d)


class Run:
    """A prefill or a series of steps on the GPU with guard rows around what may be written."""

    def __init__(self, dtype, H, Hk, D, rule, lengths, seed=0, spare=2, fused=False, **kw):
        import torch
        self.dtype, self.rule, self.H, self.D = dtype, rule, H, D
        self.lengths = list(lengths)
        self.cu = np.r_[0, np.cumsum(lengths)].astype(np.int32)
        T, B = int(self.cu[-1]), len(self.lengths)
        a = inputs(seed, T, H, Hk, D, **kw)
        td = torch_dtype(dtype)
        dev = {n: torch.from_numpy(a[n]).cuda() for n in a}
        q, k, v = (dev[n].to(td) for n in "qkv")
        if fused:        # slices of one projection: tokens lie (2 Hk + H) D elements apart
            x = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1).contiguous()
            q = x[:, :Hk * D].unflatten(1, (Hk, D))
            k = x[:, Hk * D:2 * Hk * D].unflatten(1, (Hk, D))
            v = x[:, 2 * Hk * D:].unflatten(1, (H, D))
            wide = torch.full((T, 2, H, D), 7.0, dtype=td, device="cuda")
            o = wide[:, 0]
            self.untouched = wide[:, 1]
        else:
            guard = torch.full((T + 2, H, D), 7.0, dtype=td, device="cuda")
            o = guard[1:-1]
            self.untouched = guard[::T + 1]
        self.q, self.k, self.v, self.o = q, k, v, o
        self.beta = dev["beta"] if rule == "delta" else None
        self.gate = dev["gate"]
        g = np.random.default_rng(seed + 1)
        self.num_slots = B + spare
        self.slots = g.permutation(self.num_slots)[:B].astype(np.int32)
        self.state = torch.from_numpy(g.standard_normal((self.num_slots, H, D, D)).astype(np.float32) * 0.3).cuda()
        self.before = self.state.cpu().numpy()
        self.att = LN.LinearAttention(H, D, num_qk_heads=Hk, rule=rule, dtype=td)

    def host(self):
        """The inputs as the kernels see them, in float64."""
        f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        return f(self.q), f(self.k), f(self.v), f(self.beta), f(self.gate)

    def prefill(self, resume=None, slots=None, stream=None):
        import torch
        ws = self.att.workspace(len(self.lengths), int(self.cu[-1]))
        ws.fill_(0xFF)                                   # NaN wherever something unwritten is read
        r = None if resume is None else torch.from_numpy(np.asarray(resume, np.uint8)).cuda()
        s = torch.from_numpy(self.slots if slots is None else slots).cuda()
        self.att.prefill(torch.from_numpy(self.cu).cuda(), self.q, self.k, self.v, self.beta, self.gate, s, self.state,
                         self.o, resume=r, workspace=ws, stream=stream)
        torch.cuda.synchronize()

    def check(self, resume=None, factor=1.0):
        q, k, v, beta, gate = self.host()
        o, state = self.o.double().cpu().numpy(), self.state.cpu().numpy()
        for b, slot in enumerate(self.slots):
            at = slice(self.cu[b], self.cu[b + 1])
            m = self.before[slot] if resume is not None and resume[b] else np.zeros_like(self.before[slot])
            ro, rm = recurrence(q[at], k[at], v[at], None if beta is None else beta[at], gate[at], m)
            for h in range(self.H):
                assert far(state[slot, h], rm[h]) <= factor * STATE_TOL[self.dtype], (b, h)
                if self.lengths[b]:
                    assert far(o[at][:, h], ro[:, h]) <= factor * OUT_TOL[self.dtype], (b, h)
        rest = [s for s in range(self.num_slots) if s not in set(self.slots.tolist())]
        assert np.array_equal(state[rest], self.before[rest])
        assert bool((self.untouched == 7.0).all())


LENGTHS = [[1], [2, 1], [64], [63, 65, 1, 128], [0, 5, 0, 0, 130, 1], [200, 17]]


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("rule", ["additive", "delta"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_prefill_lengths(dtype, rule, lengths):
    r = Run(dtype, 4, 2, 64, rule, lengths, seed=len(lengths))
    resume = [b % 2 for b in range(len(lengths))]
    r.prefill(resume)
    r.check(resume)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (3, 1), (6, 2), (5, 5)], ids=str)
@pytest.mark.parametrize("rule", ["additive", "delta"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_prefill_head_layouts(dtype, rule, heads, D):
    r = Run(dtype, *heads, D, rule, [70, 33], seed=D)
    r.prefill()
    r.check()


@pytest.mark.gpu
@pytest.mark.parametrize("gates", ["one", "strong", "clearing"])
@pytest.mark.parametrize("rule", ["additive", "delta"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_gates(dtype, rule, gates):
    """No forgetting at all, retentions down to 1e-30, and retentions of exactly zero."""
    r = Run(dtype, 2, 2, 32, rule, [150, 64], seed=5, gates=gates)
    r.prefill([1, 0])
    r.check([1, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_prefill_keys_that_all_but_coincide(dtype):
    r = Run(dtype, 2, 1, 128, "delta", [200], seed=6, correlated=3.0, gates="one")
    r.prefill([1])
    r.check([1], factor=4.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [32, 128])
def test_slices_of_a_fused_projection(dtype, D):
    r = Run(dtype, 4, 2, D, "delta", [90, 40], seed=7, fused=True)
    r.prefill([0, 1])
    r.check([0, 1])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("rule", ["additive", "delta"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_many_requests(dtype, rule, D):
    """More (request, head) pairs than compute units: a head is not split over workgroups."""
    g = np.random.default_rng(D)
    lengths = [int(x) for x in g.choice([0, 1, 3, 40, 64, 70, 130], size=90)]
    r = Run(dtype, 3, 3, D, rule, lengths, seed=D, fused=D == 64)
    resume = (g.random(90) < 0.5).astype(np.uint8)
    r.prefill(resume)
    r.check(resume)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("gates", ["mixed", "strong"])
@pytest.mark.parametrize("rule", ["additive", "delta"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_long_prompts_of_few_heads(dtype, rule, gates, D):
    """Long on the average, an empty and a short one among them, some resuming, one
    without a slot: under the additive rule these are walked in segments."""
    r = Run(dtype, 2, 1, D, rule, [1500, 3, 0, 1023, 256, 700], seed=D, gates=gates)
    resume = [1, 0, 1, 0, 1, 1]
    slots = r.slots.copy()
    slots[4] = -3
    r.prefill(resume, slots=slots)
    o = r.o.float().cpu().numpy()
    lo, hi = r.cu[4], r.cu[5]
    assert np.isnan(o[lo:hi]).all() and np.array_equal(r.state[int(r.slots[4])].cpu().numpy(), r.before[r.slots[4]])
    r.prefill(resume=[0, 0, 0, 0, 1, 0], slots=np.where(np.arange(6) == 4, r.slots, -1).astype(np.int32))
    r.o[:lo], r.o[hi:] = torch_like(o[:lo], r.o), torch_like(o[hi:], r.o)
    r.check(resume)


def torch_like(x, t):
    import torch
    return torch.from_numpy(x).to(t.device, t.dtype)


def test_workspace_of_segments_grows_with_tokens_and_requests():
    att = LN.LinearAttention(8, 64, rule="additive", dtype=torch_dtype("bf16"))
    size = [att.workspace_bytes(b, t) for b, t in ((1, 100), (1, 5000), (3, 5000), (3, 60000), (40, 60000), (40, 10 ** 6))]
    assert size == sorted(size) and size[0] > 0


@pytest.mark.gpu
@pytest.mark.parametrize("rule", ["additive", "delta"])
def test_long_prompt_many_chunks(rule):
    r = Run("bf16", 2, 1, 128, rule, [3001, 5], seed=8)
    r.prefill()
    r.check()


@pytest.mark.gpu
@pytest.mark.parametrize("rule", ["additive", "delta"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_prompt_in_pieces_equals_prompt_at_once(dtype, rule):
    """A prompt admitted in three pieces, the later ones resuming, against the recurrence over all of it."""
    import torch
    whole = Run(dtype, 3, 1, 64, rule, [157], seed=9)
    q, k, v, beta, gate = whole.host()
    ro, rm = recurrence(q, k, v, beta, gate, np.zeros((3, 64, 64)))
    slots = torch.from_numpy(whole.slots).cuda()
    for n, (lo, hi) in enumerate([(0, 50), (50, 51), (51, 157)]):
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        whole.att.prefill(cu, whole.q[lo:hi], whole.k[lo:hi], whole.v[lo:hi],
                          None if beta is None else whole.beta[lo:hi].clone(), whole.gate[lo:hi].clone(), slots,
                          whole.state, whole.o[lo:hi], resume=torch.tensor([int(n > 0)], dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    for h in range(3):
        assert far(whole.state[int(whole.slots[0]), h].cpu().numpy(), rm[h]) <= STATE_TOL[dtype]
        assert far(whole.o[:, h].double().cpu().numpy(), ro[:, h]) <= OUT_TOL[dtype]


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1, 99, 2 ** 31 - 1])
def test_requests_without_a_slot(bad):
    r = Run("bf16", 2, 2, 32, "delta", [70, 3, 66], seed=10)
    slots = r.slots.copy()
    slots[1] = bad
    r.prefill(slots=slots)
    o = r.o.float().cpu().numpy()
    assert np.isnan(o[70:73]).all() and np.isfinite(o[:70]).all() and np.isfinite(o[73:]).all()
    state = r.state.cpu().numpy()
    kept = [s for s in range(r.num_slots) if s not in (slots[0], slots[2])]
    assert np.array_equal(state[kept], r.before[kept])


@pytest.mark.gpu
def test_non_finite_values_stay_with_their_request_and_column():
    r = Run("bf16", 2, 2, 32, "delta", [70, 40, 66], seed=11)
    clean = Run("bf16", 2, 2, 32, "delta", [70, 40, 66], seed=11)
    clean.prefill()
    r.v[75, 1, 3] = float("inf")
    r.v[90, 0, 5] = float("nan")
    r.prefill()
    same = (r.o == clean.o).cpu().numpy()
    assert same[:70].all() and same[110:].all()
    cols = np.ones((2, 32), bool)
    cols[1, 3] = cols[0, 5] = False
    assert same[:, cols].all()
    assert not np.isfinite(r.o[109, 1, 3].item()) and not np.isfinite(r.o[109, 0, 5].item())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,batch", [((1, 1), 1), ((6, 2), 3), ((3, 3), 40)], ids=str)
@pytest.mark.parametrize("rule", ["additive", "delta"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_steps(dtype, rule, heads, batch, D):
    """Three single tokens of every request.  A step is binary32 throughout, so
    its state has the binary32 tolerance whatever the inputs' type."""
    import torch
    r = Run(dtype, *heads, D, rule, [3] * batch, seed=D + batch, fused=batch == 3)
    q, k, v, beta, gate = r.host()
    slots = torch.from_numpy(r.slots).cuda()
    for t in range(3):
        at = slice(t, None, 3)
        r.att.step(slots, r.q[at], r.k[at], r.v[at], None if beta is None else r.beta[at].contiguous(),
                   r.gate[at].contiguous(), r.state, r.o[at])
    torch.cuda.synchronize()
    o, state = r.o.double().cpu().numpy(), r.state.cpu().numpy()
    for b, slot in enumerate(r.slots):
        at = slice(3 * b, 3 * b + 3)
        ro, rm = recurrence(q[at], k[at], v[at], None if beta is None else beta[at], gate[at], r.before[slot])
        assert far(state[slot], rm) <= STATE_TOL["f32"]
        assert far(o[at], ro) <= OUT_TOL[dtype]
    rest = [s for s in range(r.num_slots) if s not in set(r.slots.tolist())]
    assert np.array_equal(state[rest], r.before[rest])
    assert bool((r.untouched == 7.0).all())


@pytest.mark.gpu
def test_step_without_a_slot():
    import torch
    r = Run("f32", 2, 1, 64, "additive", [1, 1, 1], seed=12)
    slots = r.slots.copy()
    slots[1] = r.num_slots
    r.att.step(torch.from_numpy(slots).cuda(), r.q, r.k, r.v, None, r.gate, r.state, r.o)
    torch.cuda.synchronize()
    assert bool(r.o[1].isnan().all()) and bool(r.o[::2].isfinite().all())


@pytest.mark.gpu
def test_state_slots_past_32_bits_of_bytes():
    """A pool of more than 2^32 bytes and more than 2^31 elements of v's offsets is
    addressed in 64 bits: the last slot of 40000 slots of two heads of 128."""
    import torch
    att = LN.LinearAttention(2, 128, rule="delta", dtype=torch.bfloat16)
    n = 40000
    state = att.states(n)
    a = inputs(13, 80, 2, 2, 128)
    d = {x: torch.from_numpy(a[x]).cuda() for x in a}
    q, k, v = (d[x].bfloat16() for x in "qkv")
    o = torch.empty_like(v)
    slots = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    att.prefill(torch.tensor([0, 79], dtype=torch.int32, device="cuda"), q, k, v, d["beta"], d["gate"], slots, state, o)
    att.step(slots, q[79:], k[79:], v[79:], d["beta"][79:].clone(), d["gate"][79:].clone(), state, o[79:])
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    ro, rm = recurrence(f(q), f(k), f(v), f(d["beta"]), f(d["gate"]), np.zeros((2, 128, 128)))
    assert far(f(state[n - 1]), rm) <= STATE_TOL["bf16"] and far(f(o), ro) <= OUT_TOL["bf16"]
    assert float(state[:n - 1].abs().max()) == 0.0


@pytest.mark.gpu
def test_another_stream_and_graph_replays():
    """A prefill and a step recorded into a graph on a stream of their own: every
    replay gives what the eager calls give, bit for bit."""
    import torch
    r = Run("bf16", 4, 2, 128, "delta", [100, 30], seed=14)
    ws = r.att.workspace(2, 130)
    cu, slots = torch.from_numpy(r.cu).cuda(), torch.from_numpy(r.slots).cuda()
    token = [x[:2].clone() for x in (r.q, r.k, r.v, r.beta, r.gate)]
    o1 = torch.empty_like(token[2])

    def both():
        r.att.prefill(cu, r.q, r.k, r.v, r.beta, r.gate, slots, r.state, r.o, workspace=ws)
        r.att.step(slots, *token, r.state, o1)

    both()
    torch.cuda.synchronize()
    want = [x.clone() for x in (r.o, o1, r.state)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both()
    for _ in range(3):
        r.o.fill_(7.0), o1.fill_(7.0), r.state.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        used = slots.long()
        assert torch.equal(r.o, want[0]) and torch.equal(o1, want[1]) and torch.equal(r.state[used], want[2][used])


@pytest.mark.gpu
def test_prefilled_states_go_into_the_packed_pool():
    """Prompt, pack, decode: with every row 32 bits wide the pool is the prefill's
    own output, and stepq_decode_step continues the same recurrence."""
    import torch
    H, D, n = 3, 64, 50
    r = Run("f32", H, H, D, "delta", [n, n - 9], seed=15, spare=0)
    r.slots = np.arange(2, dtype=np.int32)
    r.prefill()
    L = S.Layout(H, D, 0, np.full(H, 32, np.uint8), np.ones(H * D, np.float32), S.ROW_SCALES_REFIT)
    pool, scales = L.alloc(2)
    slots = torch.arange(2, dtype=torch.int32, device="cuda")
    S.stepq_pack(L.handle, 2, slots, 2, r.state, pool, scales)
    torch.cuda.synchronize()
    assert torch.equal(pool.view(torch.float32).view(2, H, D, D), r.state)
    a = inputs(16, 2, H, H, D)
    d = {x: torch.from_numpy(a[x]).cuda() for x in a}
    o = torch.empty(2, H, D, device="cuda")
    S.stepq_decode_step(L.handle, 2, slots, 2, d["q"], d["k"], d["v"], d["beta"], d["gate"], pool, scales, o)
    o2 = torch.empty_like(o)
    r.att.step(slots, d["q"], d["k"], d["v"], d["beta"], d["gate"], r.state, o2)
    torch.cuda.synchronize()
    assert far(pool.view(torch.float32).view(2, H, D, D).cpu().numpy(), r.state.double().cpu().numpy()) <= 1e-6
    assert far(o.cpu().numpy(), o2.double().cpu().numpy()) <= 1e-6


@pytest.mark.gpu
def test_binding_refuses_what_the_kernels_could_not_hold():
    import torch
    r = Run("f32", 4, 2, 32, "delta", [5, 6], seed=17)
    cu, slots = torch.from_numpy(r.cu).cuda(), torch.from_numpy(r.slots).cuda()
    good = dict(cu_seqlens=cu, q=r.q, k=r.k, v=r.v, beta=r.beta, gate=r.gate, slot_ids=slots, state=r.state, o=r.o)
    bad = [dict(cu_seqlens=cu[:2]), dict(cu_seqlens=cu.long()), dict(q=r.q[:-1]), dict(q=r.q.half()), dict(k=r.k.cpu()),
           dict(v=r.v[:, :2]), dict(v=r.v.transpose(1, 2)), dict(beta=None), dict(beta=r.beta[:-1]),
           dict(gate=r.gate.double()), dict(state=r.state.transpose(2, 3)), dict(o=r.o[:, :, :16]),
           dict(o=r.o.expand(11, 4, 32)[:1].expand(11, 4, 32)), dict(slot_ids=slots.long()),
           dict(resume=torch.ones(3, dtype=torch.uint8, device="cuda")), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    for change in bad:
        with pytest.raises(S.StepqError) as e:
            r.att.prefill(**{**good, **change})
        assert e.value.status == S.STEPQ_ERR_INVALID_ARG, change
    with pytest.raises(S.StepqError, match="workspace of its own"):
        r.att.prefill(**good, stream=torch.cuda.Stream())
    r.att.prefill(**good)
    torch.cuda.synchronize()

"""Beam selection and state reordering against plain implementations, their
refusals and their ABI.

Scores: cum + ((x - max) - log sum).  Each of the three operations rounds a value
of at most 64 in size to binary32, 2^-19 at worst each, and the sum of
exponentials is good to 2e-6 of itself: 1e-5 in all.  Tokens and parents have to
be equal; the inputs are drawn so that no two candidates of different beams that
matter lie within 2.5 times that of each other unless they tie exactly.
"""
import re
from pathlib import Path

import numpy as np
import pytest

from quantized_recurrent_state_packed_amd import beam as B
from quantized_recurrent_state_packed_amd import build_lib
from quantized_recurrent_state_packed_amd import stepq as S

HEADER = Path(__file__).resolve().parents[1] / "include" / "stepq_seq.h"
SCORE_TOL = 1e-5
GOOD = 4096          # an address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not S.LIB_PATH.exists():
        build_lib.build()
    return B.lib()


# ------------------------------------------------------------ plain versions

def select(x, scores, finished, eos, n):
    """x [B, K, V] float64 -> tokens, parents [B, n] int, scores [B, n] float64, smallest gap between
    neighbouring candidates of different beams among the first n + 1 (exact ties do not count)."""
    tokens, parents = np.full((x.shape[0], n), -1), np.full((x.shape[0], n), -1)
    out, gap = np.full((x.shape[0], n), -np.inf), np.inf
    x = np.where(np.isnan(x), -np.inf, x)
    for b in range(x.shape[0]):
        cands = []
        for k in range(x.shape[1]):
            s = float(scores[b, k])
            if np.isnan(s) or s == -np.inf:
                continue
            if finished is not None and finished[b, k]:
                cands.append((-s, k, 0, eos))
                continue
            row, m = x[b, k], x[b, k].max()
            if m == -np.inf:
                continue
            with np.errstate(invalid="ignore"):
                e = np.where(row == m, 1.0, np.exp(np.minimum(row - m, 0.0)))
            lse = np.log(e[row > -np.inf].sum())
            order = np.argsort(-row, kind="stable")[:n]
            for r, t in enumerate(order):
                if row[t] > -np.inf and not (m == np.inf and row[t] < m):
                    cands.append((-(s + ((row[t] - m if row[t] < m else 0.0) - lse)), k, r, int(t)))
        cands.sort()
        for i, (s, k, _, t) in enumerate(cands[:n]):
            tokens[b, i], parents[b, i], out[b, i] = t, k, -s
        for p, q in zip(cands[:n], cands[1:n + 1]):
            if p[1] != q[1] and q[0] != p[0]:
                gap = min(gap, q[0] - p[0])
    return tokens, parents, out, gap


def reorder(slots, parents):
    """[B, K] each -> new slots [B, K], copies [(from, to)]."""
    new, copies = np.empty_like(slots), []
    for b in range(slots.shape[0]):
        K = slots.shape[1]
        dead = [i for i in range(K) if i not in set(parents[b].tolist())]
        seen = set()
        for j in range(K):
            p = int(parents[b, j])
            if 0 <= p < K and p not in seen:
                seen.add(p)
                new[b, j] = slots[b, p]
            else:
                new[b, j] = slots[b, dead.pop(0)]
                if 0 <= p < K:
                    copies.append((int(slots[b, p]), int(new[b, j])))
    return new, copies


# ------------------------------------------------------------------ ABI, CPU

def test_header_and_library_agree_on_the_beam_entry_points(lib):
    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    names = set(re.findall(r"\b(stepq_beam_[a-z_]+)\s*\(", text))
    assert names == set(B.EXPORTED)
    for n in names:
        assert hasattr(lib, n)
    assert int(re.search(r"STEPQ_MAX_REGIONS (\d+)", text).group(1)) == B.MAX_REGIONS


def select_status(lib, batch=2, beams=4, vocab=100, n=4, logits=GOOD, dtype=0, stride=100, scores=GOOD, finished=None,
                  tokens=GOOD, parents=GOOD, out=GOOD, ws=GOOD, nbytes=0):
    return lib.stepq_beam_select(batch, beams, vocab, n, logits, dtype, stride, scores, finished, 0, tokens, parents, out,
                                 ws, nbytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(batch=-1), 1), (dict(beams=0), 1), (dict(vocab=0), 1), (dict(n=0), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1),
    (dict(logits=None), 1), (dict(scores=None), 1), (dict(tokens=None), 1), (dict(parents=None), 1), (dict(out=None), 1),
    (dict(ws=None), 1), (dict(logits=GOOD + 2), 1), (dict(tokens=GOOD + 2), 1), (dict(stride=99), 1),
    (dict(dtype=1, logits=GOOD + 1), 1), (dict(nbytes=0), 1), (dict(nbytes=2 * 4 * 40 - 1), 1),
    (dict(beams=65), 2), (dict(n=65), 2), (dict(vocab=2 ** 31 - 1), 2), (dict(batch=2 ** 22, beams=8), 2),
    (dict(batch=2 ** 23 + 1, beams=1), 2),
])
def test_selection_arguments_that_are_refused(lib, bad, status):
    assert select_status(lib, **bad) == status


def reorder_status(lib, batch=2, beams=4, slots=GOOD, parents=GOOD, num_slots=8, regions=((GOOD, 64),), new=2 * GOOD,
                   count=None):
    r = None if regions is None else (B.stepq_region * max(1, len(regions)))(*regions)
    return lib.stepq_beam_reorder(batch, beams, slots, parents, num_slots, r,
                                  (0 if regions is None else len(regions)) if count is None else count, new, None)


@pytest.mark.parametrize("bad,status", [
    (dict(batch=-1), 1), (dict(beams=0), 1), (dict(num_slots=0), 1), (dict(count=-1), 1), (dict(slots=None), 1),
    (dict(parents=None), 1), (dict(new=None), 1), (dict(new=GOOD), 1), (dict(slots=GOOD + 2), 1),
    (dict(regions=None, count=1), 1), (dict(regions=((None, 64),)), 1), (dict(regions=((GOOD + 8, 64),)), 1),
    (dict(regions=((GOOD, 0),)), 1), (dict(regions=((GOOD, 72),)), 1), (dict(regions=((GOOD, 64), (GOOD, 8))), 1),
    (dict(beams=65), 2), (dict(count=129), 2), (dict(batch=2 ** 22, beams=8), 2), (dict(regions=((GOOD, 2 ** 32),)), 2),
])
def test_reordering_arguments_that_are_refused(lib, bad, status):
    assert reorder_status(lib, **bad) == status


def test_empty_batches_and_workspace_sizes(lib):
    assert select_status(lib, batch=0, logits=None, ws=None) == S.STEPQ_OK
    assert reorder_status(lib, batch=0, slots=None) == S.STEPQ_OK
    size = lib.stepq_beam_workspace_bytes
    assert size(0, 4, 100, 4) == 0 and size(1, 65, 100, 4) == 0 and size(1, 4, 0, 4) == 0
    assert size(1, 4, 100, 4) == 4 * 40 and size(1, 4, 1025, 4) == 2 * 4 * 40
    assert size(64, 64, 200000, 64) == 64 * 64 * 4 * 130


def test_binding_refuses_bad_tensors_before_the_library(lib):
    import torch
    for args in ((1, 65, 10), (0, 4, 10), (1, 4, 0)):
        with pytest.raises(S.StepqError):
            B.BeamSelect(*args, device="cpu")
    with pytest.raises(S.StepqError, match="not float32"):
        B.BeamSelect(1, 4, 10, dtype=torch.int32, device="cpu")
    sel = B.BeamSelect(1, 2, 10, device="cpu")
    with pytest.raises(S.StepqError, match="logits must be"):
        sel(torch.zeros(2, 10).half(), torch.zeros(2))
    with pytest.raises(S.StepqError, match="device tensor"):
        sel(torch.zeros(2, 10), torch.zeros(2))
    ids = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(S.StepqError, match="device tensor"):
        B.reorder(2, ids, ids, [torch.zeros(4, 16)], ids.clone())
    with pytest.raises(S.StepqError, match="num_slots"):
        B.reorder(2, ids, ids, [], ids.clone())
    with pytest.raises(S.StepqError) as e:
        B.reorder(2, ids, ids, [torch.zeros(4, 16)] * 129, ids.clone())
    assert e.value.status == S.STEPQ_ERR_UNSUPPORTED


# ---------------------------------------------------------------------- GPU

def run_select(x, scores, finished, n, dtype="f32", eos=7, pad=0, shift=0, stream=None):
    """x [B, K, V]; rows lie `pad` elements apart, the first one `shift` elements
    into the buffer, and the gaps are filled with +inf."""
    import torch
    td = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    b, k, v = x.shape
    flat = torch.full((shift + b * k * (v + pad),), float("inf"), dtype=td, device="cuda")
    wide = flat[shift:].view(b * k, v + pad)
    wide[:, :v] = torch.from_numpy(x.reshape(b * k, v).astype(np.float32)).cuda().to(td)
    sel = B.BeamSelect(b, k, v, n, td, eos_token=eos)
    sel.workspace.fill_(0xFF)
    f = None if finished is None else torch.from_numpy(finished.reshape(-1).astype(np.uint8)).cuda()
    out = sel(wide[:, :v], torch.from_numpy(scores.reshape(-1).astype(np.float32)).cuda(), f, stream=stream)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in out], wide[:, :v].double().cpu().numpy().reshape(x.shape)


def check_select(x, scores, finished, n, exact_ties=False, **kw):
    scores = scores.astype(np.float32)
    (tokens, parents, out), seen = run_select(x, scores, finished, n, **kw)
    t, p, s, gap = select(seen, scores, finished, kw.get("eos", 7), n)
    assert exact_ties or gap > 2.5 * SCORE_TOL, "the inputs put two candidates too close together"
    assert np.array_equal(parents, p) and np.array_equal(tokens, t)
    some = np.isfinite(s)
    assert np.array_equal(out[~some], s[~some].astype(np.float32))
    if some.any():
        assert np.abs(out[some] - s[some]).max() <= SCORE_TOL


def logits(seed, b, k, v):
    g = np.random.default_rng(seed)
    return 3.0 * g.standard_normal((b, k, v)), -10.0 * g.random((b, k)), g.random((b, k))


@pytest.mark.gpu
@pytest.mark.parametrize("b,k,v,n", [
    (1, 1, 1, 1), (1, 1, 1, 4), (1, 2, 3, 8), (2, 4, 63, 4), (1, 3, 64, 64), (3, 2, 65, 5), (1, 4, 1023, 8),
    (2, 2, 1024, 16), (1, 5, 1025, 10), (1, 8, 4097, 16), (1, 64, 600, 40), (1, 4, 50001, 8), (1, 1, 200003, 64),
    (33, 8, 3001, 16),
])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_selection_sizes(dtype, b, k, v, n):
    x, s, f = logits(b * 1000 + k * 100 + v, b, k, v)
    check_select(x, s, None, n, dtype=dtype, pad=v % 3, shift=n % 9)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_finished_beams_have_one_continuation(dtype):
    x, s, f = logits(1, 6, 4, 5000)
    done = f < 0.5
    done[0], done[1] = True, False           # all, none
    check_select(x, s, done, 8, dtype=dtype)


@pytest.mark.gpu
def test_ties_go_to_the_lower_beam_and_token():
    """Rows of equal logits, rows that are copies of each other at equal scores,
    and rows at the type's lowest value, whose probabilities are equal."""
    x = np.zeros((4, 3, 3000))
    x[1] = np.random.default_rng(2).integers(0, 3, (1, 3000))       # many equal logits, three equal rows
    x[2] = -3.0e38
    x[3, 1] = -3.4028234663852886e38
    s = np.full((4, 3), -2.0)
    check_select(x, s, None, 64, exact_ties=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_banned_tokens(dtype):
    """-inf and NaN ban tokens; rows with nothing left, and scores of -inf and NaN, have no continuation."""
    x, s, _ = logits(3, 8, 3, 2100)
    inf, nan = np.inf, np.nan
    x[0, :, :2000] = -inf
    x[1] = -inf                                # nothing left in the request
    x[2, 1] = nan
    x[3, :, 3:] = nan                          # three tokens a beam: fewer than asked for
    x[4, 0, ::2] = nan
    x[5, 2, [17, 1500]] = inf                  # shares all of the probability
    s[6, 0], s[6, 2] = -inf, nan
    s[7] = -inf
    x[2, 0, 0] = -inf
    check_select(x, s, None, 16, dtype=dtype)


@pytest.mark.gpu
def test_large_logits_and_a_row_of_the_lowest_values_with_one_way_out():
    x = np.full((1, 2, 1500), -3.4028234663852886e38)
    x[0, 0, 1400] = 5.0
    x[0, 1] = np.linspace(1e30, 3e38, 1500)
    check_select(x, np.array([[-1.0, -2.0]]), None, 2)


@pytest.mark.gpu
def test_selection_on_another_stream_and_in_a_graph():
    import torch
    x, s, f = logits(4, 3, 4, 9000)
    td = torch.from_numpy(x.reshape(12, -1).astype(np.float32)).cuda()
    sc = torch.from_numpy(s.reshape(-1).astype(np.float32)).cuda()
    sel = B.BeamSelect(3, 4, 9000, 8)
    want = [t.clone() for t in sel(td, sc)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        sel(td, sc)
    for _ in range(3):
        for t in (sel.tokens, sel.parents, sel.scores):
            t.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip((sel.tokens, sel.parents, sel.scores), want))


PARENTS = {
    "alone": [[0, 1, 2, 3]], "swapped": [[3, 2, 1, 0]], "fork": [[0, 0, 0, 0]], "fork-last": [[3, 3, 3, 3]],
    "mixed": [[1, 1, 3, 0], [2, 0, 2, 0], [3, 3, 1, 1]], "none": [[-1, -1, -1, -1]], "some": [[2, -1, 2, 2], [-1, 1, -1, 1]],
    "outside": [[9, 0, -7, 2 ** 31 - 1]],
}


def check_reorder(parents, num_slots, sizes, seed=0, slots=None):
    import torch
    g = np.random.default_rng(seed)
    b, k = parents.shape
    if slots is None:
        slots = g.permutation(num_slots)[:b * k].astype(np.int32).reshape(b, k)
    bufs = [torch.from_numpy(g.integers(0, 256, (num_slots, n), dtype=np.uint8)).cuda() for n in sizes]
    want = [t.cpu().numpy() for t in bufs]
    new = torch.full((b * k,), -5, dtype=torch.int32, device="cuda")
    B.reorder(k, torch.from_numpy(slots.reshape(-1)).cuda(), torch.from_numpy(parents.reshape(-1).astype(np.int32)).cuda(),
              bufs, new, num_slots=num_slots)
    torch.cuda.synchronize()
    ref, copies = reorder(slots, parents)
    assert np.array_equal(new.cpu().numpy().reshape(b, k), ref)
    for t, w in zip(bufs, want):
        before = w.copy()
        for s, d in copies:
            if 0 <= s < num_slots and 0 <= d < num_slots:
                w[d] = before[s]
        assert np.array_equal(t.cpu().numpy(), w)


@pytest.mark.gpu
@pytest.mark.parametrize("case", PARENTS)
def test_reordering(case):
    p = np.array(PARENTS[case], dtype=np.int64).astype(np.int32)
    check_reorder(p, p.size + 3, [16, 4096, 32768, 32784, 100000])


@pytest.mark.gpu
@pytest.mark.parametrize("b,k", [(1, 1), (7, 2), (3, 63), (2, 64), (40, 8)])
def test_reordering_random(b, k):
    g = np.random.default_rng(b + k)
    check_reorder(g.integers(-1, k, (b, k)).astype(np.int32), b * k + 1, [1024, 48, 70000], seed=b)


@pytest.mark.gpu
def test_reordering_without_buffers_with_many_and_with_ids_outside():
    g = np.random.default_rng(5)
    check_reorder(g.integers(0, 4, (3, 4)).astype(np.int32), 12, [])
    check_reorder(g.integers(0, 4, (3, 4)).astype(np.int32), 12, [16 + 16 * (i % 5) for i in range(B.MAX_REGIONS)])
    slots = np.array([[0, -1, 2, 40], [4, 5, 6, 7]], dtype=np.int32)
    for p in ([[0, 0, 2, 2], [1, 1, 1, 3]], [[1, 1, 3, 3], [0, 0, 0, 0]]):
        check_reorder(np.array(p, dtype=np.int32), 8, [64, 40000], slots=slots)


@pytest.mark.gpu
def test_reordering_of_packed_states_past_32_bits_of_bytes():
    """Slots of a packed pool of 4.9 GB, of 48 heads in 6 bits: a beam's state is found
    in the slot that its id names afterwards."""
    import torch
    L = S.Layout(48, 128, 0, np.full(48, 6, np.uint8), np.ones(48 * 128, np.float32), S.ROW_SCALES_REFIT)
    n = 8000
    assert n * L.slot_bytes > 2 ** 32
    pool, scales = L.alloc(n)
    slots = torch.tensor([n - 1, 3, n - 5, 100], dtype=torch.int32, device="cuda")
    state = torch.randn(4, 48, 128, 128, device="cuda")
    S.stepq_pack(L.handle, 4, slots, n, state, pool, scales)
    before = torch.empty_like(state)
    S.stepq_unpack(L.handle, 4, slots, n, pool, scales, before)
    parents = torch.tensor([2, 0, 2, 0], dtype=torch.int32, device="cuda")
    new = torch.empty_like(slots)
    B.reorder(4, slots, parents, [pool, scales], new, num_slots=n)
    after = torch.empty_like(state)
    S.stepq_unpack(L.handle, 4, new, n, pool, scales, after)
    torch.cuda.synchronize()
    assert torch.equal(after, before[parents.long()])
    assert new.tolist() == [n - 5, n - 1, 3, 100]


@pytest.mark.gpu
def test_reordering_in_a_graph():
    import torch
    pool = torch.randint(0, 256, (9, 50000), dtype=torch.uint8, device="cuda")[:, :49984].contiguous()
    start = pool.clone()
    slots = torch.tensor([8, 1, 4, 2], dtype=torch.int32, device="cuda")
    parents = torch.tensor([1, 1, 3, 1], dtype=torch.int32, device="cuda")
    new = torch.empty_like(slots)
    B.reorder(4, slots, parents, [pool], new)
    torch.cuda.synchronize()
    want, ids = pool.clone(), new.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        B.reorder(4, slots, parents, [pool], new)
    for _ in range(3):
        pool.copy_(start)
        new.fill_(-1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool, want) and torch.equal(new, ids)

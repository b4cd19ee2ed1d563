"""Verification of drafted tokens against a plain one in 64 bits, and what it refuses.

Everything that is written is a whole number and has to be equal.  The inputs are drawn so that
no random number lies within GAP of a border between two outcomes (the library's sums are good to
some 1e-13 of themselves; 64 bits give 1e-14 here)."""
import re
from pathlib import Path

import numpy as np
import pytest

from quantized_recurrent_state_packed_amd import build_lib
from quantized_recurrent_state_packed_amd import draft as DR
from quantized_recurrent_state_packed_amd import stepq as S

HEADER = Path(__file__).resolve().parents[1] / "include" / "stepq_block.h"
GOOD = 4096          # an address that is never dereferenced
GAP = 1e-11


@pytest.fixture(scope="module")
def lib():
    if not S.LIB_PATH.exists():
        build_lib.build()
    return DR.lib()


# ------------------------------------------------------------ plain version

def softmax(x, t):
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    m = x.max()
    if m == -np.inf:
        return np.zeros_like(x)
    if not t > 0:
        p = np.zeros_like(x)
        p[np.argmax(x)] = 1.0
        return p
    if m == np.inf:
        e = (x == np.inf).astype(np.float64)
    else:
        with np.errstate(invalid="ignore", divide="ignore"):
            e = np.exp((x - m) / np.float64(t))
        e[x == -np.inf] = 0.0
        e[x == m] = 1.0
    return e / e.sum()


def verify(x, z, d, u, count, temp):
    """x [B, K + 1, V], z [B, K, V] or None, d [B, K], u [B, K + 1]: accepted, tokens, and the smallest distance
    of a random number from a border."""
    B, K = d.shape
    acc, tokens, gap = np.zeros(B, int), np.full((B, K + 1), -1), np.inf
    for b in range(B):
        t = np.float32(1.0) if temp is None else temp[b]
        n, c = 0, K if count is None else int(np.clip(count[b], 0, K))
        p = q = None
        rejected = False
        while n < c and 0 <= d[b, n] < x.shape[-1]:
            p = softmax(x[b, n], t)
            if z is None or not t > 0:
                q = np.zeros_like(p)
                q[d[b, n]] = 1.0
            else:
                q = softmax(z[b, n], t)
            pd, qd = p[d[b, n]], q[d[b, n]]
            if t > 0 and qd > 0 and pd > 0:
                gap = min(gap, abs(float(u[b, n]) * qd / pd - 1.0))
            if not float(u[b, n]) * qd < pd:
                rejected = True
                break
            tokens[b, n] = d[b, n]
            n += 1
        acc[b] = n
        p = softmax(x[b, n], t)
        w = np.maximum(p - q, 0.0) if rejected else p
        if not w.sum() > 0:
            w = p
        if w.sum() > 0:
            run, goal = np.cumsum(w), float(u[b, K]) * w.sum()
            if np.count_nonzero(w) > 1:
                gap = min(gap, np.abs(run[w > 0][:-1] - goal).min() / w.sum())
            beyond = np.flatnonzero((run > goal) & (w > 0))
            tokens[b, n] = beyond[0] if len(beyond) else np.flatnonzero(w)[-1]
    return acc, tokens, gap


def test_the_plain_version_draws_from_the_target():
    """Whatever the draft, the first token is distributed as the target's."""
    g = np.random.default_rng(0)
    x, z = g.standard_normal((2, 6)), g.standard_normal((1, 6))
    p, q = softmax(x[0], 1.0), softmax(z[0], 1.0)
    N = 20000
    d = g.choice(6, size=(N, 1), p=q)
    _, tokens, _ = verify(np.broadcast_to(x, (N, 2, 6)), np.broadcast_to(z, (N, 1, 6)), d, g.random((N, 2)), None, None)
    got = np.bincount(tokens[:, 0], minlength=6) / N
    assert np.all(np.abs(got - p) <= 5.0 * np.sqrt(p * (1 - p) / N))


# ------------------------------------------------------------------ ABI, CPU

def test_header_and_library_agree_on_the_verify_entry_points(lib):
    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    names = set(re.findall(r"\b(stepq_verify_[a-z_]+)\s*\(", text))
    assert names == set(DR.EXPORTED)
    for n in names:
        assert hasattr(lib, n)


def status(lib, batch=2, drafts=3, vocab=100, logits=GOOD, dtype=1, stride=100, z=GOOD, zs=100, d=GOOD, count=None, temp=None,
           u=GOOD, accepted=GOOD, tokens=GOOD, ws=GOOD, nbytes=1 << 30):
    return lib.stepq_verify_drafts(batch, drafts, vocab, logits, dtype, stride, z, zs, d, count, temp, u, accepted, tokens, ws,
                                   nbytes, None)


@pytest.mark.parametrize("bad,want", [
    (dict(batch=-1), 1), (dict(drafts=-1), 1), (dict(vocab=0), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(logits=None), 1),
    (dict(logits=GOOD + 1), 1), (dict(stride=99), 1), (dict(stride=2 ** 39), 1), (dict(zs=99), 1), (dict(zs=2 ** 39), 1),
    (dict(z=GOOD + 1), 1), (dict(d=None), 1), (dict(d=GOOD + 2), 1), (dict(count=GOOD + 1), 1), (dict(temp=GOOD + 2), 1),
    (dict(u=None), 1), (dict(u=GOOD + 1), 1), (dict(accepted=None), 1), (dict(tokens=None), 1), (dict(tokens=GOOD + 2), 1),
    (dict(ws=None), 1), (dict(ws=GOOD + 8), 1), (dict(nbytes=0), 1), (dict(nbytes=14 * 16 + 2 * 48 + 2 * 16 - 1), 1),
    (dict(drafts=64), 2), (dict(vocab=2 ** 31 - 1024), 2), (dict(batch=2 ** 20), 2),
])
def test_arguments_that_are_refused(lib, bad, want):
    assert status(lib, **bad) == want


def test_empty_batches_and_workspace_sizes(lib):
    assert status(lib, batch=0, logits=None, ws=None) == S.STEPQ_OK
    size = lib.stepq_verify_workspace_bytes
    assert size(0, 4, 100) == 0 and size(1, 64, 100) == 0 and size(1, 4, 0) == 0 and size(2 ** 22, 4, 100) == 0
    assert size(2, 3, 100) == 14 * 16 + 2 * 48 + 2 * 16
    assert size(1, 0, 1025) == 2 * 16 + 48 + 2 * 16


def test_binding_refuses_bad_tensors_before_the_library(lib):
    import torch
    for args in ((1, 64, 10), (0, 4, 10), (1, 4, 0), (1, -1, 10), (2 ** 22, 4, 10)):
        with pytest.raises(S.StepqError):
            DR.DraftVerify(*args, device="cpu")
    with pytest.raises(S.StepqError, match="not float32"):
        DR.DraftVerify(1, 2, 10, torch.int32, device="cpu")
    op = DR.DraftVerify(1, 2, 10, device="cpu")
    x, d, u, z = torch.zeros(3, 10), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 3), torch.zeros(2, 10)
    for bad in (x.half(), None, 3, np.zeros((3, 10), np.float32), torch.tensor(1.0)):
        for args, kw in (((bad, d, u), {}), ((x, bad, u), {}), ((x, d, bad), {}), ((x, d, u), dict(draft_logits=bad)),
                         ((x, d, u), dict(num_drafts=bad)), ((x, d, u), dict(temperature=bad))):
            with pytest.raises(S.StepqError) as e:
                op(*args, **kw)
            assert e.value.status == S.STEPQ_ERR_INVALID_ARG


# ---------------------------------------------------------------------- GPU

TYPES = {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}


def logits(g, *shape):
    """A broad bulk and a few likely tokens, one banned."""
    x = 2.0 * g.standard_normal(shape)
    likely = g.integers(0, shape[-1], size=shape[:-1] + (min(8, shape[-1]),))
    np.put_along_axis(x, likely, 7.0 + 2.0 * g.standard_normal(likely.shape), -1)
    x[..., shape[-1] // 2] = -np.inf
    return x


def placed(x, td, pad, shift):
    """Rows [N, V] `pad` elements apart, the first one `shift` elements into a buffer of +inf."""
    import torch
    n, v = x.shape
    flat = torch.full((shift + n * (v + pad),), float("inf"), dtype=td, device="cuda")
    wide = flat[shift:].view(n, v + pad)[:, :v]
    wide.copy_(torch.from_numpy(x.astype(np.float32)).cuda().to(td))
    return wide


def run(x, z, d, u, count=None, temp=None, dtype="f32", pad=0, shift=0, stream=None):
    import torch
    td = getattr(torch, TYPES[dtype])
    B, K1, V = x.shape
    K = K1 - 1
    op = DR.DraftVerify(B, K, V, td)
    op.workspace.fill_(0xFF), op.accepted.fill_(-7), op.tokens.fill_(-7)
    xd = placed(x.reshape(B * K1, V), td, pad, shift)
    zd = None if z is None else placed(z.reshape(B * K, V), td, 2 * pad, shift // 2)

    def up(v, t):
        return None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda().to(t)

    args = (xd, up(d, torch.int32), up(u, torch.float32))
    more = dict(draft_logits=zd, num_drafts=up(count, torch.int32), temperature=up(temp, torch.float32))
    torch.cuda.synchronize()
    acc, tokens = op(*args, **more, stream=stream)
    torch.cuda.synchronize()
    back = [None if t is None else t.double().cpu().numpy() for t in (xd, zd)]
    return acc.cpu().numpy(), tokens.cpu().numpy(), back, (op, args, more)


def check(x, z, d, u, count=None, temp=None, need_gap=True, **kw):
    u = u.astype(np.float32)
    temp = None if temp is None else temp.astype(np.float32)
    acc, tokens, (xs, zs), keep = run(x, z, d, u, count, temp, **kw)
    want_acc, want_tokens, gap = verify(xs.reshape(x.shape), None if z is None else zs.reshape(z.shape), d, u, count, temp)
    assert not need_gap or gap > GAP, "the inputs put a random number too close to a border"
    assert np.array_equal(acc, want_acc) and np.array_equal(tokens, want_tokens)
    return acc, tokens, keep


def inputs(seed, B, K, V, ragged=True, temps=True):
    g = np.random.default_rng(seed)
    x = logits(g, B, K + 1, V)
    z = x[:, :K] + 0.7 * g.standard_normal((B, K, V))
    temp = (0.5 + g.random(B)).astype(np.float32)
    if temps and B > 2:
        temp[g.random(B) < 0.25] = 0.0
    d = np.empty((B, K), int)
    for b in range(B):
        for k in range(K):
            q = softmax(z[b, k], temp[b])
            d[b, k] = g.choice(V, p=q)
    count = g.integers(0, K + 1, size=B) if ragged else None
    return x, z, d, g.random((B, K + 1)).astype(np.float32), count, temp


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,K,V", [(1, 1, 2), (1, 4, 1023), (7, 3, 1025), (40, 5, 333), (3, 2, 20000), (2, 63, 70), (9, 1, 4097)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
def test_drafts_and_next_tokens(B, K, V, dtype, pad, shift):
    x, z, d, u, count, temp = inputs(B + V, B, K, V)
    check(x, z, d, u, count, temp, dtype=dtype, pad=pad, shift=shift)
    check(x, None, d, u, count, temp, dtype=dtype, pad=pad, shift=shift)
    check(x, z, d, u, dtype=dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 2, 63, 1024, 5000])
def test_drawing_without_drafts(V):
    g = np.random.default_rng(V)
    x = 2.0 * g.standard_normal((50, 1, V))
    temp = (0.3 + g.random(50)).astype(np.float32)
    temp[::7] = 0.0
    check(x, None, np.empty((50, 0), int), g.random((50, 1)), None, temp)


@pytest.mark.gpu
def test_flat_and_sharp_distributions_over_a_large_vocabulary():
    """A flat row has a border every 1 / 131072: sums in 32 bits would choose its neighbours."""
    g = np.random.default_rng(1)
    x = np.zeros((6, 3, 131072))
    x[2:4] = g.standard_normal((2, 3, 131072)) * 0.01
    x[4:, :, 100000] = 60.0
    d = g.integers(0, 131072, size=(6, 2))
    d[4:] = 100000
    check(x, x[:, :2] + 0.1 * g.standard_normal((6, 2, 131072)), d, g.random((6, 3)))
    check(x, None, d, g.random((6, 3)))


@pytest.mark.gpu
def test_a_draft_that_equals_the_target_is_kept():
    """p = q to the last bit: u q < p for every u below 1, and nothing is left of p - q."""
    x, _, d, u, _, temp = inputs(3, 20, 4, 700, ragged=False, temps=False)
    u[:] = np.float32(1.0 - 2.0 ** -24)
    acc, tokens, _ = check(x, x[:, :4].copy(), d, u, None, temp, need_gap=False)
    assert np.all(acc == 4) and np.all(tokens[:, :4] == d)


@pytest.mark.gpu
def test_random_numbers_at_their_ends():
    x, z, d, u, _, temp = inputs(4, 12, 3, 900, ragged=False, temps=False)
    for v in (0.0, 1.0 - 2.0 ** -24):
        w = np.full_like(u, v)
        check(x, z, d, w, None, temp, need_gap=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
def test_banned_tokens_and_infinities(dtype):
    g = np.random.default_rng(8)
    B, K, V = 12, 2, 3000
    x, z = logits(g, B, K + 1, V), logits(g, B, K, V)
    d = g.integers(0, V, size=(B, K))
    temp = np.ones(B, np.float32)
    x[0] = -np.inf                               # nothing is allowed at any place
    x[1, 0], x[1, 0, 17], d[1, 0] = np.nan, 1.0, 17
    x[2, 0, [5, 2999]] = np.inf                  # two tokens share all of it
    d[2, 0] = 5
    z[3, 0] = -np.inf                            # the draft's row says nothing
    z[4, 0, 9], d[4, 0] = np.inf, 9
    x[5, 1] = -np.inf
    x[6, 0, :] = np.finfo(np.float16).min if dtype == "f16" else -3e38
    d[7, 0] = -1                                 # not a token
    d[8, 1] = V
    temp[9], temp[10], temp[11] = np.inf, 1e-30, -1.0
    x[5, 0, d[5, 0]] = z[5, 0, d[5, 0]] = 30.0
    u = g.random((B, K + 1))
    check(x, z, d, u, None, temp, dtype=dtype)
    check(x, None, d, u, None, temp, dtype=dtype)
    temp[:] = 0.0
    check(x, z, d, u, None, temp, dtype=dtype)


@pytest.mark.gpu
def test_greedy_takes_the_lowest_of_equals():
    x = np.zeros((4, 3, 2050))
    x[0, :, [7, 9, 2049]] = 5.0
    x[1, :, 2049] = 1.0
    x[2, :, 1024:] = 2.0
    d = np.array([[7, 9], [2049, 2049], [1024, 1025], [0, 1]])
    acc, tokens, _ = check(x, None, d, np.full((4, 3), 0.5), None, np.zeros(4))
    assert acc.tolist() == [1, 2, 1, 1] and tokens[0].tolist() == [7, 7, -1]


@pytest.mark.gpu
def test_tokens_are_distributed_as_the_targets():
    g = np.random.default_rng(0)
    x, z = g.standard_normal((2, 6)), g.standard_normal((1, 6))
    p, q = softmax(x[0], 1.0), softmax(z[0], 1.0)
    N = 40000
    d = g.choice(6, size=(N, 1), p=q)
    acc, tokens, _, _ = run(np.broadcast_to(x, (N, 2, 6)).copy(), np.broadcast_to(z, (N, 1, 6)).copy(), d, g.random((N, 2)))
    got = np.bincount(tokens[:, 0], minlength=6) / N
    assert np.all(np.abs(got - p) <= 5.0 * np.sqrt(p * (1 - p) / N))
    second = tokens[acc == 1, 1]
    p2 = softmax(x[1], 1.0)
    got = np.bincount(second, minlength=6) / len(second)
    assert np.all(np.abs(got - p2) <= 5.0 * np.sqrt(p2 * (1 - p2) / len(second)))


@pytest.mark.gpu
def test_counts_outside_of_their_range_are_clamped():
    x, z, d, u, _, temp = inputs(6, 5, 3, 400, temps=False)
    check(x, z, d, u, np.array([-5, 0, 3, 4, 1 << 30]), temp)


@pytest.mark.gpu
def test_other_streams_and_graphs():
    import torch
    x, z, d, u, count, temp = inputs(12, 30, 4, 5000)
    acc, tokens, (op, args, more) = check(x, z, d, u, count, temp, dtype="bf16")
    others = [DR.DraftVerify(30, 4, 5000, torch.bfloat16) for _ in range(2)]
    torch.cuda.synchronize()
    for o in others:
        o(*args, **more, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    for o in others:
        assert np.array_equal(o.accepted.cpu().numpy(), acc) and np.array_equal(o.tokens.cpu().numpy(), tokens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op(*args, **more)
    for _ in range(3):
        op.tokens.fill_(9), op.accepted.fill_(9), op.workspace.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(op.accepted.cpu().numpy(), acc) and np.array_equal(op.tokens.cpu().numpy(), tokens)


@pytest.mark.gpu
def test_rows_past_32_bits():
    import torch
    V, K = 5000, 2
    stride = (1 << 30) + 8
    flat = torch.zeros(2 * stride + V, dtype=torch.bfloat16, device="cuda")
    assert flat.numel() * 2 > 1 << 32
    x, z, d, u, _, temp = inputs(2, 1, K, V, ragged=False)
    acc, tokens, (op, args, more) = check(x, z, d, u, None, temp, dtype="bf16")
    far = flat.as_strided((K + 1, V), (stride, 1))
    far.copy_(args[0])
    op(far, *args[1:], **more)
    torch.cuda.synchronize()
    assert np.array_equal(op.accepted.cpu().numpy(), acc) and np.array_equal(op.tokens.cpu().numpy(), tokens)


@pytest.mark.gpu
def test_the_largest_vocabulary():
    """2^31 - 1 - 1024 logits, all banned but some at the ends, in the middle and beside a seam of tiles; and a draft."""
    import torch
    V = 2 ** 31 - 1 - 1024
    x = torch.full((2, V), -float("inf"), dtype=torch.bfloat16, device="cuda")
    at = [0, 1023, 1024, V // 2, V - 1025, V - 1]
    for t in at:
        x[:, t] = 1.0
    op = DR.DraftVerify(1, 1, V, torch.bfloat16)
    d = torch.tensor([[V - 1]], dtype=torch.int32, device="cuda")
    for n, t in enumerate(at):
        u = torch.tensor([[0.1, (n + 0.5) / len(at)]], device="cuda")
        acc, tokens = op(x, d, u)
        assert acc.tolist() == [1] and tokens.tolist() == [[V - 1, t]]
    acc, tokens = op(x, d, torch.tensor([[0.9, 0.99]], device="cuda"))       # rejected: the last of the others
    assert acc.tolist() == [0] and tokens.tolist() == [[V - 1025, -1]]
    acc, tokens = op(x, d, u, temperature=torch.zeros(1, device="cuda"))
    assert acc.tolist() == [0] and tokens.tolist() == [[0, -1]]


@pytest.mark.gpu
def test_drawing_takes_no_drafted_tokens():
    import torch
    op = DR.DraftVerify(3, 0, 5)
    x = torch.zeros(3, 5, device="cuda")
    _, tokens = op(x, None, torch.tensor([[0.1], [0.5], [0.99]], device="cuda"))
    assert tokens[:, 0].tolist() == [0, 2, 4]


@pytest.mark.gpu
def test_refusals_that_need_a_device(monkeypatch):
    import torch
    from quantized_recurrent_state_packed_amd import linear as LN
    op = DR.DraftVerify(2, 2, 10)
    x, z, d, u = (torch.zeros(*s, device="cuda") for s in ((6, 10), (4, 10), (2, 2), (2, 3)))
    d = d.int()
    op(x, d, u, draft_logits=z)

    def refused(f, match=None):
        with pytest.raises(S.StepqError, match=match) as e:
            f()
        assert e.value.status == S.STEPQ_ERR_INVALID_ARG

    refused(lambda: op(x.t(), d, u))
    refused(lambda: op(x[:5], d, u))
    refused(lambda: op(x[:1].expand(6, 10), d, u))
    refused(lambda: op(x, d.long(), u))
    refused(lambda: op(x, d, u[:, :2]))
    refused(lambda: op(x, d, u, draft_logits=z[:3]))
    refused(lambda: op(x, d, u, num_drafts=d[0].float()))
    refused(lambda: op(x, d, u, temperature=1.0))
    refused(lambda: op(x, None, u))
    torch.cuda.synchronize()
    monkeypatch.setattr(LN, "_current_device", lambda: 1)
    refused(lambda: op(x, d, u), "current")

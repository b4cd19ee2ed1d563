"""The norms around a block against the same in 64 bits (norm_ref.py), their gradients against
the formulas and those against differences, and what they refuse.

Tolerances are those of norm_ref.py's derivation plus half a step of the output's type,
torch.finfo(t).eps / 2 of the value, or, for a float16 value below 2^-14, half of the step
2^-24 that float16's values have there."""
import ctypes
import re
from pathlib import Path

import numpy as np
import pytest

import norm_ref as ref
from quantized_recurrent_state_packed_amd import build_lib
from quantized_recurrent_state_packed_amd import norm as NM
from quantized_recurrent_state_packed_amd import stepq as S

HEADER = Path(__file__).resolve().parents[1] / "include" / "stepq_block.h"
GOOD = 4096          # an address that is never dereferenced
EPS = 1e-6


@pytest.fixture(scope="module")
def lib():
    if not S.LIB_PATH.exists():
        build_lib.build()
    return NM.lib()


# ------------------------------------------------------------------ ABI, CPU

def test_header_and_library_agree_on_the_norm_entry_points(lib):
    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    names = set(re.findall(r"\b(stepq_norm_[a-z_]+)\s*\(", text))
    assert names == set(NM.EXPORTED)
    for n in names:
        assert hasattr(lib, n)


def desc(width=100, heads=1, dtype=1, act=0, post=1, pre=1, eps=EPS):
    return ctypes.byref(NM.stepq_norm_desc(width, heads, dtype, act, post, pre, eps))


def forward_status(lib, d=None, tokens=2, block=GOOD, bs=100, gate=GOOD, gs=100, res=GOOD, rs=100, w1=GOOD, sc=GOOD, w2=GOOD,
                   out=GOOD, os=100, normed=2 * GOOD, ns=100, **kw):
    return lib.stepq_norm_forward(desc(**kw) if d is None else d, tokens, block, bs, gate, gs, res, rs, w1, sc, w2, out, os, normed,
                                  ns, None)


BAD = [
    (dict(d=ctypes.c_void_p()), 1), (dict(width=0), 1), (dict(heads=0), 1), (dict(dtype=3), 1), (dict(act=2), 1), (dict(act=-1), 1),
    (dict(post=2), 1), (dict(pre=-1), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(eps=-1.0), 1), (dict(eps=1e-40), 1), (dict(tokens=-1), 1), (dict(block=None), 1), (dict(block=GOOD + 1), 1), (dict(dtype=0, gate=GOOD + 2), 1),
    (dict(bs=99), 1), (dict(heads=2), 1), (dict(w1=GOOD + 2), 1), (dict(sc=GOOD + 1), 1), (dict(w2=GOOD + 2), 1),
    (dict(bs=2 ** 41), 1), (dict(width=16385), 2), (dict(tokens=2 ** 31), 2), (dict(tokens=2 ** 30, heads=2), 2),
]


@pytest.mark.parametrize("bad,status", BAD + [
    (dict(res=GOOD + 1), 1), (dict(rs=5), 1), (dict(out=None, normed=None, pre=0, w2=None), 1), (dict(normed=None), 1),
    (dict(pre=0, w2=None), 1), (dict(pre=0, normed=None), 1), (dict(post=0), 1), (dict(normed=GOOD), 1), (dict(ns=99), 1),
    (dict(os=99), 1), (dict(res=GOOD, out=GOOD, rs=108), 1), (dict(normed=3 * GOOD, gate=3 * GOOD, ns=104), 1),
])
def test_forward_arguments_that_are_refused(lib, bad, status):
    assert forward_status(lib, **bad) == status


def backward_status(lib, d=None, tokens=2, block=GOOD, bs=100, gate=GOOD, gs=100, out=GOOD, os=100, w1=GOOD, sc=GOOD, w2=GOOD,
                    d_out=GOOD, dos=100, d_normed=GOOD, dns=100, d_block=GOOD, dbs=100, d_gate=2 * GOOD, dgs=100, d_res=3 * GOOD,
                    drs=100, d_w1=GOOD, d_sc=GOOD, d_w2=GOOD, ws=GOOD, nbytes=1 << 30, **kw):
    return lib.stepq_norm_backward(desc(**kw) if d is None else d, tokens, block, bs, gate, gs, out, os, w1, sc, w2, d_out, dos,
                                   d_normed, dns, d_block, dbs, d_gate, dgs, d_res, drs, d_w1, d_sc, d_w2, ws, nbytes, None)


@pytest.mark.parametrize("bad,status", BAD + [
    (dict(out=None), 1), (dict(d_normed=None), 1), (dict(d_block=None), 1), (dict(d_gate=None), 1), (dict(gate=None), 1),
    (dict(pre=0), 1), (dict(pre=0, w2=None, d_w2=None), 1), (dict(pre=0, w2=None, d_w2=None, d_normed=None, d_out=None), 1),
    (dict(w1=None), 1), (dict(sc=None), 1), (dict(w2=None), 1), (dict(d_w1=GOOD + 1), 1), (dict(d_block=2 * GOOD), 1),
    (dict(d_res=GOOD), 1), (dict(d_res=2 * GOOD), 1), (dict(ws=None), 1), (dict(ws=GOOD + 8), 1), (dict(nbytes=3 * 400 - 1), 1),
    (dict(drs=99), 1), (dict(dns=99), 1), (dict(dbs=108), 1), (dict(d_res=5 * GOOD, d_out=5 * GOOD, dos=120), 1),
])
def test_backward_arguments_that_are_refused(lib, bad, status):
    assert backward_status(lib, **bad) == status


def test_empty_calls_and_workspace_sizes(lib):
    assert forward_status(lib, tokens=0, block=None) == S.STEPQ_OK
    size = lib.stepq_norm_workspace_bytes
    assert size(None, 1) == 0 and size(desc(width=0), 1) == 0 and size(desc(), -1) == 0 and size(desc(), 2 ** 31) == 0
    for heads in (1, 3):
        for width in (1, 100, 1000, 5000, 16384):
            sizes = [size(desc(width=width, heads=heads), n) for n in (0, 1, 2, 50, 1000, 100000)]
            assert sizes[0] == 0 and sizes == sorted(sizes) and sizes[1] >= 12 * width


def test_binding_refuses_bad_tensors_before_the_library(lib):
    import torch
    for args in ((0,), (4, 0), (4, 1, torch.int32), (16385,), (4, 1, None, "relu"), (4, 1, None, "silu", True, True, 0.0)):
        with pytest.raises(S.StepqError):
            NM.BlockNorm(*args)
    n = NM.BlockNorm(4)
    x = torch.zeros(3, 4)
    for bad in (x, None, 3, np.zeros((3, 4), np.float32), torch.tensor(1.0)):
        for f in (lambda: n.forward(bad, x, x), lambda: n.backward(bad, x, x, x, x)):
            with pytest.raises(S.StepqError) as e:
                f()
            assert e.value.status == S.STEPQ_ERR_INVALID_ARG


# ------------------------------------------------- the formulas, CPU

@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_gradients_equal_differences(act, post, pre):
    g = np.random.default_rng(3)
    N, D = 3, 6
    o, z, x, dt, dy = (g.standard_normal((N, D)) for _ in range(5))
    w1, sc, w2 = (1.0 + 0.3 * g.standard_normal(D) for _ in range(3))

    def loss(o, z, x, w1, sc, w2):
        t, y, _, _ = ref.forward(o, z, x, w1, sc, w2, act, post, pre, EPS)
        return (t * dt).sum() + ((y * dy).sum() if pre else 0.0)

    t = ref.forward(o, z, x, w1, sc, w2, act, post, pre, EPS)[0]
    grads, _ = ref.backward(o, z, t, w1, sc, w2, act, post, pre, EPS, dt, dy)
    args = dict(o=o, z=z, x=x, w1=w1, sc=sc, w2=w2)
    names = dict(o="dblock", z="dgate", x="dresidual", w1="dpost", sc="dscale", w2="dpre")
    for name, v in args.items():
        if names[name] not in grads:
            continue
        flat = grads[names[name]].ravel()
        for i in range(v.size):
            d = np.zeros(v.size)
            d[i] = 1e-5
            d = d.reshape(v.shape)
            diff = (loss(**{**args, name: v + d}) - loss(**{**args, name: v - d})) / 2e-5
            assert abs(diff - flat[i]) <= 1e-7 * (1.0 + abs(flat[i])), (name, i)


# ---------------------------------------------------------------------- GPU

DTYPES = {"f32": ("float32", 2.0 ** -24, 0.0), "bf16": ("bfloat16", 2.0 ** -8, 0.0), "f16": ("float16", 2.0 ** -11, 2.0 ** -25)}


class Case:
    def __init__(self, tokens, width, dtype="f32", heads=1, act="silu", post=True, pre=True, gate=True, residual=True, scale=True,
                 weights=True, pad=0, shift=0, seed=0):
        import torch
        self.torch = torch
        name, self.step, self.small = DTYPES[dtype]
        self.td = getattr(torch, name)
        g = np.random.default_rng(seed)
        self.g, self.tokens, self.heads, self.width, self.row, self.pad, self.shift = g, tokens, heads, width, heads * width, pad, shift
        self.act, self.post, self.pre = act, post, pre
        self.op = NM.BlockNorm(width, heads, self.td, act, post, pre, EPS)
        scales = 0.3 + g.random((tokens, 1))
        self.block = self.rows(g.standard_normal((tokens, self.row)) * scales)
        self.gate = self.rows(2.0 * g.standard_normal((tokens, self.row))) if gate else None
        self.residual = self.rows(2.0 * g.standard_normal((tokens, self.row))) if residual else None
        self.w1 = self.weight() if post and weights else None
        self.sc = self.weight() if scale else None
        self.w2 = self.weight() if pre and weights else None

    def rows(self, v=None):
        """[tokens, heads * width] with tokens `pad` elements further apart, `shift` elements into a buffer of NaN."""
        torch = self.torch
        flat = torch.full((self.shift + self.tokens * (self.row + self.pad),), float("nan"), dtype=self.td, device="cuda")
        t = flat[self.shift:].view(self.tokens, self.row + self.pad)[:, :self.row]
        if v is not None:
            t.copy_(torch.from_numpy(v).cuda().to(self.td))
        return t

    def weight(self):
        return self.torch.from_numpy((1.0 + 0.3 * self.g.standard_normal(self.width)).astype(np.float32)).cuda()

    def host(self, t):
        return None if t is None else t.double().cpu().numpy().reshape(-1, self.width)

    def vector(self, t):
        return 1.0 if t is None else t.double().cpu().numpy()

    def near(self, got, want, bound, what):
        got = self.host(got)
        room = bound + np.maximum(self.step * (np.abs(want) + bound), self.small)
        assert np.all(np.abs(got - want) <= room), (what, float(np.nanmax(np.abs(got - want) / room)))

    def params(self):
        return [self.vector(t) for t in (self.w1, self.sc, self.w2)] + [self.act, self.post, self.pre, EPS]

    def gaps(self, t):
        """What lies between the tokens of a strided output."""
        flat = t.as_strided((self.shift + self.tokens * (self.row + self.pad),), (1,), 0).view(-1)
        rest = self.torch.ones_like(flat, dtype=self.torch.bool)
        rest[self.shift:].view(self.tokens, self.row + self.pad)[:, :self.row] = False
        return flat[rest]

    def check_forward(self, no_out=False):
        out, normed = (None if no_out else self.rows()), (self.rows() if self.pre else None)
        self.op.forward(self.block, out, normed, self.gate, self.residual, self.w1, self.sc, self.w2)
        self.torch.cuda.synchronize()
        t, y, bt, by = ref.forward(self.host(self.block), self.host(self.gate), self.host(self.residual), *self.params())
        for got, want, bound, what in ((out, t, bt, "out"), (normed, y, by, "normed")):
            if got is not None:
                self.near(got, want, bound, what)
                assert self.torch.isnan(self.gaps(got)).all()

    def check_backward(self, d_out=True, weights=True, d_residual=True):
        torch, g = self.torch, self.g
        out = self.rows(2.0 * g.standard_normal((self.tokens, self.row))) if self.pre else None
        dt = self.rows(g.standard_normal((self.tokens, self.row))) if d_out else None
        dy = self.rows(g.standard_normal((self.tokens, self.row))) if self.pre else None
        got = dict(dblock=self.rows(), dgate=self.rows() if self.gate is not None else None,
                   dresidual=self.rows() if d_residual else None)
        for name, w in (("dpost", self.w1), ("dscale", self.sc), ("dpre", self.w2)):
            got[name] = torch.full_like(w, float("nan")) if weights and w is not None else None
        ws = self.op.workspace(self.tokens)
        ws.fill_(0xFF)
        self.op.backward(self.block, out, dt, got["dblock"], dy, self.gate, got["dgate"], got["dresidual"], self.w1, got["dpost"],
                         self.sc, got["dscale"], self.w2, got["dpre"], workspace=ws)
        torch.cuda.synchronize()
        want, room = ref.backward(self.host(self.block), self.host(self.gate), self.host(out), *self.params(), self.host(dt),
                                  self.host(dy))
        for name, t in got.items():
            if t is None:
                continue
            if name in ("dblock", "dgate", "dresidual"):
                self.near(t, want[name], room[name], name)
                assert torch.isnan(self.gaps(t)).all()
            else:
                v = t.double().cpu().numpy()
                assert np.all(np.abs(v - want[name]) <= room[name] + ref.EPS * np.abs(want[name])), name


# a width for every split of a row over lanes, with and without whole pieces of 16 bytes
WIDTHS = [1, 7, 16, 32, 48, 64, 100, 128, 256, 520, 1000, 1024, 2048, 4090, 4096, 8192, 16384]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("width", WIDTHS)
def test_block_norms_and_their_gradients(width, dtype):
    for tokens in (1, 37):
        c = Case(tokens, width, dtype, seed=width)
        c.check_forward()
        c.check_backward()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("heads,width", [(3, 16), (48, 128), (2, 100), (5, 1)])
@pytest.mark.parametrize("pad", [0, 8])
def test_heads_side_by_side(heads, width, pad, dtype):
    c = Case(33, width, dtype, heads=heads, pre=False, residual=False, scale=False, pad=pad)
    c.check_forward()
    c.check_backward(d_residual=False)
    c = Case(5, width, dtype, heads=heads, pad=pad, act="sigmoid")
    c.check_forward()
    c.check_backward()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (8, 8), (5, 3)])
@pytest.mark.parametrize("width", [64, 4096])
def test_rows_at_any_distance_and_boundary(dtype, pad, shift, width):
    c = Case(9, width, dtype, pad=pad, shift=shift)
    c.check_forward()
    c.check_backward()


FORMS = [dict(gate=False), dict(residual=False), dict(scale=False), dict(weights=False), dict(post=False), dict(pre=False),
         dict(post=False, pre=False), dict(post=False, gate=False, scale=False), dict(post=False, pre=False, gate=False, scale=False),
         dict(post=True, pre=False, gate=False, residual=False, scale=False, weights=False)]


@pytest.mark.gpu
@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("width", [96, 4096])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_what_is_not_given_is_left_out(form, width, act):
    c = Case(40, width, "f32", act=act, **FORMS[form])
    c.check_forward(no_out=c.pre)
    c.check_forward()
    c.check_backward(d_out=not c.pre)
    c.check_backward(weights=False, d_residual=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,width", [("f32", 8), ("bf16", 128), ("bf16", 1000)])
def test_more_rows_than_workgroups(dtype, width):
    c = Case(9001, width, dtype)
    c.check_forward()
    c.check_backward()


@pytest.mark.gpu
@pytest.mark.parametrize("width", [100, 128, 4096])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_outputs_in_the_buffers_of_inputs(width, dtype):
    import torch
    c = Case(70, width, dtype)
    out, normed = c.rows(), c.rows()
    c.op.forward(c.block, out, normed, c.gate, c.residual, c.w1, c.sc, c.w2)
    b, r = c.block.clone(), c.residual.clone()
    c.op.forward(b, r, b, c.gate, r, c.w1, c.sc, c.w2)
    assert torch.equal(r, out) and torch.equal(b, normed)
    dt, dy = (c.rows(c.g.standard_normal((70, width))) for _ in range(2))
    db, dg, dr = c.rows(), c.rows(), c.rows()
    w = [torch.empty(width, device="cuda") for _ in range(6)]
    c.op.backward(c.block, out, dt, db, dy, c.gate, dg, dr, c.w1, w[0], c.sc, w[1], c.w2, w[2])
    b, g, d = c.block.clone(), c.gate.clone(), dt.clone()
    c.op.backward(b, out, d, b, dy, g, g, d, c.w1, w[3], c.sc, w[4], c.w2, w[5])
    torch.cuda.synchronize()
    for p, q in ((b, db), (g, dg), (d, dr), *zip(w[:3], w[3:])):
        assert torch.equal(p, q)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("width", [64, 4096])
def test_gates_at_their_ends(act, width):
    """Gates of -inf and the type's lowest value shut, of +inf open (sigmoid) and have no slope; rows of zeros stay zero."""
    import torch
    c = Case(6, width, "f32", act=act, pre=False)
    c.gate[0, 0], c.gate[0, 1], c.gate[1] = -float("inf"), torch.finfo(torch.float32).min, -float("inf")
    c.block[2] = 0.0
    if act == "sigmoid":
        c.gate[3] = float("inf")
    out, db, dg, dr = (c.rows() for _ in range(4))
    c.op.forward(c.block, out, None, c.gate, c.residual, c.w1, c.sc)
    d = c.rows(np.ones((6, width)))
    w = [torch.empty(width, device="cuda") for _ in range(2)]
    c.op.backward(c.block, out, d, db, None, c.gate, dg, dr, c.w1, w[0], c.sc, w[1])
    torch.cuda.synchronize()
    for t in (out, db, dg, dr, *w):
        assert torch.isfinite(t).all()
    assert torch.equal(out[0, :2], c.residual[0, :2]) and torch.equal(out[1:3], c.residual[1:3])
    assert float(dg[0, :2].abs().max()) == 0.0 and float(dg[1].abs().max()) == 0.0 and float(db[1].abs().max()) == 0.0
    if act == "sigmoid":
        assert float(dg[3].abs().max()) == 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("width", [64, 4096])
def test_a_value_that_is_not_finite_spoils_its_row_alone(width):
    import torch
    c = Case(8, width, "bf16")
    outs = []
    for bad in (False, True):
        if bad:
            c.block[3, width // 2] = float("nan")
        out, normed = c.rows(), c.rows()
        c.op.forward(c.block, out, normed, c.gate, c.residual, c.w1, c.sc, c.w2)
        outs.append((out, normed))
    torch.cuda.synchronize()
    rest = [0, 1, 2, 4, 5, 6, 7]
    for a, b in zip(*outs):
        assert torch.equal(a[rest], b[rest]) and torch.isnan(b[3]).any()


@pytest.mark.gpu
def test_no_tokens():
    import torch
    c = Case(0, 64, "f32")
    c.op.forward(c.block, c.rows(), c.rows(), c.gate, c.residual, c.w1, c.sc, c.w2)
    w = [torch.full((64,), 3.0, device="cuda") for _ in range(3)]
    e = c.rows()
    c.op.backward(c.block, e, e, e, e, c.gate, e, e, c.w1, w[0], c.sc, w[1], c.w2, w[2])
    torch.cuda.synchronize()
    assert all(float(t.abs().max()) == 0.0 for t in w)


@pytest.mark.gpu
@pytest.mark.parametrize("width,dtype", [(4096, "bf16"), (64, "f32")])
def test_same_bits_again_on_another_stream_and_in_a_graph(width, dtype):
    import torch
    c = Case(700, width, dtype)
    dt, dy = (c.rows(c.g.standard_normal((700, width))) for _ in range(2))

    def buffers():
        return ([c.rows() for _ in range(5)], [torch.empty(width, device="cuda") for _ in range(3)], c.op.workspace(700))

    def run(b, stream=None):
        (out, normed, db, dg, dr), w, ws = b
        c.op.forward(c.block, out, normed, c.gate, c.residual, c.w1, c.sc, c.w2, stream=stream)
        c.op.backward(c.block, out, dt, db, dy, c.gate, dg, dr, c.w1, w[0], c.sc, w[1], c.w2, w[2], workspace=ws, stream=stream)

    first, others = buffers(), [buffers() for _ in range(2)]
    run(first)
    torch.cuda.synchronize()
    for b in others:
        run(b, torch.cuda.Stream())
    torch.cuda.synchronize()

    def same(b):
        for p, q in zip(b[0] + b[1], first[0] + first[1]):
            assert torch.equal(p, q)

    for b in others:
        same(b)
    b = buffers()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b)
    for _ in range(3):
        for t in b[0] + b[1]:
            t.fill_(7.0)
        b[2].fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        same(b)


@pytest.mark.gpu
def test_rows_past_32_bits():
    import torch
    tokens, width, stride = 70, 64, (1 << 31) // 64 + 64
    flat = torch.zeros((tokens - 1) * stride + width, dtype=torch.bfloat16, device="cuda")
    c = Case(tokens, width, "bf16")
    far = flat.as_strided((tokens, width), (stride, 1))
    far.copy_(c.block)
    out, out2, normed = c.rows(), c.rows(), c.rows()
    c.op.forward(c.block, out, normed, c.gate, c.residual, c.w1, c.sc, c.w2)
    c.op.forward(far, out2, far, c.gate, c.residual, c.w1, c.sc, c.w2)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(far, normed)


@pytest.mark.gpu
def test_refusals_that_need_a_device(monkeypatch):
    import torch
    from quantized_recurrent_state_packed_amd import linear as LN
    c = Case(6, 8, "f32")
    x, y = c.rows(), c.rows()
    w = torch.empty(8, device="cuda")

    def refused(f, match=None):
        with pytest.raises(S.StepqError, match=match) as e:
            f()
        assert e.value.status == S.STEPQ_ERR_INVALID_ARG

    def forward(block=c.block, out=x, normed=y, **kw):
        c.op.forward(block, out, normed, **kw)

    def backward(out=c.residual, d=c.block, db=x, dy=c.block, **kw):
        c.op.backward(c.block, out, d, db, dy, **kw)

    forward(), backward()
    refused(lambda: forward(normed=None), "normed")
    refused(lambda: forward(normed=x))
    refused(lambda: forward(out=x.half()))
    refused(lambda: forward(gate=c.gate[:5]))
    refused(lambda: forward(gate=c.gate.cpu()))
    refused(lambda: forward(residual=c.gate.t()))
    refused(lambda: forward(residual=c.gate[:1].expand(6, 8)), "overlap")
    refused(lambda: forward(post_weight=w.double()))
    refused(lambda: forward(scale=w[:7]))
    refused(lambda: forward(scale=1.0))
    refused(lambda: backward(dy=None))
    refused(lambda: backward(out=None))
    refused(lambda: backward(gate=c.gate))
    refused(lambda: backward(d_gate=y))
    refused(lambda: backward(d_post_weight=w))
    refused(lambda: backward(post_weight=w, d_post_weight=torch.empty(8, device="cuda"), stream=torch.cuda.Stream()), "workspace of its own")
    refused(lambda: backward(post_weight=w, d_post_weight=torch.empty(8, device="cuda"), workspace=torch.empty(4, dtype=torch.uint8, device="cuda")))
    refused(lambda: backward(workspace=3))
    refused(lambda: backward(d_residual=x))
    torch.cuda.synchronize()
    monkeypatch.setattr(LN, "_current_device", lambda: 1)
    refused(forward, "current")
    refused(backward, "current")


@pytest.mark.gpu
def test_what_a_group_without_a_row_works_out_is_not_added():
    """5 tokens of 64 leave 11 of a workgroup's 16 groups without a row.  An infinite gate in the last token makes its
    column's sums infinite, as the formula does, and leaves the other columns as they are with a finite gate."""
    import torch
    c = Case(5, 64, "f32", pre=False)
    d = c.rows(c.g.standard_normal((5, 64)))
    sums = []
    for last in (1.0, float("inf")):
        c.gate[4, 7] = last
        out, db, dg = c.rows(), c.rows(), c.rows()
        w = [torch.empty(64, device="cuda") for _ in range(2)]
        c.op.backward(c.block, out, d, db, None, c.gate, dg, None, c.w1, w[0], c.sc, w[1])
        sums.append(w)
    torch.cuda.synchronize()
    rest = torch.arange(64, device="cuda") != 7
    for a, b in zip(*sums):
        assert torch.isfinite(a).all() and torch.isinf(b[7]) and torch.equal(a[rest], b[rest])


@pytest.mark.gpu
@pytest.mark.parametrize("width,tokens", [(16, 65), (32, 257), (128, 17), (512, 5), (1000, 3)])
def test_gradients_beyond_binary16_in_the_buffers_of_inputs(width, tokens):
    """The last token's gradient of block is infinite in binary16 and overwrites block, whose values other groups of
    the workgroup must not see: the weights' gradients are finite and those of outputs in buffers of their own."""
    import torch
    c = Case(tokens, width, "f16")
    c.block[-1] = (c.block[-1].sign() + 0.5) * 2.0 ** -14          # its reciprocal root is 1000 and more
    dt, dy = (c.rows(c.g.standard_normal((tokens, width))) for _ in range(2))
    dt[-1] = 6e4
    out = c.rows(2.0 * c.g.standard_normal((tokens, width)))
    w = [torch.empty(width, device="cuda") for _ in range(6)]
    db, dg, dr = c.rows(), c.rows(), c.rows()
    c.op.backward(c.block, out, dt, db, dy, c.gate, dg, dr, c.w1, w[0], c.sc, w[1], c.w2, w[2])
    torch.cuda.synchronize()
    assert torch.isinf(db[-1]).any() and all(torch.isfinite(t).all() for t in w[:3])
    for _ in range(5):
        b, g, d, t = c.block.clone(), c.gate.clone(), dt.clone(), out.clone()
        c.op.backward(b, t, d, b, dy, g, g, d, c.w1, w[3], c.sc, w[4], c.w2, w[5])
        torch.cuda.synchronize()
        for p, q in ((b, db), (g, dg), (d, dr), *zip(w[:3], w[3:])):
            assert torch.equal(p, q)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [16, 64, 256, 512, 4096])
def test_equal_values_of_a_row_have_equal_results(width):
    """Whatever lane holds them: every lane scales by the same reciprocal root."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(width)
    x = torch.randn(500, width, generator=g, device="cuda")
    x[:, ::4] = 1.5                     # a lane's first value of its four
    out, normed = torch.empty_like(x), torch.empty_like(x)
    NM.BlockNorm(width, eps=EPS).forward(x, out, normed)
    torch.cuda.synchronize()
    for t in (out, normed):
        assert torch.equal(t[:, ::4], t[:, :1].expand(500, width // 4))


@pytest.mark.gpu
@pytest.mark.parametrize("width", [4, 64, 256, 1000, 4096, 16384])
def test_rows_whose_sum_of_squares_binary32_does_not_hold(width):
    """Rows of values whose squares add up to 2^126 and to 2^130: the former are normalised, the latter are 0, also
    where their mean is in range."""
    import torch
    x = torch.ones(8, width, device="cuda")
    x[::2] *= (2.0 ** 126 / width) ** 0.5
    x[1::2] *= (2.0 ** 130 / width) ** 0.5
    out, normed = torch.empty_like(x), torch.empty_like(x)
    NM.BlockNorm(width, pre=False, eps=EPS).forward(x, out)
    NM.BlockNorm(width, post=False, eps=EPS).forward(x, None, normed)
    torch.cuda.synchronize()
    for t in (out, normed):
        # sums of equal squares, a reciprocal root (one step) and a product
        assert float((t[::2] - 1.0).abs().max()) <= 40 * 2.0 ** -24 and float(t[1::2].abs().max()) == 0.0

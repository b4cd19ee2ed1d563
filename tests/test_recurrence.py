"""The gated linear recurrence against the recurrence in 64 bits (scan_ref.py), its
gradients against the adjoint recurrence and that against differences, and what it refuses.

Tolerances are those of scan_ref.py's derivation plus half a step of the output's type,
torch.finfo(t).eps / 2 of the value, or, for a float16 value below 2^-14, half of the step
2^-24 that float16's values have there."""
import ctypes
import re
from pathlib import Path

import numpy as np
import pytest

import scan_ref as ref
from quantized_recurrent_state_packed_amd import build_lib
from quantized_recurrent_state_packed_amd import recurrence as RC
from quantized_recurrent_state_packed_amd import stepq as S

HEADER = Path(__file__).resolve().parents[1] / "include" / "stepq_block.h"
GOOD = 4096          # an address that is never dereferenced
RATE = 8.0
PIECE = 128          # tokens of a workgroup of a large forward pass, twice those of a small one and of the backward pass


@pytest.fixture(scope="module")
def lib():
    if not S.LIB_PATH.exists():
        build_lib.build()
    return RC.lib()


# ------------------------------------------------------------------ ABI, CPU

def test_header_and_library_agree_on_the_scan_entry_points(lib):
    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    names = set(re.findall(r"\b(stepq_scan_[a-z_]+)\s*\(", text))
    assert names == set(RC.EXPORTED)
    for n in names:
        assert hasattr(lib, n)


def desc(width=100, dtype=1, rate=RATE):
    return ctypes.byref(RC.stepq_scan_desc(width, dtype, rate))


def forward_status(lib, d=None, batch=2, tokens=70, cu=GOOD, x=GOOD, xs=100, ga=GOOD, gas=100, gx=GOOD, gxs=100, decay=GOOD,
                   slots=GOOD, num_slots=3, resume=None, state=GOOD, y=GOOD, ys=100, saved=None, saved_bytes=0, ws=GOOD,
                   nbytes=1 << 30, **kw):
    return lib.stepq_scan_forward(desc(**kw) if d is None else d, batch, tokens, cu, x, xs, ga, gas, gx, gxs, decay, slots,
                                  num_slots, resume, state, y, ys, saved, saved_bytes, ws, nbytes, None)


BAD = [
    (dict(d=ctypes.c_void_p()), 1), (dict(width=0), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(rate=0.0), 1),
    (dict(rate=-1.0), 1), (dict(rate=float("nan")), 1), (dict(rate=float("inf")), 1), (dict(batch=-1), 1), (dict(tokens=-1), 1),
    (dict(cu=None), 1), (dict(cu=GOOD + 2), 1), (dict(x=None), 1), (dict(x=GOOD + 1), 1), (dict(xs=99), 1), (dict(gas=99), 1),
    (dict(gxs=-100), 1), (dict(ga=None), 1), (dict(gx=None), 1), (dict(decay=None), 1), (dict(decay=GOOD + 2), 1),
    (dict(dtype=0, x=GOOD + 2), 1), (dict(xs=2 ** 24 + 1), 1), (dict(slots=None), 1), (dict(slots=GOOD + 1), 1), (dict(state=None), 1),
    (dict(state=GOOD + 2), 1), (dict(num_slots=0), 1), (dict(width=2 ** 20 + 1), 2),
    (dict(tokens=2 ** 31), 2), (dict(batch=2 ** 23), 2),
]


@pytest.mark.parametrize("bad,status", BAD + [
    (dict(y=None), 1), (dict(y=GOOD + 1), 1), (dict(ys=99), 1), (dict(saved=GOOD + 8, saved_bytes=1 << 30), 1),
    (dict(saved=GOOD, saved_bytes=10 * 400 - 1), 1),
])
def test_forward_arguments_that_are_refused(lib, bad, status):
    assert forward_status(lib, **bad) == status


def backward_status(lib, d=None, batch=2, tokens=70, cu=GOOD, x=GOOD, xs=100, ga=GOOD, gas=100, gx=GOOD, gxs=100, decay=GOOD,
                    saved=GOOD, saved_bytes=1 << 30, dy=GOOD, dys=100, slots=GOOD, num_slots=3, resume=None, state=GOOD, dx=GOOD,
                    dxs=100, dga=GOOD, dgas=100, dgx=GOOD, dgxs=100, ddecay=GOOD, ws=GOOD, nbytes=1 << 30, **kw):
    return lib.stepq_scan_backward(desc(**kw) if d is None else d, batch, tokens, cu, x, xs, ga, gas, gx, gxs, decay, saved,
                                   saved_bytes, dy, dys, slots, num_slots, resume, state, dx, dxs, dga, dgas, dgx, dgxs, ddecay,
                                   ws, nbytes, None)


@pytest.mark.parametrize("bad,status", BAD + [
    (dict(saved=None), 1), (dict(saved=GOOD + 4), 1), (dict(saved_bytes=10 * 400 - 1), 1), (dict(dy=None), 1),
    (dict(dys=99), 1), (dict(dx=None), 1), (dict(dga=GOOD + 1), 1), (dict(dgxs=50), 1), (dict(ddecay=None), 1),
    (dict(ddecay=GOOD + 2), 1), (dict(ws=None), 1), (dict(ws=GOOD + 8), 1), (dict(nbytes=0), 1),
])
def test_backward_arguments_that_are_refused(lib, bad, status):
    assert backward_status(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(batch=-1), 1), (dict(num_slots=0), 1), (dict(slots=None), 1), (dict(state=None), 1), (dict(x=None), 1),
    (dict(xs=99), 1), (dict(ga=GOOD + 1), 1), (dict(decay=None), 1), (dict(y=None), 1), (dict(batch=2 ** 23), 2),
    (dict(state=GOOD + 2), 1),
])
def test_step_arguments_that_are_refused(lib, bad, status):
    a = dict(batch=2, slots=GOOD, num_slots=3, x=GOOD, xs=100, ga=GOOD, gas=100, gx=GOOD, gxs=100, decay=GOOD, state=GOOD, y=GOOD,
             ys=100)
    a.update(bad)
    assert lib.stepq_scan_step(desc(), *a.values(), None) == status


def test_empty_batches_and_sizes(lib):
    assert forward_status(lib, batch=0, x=None, ws=None) == S.STEPQ_OK
    size, saved = lib.stepq_scan_workspace_bytes, lib.stepq_scan_saved_bytes
    for f in (size, saved):
        assert f(None, 1, 1) == 0 and f(desc(width=0), 1, 1) == 0 and f(desc(), -1, 1) == 0 and f(desc(), 1, 2 ** 31) == 0
    assert saved(desc(), 2, 70) == (70 // 8 + 2) * 400
    sizes = [size(desc(), b, t) for t in (0, 1, 64, 65, 1000, 100000) for b in (0, 1, 3, 50)]
    assert sizes[:4] == [max(0, 16 * -(-b * 400 // 16)) for b in (0, 1, 3, 50)]
    for t in range(5):      # more requests or tokens never need less
        assert all(sizes[4 * t + i] <= sizes[4 * (t + 1) + i] for i in range(4))


def test_binding_refuses_bad_tensors_before_the_library(lib):
    import torch
    for args in ((0,), (4, torch.int32), (4, None, 0.0), (4, None, float("nan"))):
        with pytest.raises(S.StepqError):
            RC.GatedRecurrence(*args)
    rec = RC.GatedRecurrence(4)
    x, d = torch.zeros(3, 4), torch.zeros(4)
    cu, ids, st = torch.tensor([0, 3], dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 4)
    saved = torch.zeros(1000, dtype=torch.uint8)
    for bad in (x, None, 3, np.zeros((3, 4), np.float32), torch.tensor(1.0)):
        for at in range(6):
            a = [x, x, x, d, ids, st]
            a[at] = bad
            with pytest.raises(S.StepqError) as e:
                rec.prefill(cu, *a, x)
            assert e.value.status == S.STEPQ_ERR_INVALID_ARG
            with pytest.raises(S.StepqError) as e:
                rec.step(ids, *a[:4], a[5], x)
            assert e.value.status == S.STEPQ_ERR_INVALID_ARG
            with pytest.raises(S.StepqError) as e:
                rec.backward(cu, *a[:4], saved, x, x, x, x, d)
            assert e.value.status == S.STEPQ_ERR_INVALID_ARG
    with pytest.raises(S.StepqError):
        rec.prefill(None, x, x, x, d, ids, st, x)
    with pytest.raises(S.StepqError):
        rec.workspace(1 << 23, 1, device="cpu")


# ------------------------------------------------- the formulas, CPU

def test_gradients_equal_differences():
    g = np.random.default_rng(5)
    T, D = 7, 5
    x, ga, gx, dy = (g.standard_normal((T, D)) for _ in range(4))
    decay, h0, dend = g.standard_normal(D) - 2.0, g.standard_normal(D), g.standard_normal(D)

    def loss(x, ga, gx, decay, h0):
        y, _ = ref.forward(x, ga, gx, decay, RATE, h0)
        return (y * dy).sum() + (y[-1] * dend).sum()

    grads, _ = ref.backward(x, ga, gx, decay, RATE, h0, dy, dend)
    args = dict(x=x, ga=ga, gx=gx, decay=decay, h0=h0)
    for name, v in args.items():
        flat = grads["d" + name].ravel()
        for i in range(v.size):
            d = np.zeros(v.size)
            d[i] = 1e-5
            d = d.reshape(v.shape)
            diff = (loss(**{**args, name: v + d}) - loss(**{**args, name: v - d})) / 2e-5
            assert abs(diff - flat[i]) <= 1e-7 * (1.0 + abs(flat[i])), (name, i)


# ---------------------------------------------------------------------- GPU

DTYPES = {"f32": ("float32", 2.0 ** -24), "bf16": ("bfloat16", 2.0 ** -8), "f16": ("float16", 2.0 ** -11)}
SMALL_STEP = {"f16": 2.0 ** -25}      # half a step among the smallest values


class Case:
    """Inputs of requests of `lengths` tokens, with rows of no request before, between nothing and behind."""

    def __init__(self, lengths, width, dtype="f32", seed=0, pad=0, shift=0, lead=2, tail=3, resume=True, slots=True, spread=1.0,
                 bad=()):
        import torch
        g = np.random.default_rng(seed)
        self.torch, self.width, self.lengths, self.batch = torch, width, list(lengths), len(lengths)
        self.td, self.step = getattr(torch, DTYPES[dtype][0]), DTYPES[dtype][1]
        self.small = SMALL_STEP.get(dtype, 0.0)
        self.T = lead + sum(lengths) + tail
        cu = np.r_[0, np.cumsum(lengths)].astype(np.int32) + lead
        self.cu_host = cu
        self.cu = torch.from_numpy(cu).cuda()
        self.rec = RC.GatedRecurrence(width, self.td, RATE)
        row = 3 * width + pad

        def rows(scale):
            flat = torch.full((shift + self.T * row,), float("nan"), dtype=self.td, device="cuda")
            wide = flat[shift:].view(self.T, row)
            v = g.standard_normal((self.T, 3 * width)) * scale
            wide[:, :3 * width] = torch.from_numpy(v).cuda().to(self.td)
            return [wide[:, i * width:(i + 1) * width] for i in range(3)]

        self.x, self.ga, self.gx = rows(spread)
        self.dy = rows(1.0)[1]
        half = 10.0 ** g.uniform(0.0, 3.0, width)
        self.decay = torch.from_numpy(np.log(np.expm1(np.log(2.0) / (0.5 * RATE * half))).astype(np.float32)).cuda()
        self.num_slots = self.batch + 2
        ids = g.permutation(self.num_slots)[:self.batch].astype(np.int32)
        for b, value in bad:
            ids[b] = value
        self.ids_host = ids
        self.ids = torch.from_numpy(ids).cuda() if slots else None
        self.state = torch.from_numpy(g.standard_normal((self.num_slots, width)).astype(np.float32)).cuda() if slots else None
        self.dstate = torch.from_numpy(g.standard_normal((self.num_slots, width)).astype(np.float32)).cuda() if slots else None
        self.res_host = (g.random(self.batch) < 0.6).astype(np.uint8) if resume and slots else None
        self.resume = None if self.res_host is None else torch.from_numpy(self.res_host).cuda()
        self.y = rows(1.0)[2]
        self.dx, self.dga, self.dgx = rows(1.0)
        self.ddecay = torch.full((width,), 7.0, device="cuda")

    def host(self, t):
        return t.double().cpu().numpy()

    def buffers(self):
        ws = self.rec.workspace(self.batch, self.T)
        saved = self.rec.saved(self.batch, self.T)
        ws.fill_(0xFF), saved.fill_(0xFF)
        return ws, saved

    def forward(self, saved=None, **kw):
        self.rec.prefill(self.cu, self.x, self.ga, self.gx, self.decay, self.ids, self.state, self.y, resume=self.resume,
                         saved=saved, **kw)

    def backward(self, saved, **kw):
        self.rec.backward(self.cu, self.x, self.ga, self.gx, self.decay, saved, self.dy, self.dx, self.dga, self.dgx, self.ddecay,
                          slot_ids=self.ids, dstate=self.dstate, resume=self.resume, **kw)

    def known(self, b):
        return self.ids is not None and 0 <= self.ids_host[b] < self.num_slots

    def near(self, got, want, bound, what):
        room = bound + np.maximum(self.step * (np.abs(want) + bound), self.small)
        assert np.all(np.abs(got - want) <= room), (what, float(np.nanmax(np.abs(got - want) / room)))

    def check(self, gradients=True):
        torch = self.torch
        ins = [self.host(t) for t in (self.x, self.ga, self.gx)]
        decay = self.host(self.decay)
        before = None if self.state is None else self.host(self.state)
        dbefore = None if self.state is None else self.host(self.dstate)
        outs = [self.y] + ([self.dx, self.dga, self.dgx] if gradients else [])
        olds = [t.clone() for t in outs]
        ws, saved = self.buffers()
        self.forward(saved if gradients else None, workspace=ws)
        if gradients:
            ws.fill_(0xFF)
            self.backward(saved, workspace=ws)
        torch.cuda.synchronize()
        cu = self.cu_host
        outside = np.r_[0:cu[0], cu[-1]:self.T]
        for t, old in zip(outs, olds):
            assert torch.equal(t[outside], old[outside])
        state, total, room = None if before is None else before.copy(), np.zeros(self.width), np.zeros(self.width)
        dstate = None if before is None else dbefore.copy()
        sb = np.zeros_like(state) if state is not None else None
        dsb = np.zeros_like(state) if state is not None else None
        got = [self.host(t) for t in outs]
        for b in range(self.batch):
            at = slice(cu[b], cu[b + 1])
            if self.ids is not None and not self.known(b):
                for t in got:
                    assert np.isnan(t[at]).all()
                continue
            h0 = np.zeros(self.width)
            cont = self.res_host is not None and self.res_host[b]
            if cont:
                h0 = before[self.ids_host[b]]
            args = [t[at] for t in ins]
            y, size = ref.forward(*args, decay, RATE, h0)
            bound = ref.state_bound(size, args[1], args[2])
            self.near(got[0][at], y, bound, f"y of request {b}")
            if self.known(b):
                state[self.ids_host[b]] = y[-1] if len(y) else h0
                sb[self.ids_host[b]] = bound[-1] if len(y) else 0.0
            if gradients:
                dend = dbefore[self.ids_host[b]] if self.known(b) else np.zeros(self.width)
                grads, bounds = ref.backward(*args, decay, RATE, h0, self.host(self.dy)[at], dend)
                for n, t in zip(("dx", "dga", "dgx"), got[1:]):
                    self.near(t[at], grads[n], bounds[n], f"{n} of request {b}")
                total, room = total + grads["ddecay"], room + bounds["ddecay"]
                if self.known(b):
                    dstate[self.ids_host[b]] = grads["dh0"] if cont else 0.0
                    dsb[self.ids_host[b]] = bounds["dh0"] if cont else 0.0
        if state is not None:
            assert np.all(np.abs(self.host(self.state) - state) <= sb + 2.0 ** -24 * np.abs(state))
        if gradients:
            if state is not None:
                assert np.all(np.abs(self.host(self.dstate) - dstate) <= dsb + 2.0 ** -24 * np.abs(dstate))
            assert np.all(np.abs(self.host(self.ddecay) - total) <= room + 2.0 ** -23 * np.abs(total))


LENGTHS = {"one": [1], "short": [37], "piece": [PIECE], "piece+1": [PIECE + 1], "half": [PIECE // 2],
           "half+1": [PIECE // 2 + 1], "ragged": [3, 0, 1, 130, 64, 65, 7, 0], "long": [1500],
           "many": [1, 2, 0, 9, 8, 7] * 23, "two long": [700, 513], "sparse": [1, 0, 0, 2] * 30, "sparser": [0, 1, 0, 0] * 40}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("width", [1, 64, 130, 203])
def test_prompts_and_their_gradients(lengths, width, dtype):
    Case(LENGTHS[lengths], width, dtype, seed=width).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[64 * PIECE + 1], [10, 70 * PIECE, 5], [20000, 0, 9000]])
def test_prompts_of_several_runs(lengths, dtype):
    """Requests longer than the 64 pieces over which states are handed on in one go."""
    Case(lengths, 6, dtype).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("pad,shift", [(1, 0), (2, 0), (0, 1), (5, 3), (8, 8)])
def test_rows_at_any_distance_and_boundary(dtype, pad, shift):
    Case([130, 5], 66, dtype, pad=pad, shift=shift).check()


@pytest.mark.gpu
@pytest.mark.parametrize("resume,slots", [(False, True), (False, False)])
def test_requests_that_start_from_zero(resume, slots):
    Case([100, 3, 0, 64], 70, "f32", resume=resume, slots=slots).check()


@pytest.mark.gpu
def test_requests_without_a_slot_of_their_own():
    Case([100, 3, 0, 64, 9], 70, "bf16", bad=((0, -1), (2, 1 << 30), (4, 7))).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_forward_pass_without_saving(dtype):
    Case([100, 3, 0, 640], 66, dtype).check(gradients=False)


@pytest.mark.gpu
def test_more_requests_than_a_wave_has_lanes():
    Case(list(np.random.default_rng(3).integers(0, 90, size=700)), 5, "f32").check()


@pytest.mark.gpu
def test_wide_gates():
    """Gates up to 40 in size: retentions of 1 and of nearly 0 among them."""
    Case([200, 65], 66, "f32", spread=12.0).check()


@pytest.mark.gpu
def test_all_requests_empty():
    c = Case([0, 0, 0], 9, "f32", lead=0, tail=0)
    c.check()
    assert float(c.ddecay.abs().max()) == 0.0


@pytest.mark.gpu
def test_no_requests():
    import torch
    rec = RC.GatedRecurrence(9)
    x, d = torch.zeros(4, 9, device="cuda"), torch.zeros(9, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    dd = torch.full((9,), 3.0, device="cuda")
    rec.prefill(cu, x, x, x, d, None, None, x.clone())
    rec.backward(cu, x, x, x, d, rec.saved(0, 4), x, x.clone(), x.clone(), x.clone(), dd)
    torch.cuda.synchronize()
    assert float(dd.abs().max()) == 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_gates_and_decays_at_their_ends(dtype):
    """Infinite gates close or open; a decay whose softplus vanishes keeps the state: no gradient is NaN."""
    import torch
    c = Case([130, 70], 6, dtype, lead=0, tail=0, resume=True)
    for t in (c.ga, c.gx):
        t[3], t[66], t[140] = float("inf"), -float("inf"), -float("inf")
    c.decay[0], c.decay[1], c.decay[2] = -200.0, 30.0, -50.0
    ws, saved = c.buffers()
    c.forward(saved, workspace=ws)
    c.backward(saved, workspace=ws)
    torch.cuda.synchronize()
    for t in (c.y, c.dx, c.dga, c.dgx, c.ddecay, c.state, c.dstate):
        assert torch.isfinite(t).all()
    for b in range(2):
        at = slice(c.cu_host[b], c.cu_host[b + 1])
        for t in (c.dga, c.dgx):
            assert float(t[at][torch.isinf(c.ga[at])].abs().max()) == 0.0     # the logistic function is flat there
    assert float(c.dx[66].abs().max()) == 0.0
    y = c.host(c.y)
    assert np.array_equal(y[66], y[65])                       # closed: the state stays


@pytest.mark.gpu
def test_gates_and_decays_that_leave_hardly_anything():
    """1 - a of the size of the smallest binary32 numbers and below: what comes in is at most their root, 1e-18, and
    every gradient is finite."""
    import torch
    c = Case([300], 8, "f32", lead=0, tail=0, resume=False)
    c.ga[:, :4] = torch.linspace(-60.0, -104.0, 300, device="cuda")[:, None]
    c.decay[:4] = torch.tensor([-5.0, 0.0, 5.0, -20.0], device="cuda")
    c.decay[4:] = torch.tensor([-85.0, -87.5, -95.0, -110.0], device="cuda")
    ws, saved = c.buffers()
    c.forward(saved, workspace=ws)
    c.backward(saved, workspace=ws)
    torch.cuda.synchronize()
    for t in (c.y, c.dx, c.dga, c.dgx, c.ddecay, c.state, c.dstate):
        assert torch.isfinite(t).all()
    assert float(c.y.abs().max()) < 1e-10 and float(c.dga.abs().max()) < 1e-10


@pytest.mark.gpu
def test_a_value_that_is_not_finite_spoils_its_own_request_and_channel_alone():
    import torch
    c, d = (Case([200, 70], 10, "f32", seed=4) for _ in range(2))
    at = int(c.cu_host[0]) + 90
    c.x[at, 3] = float("nan")
    for k in (c, d):
        ws, saved = k.buffers()
        k.forward(saved, workspace=ws)
        k.backward(saved, workspace=ws)
    torch.cuda.synchronize()
    rest = torch.ones_like(c.y, dtype=torch.bool)
    rest[c.cu_host[0]:c.cu_host[1], 3] = False
    for n in ("y", "dx", "dga", "dgx"):
        inside = slice(int(c.cu_host[0]), int(c.cu_host[-1]))
        assert torch.equal(getattr(c, n)[inside][rest[inside]], getattr(d, n)[inside][rest[inside]])
    assert torch.isnan(c.y[at:c.cu_host[1], 3]).all() and torch.equal(c.y[c.cu_host[0]:at], d.y[c.cu_host[0]:at])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("batch,width,pad", [(1, 1, 0), (5, 130, 0), (3, 1001, 1), (512, 64, 2), (4099, 64, 0)])
def test_single_tokens(dtype, batch, width, pad):
    import torch
    c = Case([1] * batch, width, dtype, pad=pad, lead=0, tail=0, bad=((batch - 1, -3),) if batch > 2 else ())
    x, ga, gx = (c.host(t) for t in (c.x, c.ga, c.gx))
    before, decay = c.host(c.state), c.host(c.decay)
    c.rec.step(c.ids, c.x, c.ga, c.gx, c.decay, c.state, c.y)
    torch.cuda.synchronize()
    want, y, state = before.copy(), c.host(c.y), c.host(c.state)
    for b in range(batch):
        if not c.known(b):
            assert np.isnan(y[b]).all()
            continue
        h, size = ref.forward(x[b:b + 1], ga[b:b + 1], gx[b:b + 1], decay, RATE, before[c.ids_host[b]])
        bound = ref.state_bound(size, ga, gx)[0]
        c.near(y[b], h[0], bound, b)
        want[c.ids_host[b]] = h[0]
        assert np.all(np.abs(state[c.ids_host[b]] - h[0]) <= bound + 2.0 ** -24 * np.abs(h[0]))
    others = [s for s in range(c.num_slots) if s not in set(c.ids_host[[c.known(b) for b in range(batch)]].tolist())]
    assert np.array_equal(state[others], before[others])


@pytest.mark.gpu
def test_a_prompt_in_parts_and_token_by_token():
    """A prompt, the same in two calls that resume, and the same token by token end alike."""
    import torch
    c = Case([150], 34, "f32", resume=False, lead=0, tail=0)
    c.forward()
    whole = c.state.clone()
    y = c.y.clone()
    ids, on = c.ids, torch.ones(1, dtype=torch.uint8, device="cuda")
    c.state.fill_(3.0)
    for n, (lo, hi) in enumerate(((0, 70), (70, 150))):
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        c.rec.prefill(cu, c.x[lo:hi], c.ga[lo:hi], c.gx[lo:hi], c.decay, ids, c.state, c.y[lo:hi], resume=on if n else None)
    assert torch.allclose(c.state[ids.long()], whole[ids.long()], rtol=1e-5, atol=1e-5) and torch.allclose(c.y, y, rtol=1e-5, atol=1e-5)
    c.state.zero_()
    for t in range(150):
        c.rec.step(ids, c.x[t:t + 1], c.ga[t:t + 1], c.gx[t:t + 1], c.decay, c.state, c.y[t:t + 1])
    torch.cuda.synchronize()
    assert torch.allclose(c.state[ids.long()], whole[ids.long()], rtol=1e-5, atol=1e-5) and torch.allclose(c.y, y, rtol=1e-5, atol=1e-5)


@pytest.mark.gpu
def test_same_bits_again_on_another_stream_and_in_a_graph():
    """Two calls at once on two streams, each with its own workspace, and replays of a captured one."""
    import torch
    cases = [Case([400, 0, 333, 64], 130, "bf16", seed=9) for _ in range(2)]
    first = Case([400, 0, 333, 64], 130, "bf16", seed=9)
    ws, saved = first.buffers()
    first.forward(saved, workspace=ws)
    first.backward(saved, workspace=ws)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    keep = []
    for s, c in zip(streams, cases):
        s.wait_stream(torch.cuda.current_stream())
        ws, saved = c.buffers()
        keep.append((ws, saved))
    torch.cuda.synchronize()
    for s, c, (ws, saved) in zip(streams, cases, keep):
        c.forward(saved, workspace=ws, stream=s)
        c.backward(saved, workspace=ws, stream=s)
    torch.cuda.synchronize()
    names = ("y", "dx", "dga", "dgx", "ddecay", "state", "dstate")

    def same(c):
        for n in names:
            a, b = getattr(c, n), getattr(first, n)
            if n in ("y", "dx", "dga", "dgx"):
                a, b = a[c.cu_host[0]:c.cu_host[-1]], b[c.cu_host[0]:c.cu_host[-1]]
            assert torch.equal(a, b), n

    for c in cases:
        same(c)
    c = Case([400, 0, 333, 64], 130, "bf16", seed=9)
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
    """Tokens so far apart that the last ones lie 2^32 bytes and more behind the first."""
    import torch
    rows, width, stride = 140, 64, 1 << 24
    flat = torch.zeros((rows - 1) * stride + width, dtype=torch.bfloat16, device="cuda")
    assert flat.numel() * 2 > 1 << 32
    rec = RC.GatedRecurrence(width, torch.bfloat16, RATE)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, ga, gx, dy = (torch.randn(rows, width, generator=g, device="cuda").bfloat16() for _ in range(4))
    far = flat.as_strided((rows, width), (stride, 1))
    far.copy_(x)
    cu = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    decay, y, z = torch.full((width,), -3.0, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    saved, dd = rec.saved(1, rows), torch.empty(width, device="cuda")
    rec.prefill(cu, x, ga, gx, decay, None, None, y, saved=saved)
    rec.prefill(cu, far, ga, gx, decay, None, None, z)
    dx, da, dg, da2, dg2 = (torch.empty_like(x) for _ in range(5))
    rec.backward(cu, x, ga, gx, decay, saved, dy, dx, da, dg, dd)
    far.copy_(dy)
    rec.backward(cu, x, ga, gx, decay, saved, far, torch.empty_like(x), da2, dg2, dd)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and torch.equal(da, da2) and torch.equal(dg, dg2)
    rec.prefill(cu, x, ga, gx, decay, None, None, far)
    torch.cuda.synchronize()
    assert torch.equal(far, y)


@pytest.mark.gpu
def test_refusals_that_need_a_device(monkeypatch):
    import torch
    from quantized_recurrent_state_packed_amd import linear as LN
    c = Case([5, 2 * PIECE], 8, "f32")
    ws, saved = c.buffers()
    calls = (lambda: c.forward(saved, workspace=ws), lambda: c.backward(saved, workspace=ws),
             lambda: c.rec.step(c.ids, c.x[:2], c.ga[:2], c.gx[:2], c.decay, c.state, c.y[:2]))
    for call in calls:
        call()

    def refused(f, match=None):
        with pytest.raises(S.StepqError, match=match) as e:
            f()
        assert e.value.status == S.STEPQ_ERR_INVALID_ARG

    refused(lambda: c.forward(saved[:8], workspace=ws))
    refused(lambda: c.forward(saved, workspace=3))
    refused(lambda: c.forward(3, workspace=ws))
    refused(lambda: c.forward(saved, workspace=ws[:0]))
    refused(lambda: c.backward(saved, workspace=ws[:16]))
    refused(lambda: c.backward(saved, stream=torch.cuda.Stream()), "workspace of its own")
    refused(lambda: c.rec.prefill(c.cu, c.x, c.ga, c.gx, c.decay, c.ids, None, c.y), "belong together")
    refused(lambda: c.rec.prefill(c.cu, c.x, c.ga, c.gx, c.decay, None, None, c.y, resume=c.resume), "resume")
    refused(lambda: c.rec.prefill(c.cu, c.x.t(), c.ga, c.gx, c.decay, c.ids, c.state, c.y))
    refused(lambda: c.rec.prefill(c.cu, c.x.half(), c.ga, c.gx, c.decay, c.ids, c.state, c.y))
    refused(lambda: c.rec.prefill(c.cu, c.x[:, ::2], c.ga, c.gx, c.decay, c.ids, c.state, c.y))
    refused(lambda: c.rec.prefill(c.cu[:0], c.x, c.ga, c.gx, c.decay, None, None, c.y))
    refused(lambda: c.rec.prefill(c.cu, c.x[:1].expand(c.T, 8), c.ga, c.gx, c.decay, c.ids, c.state, c.y), "overlap")
    refused(lambda: c.rec.step(c.ids, c.x[:2], c.ga[:2], c.gx[:2], c.decay, None, c.y[:2]))
    torch.cuda.synchronize()
    monkeypatch.setattr(LN, "_current_device", lambda: 1)
    for call in calls:
        refused(call, "current")


@pytest.mark.gpu
@pytest.mark.parametrize("rate", [0.0027, 0.0054, 0.0108, 0.0216])
def test_retentions_are_good_to_their_last_place(rate):
    """One step from a state of 1 with nothing coming in leaves the retention itself.  An open gate and decays of 16 and more,
    whose softplus is the decay in binary32, make its logarithm z = -rate log2(e) decay, in binary32 products.
    1 - a is then good to a step, 2^-24, of 2^z, or, up to |z| = 1/2, where it is -z times a polynomial s, to 1.5e-7 of itself: 1.4e-8
    of the polynomial, half a step of its last sum (2^-25 of 0.58 and more, 5.1e-8), of the product (2^-24), of its first coefficient (1.5e-8)
    and, halved and more, of the sums before (1e-8).  a is good to half a step, 2^-25, more."""
    import torch
    width = 4096
    decay = np.linspace(16.0, 32.0, width, endpoint=False).astype(np.float32)
    z = (np.float32(-rate) * np.float32(1.4426950408889634)) * decay
    assert z.dtype == np.float32 and z.min() >= -1.0
    rec = RC.GatedRecurrence(width, torch.float32, rate)
    x, ga = torch.zeros(1, width, device="cuda"), torch.full((1, width), float("inf"), device="cuda")
    state, y = torch.ones(1, width, device="cuda"), torch.empty(1, width, device="cuda")
    rec.step(torch.zeros(1, dtype=torch.int32, device="cuda"), x, ga, x, torch.from_numpy(decay).cuda(), state, y)
    torch.cuda.synchronize()
    z = z.astype(np.float64)
    error = np.abs(state[0].double().cpu().numpy() - np.exp2(z))
    room = np.where(z > -0.5, 1.5e-7 * -np.expm1(z * np.log(2.0)), 2.0 ** -24) + 2.0 ** -25
    assert np.all(error <= room), float((error / room).max())


def test_the_header_says_how_far_apart_tokens_may_lie(lib):
    text = HEADER.read_text()
    convention = text[text.index("A *_stride"):text.index("Outputs must not overlap")]
    assert "at most 2^24" in convention and RC.MAX_STRIDE == 2 ** 24 and "2^40" in convention and "2^38" in convention
    for status in (forward_status, backward_status):
        for name in ("xs", "gas", "gxs"):
            assert status(lib, **{name: RC.MAX_STRIDE + 1}) == S.STEPQ_ERR_INVALID_ARG


@pytest.mark.gpu
def test_tokens_too_far_apart_are_refused_with_the_reason():
    import torch
    c = Case([2], 8, "bf16", lead=0, tail=0)
    for stride, good in ((RC.MAX_STRIDE, True), (RC.MAX_STRIDE + 1, False)):
        far = torch.zeros(stride + 8, dtype=torch.bfloat16, device="cuda").as_strided((2, 8), (stride, 1))
        calls = (lambda: c.rec.prefill(c.cu, far, c.ga, c.gx, c.decay, c.ids, c.state, c.y),
                 lambda: c.rec.step(torch.arange(2, dtype=torch.int32, device="cuda"), far, c.ga, c.gx, c.decay, c.state, c.y))
        for call in calls:
            if good:
                call()
                continue
            with pytest.raises(S.StepqError, match="x's tokens may lie at most 16777216 elements apart") as e:
                call()
            assert e.value.status == S.STEPQ_ERR_INVALID_ARG
    torch.cuda.synchronize()

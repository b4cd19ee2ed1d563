"""Recurrence, norms and verification together: speculative sampling with random models against the same in
binary64 on the host, and a training step of two blocks against differentiation in binary64.

Sampling.  Every choice has to be the same, so no random number may lie within GAP of a border between two outcomes:
logits are good to some 1e-5 here, probabilities to the same of themselves."""
import numpy as np
import pytest

import norm_ref
import scan_ref
import test_draft
from quantized_recurrent_state_packed_amd import build_lib
from quantized_recurrent_state_packed_amd import generate as G
from quantized_recurrent_state_packed_amd import stepq as S

GAP = 3e-5
EPS = 1e-6


class Plain:
    """A RecurrentModel's logits in binary64, from the tokens alone."""

    def __init__(self, model):
        self.m = model
        self.w = {n: [t.double().cpu().numpy() for t in getattr(model, n)] for n in ("inner", "decay", "post", "scale", "pre")}
        self.embedding, self.first, self.head = (getattr(model, n).double().cpu().numpy() for n in ("embedding", "first", "head"))

    def logits(self, tokens):
        stream = self.embedding[tokens]
        y = stream * norm_ref.root(stream, EPS) * self.first
        for n in range(self.m.layers):
            x, ga, gx, z = (y @ self.w["inner"][n]).reshape(len(tokens), 4, -1).transpose(1, 0, 2)
            h, _ = scan_ref.forward(x, ga, gx, self.w["decay"][n], 8.0, np.zeros(self.m.width))
            stream, y, _, _ = norm_ref.forward(h, z, stream, self.w["post"][n], self.w["scale"][n], self.w["pre"][n], "silu", True,
                                               True, EPS)
        return y @ self.head


def models(seed, same=False, device="cuda"):
    target = G.RecurrentModel(53, 24, layers=3, seed=seed, device=device)
    return target, target.first_layers(3 if same else 2)


def prompts(seed):
    g = np.random.default_rng(seed)
    return [g.integers(0, 53, size=n).tolist() for n in (130, 1, 7, 2)]


def speculate(target, draft, prompt, uniforms, temperature, K):
    """Rounds for one request; the smallest distance of a random number from a border."""
    t = np.float32(temperature)
    seq, gap, accepted = list(prompt), np.inf, []
    for u in uniforms:
        drafts, z = [], []
        for n in range(K):
            z.append(draft.logits(np.array(seq + drafts))[-1])
            _, tok, g = test_draft.verify(z[-1][None, None], None, np.empty((1, 0), int), u[None, n:n + 1], None, np.array([t]))
            if not t > 0:
                top = np.sort(z[-1])
                g = min(g, top[-1] - top[-2])
            drafts.append(int(tok[0, 0]))
            gap = min(gap, g)
        x = target.logits(np.array(seq + drafts))[len(seq) - 1:]
        if not t > 0:
            top = np.sort(x, axis=-1)
            gap = min(gap, (top[:, -1] - top[:, -2]).min())
        acc, tok, g = test_draft.verify(x[None], np.array(z)[None], np.array([drafts]), u[None, K:], None, np.array([t]))
        gap = min(gap, g)
        seq += tok[0, :acc[0] + 1].tolist()
        accepted.append(int(acc[0]))
    return seq[len(prompt):], accepted, gap


@pytest.mark.gpu
@pytest.mark.parametrize("temperature,seed", [(1.0, 1), (0.6, 2), (0.0, 1), (0.0, 2)])
def test_speculative_sampling_equals_that_in_64_bits(temperature, seed):
    import torch
    K, rounds = 3, 4
    target, draft = models(seed)
    gen = G.DraftGenerator(target, draft, 4, K, temperature)
    u = torch.from_numpy(np.random.default_rng(seed).random((rounds, 4, 2 * K + 1)).astype(np.float32)).cuda()
    ps = prompts(seed)
    last, got = gen.prefill(ps), [[] for _ in ps]
    for r in range(rounds):
        accepted, out = gen.round(last, u[r])
        last = out.gather(1, accepted.long()[:, None])[:, 0].long()
        for s, n, row in zip(got, accepted.tolist(), out.tolist()):
            s += row[:n + 1]
    pt, pd = Plain(target), Plain(draft)
    for b, p in enumerate(ps):
        want, _, gap = speculate(pt, pd, p, u[:, b].cpu().numpy(), temperature, K)
        assert gap > GAP, "the inputs put a random number too close to a border"
        assert got[b] == want, b


@pytest.mark.gpu
def test_a_draft_model_that_is_the_target_is_accepted():
    """p and q differ by rounding alone, of 1e-5 at most here: a draft is rejected with that probability."""
    target, draft = models(3, same=True)
    sequences, share = G.DraftGenerator(target, draft, 4, 5).run(prompts(3), 40)
    assert share > 0.98 and [len(s) for s in sequences] == [40] * 4


@pytest.mark.gpu
def test_prompts_of_single_tokens():
    """Nothing to run through before the first round."""
    target, draft = models(2)
    sequences, _ = G.DraftGenerator(target, draft, 3, 2).run([[5], [0], [52]], 6)
    assert [len(s) for s in sequences] == [6] * 3 and all(0 <= t < 53 for s in sequences for t in s)


@pytest.mark.gpu
def test_greedy_sampling_is_the_targets_own_whatever_the_draft():
    target, draft = models(1)
    sequences, _ = G.DraftGenerator(target, draft, 4, 4, temperature=0.0).run(prompts(1), 8)
    plain = Plain(target)
    for p, s in zip(prompts(1), sequences):
        seq = list(p)
        for t in s:
            x = np.sort(plain.logits(np.array(seq))[-1])
            assert x[-1] - x[-2] > GAP, "two tokens lie too close together"
            seq.append(int(np.argmax(plain.logits(np.array(seq))[-1])))
        assert s == seq[len(p):]


@pytest.mark.parametrize("bad,why", [([[1], [2]], "4 non-empty"), ([[1], [2], [], [3]], "4 non-empty"),
                                     ([[1], [53], [2], [3]], "vocabulary"), ([[1], [5], [2], [-1]], "vocabulary")])
def test_prompts_that_are_refused(bad, why):
    if not S.LIB_PATH.exists():
        build_lib.build()
    gen = G.DraftGenerator(*models(0, device="cpu"), 4, 2)
    with pytest.raises(S.StepqError, match=why) as e:
        gen.prefill(bad)
    assert e.value.status == S.STEPQ_ERR_INVALID_ARG


def test_generators_that_are_refused():
    if not S.LIB_PATH.exists():
        build_lib.build()
    target, draft = models(0, device="cpu")
    other = G.RecurrentModel(54, 10, layers=1, device="cpu")
    for args in ((target, other, 4, 2), (target, draft, 4, 0), (target, draft, 0, 2), (target, draft, 4, 64)):
        with pytest.raises(S.StepqError):
            G.DraftGenerator(*args)


# ----------------------------------------------------------------- training

def plain_loss(torch, params, tokens_x, cu, weight):
    """Two blocks, each request token by token, in binary64."""
    stream = tokens_x
    normed = stream / torch.sqrt((stream * stream).mean(-1, keepdim=True) + EPS)
    for w, decay, post, scale, pre in params:
        x, ga, gx, z = (normed @ w).view(len(stream), 4, -1).unbind(1)
        a = torch.exp(-8.0 * torch.sigmoid(ga) * torch.nn.functional.softplus(decay))
        u = torch.sqrt(1.0 - a * a) * torch.sigmoid(gx) * x
        rows = []
        for lo, hi in zip(cu[:-1], cu[1:]):
            h = torch.zeros_like(u[0])
            for t in range(lo, hi):
                h = a[t] * h + u[t]
                rows.append(h)
        h = torch.stack(rows)
        p = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * post * z * torch.sigmoid(z)
        stream = stream + scale * p
        normed = stream / torch.sqrt((stream * stream).mean(-1, keepdim=True) + EPS) * pre
    return (normed * weight).sum()


@pytest.mark.gpu
def test_a_training_step_of_two_blocks():
    """Gradients of a loss over two blocks by the library's backward passes, against differentiation in binary64.

    A block's results are good to some 1e-6 of their size in binary32 and a gradient adds up products of both
    signs over 300 tokens and two blocks: 2e-4 of a gradient's norm is far above that, and far below what a wrong term
    would leave."""
    import torch
    from quantized_recurrent_state_packed_amd.norm import BlockNorm
    from quantized_recurrent_state_packed_amd.recurrence import GatedRecurrence
    D, cu_host = 40, [0, 150, 150, 151, 300]
    T = cu_host[-1]
    g = torch.Generator().manual_seed(5)

    def rand(*shape, scale=1.0, shift=0.0):
        return shift + scale * torch.randn(*shape, generator=g)

    params = [[rand(D, 4 * D, scale=D ** -0.5), rand(D, scale=1.0, shift=-4.0), rand(D, scale=0.1, shift=1.0),
               rand(D, scale=0.1, shift=0.7), rand(D, scale=0.1, shift=1.0)] for _ in range(2)]
    tokens_x, weight = rand(T, D), rand(T, D)
    want = [[p.double().requires_grad_(True) for p in layer] for layer in params]
    x64 = tokens_x.double().requires_grad_(True)
    plain_loss(torch, want, x64, cu_host, weight.double()).backward()

    dev = [[p.cuda() for p in layer] for layer in params]
    cu = torch.tensor(cu_host, dtype=torch.int32, device="cuda")
    rec, opening, norm = GatedRecurrence(D), BlockNorm(D, post=False), BlockNorm(D)
    ws, nws = rec.workspace(4, T), norm.workspace(T)
    streams, normeds, saved, inner, hs = [tokens_x.cuda()], [], [], [], []
    normeds.append(torch.empty_like(streams[0]))
    opening.forward(streams[0], None, normeds[0])
    for w, decay, post, scale, pre in dev:
        v = (normeds[-1] @ w).view(T, 4, D)
        x, ga, gx, z = v.unbind(1)
        h, out, normed = (torch.empty_like(streams[0]) for _ in range(3))
        saved.append(rec.saved(4, T))
        rec.prefill(cu, x, ga, gx, decay, None, None, h, saved=saved[-1], workspace=ws)
        norm.forward(h, out, normed, gate=z, residual=streams[-1], post_weight=post, scale=scale, pre_weight=pre)
        inner.append(v), hs.append(h), streams.append(out), normeds.append(normed)
    d_stream, d_normed, got = None, weight.cuda(), [None, None]
    for n in (1, 0):
        w, decay, post, scale, pre = dev[n]
        x, ga, gx, z = inner[n].unbind(1)
        dv = torch.empty_like(inner[n])
        dx, dga, dgx, dz = dv.unbind(1)
        dh, d_res = torch.empty_like(hs[n]), torch.empty_like(hs[n])
        dp, ds, dpre, dd = (torch.empty(D, device="cuda") for _ in range(4))
        norm.backward(hs[n], streams[n + 1], d_stream, dh, d_normed=d_normed, gate=z, d_gate=dz, d_residual=d_res, post_weight=post,
                      d_post_weight=dp, scale=scale, d_scale=ds, pre_weight=pre, d_pre_weight=dpre, workspace=nws)
        rec.backward(cu, x, ga, gx, decay, saved[n], dh, dx, dga, dgx, dd, workspace=ws)
        flat = dv.view(T, 4 * D)
        got[n] = [normeds[n].t() @ flat, dd, dp, ds, dpre]
        d_stream, d_normed = d_res, flat @ w.t()
    d_x = torch.empty_like(d_stream)
    opening.backward(streams[0], streams[0], None, d_x, d_normed=d_normed)
    torch.cuda.synchronize()
    pairs = [(d_x + d_stream, x64.grad)] + [(a, b.grad) for la, lb in zip(got, want) for a, b in zip(la, lb)]
    for a, b in pairs:
        a = a.double().cpu()
        assert float((a - b).norm()) <= 2e-4 * float(b.norm())


@pytest.mark.gpu
def test_a_rounds_results_stay_behind_the_next_one():
    import torch
    target, draft = models(2)
    gen = G.DraftGenerator(target, draft, 4, 3)
    u = torch.from_numpy(np.random.default_rng(6).random((3, 4, 7)).astype(np.float32)).cuda()
    last, results, copies = gen.prefill(prompts(2)), [], []
    for r in range(3):
        accepted, out = gen.round(last, u[r])
        results.append((accepted, out))
        copies.append((accepted.clone(), out.clone()))
        last = out.gather(1, accepted.long()[:, None])[:, 0].long()
    torch.cuda.synchronize()
    for kept, copy in zip(results, copies):
        assert all(torch.equal(a, b) for a, b in zip(kept, copy))

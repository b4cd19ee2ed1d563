"""The whole path, prompts to beams, against a plain beam search in binary64 that
gathers full states: with every row of the layout 32 bits wide the packed slots
hold the states themselves, so the sequences have to be the same.  The inputs are
such that no two candidates that matter lie within 1e-3 of each other, which is
far more than the binary32 path's error (scores agree to 1e-3)."""
import numpy as np
import pytest

from linear_ref import recurrence
from quantized_recurrent_state_packed_amd import generate as G
from quantized_recurrent_state_packed_amd import stepq as S


def plain(model, prompts, beams, steps, eos):
    """Sequences and scores by the definition, and the smallest gap between candidates that were compared."""
    w = {n: [t.double().cpu().numpy() for t in getattr(model, n)] for n in ("qkv", "rates", "out")}
    emb, head = (t.double().cpu().numpy() for t in (model.embedding, model.head))
    H, D = model.H, model.D

    def run(tokens, states):
        x = emb[tokens]
        new = []
        for n in range(model.layers):
            q, k, v = (x @ w["qkv"][n]).reshape(-1, 3, H, D).transpose(1, 0, 2, 3)
            q, k = (t / np.linalg.norm(t, axis=-1, keepdims=True) for t in (q, k))
            beta, gate = (1 / (1 + np.exp(-(x @ w["rates"][n])))).reshape(-1, 2, H).transpose(1, 0, 2)
            o, m = recurrence(q, k, v, beta, 0.5 + 0.5 * gate, states[n])
            new.append(m)
            y = x + o.reshape(len(tokens), -1) @ w["out"][n]
            x = y / np.sqrt((y ** 2).mean(-1, keepdims=True))
        z = x[-1] @ head
        z -= z.max()
        return z - np.log(np.exp(z).sum()), new

    out, gap = [], np.inf
    for p in prompts:
        logp, st = run(np.array(p), [np.zeros((H, D, D))] * model.layers)
        alive = [(0.0, [], logp, st, False)]
        for t in range(steps):
            cands = []
            for i, (s, seq, lp, st, done) in enumerate(alive):
                if done:
                    cands.append((s, i, eos))
                else:
                    cands += [(s + lp[v], i, v) for v in range(len(lp))]
            cands.sort(key=lambda c: -c[0])
            top = cands[:beams + 1]
            gap = min([gap] + [a[0] - b[0] for a, b in zip(top, top[1:])])
            nxt = []
            for s, i, v in cands[:beams]:
                _, seq, _, st, done = alive[i]
                lp, new = (None, st) if done or v == eos else run(np.array([v]), st)
                nxt.append((s, seq + [v], lp, new, done or v == eos))
            alive = nxt
        out.append(alive)
    return [[a[1] for a in x] for x in out], np.array([[a[0] for a in x] for x in out]), gap


def make(beams, eos, seed, device="cuda"):
    model = G.RandomModel(vocab=61, width=24, layers=2, heads=3, d=16, seed=seed, device=device)
    g = np.random.default_rng(seed)
    prompts = [g.integers(1, 61, size=n).tolist() for n in (70, 1, 5)]
    return model, prompts


@pytest.mark.gpu
@pytest.mark.parametrize("beams,eos,seed", [(1, 25, 1), (3, 55, 3), (4, 42, 2)])
def test_sequences_equal_those_of_a_plain_beam_search(beams, eos, seed):
    model, prompts = make(beams, eos, seed)
    want, scores, gap = plain(model, prompts, beams, 6, eos)
    assert gap > 1e-3, "the inputs put two candidates too close together"
    layout = S.Layout(3, 16, 0, np.full(3, 32, np.uint8), np.ones(48, np.float32), S.ROW_SCALES_REFIT)
    got, s = G.BeamGenerator(model, len(prompts), beams, layout, eos_token=eos).run(prompts, 6)
    assert got.cpu().tolist() == want
    assert np.abs(s.cpu().numpy() - scores).max() <= 1e-3


@pytest.mark.gpu
def test_six_bit_slots_stay_close_to_full_states():
    """Six-bit states give scores near those of full states on a short run (the
    quantised states are another model: only closeness is asked for)."""
    model, prompts = make(3, 0, 3)
    s = []
    for bits in (32, 6):
        layout = S.Layout(3, 16, 0, np.full(3, bits, np.uint8), np.ones(48, np.float32), S.ROW_SCALES_REFIT)
        s.append(G.BeamGenerator(model, len(prompts), 3, layout, eos_token=0).run(prompts, 4)[1].cpu().numpy())
    assert np.isfinite(s[1]).all() and np.abs(s[0] - s[1]).max() < 1.0

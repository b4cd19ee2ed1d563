"""Linear attention with one decay per head, token by token in binary64, and its
inputs: the plain implementation the chunked and single-token kernels are tested
against."""
import numpy as np


def recurrence(q, k, v, beta, gate, m):
    """q, k [T, Hk, D], v [T, H, D], beta [T, H] or None, gate [T, H], m [H, D, D] -> (o, m), all float64."""
    h = v.shape[1]
    rep = h // q.shape[1]
    q, k, v, gate = (np.asarray(x, np.float64) for x in (q, k, v, gate))
    m = np.array(m, np.float64)
    o = np.zeros_like(v)
    for t in range(v.shape[0]):
        kt, qt = np.repeat(k[t], rep, 0), np.repeat(q[t], rep, 0)
        m = gate[t][:, None, None] * m
        u = v[t] if beta is None else np.asarray(beta[t], np.float64)[:, None] * (v[t] - np.einsum("hij,hi->hj", m, kt))
        m = m + kt[:, :, None] * u[:, None, :]
        o[t] = np.einsum("hij,hi->hj", m, qt)
    return o, m


def inputs(seed, tokens, H, Hk, D, correlated=0.0, gates="mixed"):
    """float32 arrays: unit q and k (sharing a direction where `correlated`), normal v."""
    g = np.random.default_rng(seed)

    def unit(n):
        x = g.standard_normal((tokens, n, D)) + correlated * np.sqrt(D)
        return (x / np.linalg.norm(x, axis=-1, keepdims=True)).astype(np.float32)

    gate = {"mixed": lambda: 2.0 ** (-1.0 / 10.0 ** g.uniform(0, 3, (tokens, H))),
            "one": lambda: np.ones((tokens, H)),
            "strong": lambda: 10.0 ** g.uniform(-30, -1, (tokens, H)),
            "clearing": lambda: np.where(g.random((tokens, H)) < 0.1, 0.0, g.uniform(0.5, 1.0, (tokens, H)))}[gates]()
    return dict(q=unit(Hk), k=unit(Hk), v=g.standard_normal((tokens, H, D)).astype(np.float32),
                beta=(1.0 / (1.0 + np.exp(-g.standard_normal((tokens, H))))).astype(np.float32),
                gate=gate.astype(np.float32))

"""The norms around a block in 64 bits, their gradients, and bounds of both's rounding
errors in binary32.

Bounds.  With e = 2^-24 and z the gate: a sum of squares takes at most 32 additions in a lane
and 14 across lanes, so it is good to 46 e and a reciprocal root to 23 e + 4 e; act(z) is good
to (|z| + 6) e (the product with log2 e, exp2, a quotient, a product).  So p = n act(z) is good to
A = (40 + max |z|) e, t to A |scale p| + e |t|, and y to that times r2 weight plus 30 e and the relative
change of the root.  A gradient adds a sum over products of both signs, good to 46 e of the sum
of sizes, and three times as many factors: 4 A + 150 e of the same formula over sizes.
z (1 - s(z)) in silu's slope is off by |z| times the error of s."""
import numpy as np

EPS = 2.0 ** -24


def sigmoid(x):
    return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def act_of(z, name):
    """act(z), its slope, and the sizes of the slope's terms."""
    if z is None:
        return 1.0, 0.0, 0.0
    s = sigmoid(z)
    if name == "sigmoid":
        return s, s * (1 - s), s * (1 - s) + 16 * s
    return z * s, s * (1 + z * (1 - s)), s * (1 + np.abs(z) * (1 - s)) + s * np.abs(z) * (np.abs(z) + 16)


def root(x, eps):
    return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def forward(o, z, x, w1, sc, w2, act, post, pre, eps):
    """Rows [N, width]: t, y (None without pre) and bounds of their errors."""
    r1 = root(o, eps) if post else 1.0
    p = o * r1 * w1 * act_of(z, act)[0]
    t = sc * p + (0.0 if x is None else x)
    A = (40.0 + (0.0 if z is None else np.abs(z).max())) * EPS
    dt = A * np.abs(sc * p) + EPS * np.abs(t)
    if not pre:
        return t, None, dt, None
    r2 = root(t, eps)
    norm = np.sqrt((t * t).sum(-1, keepdims=True))
    change = np.sqrt((dt * dt).sum(-1, keepdims=True)) / np.maximum(norm, 1e-300)
    return t, t * r2 * w2, dt, np.abs(w2) * r2 * (dt + np.abs(t) * (32 * EPS + change))


def backward(o, z, t, w1, sc, w2, act, post, pre, eps, dt, dy):
    """Gradients and bounds of their errors; t is what the forward pass wrote."""
    n_rows, width = o.shape
    g = np.zeros_like(o) if dt is None else dt.astype(np.float64)
    G = np.abs(g)
    out, room = {}, {}
    A = (40.0 + (0.0 if z is None else np.abs(z).max())) * EPS
    F = 4 * A + 150 * EPS
    S = F + n_rows * EPS              # of sums over rows
    if pre:
        r2 = root(t, eps)
        v = w2 * dy
        g = g + r2 * v - t * r2 ** 3 * (t * v).mean(-1, keepdims=True)
        G = G + r2 * np.abs(v) + np.abs(t) * r2 ** 3 * np.abs(t * v).mean(-1, keepdims=True)
        out["dpre"], room["dpre"] = (dy * t * r2).sum(0), S * np.abs(dy * t * r2).sum(0)
    out["dresidual"], room["dresidual"] = g, F * G
    r1 = root(o, eps) if post else np.ones((n_rows, 1))
    a, slope, slopes = act_of(z, act)
    n = o * r1 * w1
    out["dscale"], room["dscale"] = (g * n * a).sum(0), S * (G * np.abs(n * a)).sum(0)
    q, Q = g * sc, G * np.abs(sc)
    if z is not None:
        out["dgate"], room["dgate"] = q * n * slope, np.abs(n) * Q * (F * np.abs(slope) + (A + 16 * EPS) * slopes)
    k, K = q * a, Q * np.abs(a)
    out["dpost"], room["dpost"] = (k * o * r1).sum(0), S * (K * np.abs(o * r1)).sum(0)
    m, M = k * w1, K * np.abs(w1)
    back, Back = 0.0, 0.0
    if post:
        back = o * r1 ** 3 * (o * m).mean(-1, keepdims=True)
        Back = np.abs(o) * r1 ** 3 * np.abs(o * M).mean(-1, keepdims=True)
    out["dblock"], room["dblock"] = r1 * m - back, F * (r1 * M + Back)
    return out, room

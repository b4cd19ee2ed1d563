"""The gated linear recurrence in 64 bits, token by token, its gradients by the
adjoint recurrence, and bounds of both's rounding errors in binary32.

Bounds.  With e = 2^-24 and m the largest gate in size: a logistic function's relative
error is at most (m + 4) e (the product with log2 e, exp2 and the quotient), so 1 - a and the inputs u are
good to F = (40 + 2 m) e of themselves, and after n tokens a state to (2 F + 2 n e) times the
same sum of absolute values: the retentions' errors act over at most 1 / (1 - a) tokens, and
every token rounds twice.  Gradients are products of two such sums and twice as many factors.
"""
import numpy as np

EPS = 2.0 ** -24


def sigmoid(x):
    with np.errstate(over="ignore"):
        return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def softplus(x):
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def gates(x, ga, gx, decay, rate):
    ra, ri = sigmoid(ga), sigmoid(gx)
    la = -rate * ra * softplus(decay)
    a, b = np.exp(la), np.sqrt(-np.expm1(2.0 * la))
    return ra, ri, la, a, b, b * ri * x


def forward(x, ga, gx, decay, rate, h0):
    """[T, D] each, h0 [D]: (y [T, D], the same recurrence over absolute values)."""
    _, _, _, a, _, u = gates(x, ga, gx, decay, rate)
    h, m = h0.astype(np.float64).copy(), np.abs(h0)
    y, size = np.empty_like(u), np.empty_like(u)
    for t in range(len(u)):
        h, m = a[t] * h + u[t], a[t] * m + np.abs(u[t])
        y[t], size[t] = h, m
    return y, size


def factor(ga, gx):
    both = np.concatenate([np.abs(ga).ravel(), np.abs(gx).ravel(), [0.0]])
    return 40.0 + 2.0 * both[np.isfinite(both)].max()


def state_bound(size, ga, gx):
    return (2.0 * factor(ga, gx) + 2.0 * len(ga)) * EPS * size


def backward(x, ga, gx, decay, rate, h0, dy, dend):
    """Gradients (dx, dga, dgx, ddecay, dh0) and bounds of their errors."""
    ra, ri, la, a, b, u = gates(x, ga, gx, decay, rate)
    y, size = forward(x, ga, gx, decay, rate, h0)
    prior, prior_size = np.concatenate([h0[None], y[:-1]])[:len(u)], np.concatenate([np.abs(h0)[None], size[:-1]])[:len(u)]
    with np.errstate(divide="ignore", invalid="ignore"):
        slope = np.where(b > 0, la / b, 0.0)
    g, gs = np.empty_like(u), np.empty_like(u)
    c, cs = dend.astype(np.float64).copy(), np.abs(dend)
    for t in range(len(u) - 1, -1, -1):
        g[t], gs[t] = dy[t] + c, np.abs(dy[t]) + cs
        c, cs = a[t] * g[t], a[t] * gs[t]
    gain = ri * x
    P = g * a * (prior * la - a * gain * slope)
    Ps = gs * a * (prior_size * np.abs(la) + a * np.abs(gain * slope))
    soft, open_ = softplus(decay), sigmoid(decay)
    ratio = np.where(soft > 0, open_ / np.where(soft > 0, soft, 1.0), 1.0)
    grads = dict(dx=g * b * ri, dga=P * (1 - ra), dgx=g * u * (1 - ri), ddecay=P.sum(0) * ratio, dh0=c)
    F = (4.0 * factor(ga, gx) + 4.0 * len(u)) * EPS if len(u) else 0.0
    # 1 - s is off by the error of s where s is close to 1
    bounds = dict(dx=F * gs * b * ri, dga=Ps * (F * (1 - ra) + 16 * EPS), dgx=gs * np.abs(u) * (F * (1 - ri) + 16 * EPS),
                  ddecay=F * Ps.sum(0) * ratio, dh0=F * cs)
    return grads, bounds

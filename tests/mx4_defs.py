"""Microscaled 4-bit floats and the balance loss by their definitions, in numpy and 64 bits. Shares no code with
the package."""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode(v):
    """Codes [rows, K/2] and scales [rows, K/32] of values [rows, K] in 64 bits; a value of 2^128 or more, an infinity
    or a NaN makes its block NaN."""
    v = np.asarray(v, np.float64)
    rows, K = v.shape
    b = v.reshape(rows, K // 32, 32)
    bad = ~(np.abs(b) < 2.0 ** 128).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    m = np.abs(b).max(axis=2)
    e = np.where(m > 0, np.frexp(np.where(m > 0, m, 1.0))[1] - 1, -200)
    e = np.maximum(e - 2, -127)
    y = np.ldexp(np.abs(b), -e[:, :, None])
    # the nearest magnitude: of two that are equally near, the one whose code is even
    d = np.abs(y[..., None] - MAGNITUDES)
    near = d.argmin(axis=-1)  # (the lower of two)
    up = np.minimum(near + 1, 7)
    tie = np.take_along_axis(d, up[..., None], -1)[..., 0] == np.take_along_axis(d, near[..., None], -1)[..., 0]
    code = np.where(tie & (near % 2 == 1), up, near) + 8 * np.signbit(b)
    code = np.where(bad[:, :, None], 0, code).astype(np.uint8).reshape(rows, K // 2, 2)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, :, 0] | code[:, :, 1] << 4, scales


def decode(q, s):
    """The values [rows, K] of codes and scales, in 64 bits."""
    q, s = np.asarray(q), np.asarray(s)
    c = np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return v * np.repeat(scale, 32, axis=-1)


def silu_mul(x):
    g, u = np.split(np.asarray(x, np.float64), 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def balance(logits, ids, mask, sigmoid, alpha, up=1.0, counts=None):
    """(loss, counts [E + 1], prob_sums, gradient) of a batch; counts: others than the batch's own for the gradient."""
    l = np.asarray(logits, np.float64)
    M, E = l.shape
    k = ids.shape[1]
    there = ~np.isnan(l) & (l > -np.inf)
    use = there.any(axis=1) & (True if mask is None else np.asarray(mask, bool))
    p, q = np.zeros((M, E)), np.ones((M, E))
    for m in np.flatnonzero(use):
        x = l[m, there[m]]
        if sigmoid:
            # sigmoids over exp(min(max, 0)), which leaves their ratios
            sh = min(x.max(), 0.0)
            with np.errstate(over="ignore"):
                w = np.where(x > 0, 1 / (1 + np.exp(-x)), np.exp(np.minimum(x, 0) - sh) / (1 + np.exp(np.minimum(x, 0))))
                q[m, there[m]] = 1 / (1 + np.exp(x))
        elif x.max() == np.inf:
            w = (x == np.inf).astype(float)
        else:
            w = np.exp(x - x.max())
        p[m, there[m]] = w / w.sum()
    own = np.zeros(E + 1, np.int64)
    for m in np.flatnonzero(use):
        for e in ids[m]:
            if 0 <= e < E:
                own[e] += 1
    own[E] = use.sum()
    n = own[E]
    loss = alpha * E / (k * n * n) * (own[:E] * p.sum(axis=0)).sum() if n else 0.0
    c = own if counts is None else np.asarray(counts, np.int64)
    a = up * alpha * E / (k * float(c[E]) ** 2) * c[:E] if c[E] > 0 else np.zeros(E)
    grad = p * q * (a - (p @ a)[:, None])
    return loss, own, p.sum(axis=0), grad

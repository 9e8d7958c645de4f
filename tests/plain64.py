"""Plain 64-bit definitions (numpy) of the routed operators around the delta path, written from
their formulas: the router, 4-bit weights, and a whole mixture-of-experts layer. Test-only."""
import numpy as np


def router(logits, topk, sigmoid=False, renorm=True, scale=1.0, first=0, local=None):
    """ids int64 [M, topk], weights float64 [M, topk] of logits [M, E] (any float values)."""
    l = np.asarray(logits, np.float64)
    M, E = l.shape
    local = E if local is None else local
    ids = np.full((M, topk), -1, np.int64)
    w = np.zeros((M, topk))
    for i in range(M):
        cand = [e for e in range(E) if not np.isnan(l[i, e]) and l[i, e] != -np.inf]
        if not cand:
            continue
        order = sorted(cand, key=lambda e: (-l[i, e], e))[:topk]
        lo = l[i, order]
        m = l[i, cand].max()
        if sigmoid:
            with np.errstate(over="ignore"):
                p = 1.0 / (1.0 + np.exp(-lo))
            if renorm and p.sum() == 0:  # ratios survive: exp(l - m) / (1 + exp(l))
                p = np.exp(lo - m)
        elif np.isinf(m):
            p = (lo == m) / np.sum(l[i, cand] == m)
        else:
            p = np.exp(lo - m) / np.exp(l[i, cand] - m).sum()
        if renorm:
            p = p / p.sum()
        for j, e in enumerate(order):
            if first <= e < first + local:
                ids[i, j], w[i, j] = e - first, p[j] * scale
    return ids, w


def dequantise(W, scales, zeros=None):
    """float64 weights [.., N, K] of packed 4-bit W [.., N, K/2], and |q + c| + |c + z| times the
    scale with c = 16: the largest magnitudes the sums of a group may run through."""
    W = np.asarray(W, np.uint8)
    s = np.asarray(scales, np.float64)
    q = np.stack((W % 16, W // 16), axis=-1).reshape(*W.shape[:-1], -1).astype(np.float64)
    G = q.shape[-1] // s.shape[-1]
    z = np.full(s.shape, 8.0) if zeros is None else np.asarray(zeros, np.float64)
    s, z = np.repeat(s, G, axis=-1), np.repeat(z, G, axis=-1)
    return (q - z) * s, (q + 32 + z) * np.abs(s)


U24 = 2.0 ** -24  # half an ulp of fp32, relative


def product(W, mag, x):
    """x W^T in 64 bits, and a bound on the fp32 sum's error: every one of the K products and
    sums rounds at most once to half a unit of a partial sum no larger than sum |W| |x|; a few
    more roundings for the scales and the cross-wave sum."""
    K = x.shape[-1]
    return x @ W.T, (K + 16) * U24 * (np.abs(x) @ mag.T)


def layer(x, gate_up, down, ids, weights, eps, adapters=None, lora=None, rows_rounded=False):
    """y [M, H] of a whole layer in 64 bits, and a bound on what an implementation with fp32 sums
    and y rounded to a type of half-ulp eps / 2 may be off by. Where that type is bf16, h and the
    adapters' s enter their products as two bf16 terms: the first is cut off to 8 bits, which
    leaves less than 2^-7 of the value, and that is rounded to 8 bits, so 2^-16 of the value is
    lost at most (or, as the second term may fall below the smallest normal number, 2^-126).
    gate_up and down: functions
    from an expert to (W, magnitudes). adapters: (A1, B1, A2, B2, scale, ranks or None). rows_rounded: each
    stage's rows, and h, are rounded to the type before and after the adapter part is added."""
    M, k = ids.shape
    half = eps / 2
    cut = 2.0 ** -16 if eps > 1e-6 else 0.0
    tiny = 2.0 ** -126
    y = err = None
    for m in range(M):
        for j in range(k):
            t = int(ids[m, j])
            W1, mag1 = gate_up(t) if t >= 0 else (None, None)
            if W1 is None:
                continue
            W2, mag2 = down(t)
            if y is None:
                y, err = np.zeros((M, W2.shape[0])), np.zeros((M, W2.shape[0]))
            I = W2.shape[1]
            gu, egu = product(W1, mag1, x[m])
            if rows_rounded:
                egu = egu * (1 + half) + half * np.abs(gu)
            l = -1 if lora is None else int(lora[m])
            rl = 0
            if adapters is not None and 0 <= l < len(adapters[4]):
                A1, B1, A2, B2, scale, ranks = adapters
                E, r = A1.shape[0] // len(scale), A2.shape[1]
                rl = r if ranks is None else min(max(int(ranks[l]), 0), r)
            if rl:
                v, c = t + l * E, float(scale[l])
                for part, rows in ((slice(0, I), slice(0, rl)), (slice(I, 2 * I), slice(r, r + rl))):
                    s, es = product(A1[v, rows], np.abs(A1[v, rows]), x[m])
                    es = es + cut * (np.abs(s) + es) + tiny
                    d, ed = product(B1[v, part, :rl], np.abs(B1[v, part, :rl]), s)
                    gu[part] += c * d
                    egu[part] += abs(c) * (ed + es @ np.abs(B1[v, part, :rl]).T) + 2 * U24 * np.abs(c * d)
            if rows_rounded:
                egu = egu * (1 + half) + half * np.abs(gu)
            g, u = gu[:I], gu[I:]
            with np.errstate(over="ignore"):
                silu = g / (1 + np.exp(-g))
            h = silu * u
            eh = (1.1 * egu[:I] * np.abs(u) + np.abs(silu) * egu[I:] + 1.1 * egu[:I] * egu[I:] +
                  16 * U24 * np.abs(h))
            eh = eh + (half if rows_rounded else cut) * (np.abs(h) + eh) + tiny
            z, ez = product(W2, mag2, h)
            ez = ez + eh @ np.abs(W2).T * (1 + 1e-3)
            if rows_rounded:
                ez = ez * (1 + half) + half * np.abs(z)
            if rl:
                s, es = product(A2[v, :rl], np.abs(A2[v, :rl]), h)
                es = es + eh @ np.abs(A2[v, :rl]).T
                es = es + cut * (np.abs(s) + es) + tiny
                d, ed = product(B2[v, :, :rl], np.abs(B2[v, :, :rl]), s)
                z = z + c * d
                ez = ez + abs(c) * (ed + es @ np.abs(B2[v, :, :rl]).T) + 2 * U24 * np.abs(c * d)
            if rows_rounded:
                ez = ez * (1 + half) + half * np.abs(z)
            w = float(weights[m, j])
            y[m] += w * z
            err[m] += abs(w) * ez + (k + 4) * U24 * np.abs(w * z)
    if y is None:
        return None, None
    # the last rounding, a denormal's absolute step included
    return y, err * (1 + half) + half * np.abs(y) + 2.0 ** -134


def within(got, ref, bound, what=""):
    """got is finite and within bound of ref, element by element."""
    got = np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), what
    off = np.abs(got - ref) - bound
    at = np.unravel_index(np.argmax(off), off.shape)
    assert off[at] <= 0, f"{what}: at {at} got {got[at]}, want {ref[at]} +- {bound[at]}"

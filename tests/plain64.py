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

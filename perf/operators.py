"""The routed mixture-of-experts operators that are timed: their cases, inputs, plain forms and 64-bit definitions.

Three operators of one layer, in the order a serving step runs them:

  router  logits -> the top-k experts of each token and their weights (mol_router_topk)
  q4      the base grouped product of one stage over 4-bit weights with group scales (mol_moe_gemm_q4)
  layer   a whole layer for a few tokens: gate/up, SiLU, down and combine, with LoRA adapters (mol_moe_layer)

Sizes are those of this repository's synthetic layers (hidden 2048 with 128 experts of 768, top-8, 8 or 16 adapter slots of
rank 32; hidden 6144 with 160 experts of 256; the 64-wide fp32 layer) and odd ones near them.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK_M = 64


def _binding():
    from virtual_expert_routed_amd import binding
    return binding


# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # one decoding token: the latency of the launch
        dict(name="router_1", op="router", dtype="bf16", M=1, E=128, topk=8, scoring="softmax", renorm=True, scale=1.0,
             masked=0.0, first=0, local=128),
        # a decode batch on one of two expert-parallel GPUs, sigmoid scores, an odd batch and some masked experts
        dict(name="router_138_ep", op="router", dtype="f32", M=138, E=160, topk=8, scoring="sigmoid", renorm=True, scale=2.5,
             masked=0.1, first=80, local=80),
        # a prefill chunk
        dict(name="router_16384", op="router", dtype="bf16", M=16384, E=128, topk=8, scoring="softmax", renorm=True,
             scale=1.0, masked=0.0, first=0, local=128),
        # one token's gate/up product: eight experts' weights, each used once
        dict(name="q4_gate_up_1", op="q4", dtype="bf16", M=1, E=128, topk=8, K=2048, N=1536, group=128, zeros=False,
             pair_rows=False, dist="uniform"),
        # the down product of a small decode batch, over per-pair rows, with zero points
        dict(name="q4_down_23", op="q4", dtype="bf16", M=23, E=128, topk=8, K=768, N=2048, group=64, zeros=True,
             pair_rows=True, dist="uniform"),
        # a full decode batch whose popular experts hold most pairs
        dict(name="q4_gate_up_128_zipf", op="q4", dtype="bf16", M=128, E=128, topk=8, K=2048, N=1536, group=128,
             zeros=False, pair_rows=False, dist="zipf"),
        # one matrix of a dense layer (a single "expert"), an odd number of rows and columns, fp32 beside the weights
        dict(name="q4_dense_f32_7", op="q4", dtype="f32", M=7, E=1, topk=1, K=2080, N=1001, group=32, zeros=True,
             pair_rows=False, dist="uniform"),
        # one decoding token without an adapter
        dict(name="layer_1", op="layer", dtype="bf16", M=1, hidden=2048, inter=768, E=128, topk=8, S=0, rank=0, group=0,
             dist="uniform"),
        # a small decode batch, eight adapters
        dict(name="layer_23_lora", op="layer", dtype="bf16", M=23, hidden=2048, inter=768, E=128, topk=8, S=8, rank=32,
             group=0, dist="uniform"),
        # the same batch over 4-bit base weights
        dict(name="layer_23_lora_q4", op="layer", dtype="bf16", M=23, hidden=2048, inter=768, E=128, topk=8, S=8, rank=32,
             group=128, dist="uniform"),
        # a full decode batch, sixteen adapters, popular experts
        dict(name="layer_128_lora_zipf", op="layer", dtype="bf16", M=128, hidden=2048, inter=768, E=128, topk=8, S=16,
             rank=32, group=0, dist="zipf"),
        # fp32, ragged sizes, a low rank
        dict(name="layer_5_f32", op="layer", dtype="f32", M=5, hidden=516, inter=132, E=9, topk=3, S=3, rank=12, group=0,
             dist="uniform"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("router", "q4", "layer"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "router":
        E = _log(rng, 8, 512)
        local = rng.choice((E, max(1, E // 2)))
        return dict(op=op, dtype=dtype, M=_log(rng, 1, 12000), E=E, topk=min(E, rng.randint(1, 12)),
                    scoring=rng.choice(("softmax", "sigmoid")), renorm=rng.random() < 0.6, scale=rng.choice((1.0, 2.5)),
                    masked=rng.choice((0.0, 0.3, 0.9)), first=rng.randint(0, E - local), local=local)
    E = _log(rng, 1, 128)
    topk = min(E, rng.randint(1, 8))
    dist = rng.choice(("uniform", "zipf"))
    if op == "q4":
        group = rng.choice((32, 64, 128))
        return dict(op=op, dtype=dtype, M=_log(rng, 1, 120), E=E, topk=topk, K=group * _log(rng, 2, 2048 // group),
                    N=_log(rng, 24, 1536), group=group, zeros=rng.random() < 0.5, pair_rows=rng.random() < 0.5, dist=dist)
    group = rng.choice((0, 0, 32, 64, 128))
    unit = group or (8 if dtype == "bf16" else 4)
    S = rng.choice((0, 3, 8))
    return dict(op=op, dtype=dtype, M=_log(rng, 1, 120), hidden=unit * _log(rng, 2, 2048 // unit),
                inter=unit * _log(rng, 1, 768 // unit), E=E, topk=topk, S=S, rank=rng.choice((8, 16, 32)) if S else 0,
                group=group, dist=dist)


# ------------------------------------------------------------------------------ inputs


def _route(case, gen, dev):
    """Top-k ids of a batch (a few slots are -1: experts on another GPU) and router weights."""
    M, E, k = case["M"], case["E"], case["topk"]
    score = -torch.log(-torch.log(torch.rand(M, E, generator=gen, device=dev).clamp(1e-9, 1 - 1e-6)))
    if case["dist"] == "zipf":
        score = score - 1.1 * torch.log(torch.arange(1, E + 1, device=dev, dtype=torch.float32))
    ids = torch.argsort(score, dim=1, descending=True)[:, :k].to(torch.int32).contiguous()
    if M * k > 16:
        drop = torch.rand(M, k, generator=gen, device=dev) < 0.03
        ids = torch.where(drop, torch.full_like(ids, -1), ids)
    w = torch.softmax(torch.randn(M, k, generator=gen, device=dev), dim=1)
    return ids, w


def _quantised(E, N, K, group, zeros, dt, gen, dev):
    """4-bit weights of sigma about 0.02: two per byte, the even k in the low half, with a scale for each group of a row."""
    q = torch.randint(0, 256, (E, N, K // 2), generator=gen, device=dev, dtype=torch.uint8)
    s = (0.003 + 0.003 * torch.rand(E, N, K // group, generator=gen, device=dev)).to(dt)
    z = torch.randint(5, 11, (E, N, K // group), generator=gen, device=dev, dtype=torch.uint8) if zeros else None
    return q, s, z


def _aligned(ids, E):
    """The pairs of a batch bucketed by expert in blocks of BLOCK_M, as mol_align_block_size lays them out."""
    flat = ids.reshape(-1).long()
    numel = flat.numel()
    bucket = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    count = torch.bincount(bucket, minlength=E + 1)
    padded = (count + BLOCK_M - 1) // BLOCK_M * BLOCK_M
    start = torch.cumsum(padded, 0) - padded
    order = torch.argsort(bucket, stable=True)
    within = torch.arange(numel, device=ids.device) - (torch.cumsum(count, 0) - count)[bucket[order]]
    blocks = -(-(numel + min(numel, E + 1) * (BLOCK_M - 1)) // BLOCK_M)
    srt = torch.full((blocks * BLOCK_M,), numel, dtype=torch.int32, device=ids.device)
    srt[start[bucket[order]] + within] = order.to(torch.int32)
    of = torch.repeat_interleave(torch.arange(E + 1, device=ids.device), padded // BLOCK_M)
    eid = torch.full((blocks,), -1, dtype=torch.int32, device=ids.device)
    eid[:of.numel()] = torch.where(of < E, of, torch.full_like(of, -1)).to(torch.int32)
    return srt, eid, padded.sum().to(torch.int32).reshape(1)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, dtype=dt):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype) * sigma

    st = dict(case=case)
    if case["op"] == "router":
        logits = normal(case["M"], case["E"], sigma=2.0)
        if case["masked"]:
            gone = torch.rand(case["M"], case["E"], generator=gen, device=dev) < case["masked"]
            logits = logits.masked_fill(gone, float("-inf"))
        st["logits"] = logits
        st["ids"] = torch.empty(case["M"], case["topk"], dtype=torch.int32, device=dev)
        st["w"] = torch.empty(case["M"], case["topk"], dtype=torch.float32, device=dev)
        return st
    st["ids"], st["w"] = _route(case, gen, dev)
    if case["op"] == "q4":
        rows = case["M"] * case["topk"] if case["pair_rows"] else case["M"]
        st["x"] = normal(rows, case["K"])
        st["W"] = _quantised(case["E"], case["N"], case["K"], case["group"], case["zeros"], dt, gen, dev)
        st["routing"] = _aligned(st["ids"], case["E"])
        st["out"] = torch.zeros(case["M"] * case["topk"], case["N"], dtype=dt, device=dev)
        return st
    E, H, I, S, r, G = (case[k] for k in ("E", "hidden", "inter", "S", "rank", "group"))
    st["x"] = normal(case["M"], H)
    if G:
        st["gate_up"] = _quantised(E, 2 * I, H, G, False, dt, gen, dev)
        st["down"] = _quantised(E, H, I, G, False, dt, gen, dev)
    else:
        st["gate_up"] = normal(E, 2 * I, H, sigma=0.02)
        st["down"] = normal(E, H, I, sigma=0.02)
    st["lora"] = None
    if S:
        V = E * S
        st["lora"] = torch.randint(-1, S, (case["M"],), generator=gen, device=dev, dtype=torch.int32)
        st["slot_scale"] = 0.5 + torch.rand(S, generator=gen, device=dev)
        st["A1"], st["B1"] = normal(V, 2 * r, H, sigma=0.02), normal(V, 2 * I, r, sigma=0.02)
        st["A2"], st["B2"] = normal(V, r, I, sigma=0.02), normal(V, H, r, sigma=0.02)
    st["y"] = torch.empty(case["M"], H, dtype=dt, device=dev)
    return st


# ------------------------------------------------------------------------- plain forms


def _dequantised(q, s, z):
    E, N, half = q.shape
    v = torch.stack((q & 15, q >> 4), dim=-1).reshape(E, N, s.shape[2], -1).float()
    v = v - (8.0 if z is None else z.float().unsqueeze(-1))
    return (v * s.float().unsqueeze(-1)).reshape(E, N, 2 * half)


def _rows_times(W, index, x):
    """W[index[p]] x[p] for each pair p, in 32 bits."""
    if isinstance(W, tuple):  # 4-bit: the picked matrices alone are dequantised where they are fewer than the experts
        few = index.numel() < W[0].shape[0]
        W = _dequantised(*(t if t is None or not few else t[index] for t in W))
        W = W if few else W[index]
    else:
        W = W[index]
    return torch.matmul(W.float(), x.float().unsqueeze(-1)).squeeze(-1)


def _plain_router(st):
    c = st["case"]
    l = st["logits"].float()
    top, idx = torch.sort(l, dim=1, descending=True, stable=True)
    top, idx = top[:, :c["topk"]], idx[:, :c["topk"]]
    there = top > float("-inf")
    # in 64 bits: a sum over hundreds of experts, and weights that are compared with those of a definition in 64 bits
    if c["scoring"] == "softmax":
        m = l.max(dim=1, keepdim=True).values.clamp_min(-3e38)
        w = torch.exp((top - m).double()) / torch.exp((l - m).double()).sum(dim=1, keepdim=True).clamp_min(1e-300)
    else:
        w = 1.0 / (1.0 + torch.exp(-top.double()))
    w = torch.where(there, w, torch.zeros_like(w))
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp_min(1e-300)
    idx = idx - c["first"]
    here = there & (idx >= 0) & (idx < c["local"])
    return (torch.where(here, idx, torch.full_like(idx, -1)).to(torch.int32),
            torch.where(here, w * c["scale"], torch.zeros_like(w)).float())


def _plain_q4(st):
    c = st["case"]
    ids = st["ids"].reshape(-1).long()
    x = st["x"] if c["pair_rows"] else st["x"].repeat_interleave(c["topk"], dim=0)
    v = _rows_times(st["W"], ids.clamp_min(0), x)
    return torch.where((ids >= 0).unsqueeze(1), v, torch.zeros_like(v)).to(st["out"].dtype)


def _plain_layer(st):
    c = st["case"]
    M, k, I, r = c["M"], c["topk"], c["inter"], c["rank"]
    ids = st["ids"].reshape(-1).long()
    e = ids.clamp_min(0)
    x = st["x"].repeat_interleave(k, dim=0).float()
    gu = _rows_times(st["gate_up"], e, x)
    if st["lora"] is not None:
        slot = st["lora"].long().repeat_interleave(k)
        v = e + slot.clamp_min(0) * c["E"]
        scale = torch.where(slot >= 0, st["slot_scale"][slot.clamp_min(0)], torch.zeros_like(slot, dtype=torch.float32))
        s = _rows_times(st["A1"], v, x)
        gate = _rows_times(st["B1"][:, :I], v, s[:, :r])
        up = _rows_times(st["B1"][:, I:], v, s[:, r:])
        gu = gu + scale.unsqueeze(1) * torch.cat((gate, up), dim=1)
    g, u = gu[:, :I], gu[:, I:]
    h = g / (1.0 + torch.exp(-g)) * u
    z = _rows_times(st["down"], e, h)
    if st["lora"] is not None:
        z = z + scale.unsqueeze(1) * _rows_times(st["B2"], v, _rows_times(st["A2"], v, h))
    w = torch.where(ids >= 0, st["w"].reshape(-1), torch.zeros_like(st["w"].reshape(-1)))
    return (z * w.unsqueeze(1)).reshape(M, k, -1).sum(dim=1).to(st["y"].dtype)


# --------------------------------------------------------------------------------- run


def run(st):
    op = st["case"]["op"]
    if own:
        return {"router": _own_router, "q4": _own_q4, "layer": _own_layer}[op](st)
    return {"router": _plain_router, "q4": _plain_q4, "layer": _plain_layer}[op](st)


def _own_router(st):
    mb = _binding()
    c = st["case"]
    scoring = mb.MOL_SCORE_SOFTMAX if c["scoring"] == "softmax" else mb.MOL_SCORE_SIGMOID
    return mb.mol_router_topk(st["logits"], c["topk"], scoring, c["renorm"], c["scale"], c["first"], c["local"],
                              topk_ids=st["ids"], topk_weights=st["w"])


def _own_q4(st):
    mb = _binding()
    c = st["case"]
    q, s, z = st["W"]
    return mb.mol_moe_gemm_q4(st["x"], 1 if c["pair_rows"] else c["topk"], q, s, *st["routing"], c["M"] * c["topk"],
                              BLOCK_M, st["out"], zeros=z)


def _own_layer(st):
    mb = _binding()
    if "handle" not in st:  # what a program keeps beside its weights: their description and the scratch of a layer
        gu, dn = st["gate_up"], st["down"]
        w = (mb.MoeWeights(gu[0], dn[0], gu[1], dn[1], gu[2], dn[2]) if isinstance(gu, tuple) else mb.MoeWeights(gu, dn))
        ad = None
        if st["lora"] is not None:
            ad = mb.MoeAdapters(st["A1"], st["B1"], st["A2"], st["B2"], st["slot_scale"])
        st["handle"] = (w, ad, mb.new_moe_layer_workspace(w, st["case"]["M"], st["case"]["topk"], adapters=ad))
    w, ad, ws = st["handle"]
    return mb.mol_moe_layer(w, st["x"], st["ids"], st["w"], adapters=ad, lora_ids=st["lora"], y=st["y"], workspace=ws)


# -------------------------------------------------------------------------------- work


def _touched(E, pairs, topk, dist):
    """The experts that a batch is expected to touch: draws without replacement within a token, independent between tokens."""
    tokens = pairs / topk
    if dist == "uniform":
        return E * (1.0 - (1.0 - topk / E) ** tokens)
    p = [(i + 1) ** -1.1 for i in range(E)]
    total = sum(p)
    if topk >= E:
        return float(E)
    lo, hi = 0.0, 1e9  # the rate at which topk of the experts are drawn
    for _ in range(80):
        mid = (lo + hi) / 2
        lo, hi = (mid, hi) if sum(1 - math.exp(-mid * q / total) for q in p) < topk else (lo, mid)
    return sum(1.0 - math.exp(-lo * q / total * tokens) for q in p)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    M, E, k = case["M"], case["E"], case["topk"]
    if case["op"] == "router":
        return {"bytes": M * E * es + 8 * M * k, "flops": 4 * M * E}
    pairs = M * k * (0.97 if M * k > 16 else 1.0)
    touched = _touched(E, M * k, k, case["dist"])

    def matrix(N, K, group, zeros):
        return N * K * es if not group else N * K / 2 + N * (K // group) * (es + (1 if zeros else 0))

    if case["op"] == "q4":
        K, N = case["K"], case["N"]
        rows = M * k if case["pair_rows"] else M
        return {"bytes": touched * matrix(N, K, case["group"], case["zeros"]) + rows * K * es + pairs * N * es,
                "flops": 2 * pairs * N * K}
    H, I, S, r, G = (case[x] for x in ("hidden", "inter", "S", "rank", "group"))
    total = touched * (matrix(2 * I, H, G, False) + matrix(H, I, G, False)) + 2 * M * H * es + 8 * M * k
    flops = 2 * pairs * 3 * I * H
    if S:
        adapted = pairs * S / (S + 1)
        total += min(adapted, E * S) * (2 * r * H + 2 * I * r + r * I + H * r) * es
        flops += 2 * adapted * (2 * r * H + 2 * I * r + r * I + H * r)
    return {"bytes": total, "flops": flops}


# ------------------------------------------------------------------------------- exact


def _expert64(W, e):
    """One expert's matrix in 64 bits."""
    if not isinstance(W, tuple):
        return W[e].double()
    q, s, z = (None if t is None else t[e] for t in W)
    N, half = q.shape
    out = torch.empty(N, 2 * half, dtype=torch.float64, device=q.device)
    out[:, 0::2] = (q % 16).double()
    out[:, 1::2] = (q // 16).double()
    G = 2 * half // s.shape[1]
    zero = torch.full_like(s, 8.0, dtype=torch.float64) if z is None else z.double()
    return (out - zero.repeat_interleave(G, dim=1)) * s.double().repeat_interleave(G, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    dev = st["ids"].device
    k = case["topk"]
    if case["op"] == "router":
        l = st["logits"].double()
        w = torch.zeros(l.shape[0], k, dtype=torch.float64, device=dev)
        finite = l > float("-inf")
        score = (torch.where(finite, l, torch.full_like(l, -1e300)).softmax(dim=1) if case["scoring"] == "softmax"
                 else torch.sigmoid(l)) * finite
        left = l.clone()
        for j in range(k):  # one expert after another: the largest that is left, the first of equals
            best = left.max(dim=1, keepdim=True).values
            at = (left == best).to(torch.int8).argmax(dim=1, keepdim=True)
            got = torch.where(best > float("-inf"), score.gather(1, at), torch.zeros_like(best))
            w[:, j:j + 1] = torch.where((at >= case["first"]) & (at < case["first"] + case["local"]), got, -got)
            left.scatter_(1, at, float("-inf"))
        if case["renorm"]:
            w = w / w.abs().sum(dim=1, keepdim=True).clamp_min(1e-300)
        return None, w.clamp_min(0.0) * case["scale"]
    ids = st["ids"].reshape(-1)
    experts = [int(e) for e in torch.unique(ids).tolist() if e >= 0]
    x = st["x"].double()
    if case["op"] == "q4":
        out = torch.zeros(ids.numel(), case["N"], dtype=torch.float64, device=dev)
        for e in experts:
            p = torch.nonzero(ids == e).reshape(-1)
            out[p] = x[p if case["pair_rows"] else p // k] @ _expert64(st["W"], e).t()
        return out
    M, I, r = case["M"], case["inter"], case["rank"]
    y = torch.zeros(M, case["hidden"], dtype=torch.float64, device=dev)
    slots = [-1] * M if st["lora"] is None else st["lora"].tolist()
    w = st["w"].double().reshape(-1)
    for e in experts:
        p = torch.nonzero(ids == e).reshape(-1)
        gu = x[p // k] @ _expert64(st["gate_up"], e).t()
        mine = [(i, slots[q // k]) for i, q in enumerate(p.tolist()) if slots[q // k] >= 0]
        for i, l in mine:
            v, c = e + l * case["E"], st["slot_scale"][l].double()
            s = st["A1"][v].double() @ x[p[i] // k]
            gu[i, :I] += c * (st["B1"][v, :I].double() @ s[:r])
            gu[i, I:] += c * (st["B1"][v, I:].double() @ s[r:])
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        z = h @ _expert64(st["down"], e).t()
        for i, l in mine:
            v, c = e + l * case["E"], st["slot_scale"][l].double()
            z[i] += c * (st["B2"][v].double() @ (st["A2"][v].double() @ h[i]))
        y.index_add_(0, p // k, z * w[p].unsqueeze(1))
    return y

"""A whole layer for a few tokens through the C ABI against its 64-bit definition, element by
element, within the bound that fp32 sums and the roundings of h and y allow (plain64.layer)."""
import numpy as np
import pytest
import torch

from tests import plain64
from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Layer:
    """One layer's host tensors, and the same on the GPU behind MoeWeights / MoeAdapters."""

    def __init__(self, dtype, H, I, E, S=0, r=0, group=0, ranks=None, zeros=False, seed=0):
        g = torch.Generator().manual_seed(seed)
        dt = self.dt = DT[dtype]
        self.H, self.I, self.E, self.S, self.r, self.ranks = H, I, E, S, r, ranks
        self.group = group

        def normal(*shape, sigma=0.05):
            return (torch.randn(*shape, generator=g) * sigma).to(dt)

        def packed(N, K):
            return (torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8),
                    normal(E, N, K // group, sigma=0.01),
                    torch.randint(0, 16, (E, N, K // group), generator=g, dtype=torch.uint8)
                    if zeros else None)

        if group:
            self.gu, self.dn = packed(2 * I, H), packed(H, I)
            up = [t if t is None else t.cuda() for t in (*self.gu, *self.dn)]
            self.w = mb.MoeWeights(up[0], up[3], up[1], up[4], up[2], up[5])
        else:
            self.gu, self.dn = normal(E, 2 * I, H), normal(E, H, I)
            self.w = mb.MoeWeights(self.gu.cuda(), self.dn.cuda())
        self.ad = self.ad64 = None
        if S:
            V = E * S
            A1, B1 = normal(V, 2 * r, H), normal(V, 2 * I, r)
            A2, B2 = normal(V, r, I), normal(V, H, r)
            scale = torch.linspace(0.5, 2.0, S)
            self.ad64 = tuple(t.double().numpy() for t in (A1, B1, A2, B2)) + (
                scale.double().numpy(), ranks)
            for l, rl in enumerate(ranks or ()):  # weights past a slot's rank are never read
                rl = min(max(rl, 0), r)
                v = slice(l * E, (l + 1) * E)
                A1[v, rl:r], A1[v, r + rl:] = float("nan"), float("nan")
                B1[v, :, rl:], A2[v, rl:], B2[v, :, rl:] = (float("nan"),) * 3
            dev_ranks = None if ranks is None else torch.tensor(ranks, dtype=torch.int32).cuda()
            self.ad = mb.MoeAdapters(A1.cuda(), B1.cuda(), A2.cuda(), B2.cuda(), scale.cuda(),
                                     dev_ranks)

    def expert(self, W):
        def get(t):
            if not 0 <= t < self.E:
                return None, None
            if self.group:
                return plain64.dequantise(W[0][t].numpy(), W[1][t].double().numpy(),
                                          None if W[2] is None else W[2][t].numpy())
            w = W[t].double().numpy()
            return w, np.abs(w)
        return get

    def step(self, M, topk, seed=1, sentinels=True):
        """One batch: x, ids, weights, slots (host)."""
        g = torch.Generator().manual_seed(seed)
        x = torch.randn(M, self.H, generator=g).to(self.dt)
        if topk <= self.E:
            ids = torch.stack([torch.randperm(self.E, generator=g)[:topk] for _ in range(M)])
        else:
            ids = torch.randint(0, self.E, (M, topk), generator=g)
        if sentinels and M * topk > 4:
            ids.view(-1)[torch.randperm(M * topk, generator=g)[:M * topk // 10 + 1]] = -1
        w = torch.softmax(torch.randn(M, topk, generator=g), 1)
        lora = torch.randint(-1, self.S, (M,), generator=g).int() if self.S else None
        return x, ids.int(), w, lora

    def call(self, x, ids, w, lora, **kw):
        return mb.mol_moe_layer(self.w, x.cuda(), ids.cuda(), w.cuda(), self.ad,
                                None if lora is None else lora.cuda(), **kw)

    def check(self, x, ids, w, lora, got):
        got = got.float().cpu().numpy()
        assert got.shape == (x.shape[0], self.H)
        ref, bound = plain64.layer(x.double().numpy(), self.expert(self.gu), self.expert(self.dn),
                                   ids.numpy(), w.double().numpy(), torch.finfo(self.dt).eps,
                                   self.ad64, None if lora is None else lora.numpy())
        if ref is None:
            assert np.all(got == 0)
            return
        plain64.within(got, ref, bound)
        empty = np.all((ids.numpy() < 0) | (ids.numpy() >= self.E), axis=1)
        assert np.all(got[empty] == 0)

    def run(self, M, topk, seed=1):
        b = self.step(M, topk, seed)
        got = self.call(*b)
        self.check(*b, got)
        return b, got


@pytest.mark.parametrize("dtype,H,I,group,zeros", [
    ("bf16", 64, 40, 0, False), ("bf16", 136, 96, 0, False), ("f32", 68, 20, 0, False),
    ("bf16", 96, 32, 32, True), ("bf16", 192, 64, 64, False), ("bf16", 256, 128, 128, True),
    ("f32", 160, 96, 32, False), ("f32", 128, 256, 128, True)])
@pytest.mark.parametrize("M,topk,E", [(1, 1, 1), (1, 8, 16), (2, 2, 3), (5, 3, 7), (23, 8, 16),
                                      (33, 2, 5), (70, 9, 12)])
@pytest.mark.parametrize("adapters", [False, True])
def test_sizes(dtype, H, I, group, zeros, M, topk, E, adapters):
    r = 16 if dtype == "bf16" else 12
    S = 3 if adapters else 0
    Layer(dtype, H, I, E, S, r if S else 0, group, zeros=zeros, seed=H + I).run(M, topk, seed=M)


@pytest.mark.parametrize("dtype,r,ranks", [("bf16", 32, (32, 5, 0, 17)), ("f32", 8, (1, 8, -3, 99)),
                                           ("bf16", 128, (128, 71)), ("f32", 64, (64, 33))])
@pytest.mark.parametrize("M", [4, 40])
def test_slot_ranks(dtype, r, ranks, M):
    Layer(dtype, 64, 48, 6, len(ranks), r, ranks=ranks, seed=3).run(M, 4)


@pytest.mark.parametrize("M", [20, 200])
def test_one_expert_takes_most_pairs(M):
    """More pairs of one matrix than a pass of 64, by pair and by expert."""
    for E in (2, 512):
        la = Layer("bf16", 64, 32, E, 2, 8, seed=4)
        x, ids, w, lora = la.step(M, 2)
        ids[:, 0] = 1
        la.check(x, ids, w, lora, la.call(x, ids, w, lora))


@pytest.mark.parametrize("M,E", [(10, 2), (20, 2), (45, 3), (300, 5)])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_many_pairs_over_long_rows(M, E, group):
    """Columns of every width class over rows whose x takes several stages, the pairs found by
    every wave itself (up to 512 of them) and in quarters."""
    if M == 300:
        la = Layer("bf16", 2048, 128, E, 2, 8, group=group, seed=M)
        x, ids, w, lora = la.step(M, 2)
        rows = torch.tensor([0, 1, 57, 150, 299])
        got = la.call(x, ids, w, lora)[rows.cuda()]
        la.check(x[rows], ids[rows], w[rows], lora[rows], got)
        return
    Layer("bf16", 2048, 256, E, 2, 8, group=group, seed=M).run(M, 2)
    if group == 0:
        Layer("f32", 1040, 516, E, 2, 8, seed=M).run(M, 2)


@pytest.mark.parametrize("dtype,group", [("bf16", 0), ("bf16", 32), ("bf16", 64), ("bf16", 128),
                                         ("f32", 0), ("f32", 32)])
@pytest.mark.parametrize("M,topk,E", [(1, 64, 70), (1, 17, 5), (1, 1, 3), (2, 8, 9), (3, 8, 6),
                                      (3, 2, 4), (3, 64, 64), (4, 8, 9)])
def test_few_tokens_without_adapters(dtype, group, M, topk, E):
    """Down per token, over one tile of experts to sixteen, and the counts around its choice."""
    Layer(dtype, 128, 1152, E, group=group, zeros=True, seed=topk).run(M, topk, seed=M)


@pytest.mark.parametrize("M,topk", [(64, 64), (4096, 1), (1365, 3)])
@pytest.mark.parametrize("adapters", [False, True])
def test_the_most_pairs(M, topk, adapters):
    la = Layer("bf16", 64, 32, 70, 3 if adapters else 0, 8, ranks=(8, 0, 3), seed=M)
    x, ids, w, lora = la.step(M, topk)
    ids[M // 2:, 0] = 4                           # an expert of very many pairs
    got = la.call(x, ids, w, lora)
    rows = torch.cat((torch.arange(0, 20), torch.arange(M - 20, M)))
    la.check(x[rows], ids[rows], w[rows], None if lora is None else lora[rows], got[rows.cuda()])


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("M", [2, 50])
def test_the_most_virtual_experts(group, M):
    Layer("bf16", 32, 32, 4095, 2, 8, group=group, seed=5).run(M, 8)
    Layer("f32", 32, 32, 2, 4095, 4, group=group, seed=6).run(M, 2)


def test_a_workspace_of_more_tokens():
    la = Layer("bf16", 96, 64, 6, 2, 16, seed=18)
    ws = mb.new_moe_layer_workspace(la.w, 50, 4, la.ad)
    for M, topk in ((50, 4), (1, 4), (7, 2), (100, 2)):
        b = la.step(M, topk, seed=M)
        assert torch.equal(la.call(*b, workspace=ws), la.call(*b))


@pytest.mark.parametrize("M", [1, 2, 9])
@pytest.mark.parametrize("group", [0, 128])
def test_router_and_layer_in_one_graph(M, group):
    """A decode step without adapters, captured once, replayed over new inputs between eager
    steps that use the same workspace."""
    la = Layer("bf16", 256, 1024, 16, group=group, seed=19)
    x = torch.zeros(M, 256, dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros(M, 16, device="cuda")
    ids = torch.zeros(M, 8, dtype=torch.int32, device="cuda")
    w = torch.zeros(M, 8, device="cuda")
    y = torch.zeros_like(x)
    ws = mb.new_moe_layer_workspace(la.w, M, 8)

    def step(y):
        mb.mol_router_topk(logits, 8, topk_ids=ids, topk_weights=w)
        return mb.mol_moe_layer(la.w, x, ids, w, y=y, workspace=ws)
    step(y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(y)
    gen = torch.Generator().manual_seed(20)
    for _ in range(4):
        x.copy_(torch.randn(M, 256, generator=gen))
        logits.copy_(torch.randn(M, 16, generator=gen))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, step(torch.empty_like(y)))
        la.check(x.cpu(), ids.cpu(), w.cpu(), None, got)


def test_decode_layer_width():
    Layer("bf16", 2048, 768, 10, 2, 32, seed=5).run(3, 8)
    Layer("bf16", 6144, 256, 9, 2, 32, seed=6).run(2, 8)
    Layer("bf16", 2048, 768, 10, 2, 32, group=128, seed=7).run(2, 8)


@pytest.mark.parametrize("M", [6, 40])
def test_odd_routings(M):
    la = Layer("bf16", 64, 48, 5, 2, 8, seed=8)
    x, ids, w, lora = la.step(M, 4, sentinels=False)
    ids[0] = -1                                   # a token without experts: zeros
    ids[1] = torch.tensor([5, -9, 2**31 - 1, -2**31])
    ids[2] = 3                                    # the same expert in every slot
    ids[3] = torch.tensor([1, 1, 4, 1])
    w[4] = torch.tensor([0.0, -1.5, 2.0, 0.0])
    lora[:] = torch.tensor([0, 7, 1, -5, 0, 1])[torch.arange(M) % 6].int()
    la.check(x, ids, w, lora, la.call(x, ids, w, lora))
    ids[:] = -1
    la.check(x, ids, w, lora, la.call(x, ids, w, lora))


@pytest.mark.parametrize("M", [5, 40])
@pytest.mark.parametrize("group", [0, 32])
def test_bad_values_stay_in_their_token(M, group):
    la = Layer("bf16", 64, 32, 4, 2, 8, group=group, seed=9)
    x, ids, w, lora = la.step(M, 3, sentinels=False)
    clean = la.call(x, ids, w, lora)
    x[1, 5], x[3, 63] = float("nan"), float("inf")
    got = la.call(x, ids, w, lora)
    keep = torch.ones(M, dtype=torch.bool)
    keep[[1, 3]] = False
    assert torch.equal(got[keep.cuda()], clean[keep.cuda()])
    assert torch.all(torch.isnan(got[1]))


def test_an_expert_no_token_uses_may_hold_anything():
    for M in (5, 40):
        la = Layer("bf16", 64, 32, 4, seed=10)
        x, ids, w, lora = la.step(M, 2)
        ids[ids == 2] = 1
        want = la.call(x, ids, w, lora)
        la.w.tensors[0][2] = float("nan")
        la.w.tensors[1][2] = float("inf")
        assert torch.equal(want, la.call(x, ids, w, lora))


@pytest.mark.parametrize("M", [7, 40])
@pytest.mark.parametrize("group", [0, 32])
def test_strides_guards_and_dirty_workspace(M, group):
    la = Layer("bf16", 96, 64, 6, 2, 16, group=group, seed=11)
    x, ids, w, lora = la.step(M, 3)
    want = la.call(x, ids, w, lora)
    wide = torch.full((M, 96 + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 16:112] = x.cuda()
    raw = torch.full((M * 101 + 300,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = raw[150:150 + M * 101].view(M, 101)[:, 2:98]
    n = mb.mol_moe_layer_workspace_bytes(la.w, M, 3, la.ad)
    ws = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN as any float
    mb.mol_moe_layer(la.w, wide[:, 16:112], ids.cuda(), w.cuda(), la.ad, lora.cuda(), y=y,
                     workspace=ws[256:256 + n])
    assert torch.equal(y, want)
    assert torch.all(ws[:256] == 0xFF) and torch.all(ws[256 + n:] == 0xFF)
    keep = torch.ones_like(raw, dtype=torch.bool)
    keep[150:150 + M * 101].view(M, 101)[:, 2:98] = False
    assert torch.all(raw[keep] == 7.0)


def test_no_tokens():
    la = Layer("bf16", 64, 32, 4, 2, 8, seed=12)
    y = la.call(torch.empty(0, 64, dtype=torch.bfloat16), torch.empty(0, 2, dtype=torch.int32),
                torch.empty(0, 2), torch.empty(0, dtype=torch.int32))
    assert y.shape == (0, 64)


@pytest.mark.parametrize("M", [3, 40])
def test_streams_and_graphs(M):
    """Two calls at once on two streams with a workspace each, and a replayed graph."""
    la = Layer("bf16", 128, 64, 8, 2, 16, seed=13)
    a, b = la.step(M, 4, seed=1), la.step(M, 4, seed=2)
    da, db = ([None if t is None else t.cuda() for t in s] for s in (a, b))
    wa, wb = la.call(*a), la.call(*b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws = [mb.new_moe_layer_workspace(la.w, M, 4, la.ad) for _ in range(2)]
    ya, yb = torch.zeros_like(wa), torch.zeros_like(wb)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            mb.mol_moe_layer(la.w, da[0], da[1], da[2], la.ad, da[3], y=ya, workspace=ws[0])
        with torch.cuda.stream(s2):
            mb.mol_moe_layer(la.w, db[0], db[1], db[2], la.ad, db[3], y=yb, workspace=ws[1])
    torch.cuda.synchronize()
    assert torch.equal(ya, wa) and torch.equal(yb, wb)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mb.mol_moe_layer(la.w, da[0], da[1], da[2], la.ad, da[3], y=ya, workspace=ws[0])
    for seed in (3, 4, 5):
        c = la.step(M, 4, seed=seed)
        for d, h in zip(da, c):
            d.copy_(h)
        ya.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ya, la.call(*c))


@pytest.mark.parametrize("M", [6, 40])
def test_router_then_layer_matches_the_aligned_path(M):
    """A serving step: router, then the layer in one call; and the same step through the aligned
    path (align, 4-bit grouped GEMM, LoRA delta, activation, again, combine), both within the
    bound of the 64-bit layer (the aligned path rounds its rows to bf16 in between)."""
    la = Layer("bf16", 256, 128, 16, 3, 16, group=64, seed=14)
    x, _, _, lora = la.step(M, 4)
    logits = torch.randn(M, 16, generator=torch.Generator().manual_seed(15)).cuda()
    ids, w = mb.mol_router_topk(logits, 4)
    y = mb.mol_moe_layer(la.w, x.cuda(), ids, w, la.ad, lora.cuda())
    la.check(x, ids.cpu(), w.cpu(), lora, y)
    numel, dev = M * 4, "cuda"
    gu, dn, gus, dns, _, _ = la.w.tensors
    A1, B1, A2, B2, scale, _ = la.ad.tensors
    base = mb.mol_align_block_size(ids, None, 16, 1, 64)
    virt = mb.mol_align_block_size(ids, lora.cuda(), 16, 3, 64)
    rows = torch.zeros(numel, 256, dtype=torch.bfloat16, device=dev)
    mb.mol_moe_gemm_q4(x.cuda(), 4, gu, gus, *base, numel, 64, rows)
    mb.mol_lora_delta(x.cuda(), 4, A1, 2, B1, scale, 16, *virt, numel, 48, 64, rows,
                      mb.new_delta_workspace(numel, 32, 48, 64, dev))
    g, u = rows.float()[:, :128], rows.float()[:, 128:]
    h = (torch.nn.functional.silu(g) * u).bfloat16()
    out = torch.zeros(numel, 256, dtype=torch.bfloat16, device=dev)
    mb.mol_moe_gemm_q4(h, 1, dn, dns, *base, numel, 64, out)
    mb.mol_lora_delta(h, 1, A2, 1, B2, scale, 16, *virt, numel, 48, 64, out,
                      mb.new_delta_workspace(numel, 16, 48, 64, dev))
    y2 = mb.mol_moe_combine(out, ids, w, 16)
    ref, bound = plain64.layer(x.double().numpy(), la.expert(la.gu), la.expert(la.dn),
                               ids.cpu().numpy(), w.cpu().double().numpy(), 2.0 ** -7,
                               la.ad64, lora.numpy(), rows_rounded=True)
    plain64.within(y2.float().cpu().numpy(), ref, bound)


@pytest.mark.parametrize("M", [1, 6])
def test_weights_past_32_bits(M):
    """Experts whose rows lie more than 4 GiB into the weights: bit for bit what they give alone."""
    E, H, I = 400, 2048, 1408
    gu = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    dn = torch.zeros(E, H, I, dtype=torch.bfloat16, device="cuda")
    assert gu.numel() * 2 > 2**32
    gen = torch.Generator("cuda").manual_seed(21)
    gu[E - 1].normal_(0, 0.05, generator=gen)
    dn[E - 1].normal_(0, 0.05, generator=gen)
    x = torch.randn(M, H, generator=gen, device="cuda").bfloat16()
    w = torch.ones(M, 1, device="cuda")
    ids = torch.full((M, 1), E - 1, dtype=torch.int32, device="cuda")
    got = mb.mol_moe_layer(mb.MoeWeights(gu, dn), x, ids, w)
    alone = mb.mol_moe_layer(mb.MoeWeights(gu[E - 1:].clone(), dn[E - 1:].clone()), x,
                             torch.zeros_like(ids), w)
    assert torch.equal(got, alone) and torch.all(torch.isfinite(got)) and got.abs().max() > 0


def test_refusals():
    la = Layer("bf16", 64, 32, 4, 2, 8, seed=16)
    b = [t.cuda() for t in la.step(3, 2)]

    def go(x=b[0], ids=b[1], w=b[2], ad=la.ad, lora=b[3], **kw):
        return mb.mol_moe_layer(la.w, x, ids, w, ad, lora, **kw)
    go()
    for kw in (dict(x=b[0][:2]), dict(x=b[0][:, :56]), dict(x=b[0].cpu()), dict(lora=None),
               dict(ad=None), dict(w=b[2][:, :1]), dict(lora=b[3][:2]),
               dict(y=torch.zeros(3, 63, dtype=torch.bfloat16, device="cuda")),
               dict(ad=Layer("bf16", 72, 32, 4, 2, 8).ad)):
        with pytest.raises(ValueError):
            go(**kw)
    for kw in (dict(x=b[0].float()), dict(ids=b[1].long()), dict(w=b[2].double())):
        with pytest.raises(TypeError):
            go(**kw)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(mb.MolError) as e:
        go(workspace=small)
    assert e.value.status == mb.MOL_E_WORKSPACE
    with pytest.raises(mb.MolError) as e:
        la.call(*la.step(2050, 2))
    assert e.value.status == mb.MOL_E_LIMIT

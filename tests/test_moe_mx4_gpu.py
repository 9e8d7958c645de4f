"""The base grouped GEMM over microscaled 4-bit weights, element by element against the product in 64 bits of the
values that codes and scales stand for. Those and their products are exact in fp32 (products of two codes and
two powers of two; a bf16 or fp32 row times a code: 26 bits, half a unit of 2^-24 lost at most), and any order of K
fp32 additions loses at most K 2^-24 of the sum of magnitudes: (K + 1) 2^-24 of it for the sum, and half a step of
the output type of the value."""
import pytest
import torch

from tests import mx4_cases as mc
from tests import mx4_defs as d
from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
FORMS = pytest.mark.parametrize("x,dtype", [("codes", torch.bfloat16), ("codes", torch.float32), ("rows", torch.bfloat16),
                                            ("rows", torch.float32)], ids=["codes_bf16", "codes_f32", "bf16", "f32"])


def value(q, s):
    return torch.from_numpy(d.decode(q.cpu().numpy(), s.cpu().numpy())).cuda()


def codes(rows, K, gen, sigma=1.0):
    return mb.mol_mx4_quantize(torch.randn(rows, K, generator=gen, device="cuda") * sigma)


class Case:
    def __init__(self, M, E, topk, K, N, x, dtype, block=64, per_pair=False, seed=0, skew=False, pad_out=0):
        g = torch.Generator(device="cuda").manual_seed(seed + M + 7 * N + K)
        self.E, self.N, self.K, self.block, self.dtype = E, N, K, block, dtype
        self.numel = M * topk
        score = torch.rand(M, E, generator=g, device="cuda")
        if skew:
            score = score + 3.0 / torch.arange(1, E + 1, device="cuda")
        self.ids = score.argsort(dim=1, descending=True)[:, :topk].to(torch.int32).contiguous()
        if M * topk > 8:
            self.ids[torch.rand(M, topk, generator=g, device="cuda") < 0.1] = -1
            self.ids[M // 2, 0] = E  # not an expert either
        self.row_div = 1 if per_pair else topk
        rows = self.numel if per_pair else M
        if x == "codes":
            self.x, self.xs = codes(rows, K, g)
        else:
            self.x, self.xs = torch.randn(rows, K, generator=g, device="cuda").to(dtype), None
        W, s = codes(E * N, K, g, 0.05)
        self.W, self.s = W.view(E, N, K // 2), s.view(E, N, K // 32)
        self.out = torch.full((self.numel, N + pad_out), 7.0, dtype=dtype, device="cuda")[:, :N]
        self.route()

    def route(self):
        self.routing = mb.mol_align_block_size(self.ids, None, self.E, 1, self.block)

    def run(self):
        return mb.mol_moe_gemm_mx4(self.x, self.row_div, self.W, self.s, *self.routing, self.numel, self.block, self.out,
                                   x_scales=self.xs)

    def check(self):
        self.run()
        x = self.x.double() if self.xs is None else value(self.x, self.xs)
        flat = self.ids.reshape(-1)
        for e in range(self.E):
            p = (flat == e).nonzero().reshape(-1)
            if p.numel() == 0:
                continue
            xr, w = x[p // self.row_div], value(self.W[e], self.s[e])
            ref, mag = xr @ w.t(), xr.abs() @ w.abs().t()
            got = self.out[p].double()
            err = (got - ref).abs() - ((self.K + 1) * 2.0 ** -24 * mag * (1 + HALF[self.dtype]) + HALF[self.dtype] * ref.abs())
            assert bool((err <= 0).all()), (e, err.max().item())
        rest = ((flat < 0) | (flat >= self.E)).nonzero().reshape(-1)
        assert bool((self.out[rest] == 7.0).all())


@FORMS
@pytest.mark.parametrize("M,E,topk,K,N", [(1, 1, 1, 32, 1), (1, 8, 2, 64, 16), (1, 128, 8, 2048, 128), (3, 4, 2, 96, 17),
                                          (7, 1, 1, 2080, 101), (23, 16, 4, 160, 100), (5, 9, 3, 288, 65),
                                          (40, 5, 2, 544, 130), (2, 3, 3, 4128, 33)])
@pytest.mark.parametrize("per_pair", [False, True])
def test_few_pairs(x, dtype, M, E, topk, K, N, per_pair):
    Case(M, E, topk, K, N, x, dtype, per_pair=per_pair).check()


@FORMS
@pytest.mark.parametrize("M,E,topk,K,N,block", [(200, 3, 2, 256, 300, 128), (130, 1, 1, 2048, 256, 128),
                                                (600, 4, 2, 96, 70, 64), (333, 2, 1, 1056, 515, 1024),
                                                (129, 1, 1, 32, 5, 16), (500, 7, 3, 768, 264, 200)])
def test_many_pairs(x, dtype, M, E, topk, K, N, block):
    Case(M, E, topk, K, N, x, dtype, block=block, skew=True).check()
    Case(M, E, topk, K, N, x, dtype, block=block, per_pair=True, seed=1).check()


@pytest.mark.parametrize("x,M,E,topk,K,N,block,form", mc.FORMS)
@pytest.mark.parametrize("per_pair", [False, True])
def test_every_form(x, M, E, topk, K, N, block, form, per_pair):
    for dtype in (torch.bfloat16, torch.float32) if x == "codes" else ({"bf16": torch.bfloat16, "f32": torch.float32}[x],):
        Case(M, E, topk, K, N, "codes" if x == "codes" else "rows", dtype, block=block, per_pair=per_pair,
             pad_out=8 if per_pair else 0).check()


@pytest.mark.parametrize("x,M,E,topk,K,N,block,form", mc.POPULAR)
def test_popular_experts_in_several_passes(x, M, E, topk, K, N, block, form):
    c = Case(M, E, topk, K, N, "codes" if x == "codes" else "rows", torch.bfloat16, block=block, skew=True)
    assert int((c.ids == 0).sum()) > 3 * block
    c.check()


@pytest.mark.parametrize("x,dtype", [("codes", torch.bfloat16), ("rows", torch.bfloat16)], ids=["codes", "bf16"])
@pytest.mark.parametrize("block", [16, 32, 64])
def test_small_blocks_in_any_order(x, dtype, block):
    """Blocks of an expert that are partly filled, empty or apart from each other, of the widest form."""
    c = Case(1200, 3, 1, 160, 4400, x, dtype, block=block)
    c.ids[torch.rand(1200, 1, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") < 0.5] = -1
    ahead, behind = [], []
    for e in range(3):
        pairs = (c.ids.reshape(-1) == e).nonzero().reshape(-1).tolist()
        mine = []
        for size in (block, block, 3, block, 0, block - 1) + (block,) * 99:
            if pairs:
                mine.append((pairs[:size] + [c.numel] * (block - size))[:block])
                pairs = pairs[size:]
        mine[-1] += [c.numel] * (block - len(mine[-1]))
        ahead += [(b, e) for b in mine[:5]]
        behind += [(b, e) for b in mine[5:]]
    blocks = ahead + behind
    srt, ids, npp = c.routing
    assert len(blocks) <= ids.numel()
    srt[:len(blocks) * block] = torch.tensor([b for b, _ in blocks], dtype=torch.int32).reshape(-1)
    ids[:len(blocks)] = torch.tensor([e for _, e in blocks], dtype=torch.int32)
    npp.fill_(len(blocks) * block)
    c.check()


@FORMS
@pytest.mark.parametrize("block", [1, 16, 48, 64, 128, 256])
def test_blocks(x, dtype, block):
    Case(61, 6, 2, 320, 192, x, dtype, block=block, skew=True).check()


@FORMS
@pytest.mark.parametrize("M,E", [(90, 100), (300, 100), (2000, 100)])
def test_many_experts(x, dtype, M, E):
    Case(M, E, 4, 512, 520, x, dtype, block=64, skew=True).check()


@FORMS
def test_no_pairs_and_no_local_experts(x, dtype):
    c = Case(4, 4, 2, 64, 32, x, dtype)
    c.ids.fill_(-1)
    c.route()
    c.run()
    assert bool((c.out == 7.0).all())
    c.numel, c.ids, c.out = 0, c.ids[:0], c.out[:0]
    c.route()
    c.run()


@FORMS
@pytest.mark.parametrize("pad_out,N", [(0, 66), (1, 64), (4, 64), (3, 61)])
def test_strided_outputs(x, dtype, pad_out, N):
    Case(33, 4, 2, 128, N, x, dtype, pad_out=pad_out).check()
    Case(300, 2, 2, 128, N, x, dtype, pad_out=pad_out, block=128).check()


@FORMS
@pytest.mark.parametrize("M", [9, 400])
def test_strided_rows(x, dtype, M):
    c = Case(M, 3, 2, 160, 40, x, dtype, block=128)
    if c.xs is None:
        wide = torch.full((M, 160 + 24), float("nan"), dtype=dtype, device="cuda")
        wide[:, 8:168] = c.x
        c.x = wide[:, 8:168]
    else:
        wide, ws = (torch.full((M, n), 255, dtype=torch.uint8, device="cuda") for n in (160, 10))
        wide[:, 16:96], ws[:, 3:8] = c.x, c.xs
        c.x, c.xs = wide[:, 16:96], ws[:, 3:8]
    c.check()


@FORMS
@pytest.mark.parametrize("M,block", [(6, 16), (300, 128)])
def test_nan_and_extreme_scales(x, dtype, M, block):
    """NaN blocks of weights and of rows reach the sums that hold them and no others; scales at both ends."""
    c = Case(M, 2, 1, 224, 50, x, dtype, block=block)
    c.s[0, 3, 6], c.s[1, 0, 0], c.s[1, 49, 2] = 255, 255, 255
    c.s[0, 20], c.s[0, 21] = 0, 1
    c.s[1, 20] = 200
    if c.xs is not None:
        c.xs[2, 1] = 255
        c.xs[3] = 20
        c.xs[4] = 160
    c.run()
    xv = c.x.double() if c.xs is None else value(c.x, c.xs)
    wv = value(c.W.view(-1, 112), c.s.view(-1, 7)).view(2, 50, 224)
    flat = c.ids.reshape(-1)
    for p in range(c.numel):
        e = int(flat[p])
        if not 0 <= e < 2:
            continue
        ref, mag = wv[e] @ xv[p], wv[e].abs() @ xv[p].abs()
        got = c.out[p].double()
        assert torch.equal(got.isnan(), ref.isnan())
        ok = ~ref.isnan()
        tiny = 225 * 2.0 ** -149 + torch.finfo(dtype).smallest_normal * HALF[dtype] * 2
        bound = 225 * 2.0 ** -24 * mag * (1 + HALF[dtype]) + HALF[dtype] * ref.abs() + tiny
        assert bool(((got - ref).abs() <= bound)[ok].all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,block", [(6, 16), (300, 128)])
def test_infinite_and_nan_rows(dtype, M, block):
    c = Case(M, 2, 1, 160, 48, "rows", dtype, block=block)
    inf, nan = float("inf"), float("nan")
    c.x[0, 7], c.x[1, 159], c.x[2, 0], c.x[2, 1], c.x[3, 40] = inf, -inf, inf, -inf, nan
    c.run()
    wv = value(c.W.view(-1, 80), c.s.view(-1, 5)).view(2, 48, 160)
    flat = c.ids.reshape(-1)
    for p in range(M):
        e = int(flat[p])
        if not 0 <= e < 2:
            continue
        ref = (wv[e] * c.x[p].double()).sum(dim=1)
        got = c.out[p].double()
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(got.isinf(), ref.isinf()) and torch.equal(got[ref.isinf()], ref[ref.isinf()])
        ok = ref.isfinite()
        mag = wv[e].abs() @ torch.nan_to_num(c.x[p].double().abs(), posinf=0.0)
        assert bool(((got - ref).abs() <= 161 * 2.0 ** -24 * mag * 2 + HALF[dtype] * ref.abs())[ok].all())


@FORMS
@pytest.mark.parametrize("M,block", [(23, 64), (500, 128)])
def test_repeats_streams_and_graphs(x, dtype, M, block):
    c = Case(M, 8, 2, 352, 130, x, dtype, block=block)
    first = c.run().clone()
    assert torch.equal(c.run(), first)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.out.zero_()
    c.run()
    first = c.out.clone()
    c.out.zero_()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        c.run()
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(c.out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for turn in range(3):
        c.ids.copy_(c.ids.roll(turn, dims=0))
        c.W.copy_(c.W.roll(1, dims=1))
        r = mb.mol_align_block_size(c.ids, None, c.E, 1, block)
        for a, b in zip(c.routing, r):
            a.copy_(b)
        c.out.zero_()
        want = c.run().clone()
        c.out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)


def test_weights_past_32_bits():
    """Experts whose weights begin past 4 GiB."""
    E, N, K = 3, 1 << 20, 4064
    W = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    assert W.numel() > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.tensor([0, 5, N // 2, N - 17, N - 1], device="cuda")
    for e in range(E):
        W[e, rows], s[e, rows] = codes(5, K, g)
    for M, block in ((6, 16), (60, 128)):
        x, xs = codes(M, K, g)
        ids = (torch.arange(M, device="cuda") % E).to(torch.int32).view(M, 1)
        out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        r = mb.mol_align_block_size(ids, None, E, 1, block)
        mb.mol_moe_gemm_mx4(x, 1, W, s, *r, M, block, out, x_scales=xs)
        xv = value(x, xs)
        for p in range(M):
            w = value(W[p % E, rows], s[p % E, rows])
            ref, mag = w @ xv[p], w.abs() @ xv[p].abs()
            assert bool(((out[p, rows].double() - ref).abs() <= (K + 1) * 2.0 ** -24 * mag * 2 + 2.0 ** -8 * ref.abs()).all())
            assert int((out[p] != 0).sum()) <= 5


@FORMS
def test_wide_form_of_strided_rows_with_nan_and_infinity(x, dtype):
    """The widest form: rows of x and of out apart from each other, NaN blocks of weights and rows, infinite rows, and
    a graph's replay."""
    c = Case(1000, 2, 1, 224, 6401, x, dtype, block=128, pad_out=7)
    c.s[0, 3, 6], c.s[1, 0, 0], c.s[1, 6400, 2] = 255, 255, 255
    c.s[0, 20], c.s[1, 21] = 0, 200
    if c.xs is None:
        wide = torch.full((1000, 224 + 24), float("nan"), dtype=dtype, device="cuda")
        wide[:, 8:232] = c.x
        c.x = wide[:, 8:232]
        c.x[3, 5], c.x[4, 223], c.x[5, 100] = float("inf"), -float("inf"), float("nan")
        xv = c.x.double()
    else:
        wide, ws = (torch.full((1000, n), 255, dtype=torch.uint8, device="cuda") for n in (160, 10))
        wide[:, 16:128], ws[:, 2:9] = c.x, c.xs
        c.x, c.xs = wide[:, 16:128], ws[:, 2:9]
        c.xs[2, 1], c.xs[3], c.xs[4] = 255, 20, 160
        xv = value(c.x.contiguous(), c.xs.contiguous())
    wv = value(c.W.view(-1, 112), c.s.view(-1, 7)).view(2, 6401, 224)
    first = c.run().clone()
    flat = c.ids.reshape(-1)
    for e in range(2):
        p = (flat == e).nonzero().reshape(-1)
        odd = ~xv[p].isfinite().all(dim=1)
        for q in p[odd].tolist():  # term by term: a product of matrices may meet infinities in another order
            ref = (wv[e] * xv[q]).sum(dim=1)
            assert torch.equal(first[q].isnan(), ref.isnan()) and torch.equal(first[q].isinf(), ref.isinf())
            assert torch.equal(first[q].double()[ref.isinf()], ref[ref.isinf()])
        p = p[~odd]
        w0 = torch.nan_to_num(wv[e])
        ref, mag = xv[p] @ w0.t(), xv[p].abs() @ w0.abs().t()
        nan = wv[e].isnan().any(dim=1)
        got = first[p].double()
        assert bool(got[:, nan].isnan().all())
        tiny = 225 * 2.0 ** -149 + torch.finfo(dtype).smallest_normal * HALF[dtype] * 2
        err = (got - ref).abs() - (225 * 2.0 ** -24 * mag * (1 + HALF[dtype]) + HALF[dtype] * ref.abs() + tiny)
        assert bool((err[:, ~nan] <= 0).all())
    assert bool((first[(flat < 0) | (flat >= 2)] == 7.0).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for _ in range(3):
        c.out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out.nan_to_num(123.0), first.nan_to_num(123.0))

"""The grouped GEMM over 4-bit weights through the C ABI against its 64-bit definition, element by
element, within the bound of fp32 sums and one rounding (plain64.product)."""
import numpy as np
import pytest
import torch

from tests import plain64
from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def draw(M, E, topk, K, N, group, zeros, dtype, row_div, seed, ids=None, sentinels=True):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    numel = M * topk
    if ids is None:
        ids = torch.stack([torch.randperm(E, generator=g)[:topk] for _ in range(M)]) if M else \
            torch.empty(0, topk, dtype=torch.int64)
        if sentinels and numel > 4:
            ids.view(-1)[torch.randperm(numel, generator=g)[:numel // 8 + 1]] = -1
    st = dict(ids=ids.to(torch.int32), E=E, numel=numel, row_div=row_div, group=group,
              x=torch.randn(-(-numel // row_div), K, generator=g).to(dt),
              W=torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8),
              s=(torch.randn(E, N, K // group, generator=g) * 0.01).to(dt),
              z=torch.randint(0, 256, (E, N, K // group), generator=g, dtype=torch.uint8)
              if zeros else None)
    return st


def call(st, block_m=64, out=None, x=None):
    dev = {k: v.cuda() if torch.is_tensor(v) else v for k, v in st.items()}
    r = mb.mol_align_block_size(dev["ids"], None, st["E"], 1, block_m)
    if out is None:
        out = torch.full((st["numel"], st["W"].shape[1]), 3.0, dtype=st["x"].dtype, device="cuda")
    return mb.mol_moe_gemm_q4(dev["x"] if x is None else x, st["row_div"], dev["W"], dev["s"], *r,
                              st["numel"], block_m, out, zeros=dev["z"])


def check(st, got, fill=3.0):
    got = got.float().cpu().numpy().astype(np.float64)
    ids = st["ids"].reshape(-1).numpy()
    x = st["x"].double().numpy()
    half = torch.finfo(st["x"].dtype).eps / 2
    for p, t in enumerate(ids):
        if not 0 <= t < st["E"]:
            assert np.all(got[p] == fill), f"row {p} of a pair without an expert was written"
            continue
        W, mag = plain64.dequantise(st["W"][t].numpy(), st["s"][t].double().numpy(),
                                    None if st["z"] is None else st["z"][t].numpy())
        ref, e = plain64.product(W, mag, x[p // st["row_div"]])
        plain64.within(got[p], ref, e * (1 + half) + half * np.abs(ref) + 2.0 ** -134, f"pair {p}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,E,topk,chunks,N,pair_rows", [
    (1, 8, 2, 1, 1, False),        # one group a row, one column
    (1, 128, 8, 4, 40, False),
    (3, 1, 1, 5, 17, False),       # a single matrix; rows that end inside a 128-wide step
    (7, 5, 3, 7, 31, True),
    (40, 4, 2, 3, 48, False),      # more than 16 pairs an expert
])
def test_sizes(dtype, group, zeros, M, E, topk, chunks, N, pair_rows):
    st = draw(M, E, topk, group * chunks, N, group, zeros, dtype, 1 if pair_rows else topk,
              seed=M + N)
    check(st, call(st))


@pytest.mark.parametrize("block_m", [1, 16, 48, 64, 200, 1024])
def test_many_pairs_of_one_expert(block_m):
    """Blocks of every length: up to 150 pairs of an expert, several passes of 64."""
    st = draw(150, 3, 1, 160, 24, 32, True, "bf16", 1, seed=3)
    st["ids"][:] = torch.tensor([1, 1, 1, 1, 2])[torch.arange(150) % 5].view(150, 1).int()
    check(st, call(st, block_m))


def test_hidden_sizes_of_the_decode_layers():
    check(*(lambda s: (s, call(s)))(draw(3, 16, 8, 2048, 96, 128, False, "bf16", 8, seed=5)))
    check(*(lambda s: (s, call(s)))(draw(2, 16, 8, 6144, 32, 64, True, "bf16", 8, seed=6)))
    check(*(lambda s: (s, call(s)))(draw(1, 4, 2, 8192, 16, 32, True, "f32", 2, seed=7)))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs,block_m", [(3, 16), (70, 1), (70, 64)])
def test_the_longest_rows(group, dtype, pairs, block_m):
    """256 groups a row: scales and x in many stages, split k's and whole (blocks of one pair make
    enough items for that)."""
    st = draw(1100 if block_m == 1 else pairs, 2, 1, 256 * group, 72, group, True, dtype, 1,
              seed=group)
    st["ids"][pairs:] = -1
    check(st, call(st, block_m))


def test_weights_past_32_bits():
    """An expert more than 4 GiB into the weights: bit for bit what it gives alone."""
    E, N, K, G = 520, 4096, 4096, 128
    W = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(E, N, K // G, dtype=torch.bfloat16, device="cuda")
    assert W.numel() > 2**32
    gen = torch.Generator("cuda").manual_seed(22)
    W[E - 1].random_(0, 256, generator=gen)
    sc[E - 1].normal_(0, 0.01, generator=gen)
    x = torch.randn(5, K, generator=gen, device="cuda").bfloat16()
    outs = []
    for w, s in ((W, sc), (W[E - 1:].clone(), sc[E - 1:].clone())):
        ids = torch.full((5, 1), w.shape[0] - 1, dtype=torch.int32, device="cuda")
        out = torch.zeros(5, N, dtype=torch.bfloat16, device="cuda")
        outs.append(mb.mol_moe_gemm_q4(x, 1, w, s, *mb.mol_align_block_size(ids, None,
                                                                           w.shape[0], 1, 16),
                                       5, 16, out))
    assert torch.equal(*outs) and outs[0].abs().max() > 0


def test_two_calls_at_once():
    a, b = (draw(23, 16, 8, 256, 64, 128, True, "bf16", 8, seed=s) for s in (21, 22))
    wa, wb = call(a), call(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        ga = call(a)
    with torch.cuda.stream(s2):
        gb = call(b)
    torch.cuda.synchronize()
    assert torch.equal(ga, wa) and torch.equal(gb, wb)


def test_ids_past_the_experts_and_no_pairs():
    st = draw(4, 5, 2, 64, 20, 32, False, "f32", 2, seed=8)
    st["ids"] = torch.tensor([[5, -7], [100, 2], [-1, -1], [0, 4]], dtype=torch.int32)
    check(st, call(st))
    st["ids"][:] = -1
    check(st, call(st))
    empty = draw(0, 5, 2, 64, 20, 32, False, "f32", 2, seed=9)
    assert call(empty).shape == (0, 20)


def test_strided_rows_and_guards():
    st = draw(9, 6, 2, 96, 23, 32, True, "bf16", 2, seed=10)
    wide = torch.full((9, 96 + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:104] = st["x"].cuda()
    raw = torch.full((18 * 31 + 200,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = raw[100:100 + 18 * 31].view(18, 31)[:, 3:26]
    call(st, out=out, x=wide[:, 8:104])
    check(st, out)
    keep = torch.ones_like(raw, dtype=torch.bool)
    keep[100:100 + 18 * 31].view(18, 31)[:, 3:26] = False
    assert torch.all(raw[keep] == 3.0)


def test_a_bad_row_stays_in_its_row():
    st = draw(5, 2, 2, 128, 32, 64, False, "bf16", 2, seed=11)
    clean = call(st)
    st["x"][2, 7] = float("nan")
    st["x"][3, 100] = float("inf")
    got = call(st)
    other = torch.tensor([0, 1, 2, 3, 8, 9], device="cuda")
    assert torch.equal(got[other], clean[other])
    rows = torch.tensor([p for p in (4, 5) if st["ids"].view(-1)[p] >= 0], device="cuda")
    assert torch.all(torch.isnan(got[rows]))


def test_repeats_bit_for_bit_on_a_stream_and_in_a_graph():
    st = draw(23, 16, 8, 256, 64, 128, True, "bf16", 8, seed=12)
    first = call(st)
    assert torch.equal(first, call(st))
    dev = {k: v.cuda() if torch.is_tensor(v) else v for k, v in st.items()}
    out = torch.full_like(first, 3.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = mb.mol_align_block_size(dev["ids"], None, 16, 1, 64)
        mb.mol_moe_gemm_q4(dev["x"], 8, dev["W"], dev["s"], *r, 184, 64, out, zeros=dev["z"])
    s.synchronize()
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mb.mol_moe_gemm_q4(dev["x"], 8, dev["W"], dev["s"], *r, 184, 64, out, zeros=dev["z"])
    for seed in (1, 2, 3):
        st["x"] = torch.randn(23, 256, generator=torch.Generator().manual_seed(seed)).bfloat16()
        dev["x"].copy_(st["x"])
        out.fill_(3.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call(st))


def test_refusals():
    st = {k: v.cuda() if torch.is_tensor(v) else v
          for k, v in draw(4, 3, 2, 64, 8, 32, True, "bf16", 2, seed=13).items()}
    r = mb.mol_align_block_size(st["ids"], None, 3, 1, 16)
    out = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")

    def go(**kw):
        a = dict(x=st["x"], W=st["W"], s=st["s"], z=st["z"], out=out, numel=8, r=r)
        a.update(kw)
        return mb.mol_moe_gemm_q4(a["x"], 2, a["W"], a["s"], *a["r"], a["numel"], 16, a["out"],
                                  zeros=a["z"])
    go()
    for kw in (dict(x=st["x"][:3]), dict(x=st["x"].cpu()), dict(x=st["x"][:, :32]),
               dict(out=out[:, :7]), dict(out=out[:7]), dict(z=st["z"][:2]),
               dict(s=st["s"][:, :7]), dict(W=st["W"][:, :, ::2]), dict(r=(r[0][:3], *r[1:]))):
        with pytest.raises(ValueError):
            go(**kw)
    for kw in (dict(x=st["x"].float()), dict(out=out.float()), dict(z=st["z"].int()),
               dict(W=st["W"].int())):
        with pytest.raises(TypeError):
            go(**kw)

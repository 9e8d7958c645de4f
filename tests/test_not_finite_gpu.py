"""Infinities, NaN and sums that leave fp32's range, through the C ABI: the 4-bit product and the whole
layer give what their 64-bit definitions give (the same infinities, NaN in the same places, finite values
within the bound), and every other row is bit for bit what it is beside clean rows."""
import numpy as np
import pytest
import torch

from tests import plain64
from tests.test_moe_layer_gpu import Layer
from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def agrees(got, ref, bound, what=""):
    """NaN and infinities exactly where and as the definition has them, the rest within bound."""
    got = np.asarray(got, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN\n{got}\n{ref}"
    inf = np.isinf(ref)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], ref[inf]), f"{what}: infinities"
    rest = np.isfinite(ref)
    if rest.any():
        plain64.within(got[rest], ref[rest], np.asarray(bound)[rest], what)


# few items (16 rows each, k's split), and enough of them for items of 64 rows and more; rows of x that
# fit a stage and rows that take several; experts of up to 4, 16 and 64 pairs
@pytest.mark.parametrize("E,M,topk,N,popular", [(2, 12, 2, 40, 0), (400, 20, 20, 65, 12), (400, 60, 10, 65, 60)])
@pytest.mark.parametrize("chunks", ["short", "long"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_4bit_product(dtype, group, chunks, E, M, topk, N, popular):
    K = 256 if chunks == "short" else 2304
    g = torch.Generator().manual_seed(K + group + M)
    dt = DT[dtype]
    ids = torch.stack([torch.randperm(E, generator=g)[:topk] for _ in range(M)]).int()
    ids[:popular, 0] = 1
    W = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    s = (torch.randn(E, N, K // group, generator=g) * 1e-3).to(dt)
    z = torch.randint(0, 16, (E, N, K // group), generator=g, dtype=torch.uint8)
    x = torch.randn(M, K, generator=g).to(dt)
    clean = x.clone()
    x[1, 7] = INF
    x[2, K - 1], x[2, 40] = -INF, INF
    x[4, 3] = NAN
    x[5] *= 3e37                     # (16 + q) x and the sum of x pass the largest float
    x[5].clamp_(-1e38, 1e38)
    x[7, 100] = 3e38
    x[8, 64] = -INF
    r = mb.mol_align_block_size(ids.cuda(), None, E, 1, 64)
    dev = [t.cuda() for t in (W, s, z)]

    def call(x):
        out = torch.zeros(M * topk, N, dtype=dt, device="cuda")
        return mb.mol_moe_gemm_q4(x.cuda(), topk, dev[0], dev[1], *r, M * topk, 64, out, zeros=dev[2])
    got, want = call(x).view(M, topk, N), call(clean).view(M, topk, N)
    bad = [1, 2, 4, 5, 7, 8]
    good = torch.ones(M, dtype=torch.bool)
    good[bad] = False
    assert torch.equal(got[good.cuda()], want[good.cuda()])
    got, half = got.float().cpu().numpy(), torch.finfo(dt).eps / 2
    seen = set()
    for m in bad:
        for k in range(min(topk, 3)):
            t = int(ids[m, k])
            w, mag = plain64.dequantise(W[t].numpy(), s[t].double().numpy(), z[t].numpy())
            with np.errstate(invalid="ignore"):
                ref, e = plain64.product(w, mag, x[m].double().numpy())
            agrees(got[m, k], ref, e * (1 + half) + half * np.abs(ref), f"row {m}, slot {k}")
            seen |= {"inf"} if np.isinf(ref).any() else set()
            seen |= {"finite"} if np.isfinite(ref).all() else set()
    assert seen == {"inf", "finite"}


def layer64(la, x, ids, w, lora):
    with np.errstate(invalid="ignore", over="ignore"):
        return plain64.layer(x.double().numpy(), la.expert(la.gu), la.expert(la.dn), ids.numpy(),
                             w.double().numpy(), torch.finfo(la.dt).eps, la.ad64,
                             None if lora is None else lora.numpy())


def positive_4bit(la, seed):
    """Weights of one sign a row: positive, but for odd rows of down."""
    g = torch.Generator().manual_seed(seed)
    for i, part in enumerate((la.gu, la.dn)):
        q, s, _ = part
        n = torch.randint(9, 16, (*q.shape, 2), generator=g, dtype=torch.uint8)
        if i:
            n[:, 1::2] = 16 - n[:, 1::2]
        q.copy_(n[..., 0] | (n[..., 1] << 4))
        s.copy_(s.abs() + 0.001)
        la.w.tensors[i].copy_(q)
        la.w.tensors[2 + i].copy_(s)


@pytest.mark.parametrize("M,topk,E,H,I", [(7, 3, 5, 256, 128), (60, 8, 400, 128, 128), (60, 8, 20, 2304, 128)])
@pytest.mark.parametrize("adapters", [False, True])
@pytest.mark.parametrize("dtype,group", [("bf16", 32), ("bf16", 64), ("bf16", 128), ("f32", 32), ("f32", 128)])
def test_infinite_x_over_a_4bit_layer(dtype, group, adapters, M, topk, E, H, I):
    la = Layer(dtype, H, I, E, 2 if adapters else 0, 8, group, seed=H + M)
    positive_4bit(la, 1)
    x, ids, w, lora = la.step(M, topk, sentinels=False)
    x = x.abs() * 0.1
    if adapters:
        lora[1], lora[3] = -1, -1
    clean = la.call(x, ids, w, lora)
    x[1, 9], x[3, 5] = INF, NAN
    got = la.call(x, ids, w, lora)
    keep = torch.ones(M, dtype=torch.bool)
    keep[[1, 3]] = False
    assert torch.equal(got[keep.cuda()], clean[keep.cuda()])
    rows = torch.tensor([1, 3])
    ref, bound = layer64(la, x[rows], ids[rows], w[rows], None if lora is None else lora[rows])
    assert np.isinf(ref[0]).all() and np.isnan(ref[1]).all()
    agrees(got[rows.cuda()].float().cpu().numpy(), ref, bound)


# ---- down per token (one token; up to three with large items), without adapters


@pytest.mark.parametrize("M,topk,E,I", [(1, 1, 3, 128), (1, 2, 3, 256), (1, 8, 9, 128), (1, 20, 24, 128), (2, 8, 9, 2048),
                                        (3, 8, 9, 2048)])
@pytest.mark.parametrize("dtype,group", [("bf16", 32), ("bf16", 64), ("bf16", 128), ("f32", 32), ("f32", 128)])
def test_infinite_x_of_one_token_over_a_4bit_layer(dtype, group, M, topk, E, I):
    la = Layer(dtype, 128, I, E, group=group, seed=I + topk)
    positive_4bit(la, 2)
    x, ids, w, lora = la.step(M, topk, sentinels=False)
    ids[0, topk // 2] = -1 if topk > 2 else ids[0, topk // 2]
    x = x.abs() * 0.1
    clean = la.call(x, ids, w, lora)
    la.check(x, ids, w, lora, clean)
    x[M - 1, 9] = INF
    got = la.call(x, ids, w, lora)
    assert torch.equal(got[:M - 1], clean[:M - 1])
    ref, bound = layer64(la, x[M - 1:], ids[M - 1:], w[M - 1:], None)
    assert np.isinf(ref).all()
    agrees(got[M - 1:].float().cpu().numpy(), ref, bound)
    x[M - 1, 9] = NAN
    assert torch.all(torch.isnan(la.call(x, ids, w, lora)[M - 1]))


@pytest.mark.parametrize("M", [1, 5])
@pytest.mark.parametrize("dtype,group", [("bf16", 0), ("f32", 0), ("bf16", 64), ("f32", 32)])
def test_an_infinite_router_weight(dtype, group, M):
    la = Layer(dtype, 96 if not group else 128, 64, 6, group=group, seed=33)
    x, ids, w, lora = la.step(M, 3, sentinels=False)
    w[0, 1] = INF
    ref, bound = layer64(la, x, ids, w, lora)
    assert np.isinf(ref[0]).all()
    agrees(la.call(x, ids, w, lora).float().cpu().numpy(), ref, bound)


def exact_h(M, E=4, H=64, I=32, S=0):
    """A bf16 layer and tokens whose h is exact in bf16 at one place: gate 32 and up 2 there, from x = 1 at
    its first element, so h = silu(32) * 2 = 64 and its second bf16 term is zero."""
    la = Layer("bf16", H, I, E, S, 8 if S else 0, seed=34)
    la.gu[:, 5], la.gu[:, I + 5] = 0, 0
    la.gu[:, 5, 0], la.gu[:, I + 5, 0] = 32, 2
    la.w.tensors[0].copy_(la.gu)
    x, ids, w, lora = la.step(M, 2, sentinels=False)
    x[:, 0] = 1
    return la, x, ids, w, lora


@pytest.mark.parametrize("M", [1])
def test_an_infinite_down_weight(M):
    la, x, ids, w, lora = exact_h(M)
    la.dn[:, 7, 5], la.dn[:, 9, 5], la.dn[:, 60, 4] = INF, -INF, INF
    la.w.tensors[1].copy_(la.dn)
    ref, bound = layer64(la, x, ids, w, lora)
    assert np.isinf(ref[:, [7, 9]]).all() and np.isfinite(ref).sum() == 61 * M
    agrees(la.call(x, ids, w, lora).float().cpu().numpy(), ref, bound)


# ---- an infinite weight where h or s is exact in bf16 (its second term is zero)


@pytest.mark.parametrize("M", [3, 5, 40])
def test_an_infinite_down_weight_of_more_tokens(M):
    test_an_infinite_down_weight(M)


def adapters64(la, i, t):
    """Adapter tensor i of the layer becomes t (host)."""
    la.ad.tensors[i].copy_(t)
    la.ad64 = tuple(t.double().numpy() if j == i else v for j, v in enumerate(la.ad64))


@pytest.mark.parametrize("M", [5, 40])
@pytest.mark.parametrize("which", ["gate_up_B", "down_A", "down_B"])
def test_an_infinite_adapter_weight(which, M):
    """s of the adapters is exact too: A's first rows pick x[0] = 1, and h[5] = 64."""
    la, x, ids, w, lora = exact_h(M, S=2)
    x[:, 1:] = 0
    lora[:] = torch.arange(M).int() % 3 - 1
    host = [t.cpu() for t in la.ad.tensors[:4]]
    A1, B1, A2, B2 = host
    A1[:, :, 0] = 0.5
    B1[:, (5, 32 + 5)] = 0                   # g and u of column 5 stay 32 and 2
    A2[:] = 0
    A2[:, :, 5] = 0.25                       # s = 16 exactly
    if which == "gate_up_B":
        B1[:, 11, 3] = INF                   # g = inf there: h = inf * u
        A2[:, :, 11], B2[:] = 0.25, 0.5
    elif which == "down_A":
        A2[:, 2, 5] = INF                    # s = inf at rank 2
    else:
        B2[:, 7, 1], B2[:, 9, 1] = INF, -INF
    for i, t in enumerate(host):
        adapters64(la, i, t)
    ref, bound = layer64(la, x, ids, w, lora)
    with_adapter = lora.numpy() >= 0
    assert not np.isfinite(ref[with_adapter]).all(axis=1).any() and np.isfinite(ref[~with_adapter]).all()
    assert np.isinf(ref[with_adapter]).any()
    agrees(la.call(x, ids, w, lora).float().cpu().numpy(), ref, bound)

"""The balance loss, its counts and its gradient against their definitions in 64 bits, and the gradient against
differences of the loss.

Tolerances. A score: the difference l - max rounds once (|l| < 64: an absolute 2^-19 in the exponent), exp, the
sums of at most E = 8191 scores (64 lanes of 128: 134 additions in a row), the division: 2^-17 relative in all.
Over a workgroup's tokens: at most 40 additions of 2^-24 more. P_e and the loss: 2^-16.
The gradient p q (b - sum p b): p within 2^-17, q within 2^-20, the difference within 2^-16 of max |b|; b itself from whole
numbers within 2^-23: |error| <= 2^-15 p q max |b|, and half a step of the type."""
import numpy as np
import pytest
import torch

from tests import mx4_defs as d
from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu

BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
SCORES = pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])


def draw(M, E, k, dtype, seed, sigma=2.0, skew=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn(M, E, generator=g, device="cuda") * sigma - skew * torch.arange(E, device="cuda") / E
    l = l.to(dtype)
    ids, _ = mb.mol_router_topk(l, k)
    mask = torch.rand(M, generator=g, device="cuda") < 0.8
    return l, ids, mask


def check(l, ids, mask, sigmoid, alpha=0.5, up=None, counts=None):
    sc = mb.MOL_SCORE_SIGMOID if sigmoid else mb.MOL_SCORE_SOFTMAX
    loss, cnt, sums = mb.mol_router_balance(l, ids, sc, alpha, token_mask=mask)
    use = cnt if counts is None else counts
    grad = mb.mol_router_balance_grad(l, use, ids.shape[1], sc, alpha, token_mask=mask, grad_loss=up)
    torch.cuda.synchronize()
    host = l.float().cpu().numpy()
    rl, rc, rp, rg = d.balance(host, ids.cpu().numpy(), None if mask is None else mask.cpu().numpy(), sigmoid, alpha,
                               1.0 if up is None else float(up), None if counts is None else counts.cpu().numpy())
    assert np.array_equal(cnt.cpu().numpy(), rc)
    assert np.all(np.abs(sums.double().cpu().numpy() - rp) <= 2.0 ** -16 * rp + 1e-37)
    assert abs(float(loss) - rl) <= 2.0 ** -16 * abs(rl)
    # p q and max |b| of the bound
    c = rc if counts is None else counts.cpu().numpy().astype(np.int64)
    E, k, n = l.shape[1], ids.shape[1], max(int(c[-1]), 1)
    b = np.abs((E * c[:E] - k * n) * (alpha / (k * float(n) * n)) * (1.0 if up is None else float(up))).max()
    there = ~np.isnan(host) & (host > -np.inf)
    with np.errstate(all="ignore"):
        big = np.where(there, host.astype(np.float64), -np.inf)
        m = big.max(axis=1, keepdims=True)
        if sigmoid:
            sh = np.minimum(m, 0)
            w = np.where(there, np.where(big > 0, 1 / (1 + np.exp(-big)), np.exp(np.minimum(big, 0) - sh) / (1 + np.exp(np.minimum(big, 0)))), 0)
            q = 1 / (1 + np.exp(big))
        else:
            w = np.where(there, np.where(big == m, 1.0, np.exp(big - m)), 0)
            q = 1.0
        pq = np.nan_to_num(w / w.sum(axis=1, keepdims=True) * q)
    half = 2.0 ** -8 if l.dtype is torch.bfloat16 else 2.0 ** -24
    got = grad.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - rg) <= (2.0 ** -15 * pq * b) * (1 + half) + half * np.abs(rg) + 1e-37)
    off = ~there if mask is None else ~there | ~mask.cpu().numpy()[:, None]
    assert np.all(got[off] == 0)
    return loss, cnt, sums, grad


@BOTH
@SCORES
@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 128, 8), (23, 128, 8), (7, 4, 2), (16, 64, 4), (17, 65, 5), (64, 129, 7),
                                   (65, 160, 8), (33, 256, 16), (9, 257, 3), (16, 512, 8), (17, 513, 12), (130, 1024, 8),
                                   (3, 1025, 9), (30, 2049, 9), (40, 8191, 33), (1000, 100, 6), (9001, 60, 4)])
def test_sizes(dtype, sigmoid, M, E, k):
    l, ids, mask = draw(M, E, k, dtype, M * 31 + E)
    check(l, ids, mask, sigmoid)
    check(l, ids, None, sigmoid, alpha=0.01, up=torch.tensor([2.5], device="cuda"))


@BOTH
@SCORES
def test_an_uneven_batch(dtype, sigmoid):
    l, ids, mask = draw(700, 32, 2, dtype, 3, sigma=0.5, skew=6.0)
    loss, cnt, _, _ = check(l, ids, mask, sigmoid, alpha=1.0)
    assert float(loss) > 1.2 and int(cnt[0]) > 4 * int(cnt[20])


@SCORES
def test_an_even_batch_has_loss_alpha(sigmoid):
    l = torch.zeros(64, 16, device="cuda")
    ids = (torch.arange(128, device="cuda") % 16).to(torch.int32).view(64, 2)
    loss, cnt, sums, grad = check(l, ids, None, sigmoid, alpha=0.25)
    assert float(loss) == 0.25 and bool((grad == 0).all())


@BOTH
@SCORES
@pytest.mark.parametrize("M", [40, 300])
def test_masked_rows_and_special_logits(dtype, sigmoid, M):
    inf, nan = float("inf"), float("nan")
    l, ids, mask = draw(M, 96, 5, dtype, 7)
    l[0] = -inf                       # no candidate: the token does not count
    l[1] = nan
    l[2, 3:] = -inf                   # fewer candidates than slots
    l[3, ::2] = nan
    l[4] = torch.finfo(dtype).min     # finite: candidates, evenly
    l[5, 9] = inf
    l[6, 5], l[6, 77] = inf, inf
    l[7] = -inf
    l[7, 95] = -1000.0
    l[8, :50] = torch.finfo(dtype).min
    mask[:20] = True
    mask[10] = False
    l[10] = nan
    ids, _ = mb.mol_router_topk(l, 5)
    ids[11, 2], ids[12, 0], ids[13, 4] = -1, 96, 2 ** 30  # not experts
    ids[14, 0] = ids[14, 1]           # one expert twice
    check(l, ids, mask, sigmoid)


@SCORES
def test_no_tokens(sigmoid):
    l = torch.empty(0, 16, device="cuda")
    ids = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    loss, cnt, sums = mb.mol_router_balance(l, ids)
    assert float(loss) == 0 and not cnt.any() and not sums.any()
    assert mb.mol_router_balance_grad(l, cnt, 4).shape == (0, 16)
    for M in (5, 500):  # and none that counts
        l, ids, mask = draw(M, 16, 4, torch.float32, 2)
        mask.fill_(False)
        loss, cnt, sums, grad = check(l, ids, mask, sigmoid)
        assert float(loss) == 0 and not cnt.any() and not sums.any() and not grad.any()


@BOTH
@pytest.mark.parametrize("offset,ld", [(0, 131), (1, 128), (3, 130), (8, 136)])
def test_strides_and_alignment(dtype, offset, ld):
    g = torch.Generator(device="cuda").manual_seed(offset + ld)
    flat = torch.randn(90 * ld + offset + 8, generator=g, device="cuda").to(dtype)
    l = flat[offset:offset + 90 * ld].view(90, ld)[:, :125]
    ids, _ = mb.mol_router_topk(l, 6)
    _, cnt, _, grad = check(l, ids, None, False)
    buf = torch.full_like(flat, 7.0)
    out = buf[offset:offset + 90 * ld].view(90, ld)[:, :125]
    mb.mol_router_balance_grad(l, cnt, 6, alpha=0.5, out=out)
    assert torch.equal(out, grad)
    out.fill_(7.0)
    assert bool((buf == 7.0).all())


def test_counts_of_several_ranks():
    """Two halves of a batch, their counts added, give the gradient of the whole."""
    l, ids, mask = draw(600, 40, 3, torch.float32, 5, skew=3.0)
    _, cnt, sums, grad = check(l, ids, mask, False)
    parts = [mb.mol_router_balance(l[i:i + 300], ids[i:i + 300], alpha=0.5, token_mask=mask[i:i + 300]) for i in (0, 300)]
    both = parts[0][1] + parts[1][1]
    assert torch.equal(both, cnt)
    for i in (0, 300):
        h = mb.mol_router_balance_grad(l[i:i + 300], both, 3, alpha=0.5, token_mask=mask[i:i + 300])
        assert torch.equal(h, grad[i:i + 300])
    check(l, ids, mask, True, counts=both * 3)


@SCORES
def test_gradient_against_differences(sigmoid):
    """Central differences of the loss in 64 bits with the counts held, in random directions: h^2 of the third derivative
    (below 2^-10 of the gradient's size at h = 2^-6) and nothing of fp32."""
    l, ids, mask = draw(80, 24, 3, torch.float32, 9, skew=2.0)
    sc = mb.MOL_SCORE_SIGMOID if sigmoid else mb.MOL_SCORE_SOFTMAX
    _, cnt, _ = mb.mol_router_balance(l, ids, sc, 1.0, token_mask=mask)
    grad = mb.mol_router_balance_grad(l, cnt, 3, sc, 1.0, token_mask=mask).double().cpu().numpy()
    host, hids, hm = l.double().cpu().numpy(), ids.cpu().numpy(), mask.cpu().numpy()
    rng = np.random.default_rng(4)
    for _ in range(6):
        dirn = rng.standard_normal(host.shape)
        h = 2.0 ** -6
        diff = (d.balance(host + h * dirn, hids, hm, sigmoid, 1.0)[0] - d.balance(host - h * dirn, hids, hm, sigmoid, 1.0)[0]) / (2 * h)
        assert abs(diff - (grad * dirn).sum()) <= 2.0 ** -10 * np.abs(grad * dirn).sum()


def test_writes_only_its_outputs_and_repeats_bit_for_bit():
    l, ids, mask = draw(300, 70, 4, torch.bfloat16, 15)
    bufs = [torch.full((n + 64,), 12345, dtype=t, device="cuda") for n, t in ((71, torch.int32), (70, torch.float32), (1, torch.float32))]
    cnt, sums, loss = (b[32:-32] for b in bufs)
    ws = mb.new_router_balance_workspace(300, 70, "cuda")
    need = mb.mol_router_balance_workspace_bytes(300, 70)
    assert need > 0
    first = None
    for fill in (0, 255, 77):
        guard = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
        mb.mol_router_balance(l, ids, token_mask=mask, counts=cnt, prob_sums=sums, loss=loss, workspace=guard[256:256 + need])
        assert bool((guard[:256] == fill).all()) and bool((guard[-256:] == fill).all())
        got = (cnt.clone(), sums.clone(), loss.clone())
        assert first is None or all(torch.equal(a, b) for a, b in zip(got, first))
        first = got
    for b in bufs:
        assert bool((b[:32] == 12345).all()) and bool((b[-32:] == 12345).all())
    a = mb.mol_router_balance(l, ids, token_mask=mask.to(torch.uint8) * 7, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(a, (first[2], first[0], first[1])))


@pytest.mark.parametrize("M", [20, 2000])
def test_on_another_stream_and_in_a_graph(M):
    l, ids, mask = draw(M, 128, 8, torch.bfloat16, 17)
    ws = mb.new_router_balance_workspace(M, 128, "cuda")

    def step(out=None):
        o = mb.mol_router_balance(l, ids, token_mask=mask, workspace=ws) if out is None else mb.mol_router_balance(
            l, ids, token_mask=mask, workspace=ws, loss=out[0], counts=out[1], prob_sums=out[2])
        g = mb.mol_router_balance_grad(l, o[1], 8, token_mask=mask, grad_loss=o[0], out=None if out is None else out[3])
        return (*o, g)

    first = step()
    out = tuple(torch.zeros_like(t) for t in first)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(out)
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out)
    for seed in (18, 19, 20):
        l2, i2, m2 = draw(M, 128, 8, torch.bfloat16, seed)
        l.copy_(l2), ids.copy_(i2), mask.copy_(m2)
        want = step()
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_logits_past_32_bits():
    M, E, ld = 280_000, 16, 8192
    buf = torch.zeros(M, ld, dtype=torch.bfloat16, device="cuda")
    l = buf[:, 8:8 + E]
    l[:] = torch.randn(M, E, generator=torch.Generator().manual_seed(23)).bfloat16().cuda()
    ids, _ = mb.mol_router_topk(l, 4)
    near = l.contiguous()
    a, b = mb.mol_router_balance(l, ids), mb.mol_router_balance(near, ids)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(a[1][:E].long(), torch.bincount(ids.reshape(-1).long(), minlength=E)) and int(a[1][E]) == M
    p = torch.softmax(near.double(), dim=1).sum(dim=0)
    # 280000 tokens over 512 workgroups of 16 rows: 35 in a row
    assert bool(((a[2].double() - p).abs() <= 2.0 ** -16 * p).all())
    g = mb.mol_router_balance_grad(near, a[1], 4)
    mb.mol_router_balance_grad(l, a[1], 4, out=l)
    assert torch.equal(l, g)

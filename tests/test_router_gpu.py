"""The top-k router through the C ABI against its 64-bit definition: ids exactly, weights to
fp32. The tolerance of a weight: the difference l - max rounds once (half an ulp of up to 2^7:
absolute 2^-18 in the exponent for the logits used here, sigma 3 with |l| < 32: 2^-19 relative to
the score), expf and the sums add a few units of 2^-24, the divisions and the scale half a
unit each: 2^-17 relative covers all of it."""
import numpy as np
import pytest
import torch

from tests import plain64
from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu

REL = 2.0 ** -17


def check(logits, topk, sigmoid=False, renorm=True, scale=1.0, first=0, local=None, out=None):
    """One call on device logits; compared with the definition on the same values."""
    host = logits.float().cpu().numpy()
    ids, w = mb.mol_router_topk(logits, topk,
                                mb.MOL_SCORE_SIGMOID if sigmoid else mb.MOL_SCORE_SOFTMAX,
                                renorm, scale, first, local)
    torch.cuda.synchronize()
    rid, rw = plain64.router(host, topk, sigmoid, renorm, scale, first, local)
    assert np.array_equal(ids.cpu().numpy(), rid)
    got = w.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - rw) <= REL * np.abs(rw) + 1e-37)
    return ids, w


def draw(M, E, dtype, seed, sigma=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(M, E, generator=g, device="cuda") * sigma).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,E,topk", [
    (1, 1, 1), (1, 128, 8), (23, 128, 8), (7, 4, 2), (5, 64, 16), (3, 65, 5), (17, 129, 7),
    (40, 160, 8), (33, 256, 16), (9, 257, 3), (6, 60, 17), (4, 512, 64), (3, 513, 12),
    (2, 1024, 8), (3, 1025, 9), (2, 8191, 33), (1000, 100, 6)])
@pytest.mark.parametrize("sigmoid,renorm", [(False, True), (False, False), (True, True),
                                            (True, False)])
def test_sizes(dtype, M, E, topk, sigmoid, renorm):
    check(draw(M, E, dtype, seed=M * 31 + E), min(topk, E), sigmoid, renorm, scale=2.5)


def test_more_slots_than_experts():
    ids, w = check(draw(5, 3, torch.float32, 1), 8)
    assert torch.all(ids[:, 3:] == -1) and torch.all(w[:, 3:] == 0)


@pytest.mark.parametrize("E,topk", [(128, 8), (40, 20), (600, 5)])
def test_ties_fall_to_the_lowest_expert(E, topk):
    l = draw(64, E, torch.float32, 5).round()  # whole numbers: many equal logits
    l[0] = 0.0
    l[1, ::2] = -0.0  # equal to +0
    l[1, 1::2] = 0.0
    check(l, topk)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_masked_and_special_logits(sigmoid):
    inf, nan = float("inf"), float("nan")
    l = draw(16, 128, torch.float32, 7)
    l[0] = -inf                      # no candidate at all
    l[1] = nan
    l[2, 3:] = -inf                  # fewer candidates than slots
    l[3, ::2] = nan
    l[4] = torch.finfo(torch.float32).min   # finite: candidates
    l[5, 9] = inf                    # an infinite logit takes all of the softmax
    l[6, 5], l[6, 77] = inf, inf
    l[7] = -inf
    l[7, 127] = -1000.0              # one candidate, whose sigmoid underflows
    l[8, :64] = torch.finfo(torch.float32).min
    for renorm in (True, False):
        if sigmoid and renorm:       # rows whose scores underflow in 64 bits too have no ratio
            check(l[[0, 1, 2, 3, 5, 6, 7]].contiguous(), 8, sigmoid, renorm)
        else:
            check(l, 8, sigmoid, renorm)


def test_sigmoid_renormalized_far_below_zero():
    l = draw(8, 64, torch.float32, 9) - 200.0   # sigmoid(l) underflows in fp32
    _, w = check(l, 4, sigmoid=True, renorm=True)
    assert torch.allclose(w.sum(1), torch.ones_like(w[:, 0]), atol=1e-5)


@pytest.mark.parametrize("first,local", [(0, 64), (64, 64), (37, 11), (127, 1)])
def test_expert_parallel_window(first, local):
    ids, w = check(draw(50, 128, torch.bfloat16, 11), 8, first=first, local=local)
    assert torch.all((ids >= -1) & (ids < local)) and torch.all(w[ids < 0] == 0)


@pytest.mark.parametrize("offset,ld", [(0, 131), (1, 128), (3, 130), (8, 136)])
def test_strides_and_alignment(offset, ld):
    for dtype in (torch.bfloat16, torch.float32):
        flat = draw(1, 20 * ld + offset + 8, dtype, 13).reshape(-1)
        check(flat[offset:offset + 20 * ld].view(20, ld)[:, :125], 8)


def test_no_tokens():
    ids, w = mb.mol_router_topk(torch.empty(0, 16, device="cuda"), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def test_writes_only_its_outputs_and_repeats_bit_for_bit():
    l = draw(37, 100, torch.bfloat16, 15)
    gi = torch.full((37 * 6 + 64,), 12345, dtype=torch.int32, device="cuda")
    gw = torch.full((37 * 6 + 64,), 7.5, device="cuda")
    ids, w = gi[32:-32].view(37, 6), gw[32:-32].view(37, 6)
    mb.mol_router_topk(l, 6, topk_ids=ids, topk_weights=w)
    first = (ids.clone(), w.clone())
    mb.mol_router_topk(l, 6, topk_ids=ids, topk_weights=w)
    assert torch.equal(ids, first[0]) and torch.equal(w, first[1])
    assert torch.all(gi[:32] == 12345) and torch.all(gi[-32:] == 12345)
    assert torch.all(gw[:32] == 7.5) and torch.all(gw[-32:] == 7.5)


def test_on_another_stream_and_in_a_graph():
    l = draw(23, 128, torch.bfloat16, 17)
    ids, w = mb.mol_router_topk(l, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    i2, w2 = torch.zeros_like(ids), torch.zeros_like(w)
    with torch.cuda.stream(s):
        mb.mol_router_topk(l, 8, topk_ids=i2, topk_weights=w2)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(ids, i2) and torch.equal(w, w2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mb.mol_router_topk(l, 8, topk_ids=i2, topk_weights=w2)
    for seed in (18, 19, 20):
        l.copy_(draw(23, 128, torch.bfloat16, seed))
        ids, w = mb.mol_router_topk(l, 8)
        i2.zero_(), w2.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, i2) and torch.equal(w, w2)


def test_logits_past_32_bits():
    """Rows of a buffer of more than 4 GiB."""
    M, E, ld = 280_000, 16, 8192
    buf = torch.zeros(M, ld, dtype=torch.bfloat16, device="cuda")
    assert buf.numel() * 2 > 2**32
    logits = buf[:, 8:8 + E]
    logits[:] = torch.randn(M, E, generator=torch.Generator().manual_seed(23)).bfloat16().cuda()
    ids, w = mb.mol_router_topk(logits, 4)
    near, wn = mb.mol_router_topk(logits.contiguous(), 4)
    assert torch.equal(ids, near) and torch.equal(w, wn)
    want = logits[-1000:].float().cpu().sort(dim=1, descending=True, stable=True).indices[:, :4]
    assert torch.equal(ids[-1000:].cpu().long(), want)

"""Scales at both ends of their range in the product over microscaled 4-bit weights, against 64 bits (tolerances as in
test_moe_mx4_gpu.py; sums below the normal numbers lose up to half of fp32's and of the output's smallest step a term)."""
import pytest
import torch

from tests.test_moe_mx4_gpu import HALF, value
from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu

SCALES = [0, 1, 2, 3, 40, 126, 127, 128, 200, 250, 251, 252, 253, 254]
K = 160


def product(x, xs, dtype, block, M):
    """out [M, N], codes and scales of one matrix: row n's scales are SCALES[n % 14], with all sixteen codes."""
    N = 14 * 5
    g = torch.Generator(device="cuda").manual_seed(M + block)
    W = torch.randint(0, 256, (1, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.tensor(SCALES * 5, dtype=torch.uint8, device="cuda").view(1, N, 1).expand(1, N, K // 32).contiguous()
    ids = torch.zeros(M, 1, dtype=torch.int32, device="cuda")
    out = torch.empty(M, N, dtype=dtype, device="cuda")
    mb.mol_moe_gemm_mx4(x, 1, W, s, *mb.mol_align_block_size(ids, None, 1, 1, block), M, block, out, x_scales=xs)
    return out, value(W[0], s[0])


def near(out, x, w, dtype):
    """Where no partial sum can leave the range of fp32; returns how many."""
    ref, mag = x @ w.t(), x.abs() @ w.abs().t()
    ok = mag < 2.0 ** 127
    tiny = (K + 1) * 2.0 ** -149 + torch.finfo(dtype).smallest_normal * HALF[dtype] * 2
    bound = (K + 1) * 2.0 ** -24 * mag * (1 + HALF[dtype]) + HALF[dtype] * ref.abs() + tiny
    assert bool(((out.double() - ref).abs() <= bound)[ok].all())
    return int(ok.sum())


BLOCKS = pytest.mark.parametrize("M,block", [(14, 16), (280, 64), (4200, 128)])


@BLOCKS
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_codes_of_any_scales(dtype, M, block):
    """A product of codes is a number of the sum of both scales' exponents, however large one of them is."""
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    xs = torch.tensor([SCALES[-1 - m % 14] for m in range(M)], dtype=torch.uint8, device="cuda").view(M, 1).expand(M, K // 32).contiguous()
    out, w = product(x, xs, dtype, block, M)
    assert near(out, value(x, xs), w, dtype) > out.numel() // 2


@BLOCKS
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weights_past_the_range_are_infinite_beside_rows(dtype, M, block):
    """bf16 and fp32 rows meet the weights' values in fp32, where those of 2^128 or more are infinite."""
    g = torch.Generator(device="cuda").manual_seed(M)
    x = (torch.randn(M, K, generator=g, device="cuda") * torch.exp2(torch.arange(M, device="cuda") % 14 * 16.0 - 118).view(M, 1)).to(dtype)
    out, w = product(x, None, dtype, block, M)
    w = torch.where(w.abs() >= 2.0 ** 128, torch.copysign(torch.full_like(w, float("inf")), w), w)
    finite = w.isfinite().all(dim=1)
    assert int((~finite).sum()) == 10
    assert near(out[:, finite], x.double(), w[finite], dtype) > M * 30
    for n in (~finite).nonzero().reshape(-1).tolist():  # term by term
        ref = (x.double() * w[n]).sum(dim=1)
        got = out[:, n].double()
        assert torch.equal(got.isnan(), ref.isnan()) and torch.equal(got[~ref.isnan()], ref[~ref.isnan()])

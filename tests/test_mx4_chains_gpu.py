"""Small blocks of one expert in a long row, of the widest form of the product over microscaled 4-bit weights: their pairs, and
that a block's look for the blocks it goes together with does not grow with the row."""
import pytest
import torch

from tests.test_moe_mx4_gpu import Case, codes
from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x,dtype", [("codes", torch.bfloat16), ("rows", torch.bfloat16)], ids=["codes", "bf16"])
@pytest.mark.parametrize("block,pairs", [(16, (1010, 1030, 2100)), (16, (30, 1024, 1024)), (32, (2016, 2080, 100)),
                                         (64, (4090, 70, 4200)), (16, (5000,))])
def test_rows_of_blocks_of_many_lengths(x, dtype, block, pairs):
    """Experts whose rows of blocks begin anywhere, are shorter and longer than 64 blocks and end in a part of one."""
    M = sum(pairs)
    c = Case(M, len(pairs), 1, 96, 2500, x, dtype, block=block)
    c.ids = torch.cat([torch.full((n, 1), e, dtype=torch.int32) for e, n in enumerate(pairs)])[torch.randperm(
        M, generator=torch.Generator().manual_seed(4))].cuda().contiguous()
    c.route()
    c.check()


@pytest.mark.parametrize("x", ["codes", "bf16"])
def test_time_of_a_long_row_of_small_blocks(x):
    """65536 pairs of one expert: blocks of 16 take up to three times as long as blocks of 128, which read the same bytes
    and form the same products (with a look back over the whole row they took eleven times as long)."""
    M, K, N = 65536, 2048, 1536
    g = torch.Generator(device="cuda").manual_seed(1)
    W, s = (t.view(1, N, -1) for t in codes(N, K, g))
    rows = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    rows, xs = mb.mol_mx4_quantize(rows) if x == "codes" else (rows, None)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(M, 1, dtype=torch.int32, device="cuda")
    times = {}
    for block in (16, 128):
        r = mb.mol_align_block_size(ids, None, 1, 1, block)
        best = float("inf")
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            mb.mol_moe_gemm_mx4(rows, 1, W, s, *r, M, block, out, x_scales=xs)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        times[block] = best
    assert times[16] <= 3 * times[128], times

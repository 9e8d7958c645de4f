"""Whole numbers that the binding of the routed operators has to refuse itself, on the host: a row divisor that is
not positive, and values that a 32-bit argument would wrap (a wrapped row_div of 1 would have the product read a
row of xin for every pair, where one row is all that the checks asked for)."""
import pytest
import torch

from virtual_expert_routed_amd import binding as mb

I32 = torch.int32


def q4(row_div=1, block_m=16, rows=4, numel=4):
    W, s = torch.zeros(2, 8, 32, dtype=torch.uint8), torch.zeros(2, 8, 2)
    routing = (torch.zeros(256, dtype=I32), torch.zeros(16, dtype=I32), torch.zeros(1, dtype=I32))
    return mb.mol_moe_gemm_q4(torch.zeros(rows, 64), row_div, W, s, *routing, numel, block_m, torch.zeros(numel, 8))


@pytest.mark.parametrize("row_div", [0, -1, -2**31])
def test_q4_refuses_a_row_div_below_one(row_div):
    with pytest.raises(ValueError, match="row_div"):
        q4(row_div=row_div)

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


@pytest.mark.parametrize("kw", [dict(row_div=2**32 + 1, rows=1), dict(row_div=2**31), dict(block_m=2**32 + 16)])
def test_q4_refuses_what_32_bits_would_wrap(kw):
    with pytest.raises(ValueError, match="32 bits"):
        q4(**kw)


@pytest.mark.parametrize("kw", [dict(topk=2**32 + 2), dict(scoring=2**32), dict(first_expert=2**32),
                                dict(num_local=2**32 + 8), dict(first_expert=-2**32)])
def test_router_refuses_what_32_bits_would_wrap(kw):
    with pytest.raises(ValueError, match="32 bits"):
        mb.mol_router_topk(torch.zeros(2, 8), **{"topk": 2, **kw})


def test_router_refuses_rows_that_32_bits_would_wrap():
    logits = torch.zeros(1, 1).expand(2**32 + 1, 1)  # (no memory behind its rows)
    with pytest.raises(ValueError, match="32 bits"):
        mb.mol_router_topk(logits, 1, topk_ids=torch.zeros(1, 1, dtype=I32).expand(2**32 + 1, 1),
                           topk_weights=torch.zeros(1, 1).expand(2**32 + 1, 1))


def test_layer_refuses_rows_that_32_bits_would_wrap():
    w = mb.MoeWeights(torch.zeros(2, 16, 8), torch.zeros(2, 8, 8))
    M = 2**32 + 1
    with pytest.raises(ValueError, match="32 bits"):
        mb.mol_moe_layer(w, torch.zeros(1, 8).expand(M, 8), torch.zeros(1, 1, dtype=I32).expand(M, 1),
                         torch.zeros(1, 1).expand(M, 1))


@pytest.mark.parametrize("E,N", [(2**32 + 1, 8), (1, 2**32 + 8)])
def test_4bit_weights_refuse_what_32_bits_would_wrap(E, N):
    with pytest.raises(ValueError, match="32 bits"):
        mb.mol_moe_gemm_q4(torch.zeros(4, 64), 1, torch.zeros(1, 1, 32, dtype=torch.uint8).expand(E, N, 32),
                           torch.zeros(1, 1, 2).expand(E, N, 2), *[torch.zeros(64, dtype=I32)] * 3, 4, 16,
                           torch.zeros(4, 8))

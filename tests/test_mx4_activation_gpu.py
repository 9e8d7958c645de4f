"""Codes of the activation where a factor of SiLU(gate) * up leaves fp32's normal numbers before the value does, against
their definition in 64 bits: codes and scales exactly."""
import numpy as np
import pytest
import torch

from tests import mx4_defs as d
from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu

BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])


def uniform(rows, K, low, high, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(rows, K, generator=g, device="cuda") * (high - low) + low


def check(gate, up, dtype):
    x = torch.cat([gate, up], dim=1).to(dtype)
    q, s = mb.mol_mx4_quantize(x, mb.MOL_ACT_SILU_MUL)
    torch.cuda.synchronize()
    with np.errstate(over="ignore", invalid="ignore"):
        rq, rs = d.encode(d.silu_mul(x.double().cpu().numpy()))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    return rq, rs


@BOTH
@pytest.mark.parametrize("low,high", [(-92, -84), (-99, -93), (-104, -100), (-112, -106), (-135, -110), (-180, -130), (-300, -170)])
@pytest.mark.parametrize("size", [1e5, 1e12, 1e20, 1e38])
def test_gates_far_below_zero_beside_large_ups(dtype, low, high, size):
    up = uniform(64, 96, -1.0, 1.0, 3) * size
    rq, _ = check(uniform(64, 96, low, high, 2), up, dtype)
    if size * np.exp(float(high)) > 2.0 ** -110:
        assert (rq & 0x77).any()


@BOTH
@pytest.mark.parametrize("exponent", [-149, -140, -133, -127, -126, -124, -120])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 60, 2.0 ** 126])
def test_gates_next_to_zero_beside_large_ups(dtype, exponent, size):
    gate = uniform(40, 64, -2.0, 2.0, 4).double() * 2.0 ** exponent
    check(gate.float(), uniform(40, 64, -1.0, 1.0, 5) * size, dtype)


@BOTH
def test_a_few_such_gates_in_a_block(dtype):
    """One lane's values of a block, or one value of a lane, beside zeros and beside ordinary values."""
    gate, up = torch.zeros(64, 64, device="cuda"), uniform(64, 64, 1e20, 1e30, 6)
    for r in range(32):
        gate[r, r] = -110.0
        gate[32 + r, (r // 8) * 8:(r // 8) * 8 + 8] = -101.0 - r
        gate[32 + r, 32 + r] = -200.0
    check(gate, up, dtype)
    gate[:, 3::8] = 1.5
    up[:, 3::8] = 1e-9
    check(gate, up, dtype)


@BOTH
def test_zeros_of_either_half(dtype):
    gate, up = torch.zeros(6, 64, device="cuda"), torch.full((6, 64), 1e30, device="cuda")
    gate[1] = -0.0
    gate[2], up[2] = -120.0, 0.0
    gate[3], up[3] = 7.0, -0.0
    up[4] = -1e30
    gate[5, 40], up[5, ::2] = -500.0, 0.0
    _, s = check(gate, up, dtype)
    assert not s[:5].any()


def border_products(n, seed):
    """Gates and ups in fp32 whose product in 64 bits is within 2^-20 of 2^128, on both sides of it, and some that fp32
    rounds onto the other side."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    gate = (torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * 20 + 1.5).float()
    silu = gate.double() / (1 + torch.exp(-gate.double()))
    steps = torch.randint(-8, 9, (n,), generator=g, device="cuda").double() * 2.0 ** -25
    up = (2.0 ** 128 * (1 + steps) / silu).float()
    return gate, up


def test_products_on_either_side_of_fp32s_range():
    """2^128 in 64 bits is the border of a NaN block, not what fp32 rounds the product to: a value below it has codes, at
    the largest scale there is."""
    gate, up = border_products(4096, 7)
    value = torch.nn.functional.silu(gate.double()) * up.double()
    below = (value < 2.0 ** 128)
    rounds_up = below & (value >= 2.0 ** 128 * (1 - 2.0 ** -25))
    assert int(below.sum()) > 1000 and int((~below).sum()) > 1000 and int(rounds_up.sum()) > 100
    g, u = torch.full((4096, 64), 2.0, device="cuda"), uniform(4096, 64, -1e38, 1e38, 8)
    places = torch.arange(4096, device="cuda") % 64
    rows = torch.arange(4096, device="cuda")
    g[rows, places], u[rows, places] = gate, up * torch.where(rows % 3 == 0, -1.0, 1.0)
    _, s = check(g, u, torch.float32)
    own = s[rows.cpu().numpy(), (places // 32).cpu().numpy()]
    assert np.array_equal(own == 255, (~below).cpu().numpy()) and set(own.tolist()) == {252, 255}


@BOTH
def test_finite_inputs_past_fp32s_range_and_inputs_that_are_not_finite(dtype):
    top, inf, nan = torch.finfo(dtype).max, float("inf"), float("nan")
    gate, up = uniform(10, 64, 1.0, 3.0, 9), uniform(10, 64, -3.0, 3.0, 10)
    gate[0, 3], up[0, 3] = top, top                # past the range, beside ordinary values
    gate[1, 40], up[1, 40] = -top, top             # SiLU(-max) = -0
    gate[2, 5], up[2, 5] = 1.0, top                # 0.73 max
    gate[3, 5], up[3, 5] = 100.0, top
    gate[4, 0], up[4, 0], up[4, 1] = 100.0, top, nan
    gate[5, 0], up[5, 0], gate[5, 31] = 100.0, -top, -inf
    gate[6, 0], up[6, 0] = inf, 0.0
    gate[7, 0], up[7, 0] = 0.0, inf
    gate[8], up[8] = top, top
    gate[9], up[9] = -110.0, inf
    _, s = check(gate, up, dtype)
    assert (s == 255).tolist() == [[True, False], [False, False], [False, False], [True, False], [True, False], [True, False],
                                   [True, False], [True, False], [True, True], [True, True]]


@BOTH
@pytest.mark.parametrize("seed", [11, 12, 13])
def test_blocks_of_every_size_of_gates_and_ups(dtype, seed):
    """Gates of a block next to zero, ordinary, far below or far above it, ups of any exponent, both with a spread of their
    own; some zeros of either."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, blocks = 1500, 4

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float64)

    sign = torch.where(rand(rows, blocks, 32) < 0.5, -1.0, 1.0)
    kind = torch.randint(0, 5, (rows, blocks, 1), generator=g, device="cuda")
    near = torch.exp2(-150 + 60 * rand(rows, blocks, 1) + 6 * rand(rows, blocks, 32)) * sign
    below = -80 - 170 * rand(rows, blocks, 1) - 8 * rand(rows, blocks, 32)
    far = torch.exp2(5 + 100 * rand(rows, blocks, 1) + 2 * rand(rows, blocks, 32)) * sign
    ordinary = 6 * rand(rows, blocks, 32) - 3
    gate = torch.where(kind == 0, near, torch.where(kind == 1, below, torch.where(kind == 2, far, ordinary)))
    up = torch.exp2(-145 + 262 * rand(rows, blocks, 1) + 10 * rand(rows, blocks, 32)) * torch.where(rand(rows, blocks, 32) < 0.5, -1.0, 1.0)
    gate[rand(rows, blocks, 32) < 0.02] = 0.0
    up[rand(rows, blocks, 32) < 0.02] = 0.0
    _, s = check(gate.view(rows, 128).float(), up.view(rows, 128).float(), dtype)
    assert 0 < (s == 255).sum() < s.size // 4 and len(np.unique(s)) > 200

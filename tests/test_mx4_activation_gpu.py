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

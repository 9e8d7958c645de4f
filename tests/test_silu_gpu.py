"""The layer's activation over the whole range of g, against 64 bits: x picks one gate and one up value a
column (products of one term, exact), down is the identity, fp32 throughout.

Relative to silu(g) u: the argument's rounding is corrected to first order (what is left is below 2^-30), exp2
and the reciprocal are each within one unit of 2^-23, and four more roundings of 2^-24 follow (the correction,
1 + e, both products): 2^-21 covers them, and 2^-20 leaves room for the hardware's bound on exp2. Below the
smallest normal number, 2^-126 absolute (times u)."""
import numpy as np
import pytest
import torch

from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu


def layer_of(g, u, M=1):
    """y [M, I]: silu(g) u with H = I columns and one expert; M tokens give other launch shapes."""
    I = g.numel()
    gate_up = torch.zeros(1, 2 * I, I)
    gate_up[0, :I, 0], gate_up[0, I:, 0] = g, u
    x = torch.zeros(M, I)
    x[:, 0] = 1
    w = mb.MoeWeights(gate_up.cuda(), torch.eye(I).unsqueeze(0).cuda())
    return mb.mol_moe_layer(w, x.cuda(), torch.zeros(M, 1, dtype=torch.int32, device="cuda"),
                            torch.ones(M, 1, device="cuda")).double().cpu().numpy()


@pytest.mark.parametrize("M", [1, 9])
@pytest.mark.parametrize("lo,hi,u", [(-30, 30, 1.0), (-88, -30, 1e30), (-87.5, -87.1, 1e30), (-92, -86, 1e30),
                                     (-140, -88, 1e30), (0, 1e30, 1e-3), (-3e38, -100, 1.0)])
def test_silu(lo, hi, u, M):
    n = 256
    g = torch.linspace(lo, hi, n) + (torch.rand(n, generator=torch.Generator().manual_seed(1)) - 0.5) * (hi - lo) / n
    g = g.clamp(lo, hi).float()
    u = torch.full((n,), u)
    g64, u64 = g.double().numpy(), u.double().numpy()
    with np.errstate(over="ignore"):
        silu = g64 / (1 + np.exp(-g64))
    got = layer_of(g, u, M)
    assert np.all(np.abs(got - silu * u64) <= (2.0 ** -20 * np.abs(silu) + 2.0 ** -126) * u64)


def test_silu_of_special_values():
    inf, nan = float("inf"), float("nan")
    # an infinite column reaches every y through its zeros in down: each on its own, at its own y
    for v, want in ((0.0, 0.0), (inf, None), (-inf, None), (nan, None), (-3.4e38, 0.0), (3.4e38, 3.4e38)):
        one = torch.zeros(32)
        one[0] = v
        y = layer_of(one, torch.ones(32))[0, 0]
        if want is None:
            assert np.isnan(y) if v != inf else y == inf
        else:
            assert y == np.float64(np.float32(want))

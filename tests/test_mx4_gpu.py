"""Quantisation to microscaled 4-bit floats and back, against their definition in 64 bits: codes, scales and values
exactly (the division is by a power of two; the activation's codes are those of its value in 64 bits)."""
import numpy as np
import pytest
import torch

from tests import mx4_defs as d
from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu

BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])


def draw(rows, width, dtype, seed):
    """Normal values, rows of sizes from 2^-20 to 2^20."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, width, generator=g, device="cuda")
    return (x * torch.exp2(torch.rand(rows, 1, generator=g, device="cuda") * 40 - 20)).to(dtype)


def check(x, act=False):
    q, s = mb.mol_mx4_quantize(x, mb.MOL_ACT_SILU_MUL if act else mb.MOL_ACT_NONE)
    torch.cuda.synchronize()
    v = x.double().cpu().numpy()
    rq, rs = d.encode(d.silu_mul(v) if act else v)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    return q, s


@BOTH
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 2048), (2, 64), (7, 96), (23, 2048), (33, 160), (1000, 32), (5, 4128),
                                    (257, 768)])
def test_sizes(dtype, rows, K):
    check(draw(rows, K, dtype, rows * 7 + K))


@BOTH
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (23, 768), (184, 96), (65, 2080)])
def test_activation_sizes(dtype, rows, K):
    g = torch.Generator(device="cuda").manual_seed(rows + K)
    check((torch.randn(rows, 2 * K, generator=g, device="cuda") * 2).to(dtype), act=True)


@BOTH
def test_every_border_between_codes(dtype):
    """Values on, one step above and one step below the middles between neighbouring magnitudes, at many scales."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], device="cuda").to(dtype)
    v = torch.cat([mid, torch.nextafter(mid, mid * 2), torch.nextafter(mid, mid * 0)])
    v = torch.cat([v, -v, torch.tensor([0.0, -0.0, 1e-3, 2.0 ** -20], device="cuda").to(dtype)])
    rows = []
    for e in range(-120, 125, 5):
        for first in (4.0, 7.5, 6.0):
            row = torch.zeros(64, device="cuda", dtype=dtype)
            row[0] = row[32] = first
            row[1:32], row[33:64] = v[:31], v[-31:]
            rows.append(row * 2.0 ** e)
    check(torch.stack(rows))


@BOTH
def test_small_and_large_blocks(dtype):
    x = torch.zeros(12, 64, device="cuda", dtype=dtype)  # row 0: zeros
    x[1] = -0.0
    x[2, 5] = 2.0 ** -126
    x[3, 5], x[3, 6] = 2.0 ** -128, -(2.0 ** -129)       # subnormals: the scale stays at 2^-127
    x[4, 5] = 2.0 ** -133
    x[5, 40] = torch.finfo(dtype).max
    x[6, 3] = 2.0 ** 127
    x[7] = 2.0 ** -125
    x[8, :32], x[8, 32:] = 1e30, 1e-30
    x[9] = 1.0
    x[10, 31], x[10, 32] = -3.0, 3.0
    x[11] = torch.linspace(-7.99, 7.99, 64, device="cuda").to(dtype)
    check(x)


@BOTH
@pytest.mark.parametrize("act", [False, True])
def test_nan_and_infinity_take_their_block(dtype, act):
    x = draw(8, 256 if act else 128, dtype, 3)
    x = (x / x.abs().amax(dim=1, keepdim=True)).contiguous()
    inf, nan = float("inf"), float("nan")
    x[0, 0], x[1, 33], x[2, 127], x[3, 64], x[4, 5], x[4, 6] = nan, inf, -inf, nan, inf, -inf
    if act:
        x[5, 128 + 40], x[6, 3], x[7, 128 + 5] = inf, -200.0, nan
        x[3, 64] = -inf  # SiLU(-inf) * u is NaN
    q, s = check(x, act)
    assert (s == 255).any() and not (s == 255).all(dim=1).any()
    v = mb.mol_mx4_dequantize(q, s, dtype)
    assert torch.equal(v.isnan(), (s == 255).repeat_interleave(32, dim=1))


def test_activation_next_to_borders():
    """Products that round onto the middle between two codes in fp32, in either direction, and largest values next to
    a power of two."""
    g = torch.Generator(device="cuda").manual_seed(5)
    gate = torch.rand(400, 64, generator=g, device="cuda", dtype=torch.float64) * 6 - 2
    gate = gate.float()
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0], device="cuda", dtype=torch.float64)
    want = mid[torch.randint(0, 8, (400, 64), generator=g, device="cuda")]
    want[:, 0] = want[:, 32] = 4.0  # the block's largest: its scale is next to another one
    want = want.clamp(max=5.0)
    want[:200, 1] = want[:200, 33] = 5.0
    want[200:] = want[200:].clamp(max=4.0)
    silu = gate.double() / (1 + torch.exp(-gate.double()))
    up = (want / silu).float()
    x = torch.cat([gate, up], dim=1)
    got = torch.nn.functional.silu(gate.double()) * up.double()
    assert ((got / want - 1).abs() < 2.0 ** -22).all()
    check(x, act=True)


@BOTH
def test_activation_far_gates(dtype):
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(64, 128, generator=g, device="cuda")
    x[:, :64] *= 40
    check(x.to(dtype), act=True)


@BOTH
@pytest.mark.parametrize("offset,ld", [(0, 131), (1, 128), (3, 130), (8, 136)])
def test_strides_and_alignment(dtype, offset, ld):
    flat = draw(1, 20 * ld + offset + 8, dtype, 13).reshape(-1)
    x = flat[offset:offset + 20 * ld].view(20, ld)[:, :128]
    q, s = check(x)
    check(x, act=True)
    back = torch.full((20 * ld + offset + 8,), 7.0, dtype=dtype, device="cuda")
    out = back[offset:offset + 20 * ld].view(20, ld)[:, :128]
    mb.mol_mx4_dequantize(q, s, out=out)
    assert torch.equal(out.double(), torch.from_numpy(d.decode(q.cpu(), s.cpu())).cuda())
    assert (back == 7.0).sum() >= back.numel() - 20 * 128 and bool((back[:offset] == 7.0).all())


@BOTH
def test_every_byte_at_every_scale(dtype):
    q = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 16, 16).expand(256, 16, 16).contiguous()
    s = torch.arange(256, dtype=torch.uint8, device="cuda").view(256, 1, 1).expand(256, 16, 1).contiguous()
    v = mb.mol_mx4_dequantize(q, s, dtype)
    assert v.shape == (256, 16, 32)
    with np.errstate(over="ignore"):
        want = d.decode(q.cpu().numpy(), s.cpu().numpy()).astype(np.float32)  # (infinite past fp32's range)
    got = v.float().cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(np.signbit(got[:255]), np.signbit(want[:255]))


@BOTH
def test_values_come_back_as_they_are(dtype):
    q, s = mb.mol_mx4_quantize(draw(40, 320, dtype, 21))
    v = mb.mol_mx4_dequantize(q, s, dtype)
    q2, s2 = mb.mol_mx4_quantize(v)
    assert torch.equal(mb.mol_mx4_dequantize(q2, s2, dtype), v)


def test_weights_of_three_dimensions_and_no_rows():
    x = draw(12, 64, torch.bfloat16, 9).view(3, 4, 64)
    q, s = mb.mol_mx4_quantize(x)
    assert q.shape == (3, 4, 32) and s.shape == (3, 4, 2)
    q2, s2 = mb.mol_mx4_quantize(x.view(12, 64))
    assert torch.equal(q.view(12, 32), q2) and torch.equal(s.view(12, 2), s2)
    q, s = mb.mol_mx4_quantize(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0, 2)
    assert mb.mol_mx4_dequantize(q, s).shape == (0, 64)


def test_writes_only_its_outputs():
    x = draw(37, 96, torch.float32, 15)
    gq = torch.full((37 * 48 + 64,), 77, dtype=torch.uint8, device="cuda")
    gs = torch.full((37 * 3 + 64,), 77, dtype=torch.uint8, device="cuda")
    q, s = gq[32:-32].view(37, 48), gs[32:-32].view(37, 3)
    mb.mol_mx4_quantize(x, q=q, scales=s)
    rq, rs = mb.mol_mx4_quantize(x)
    assert torch.equal(q, rq) and torch.equal(s, rs)
    for g in (gq, gs):
        assert bool((g[:32] == 77).all()) and bool((g[-32:] == 77).all())


def test_on_another_stream_and_in_a_graph():
    x = draw(23, 1536, torch.bfloat16, 17)
    q, s = mb.mol_mx4_quantize(x, mb.MOL_ACT_SILU_MUL)
    v = mb.mol_mx4_dequantize(q, s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q2, s2, v2 = torch.zeros_like(q), torch.zeros_like(s), torch.zeros_like(v)
    with torch.cuda.stream(st):
        mb.mol_mx4_quantize(x, mb.MOL_ACT_SILU_MUL, q=q2, scales=s2)
        mb.mol_mx4_dequantize(q2, s2, out=v2)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(v, v2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mb.mol_mx4_quantize(x, mb.MOL_ACT_SILU_MUL, q=q2, scales=s2)
        mb.mol_mx4_dequantize(q2, s2, out=v2)
    for seed in (18, 19, 20):
        x.copy_(draw(23, 1536, torch.bfloat16, seed))
        q, s = mb.mol_mx4_quantize(x, mb.MOL_ACT_SILU_MUL)
        v = mb.mol_mx4_dequantize(q, s)
        q2.zero_(), s2.zero_(), v2.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(v, v2)


def test_rows_past_32_bits():
    """Rows of a buffer of more than 4 GiB, in and out."""
    rows, ld = 280_000, 8192
    buf = torch.zeros(rows, ld, dtype=torch.bfloat16, device="cuda")
    x = buf[:, 8:72]
    x[:] = torch.randn(rows, 64, generator=torch.Generator().manual_seed(23)).bfloat16().cuda()
    near = x.contiguous()
    q, s = mb.mol_mx4_quantize(x)
    q2, s2 = mb.mol_mx4_quantize(near)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    rq, rs = d.encode(near[-2000:].double().cpu().numpy())
    assert np.array_equal(q[-2000:].cpu().numpy(), rq) and np.array_equal(s[-2000:].cpu().numpy(), rs)
    mb.mol_mx4_dequantize(q, s, out=x)
    assert torch.equal(x, mb.mol_mx4_dequantize(q, s))

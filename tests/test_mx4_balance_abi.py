"""Refusals of the microscaled 4-bit operators and of the balance loss on the host, before anything is enqueued: no
call here touches a device."""
import pytest
import torch

from virtual_expert_routed_amd import binding as mb

FAKE = 0x1000  # never dereferenced: every call fails validation or enqueues nothing
I32, U8 = torch.int32, torch.uint8


def quantize(**kw):
    a = dict(dtype=mb.MOL_BF16, act=0, x=FAKE, ld=64, rows=4, K=64, q=FAKE, scales=FAKE)
    a.update(kw)
    return mb.lib().mol_mx4_quantize(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), mb.MOL_E_DTYPE), (dict(dtype=-1), mb.MOL_E_DTYPE),
    (dict(act=2), mb.MOL_E_ARG), (dict(act=-1), mb.MOL_E_ARG),
    (dict(rows=-1), mb.MOL_E_ARG), (dict(K=0), mb.MOL_E_ARG), (dict(K=-32), mb.MOL_E_ARG), (dict(K=48), mb.MOL_E_ARG),
    (dict(ld=63), mb.MOL_E_ARG), (dict(act=1), mb.MOL_E_ARG), (dict(act=1, ld=127), mb.MOL_E_ARG),
    (dict(rows=2**31), mb.MOL_E_LIMIT), (dict(rows=2**62), mb.MOL_E_LIMIT), (dict(rows=2**27 - 511), mb.MOL_E_LIMIT),
    (dict(x=None), mb.MOL_E_ARG), (dict(q=None), mb.MOL_E_ARG), (dict(scales=None), mb.MOL_E_ARG),
    (dict(x=FAKE + 1), mb.MOL_E_ALIGN), (dict(dtype=0, x=FAKE + 2), mb.MOL_E_ALIGN), (dict(q=FAKE + 8), mb.MOL_E_ALIGN),
    (dict(rows=0, x=None, q=None, scales=None), mb.MOL_OK),
])
def test_quantize_refuses(kw, status):
    assert quantize(**kw) == status


def dequantize(**kw):
    a = dict(dtype=mb.MOL_BF16, q=FAKE, scales=FAKE, rows=4, K=64, x=FAKE, ld=64)
    a.update(kw)
    return mb.lib().mol_mx4_dequantize(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), mb.MOL_E_DTYPE), (dict(rows=-1), mb.MOL_E_ARG), (dict(K=0), mb.MOL_E_ARG),
    (dict(K=33), mb.MOL_E_ARG), (dict(ld=63), mb.MOL_E_ARG), (dict(rows=2**40), mb.MOL_E_LIMIT),
    (dict(x=None), mb.MOL_E_ARG), (dict(q=None), mb.MOL_E_ARG), (dict(scales=None), mb.MOL_E_ARG),
    (dict(x=FAKE + 1), mb.MOL_E_ALIGN), (dict(dtype=0, x=FAKE + 2), mb.MOL_E_ALIGN), (dict(q=FAKE + 4), mb.MOL_E_ALIGN),
    (dict(rows=0, x=None, q=None, scales=None), mb.MOL_OK),
])
def test_dequantize_refuses(kw, status):
    assert dequantize(**kw) == status


def gemm(**kw):
    a = dict(dtype=mb.MOL_BF16, x=FAKE, ld_x=256, x_scales=None, row_div=2, W=FAKE, scales=FAKE, K=256, N=40, E=4,
             sorted=FAKE, expert=FAKE, npp=FAKE, numel=8, block_m=16, out=FAKE, ld_out=40)
    a.update(kw)
    return mb.lib().mol_moe_gemm_mx4(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), mb.MOL_E_DTYPE),
    (dict(K=0), mb.MOL_E_ARG), (dict(K=240), mb.MOL_E_ARG), (dict(K=-256), mb.MOL_E_ARG), (dict(N=0), mb.MOL_E_ARG),
    (dict(row_div=0), mb.MOL_E_ARG), (dict(ld_x=224), mb.MOL_E_ARG), (dict(ld_out=39), mb.MOL_E_ARG),
    (dict(numel=-1), mb.MOL_E_ARG), (dict(E=0), mb.MOL_E_ARG), (dict(block_m=0), mb.MOL_E_ARG),
    (dict(E=8192), mb.MOL_E_LIMIT), (dict(block_m=1025), mb.MOL_E_LIMIT),
    (dict(N=2**24, ld_out=2**24), mb.MOL_E_LIMIT),               # one expert's weights: 2 GiB
    (dict(N=2**23, ld_out=2**23, numel=2**20), mb.MOL_E_LIMIT),  # the grid
    (dict(N=2**22, ld_out=2**22, numel=2**17, E=1, block_m=1024), mb.MOL_E_LIMIT),  # 2^32 threads in groups of 512
    (dict(dtype=0, K=32, ld_x=32, N=2**20, ld_out=2**20, numel=2**20, E=1, block_m=32), mb.MOL_E_LIMIT),
    (dict(x=None), mb.MOL_E_ARG), (dict(W=None), mb.MOL_E_ARG), (dict(scales=None), mb.MOL_E_ARG),
    (dict(out=None), mb.MOL_E_ARG), (dict(sorted=None), mb.MOL_E_ARG),
    (dict(expert=None), mb.MOL_E_ARG), (dict(npp=None), mb.MOL_E_ARG),
    (dict(x=FAKE + 8), mb.MOL_E_ALIGN), (dict(W=FAKE + 8), mb.MOL_E_ALIGN), (dict(out=FAKE + 1), mb.MOL_E_ALIGN),
    (dict(dtype=0, out=FAKE + 2), mb.MOL_E_ALIGN), (dict(ld_x=260), mb.MOL_E_ALIGN),
    (dict(x_scales=FAKE, ld_x=272), mb.MOL_E_ALIGN), (dict(dtype=0, ld_x=258), mb.MOL_E_ALIGN),
    (dict(numel=0, x=None, W=None, scales=None, out=None, sorted=None, expert=None, npp=None), mb.MOL_OK),
])
def test_gemm_refuses(kw, status):
    assert gemm(**kw) == status


def balance(**kw):
    a = dict(dtype=mb.MOL_BF16, logits=FAKE, ld=64, ids=FAKE, mask=None, M=100, E=64, topk=4, scoring=0, alpha=1.0,
             counts=FAKE, sums=FAKE, loss=FAKE, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return mb.lib().mol_router_balance(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), mb.MOL_E_DTYPE), (dict(M=-1), mb.MOL_E_ARG), (dict(E=0), mb.MOL_E_ARG), (dict(topk=0), mb.MOL_E_ARG),
    (dict(ld=63), mb.MOL_E_ARG), (dict(scoring=2), mb.MOL_E_ARG), (dict(scoring=-1), mb.MOL_E_ARG),
    (dict(alpha=float("nan")), mb.MOL_E_ARG), (dict(alpha=float("inf")), mb.MOL_E_ARG),
    (dict(E=8192, ld=8192), mb.MOL_E_LIMIT), (dict(topk=65), mb.MOL_E_LIMIT), (dict(M=2**30), mb.MOL_E_LIMIT),
    (dict(logits=None), mb.MOL_E_ARG), (dict(ids=None), mb.MOL_E_ARG), (dict(counts=None), mb.MOL_E_ARG),
    (dict(sums=None), mb.MOL_E_ARG), (dict(loss=None), mb.MOL_E_ARG),
    (dict(ws=None), mb.MOL_E_WORKSPACE), (dict(bytes=256), mb.MOL_E_WORKSPACE), (dict(ws=FAKE + 8), mb.MOL_E_ALIGN),
    (dict(logits=FAKE + 1), mb.MOL_E_ALIGN), (dict(dtype=0, logits=FAKE + 2), mb.MOL_E_ALIGN),
    (dict(ids=FAKE + 2), mb.MOL_E_ALIGN), (dict(counts=FAKE + 2), mb.MOL_E_ALIGN), (dict(sums=FAKE + 1), mb.MOL_E_ALIGN),
    (dict(loss=FAKE + 2), mb.MOL_E_ALIGN),
])
def test_balance_refuses(kw, status):
    assert balance(**kw) == status


def grad(**kw):
    a = dict(dtype=mb.MOL_BF16, logits=FAKE, ld=64, mask=None, counts=FAKE, up=None, M=100, E=64, topk=4, scoring=0,
             alpha=1.0, grad=FAKE, ld_grad=64)
    a.update(kw)
    return mb.lib().mol_router_balance_grad(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), mb.MOL_E_DTYPE), (dict(M=-1), mb.MOL_E_ARG), (dict(E=0), mb.MOL_E_ARG), (dict(topk=0), mb.MOL_E_ARG),
    (dict(ld=63), mb.MOL_E_ARG), (dict(ld_grad=63), mb.MOL_E_ARG), (dict(scoring=2), mb.MOL_E_ARG),
    (dict(alpha=float("-inf")), mb.MOL_E_ARG), (dict(E=8192, ld=8192, ld_grad=8192), mb.MOL_E_LIMIT),
    (dict(topk=65), mb.MOL_E_LIMIT), (dict(M=2**30), mb.MOL_E_LIMIT),
    (dict(logits=None), mb.MOL_E_ARG), (dict(counts=None), mb.MOL_E_ARG), (dict(grad=None), mb.MOL_E_ARG),
    (dict(logits=FAKE + 1), mb.MOL_E_ALIGN), (dict(counts=FAKE + 1), mb.MOL_E_ALIGN), (dict(up=FAKE + 2), mb.MOL_E_ALIGN),
    (dict(dtype=0, grad=FAKE + 2), mb.MOL_E_ALIGN),
    (dict(M=0, logits=None, counts=None, grad=None), mb.MOL_OK),
])
def test_balance_grad_refuses(kw, status):
    assert grad(**kw) == status


def test_balance_workspace_bytes():
    f = mb.lib().mol_router_balance_workspace_bytes
    assert f(0, 8) == 0 and f(16, 128) == 0
    for E in (1, 100, 257, 8191):
        sizes = [f(m, E) for m in (0, 1, 16, 17, 64, 65, 300, 1023, 1024, 1025, 1100, 5000, 2**20, 2**31 - 1)]
        assert sizes == sorted(sizes)  # a workspace for M tokens serves fewer
        assert 0 < sizes[-1] < 9 << 20
    assert f(-1, 8) == -mb.MOL_E_ARG and f(1, 0) == -mb.MOL_E_ARG and f(1, 8192) == -mb.MOL_E_LIMIT


# ---- the binding's own checks ----


def test_binding_refuses_host_tensors():
    z = torch.zeros
    for call in (lambda: mb.mol_mx4_quantize(z(2, 32)), lambda: mb.mol_mx4_dequantize(z(2, 16, dtype=U8), z(2, 1, dtype=U8)),
                 lambda: mb.mol_router_balance(z(2, 8), z(2, 2, dtype=I32)),
                 lambda: mb.mol_router_balance_grad(z(2, 8), z(9, dtype=I32), 2)):
        with pytest.raises(ValueError, match="device"):
            call()


def bgemm(rows=4, numel=4, K=64, x_scales=None, out=None, x=None, N=8, E=2, row_div=1, block_m=16, W=None, s=None, **kw):
    W = torch.zeros(E, N, K // 2, dtype=U8) if W is None else W
    s = torch.zeros(E, N, K // 32, dtype=U8) if s is None else s
    routing = kw.get("routing") or (torch.zeros(256, dtype=I32), torch.zeros(16, dtype=I32), torch.zeros(1, dtype=I32))
    return mb.mol_moe_gemm_mx4(torch.zeros(rows, K) if x is None else x, row_div, W, s, *routing, numel, block_m,
                               torch.zeros(numel, N) if out is None else out, x_scales=x_scales)


@pytest.mark.parametrize("kw,match", [
    (dict(row_div=0), "row_div"), (dict(row_div=2**32 + 1), "32 bits"), (dict(block_m=2**32 + 16), "32 bits"),
    (dict(rows=3), "rows"), (dict(x=torch.zeros(4, 32)), "xin"), (dict(x=torch.zeros(4)), "2-d"),
    (dict(x_scales=torch.zeros(4, 2, dtype=U8)), "xin|uint8"),  # fp32 rows with scales
    (dict(x=torch.zeros(4, 32, dtype=U8)), "xin|float"),        # codes without scales
    (dict(x=torch.zeros(4, 32, dtype=U8), x_scales=torch.zeros(4, 1, dtype=U8)), "x_scales"),
    (dict(x=torch.zeros(4, 64, dtype=U8)[:, :32], x_scales=torch.zeros(4, 2, dtype=U8)), "apart"),
    (dict(s=torch.zeros(2, 8, 1, dtype=U8)), "scales"), (dict(W=torch.zeros(2, 8, 24, dtype=U8)), "whole blocks"),
    (dict(W=torch.zeros(8, 32, dtype=U8)), "W"), (dict(out=torch.zeros(4, 9)), "out"),
    (dict(routing=(torch.zeros(4, dtype=I32),) * 3), "sorted_ids"),
    (dict(W=torch.zeros(1, 1, 32, dtype=U8).expand(2**32 + 1, 8, 32)), "32 bits"),
])
def test_binding_gemm_refuses(kw, match):
    with pytest.raises((ValueError, TypeError), match=match):
        bgemm(**kw)


@pytest.mark.parametrize("call", [
    lambda: mb.mol_mx4_quantize(torch.zeros(2, 48)), lambda: mb.mol_mx4_quantize(torch.zeros(64)),
    lambda: mb.mol_mx4_quantize(torch.zeros(2, 65), mb.MOL_ACT_SILU_MUL), lambda: mb.mol_mx4_quantize(torch.zeros(2, 64), 3),
    lambda: mb.mol_mx4_quantize(torch.zeros(4, 3, 64)[:, :, ::2]), lambda: mb.mol_mx4_quantize(torch.zeros(64, 64).t()[:32, ::2]),
    lambda: mb.mol_mx4_quantize(torch.zeros(2, 32, dtype=torch.float16)),
    lambda: mb.mol_mx4_quantize(torch.zeros(2, 32), q=torch.zeros(2, 17, dtype=U8)),
    lambda: mb.mol_mx4_dequantize(torch.zeros(2, 24, dtype=U8), torch.zeros(2, 1, dtype=U8)),
    lambda: mb.mol_mx4_dequantize(torch.zeros(2, 32, dtype=U8), torch.zeros(2, 1, dtype=U8)),
    lambda: mb.mol_mx4_dequantize(torch.zeros(2, 32, dtype=U8), torch.zeros(2, 2, dtype=U8), out=torch.zeros(2, 65)),
    lambda: mb.mol_router_balance(torch.zeros(2, 8), torch.zeros(3, 2, dtype=I32)),
    lambda: mb.mol_router_balance(torch.zeros(2, 8), torch.zeros(2, 2)),
    lambda: mb.mol_router_balance(torch.zeros(2, 8), torch.zeros(2, dtype=I32)),
    lambda: mb.mol_router_balance(torch.zeros(2, 8), torch.zeros(2, 2, dtype=I32), token_mask=torch.ones(2)),
    lambda: mb.mol_router_balance(torch.zeros(2, 8), torch.zeros(2, 2, dtype=I32), token_mask=torch.ones(3, dtype=torch.bool)),
    lambda: mb.mol_router_balance(torch.zeros(2, 8), torch.zeros(2, 2, dtype=I32), scoring=2**32),
    lambda: mb.mol_router_balance(torch.zeros(8, 2).t(), torch.zeros(2, 2, dtype=I32)),
    lambda: mb.mol_router_balance_grad(torch.zeros(2, 8), torch.zeros(8, dtype=I32), 2),
    lambda: mb.mol_router_balance_grad(torch.zeros(2, 8), torch.zeros(9, dtype=I32), 2**32 + 2),
    lambda: mb.mol_router_balance_grad(torch.zeros(2, 8), torch.zeros(9, dtype=I32), 2, out=torch.zeros(2, 8).bfloat16()),
    lambda: mb.mol_router_balance_grad(torch.zeros(2, 8), torch.zeros(9, dtype=I32), 2, grad_loss=torch.zeros(2)),
])
def test_binding_refuses_shapes_and_types(call):
    with pytest.raises((ValueError, TypeError)):
        call()

"""Refusals of the routed operators (router, 4-bit grouped GEMM, whole layer) on the host, before
anything is enqueued: no call here touches a device."""
import ctypes

import pytest
import torch

from virtual_expert_routed_amd import binding as mb

P = ctypes.c_void_p
FAKE = 0x1000  # never dereferenced: every call fails validation or enqueues nothing


def router(**kw):
    a = dict(dtype=mb.MOL_BF16, logits=FAKE, ld=128, M=4, E=128, topk=8, scoring=0, renorm=1,
             scale=1.0, first=0, local=128, ids=FAKE, weights=FAKE)
    a.update(kw)
    return mb.lib().mol_router_topk(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), mb.MOL_E_DTYPE),
    (dict(M=-1), mb.MOL_E_ARG), (dict(E=0), mb.MOL_E_ARG), (dict(topk=0), mb.MOL_E_ARG),
    (dict(ld=127), mb.MOL_E_ARG), (dict(scoring=2), mb.MOL_E_ARG),
    (dict(scale=float("nan")), mb.MOL_E_ARG), (dict(scale=float("inf")), mb.MOL_E_ARG),
    (dict(first=-1), mb.MOL_E_ARG), (dict(local=0), mb.MOL_E_ARG),
    (dict(first=1), mb.MOL_E_ARG), (dict(first=2**31 - 1, local=2**31 - 1), mb.MOL_E_ARG),
    (dict(E=8192, ld=8192), mb.MOL_E_LIMIT), (dict(topk=65), mb.MOL_E_LIMIT),
    (dict(M=2**30), mb.MOL_E_LIMIT),
    (dict(logits=None), mb.MOL_E_ARG), (dict(ids=None), mb.MOL_E_ARG),
    (dict(weights=None), mb.MOL_E_ARG),
    (dict(logits=FAKE + 1), mb.MOL_E_ALIGN), (dict(dtype=0, logits=FAKE + 2), mb.MOL_E_ALIGN),
    (dict(ids=FAKE + 2), mb.MOL_E_ALIGN), (dict(weights=FAKE + 2), mb.MOL_E_ALIGN),
    (dict(M=0, logits=None, ids=None, weights=None), mb.MOL_OK),
])
def test_router_refuses(kw, status):
    assert router(**kw) == status


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError):
        mb.mol_router_topk(torch.zeros(2, 8), 2)


def q4(**kw):
    a = dict(dtype=mb.MOL_BF16, x=FAKE, ld_x=256, row_div=2, W=FAKE, scales=FAKE, zeros=None,
             group=64, K=256, N=40, E=4, sorted=FAKE, expert=FAKE, npp=FAKE, numel=8, block_m=16,
             out=FAKE, ld_out=40)
    a.update(kw)
    return mb.lib().mol_moe_gemm_q4(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), mb.MOL_E_DTYPE),
    (dict(group=16), mb.MOL_E_ARG), (dict(group=0), mb.MOL_E_ARG), (dict(group=-32), mb.MOL_E_ARG),
    (dict(K=224, ld_x=224), mb.MOL_E_ARG), (dict(K=0), mb.MOL_E_ARG), (dict(N=0), mb.MOL_E_ARG),
    (dict(row_div=0), mb.MOL_E_ARG), (dict(ld_x=255), mb.MOL_E_ARG), (dict(ld_out=39), mb.MOL_E_ARG),
    (dict(numel=-1), mb.MOL_E_ARG), (dict(E=0), mb.MOL_E_ARG), (dict(block_m=0), mb.MOL_E_ARG),
    (dict(E=8192), mb.MOL_E_LIMIT), (dict(block_m=1025), mb.MOL_E_LIMIT),
    (dict(K=64 * 257, ld_x=64 * 257), mb.MOL_E_LIMIT),
    (dict(N=2**24, ld_out=2**24), mb.MOL_E_LIMIT),      # one expert's weights: 2 GiB
    (dict(N=2**23, ld_out=2**23, numel=2**20), mb.MOL_E_LIMIT),  # the grid
    (dict(x=None), mb.MOL_E_ARG), (dict(W=None), mb.MOL_E_ARG), (dict(scales=None), mb.MOL_E_ARG),
    (dict(out=None), mb.MOL_E_ARG), (dict(sorted=None), mb.MOL_E_ARG),
    (dict(expert=None), mb.MOL_E_ARG), (dict(npp=None), mb.MOL_E_ARG),
    (dict(x=FAKE + 8), mb.MOL_E_ALIGN), (dict(W=FAKE + 8), mb.MOL_E_ALIGN),
    (dict(scales=FAKE + 1), mb.MOL_E_ALIGN), (dict(out=FAKE + 1), mb.MOL_E_ALIGN),
    (dict(ld_x=260), mb.MOL_E_ALIGN), (dict(dtype=0, ld_x=258), mb.MOL_E_ALIGN),
    (dict(numel=0, x=None, W=None, scales=None, out=None, sorted=None, expert=None, npp=None),
     mb.MOL_OK),
])
def test_q4_refuses(kw, status):
    assert q4(**kw) == status


W_OK = dict(dtype=mb.MOL_BF16, group=0, num_experts=8, hidden=64, inter=32, reserved=0,
            gate_up=FAKE, down=FAKE, gate_up_scales=None, down_scales=None, gate_up_zeros=None,
            down_zeros=None)
AD_OK = dict(num_slots=2, rank=8, gate_up_A=FAKE, gate_up_B=FAKE, down_A=FAKE, down_B=FAKE,
             slot_scale=FAKE, slot_ranks=None)
Q4 = dict(group=32, gate_up_scales=FAKE, down_scales=FAKE)


def layer(w=None, ad=None, **kw):
    """ad None: no adapters; a dict: those fields over AD_OK's."""
    wc = mb._MoeWeightsC(*{**W_OK, **(w or {})}.values())
    adc = None if ad is None else mb._MoeAdaptersC(*{**AD_OK, **ad}.values())
    a = dict(x=FAKE, ld_x=wc.hidden, ids=FAKE, weights=FAKE, lora=None if ad is None else FAKE, M=4,
             topk=2, y=FAKE, ld_y=wc.hidden, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return mb.lib().mol_moe_layer(ctypes.addressof(wc),
                                  None if adc is None else ctypes.addressof(adc), *a.values(),
                                  None)


@pytest.mark.parametrize("w,ad,kw,status", [
    (dict(dtype=3), None, {}, mb.MOL_E_DTYPE),
    (dict(group=8), None, {}, mb.MOL_E_ARG), (dict(num_experts=0), None, {}, mb.MOL_E_ARG),
    (dict(hidden=0), None, {}, mb.MOL_E_ARG), (dict(inter=0), None, {}, mb.MOL_E_ARG),
    (dict(gate_up=None), None, {}, mb.MOL_E_ARG), (dict(down=None), None, {}, mb.MOL_E_ARG),
    (dict(gate_up_scales=FAKE), None, {}, mb.MOL_E_ARG), (dict(down_zeros=FAKE), None, {}, mb.MOL_E_ARG),
    (dict(group=32), None, {}, mb.MOL_E_ARG),
    (dict(group=32, gate_up_scales=FAKE), None, {}, mb.MOL_E_ARG),
    (dict(Q4, hidden=72), None, {}, mb.MOL_E_ARG), (dict(Q4, inter=48), None, {}, mb.MOL_E_ARG),
    (dict(Q4, hidden=32 * 257), None, {}, mb.MOL_E_LIMIT),
    (dict(Q4, down_scales=FAKE + 1), None, {}, mb.MOL_E_ALIGN),
    (dict(hidden=60), None, {}, mb.MOL_E_ALIGN), (dict(inter=36), None, {}, mb.MOL_E_ALIGN),
    (dict(gate_up=FAKE + 8), None, {}, mb.MOL_E_ALIGN), (dict(down=FAKE + 2), None, {}, mb.MOL_E_ALIGN),
    (dict(num_experts=8192), None, {}, mb.MOL_E_LIMIT),
    (dict(hidden=2**16, inter=2**13), None, {}, mb.MOL_E_LIMIT),
    ({}, None, dict(M=-1), mb.MOL_E_ARG), ({}, None, dict(topk=0), mb.MOL_E_ARG),
    ({}, None, dict(topk=65), mb.MOL_E_LIMIT), ({}, None, dict(M=2049), mb.MOL_E_LIMIT),
    ({}, None, dict(ld_x=63), mb.MOL_E_ARG), ({}, None, dict(ld_y=63), mb.MOL_E_ARG),
    ({}, None, dict(ld_x=68), mb.MOL_E_ALIGN), ({}, None, dict(x=FAKE + 8), mb.MOL_E_ALIGN),
    ({}, None, dict(y=FAKE + 1), mb.MOL_E_ALIGN), ({}, None, dict(ids=FAKE + 2), mb.MOL_E_ALIGN),
    ({}, None, dict(weights=FAKE + 2), mb.MOL_E_ALIGN),
    ({}, None, dict(x=None), mb.MOL_E_ARG), ({}, None, dict(y=None), mb.MOL_E_ARG),
    ({}, None, dict(ids=None), mb.MOL_E_ARG), ({}, None, dict(weights=None), mb.MOL_E_ARG),
    ({}, None, dict(lora=FAKE), mb.MOL_E_ARG), ({}, {}, dict(lora=None), mb.MOL_E_ARG),
    ({}, None, dict(ws=None), mb.MOL_E_WORKSPACE), ({}, None, dict(bytes=511), mb.MOL_E_WORKSPACE),
    ({}, None, dict(ws=FAKE + 8), mb.MOL_E_ALIGN),
    ({}, dict(num_slots=0), {}, mb.MOL_E_ARG), ({}, dict(rank=0), {}, mb.MOL_E_ARG),
    ({}, dict(num_slots=1024), {}, mb.MOL_E_LIMIT), ({}, dict(rank=136), {}, mb.MOL_E_LIMIT),
    ({}, dict(rank=12), {}, mb.MOL_E_ALIGN),
    ({}, dict(gate_up_A=None), {}, mb.MOL_E_ARG), ({}, dict(gate_up_B=None), {}, mb.MOL_E_ARG),
    ({}, dict(down_A=None), {}, mb.MOL_E_ARG), ({}, dict(down_B=None), {}, mb.MOL_E_ARG),
    ({}, dict(slot_scale=None), {}, mb.MOL_E_ARG), ({}, dict(down_B=FAKE + 8), {}, mb.MOL_E_ALIGN),
    ({}, dict(slot_ranks=FAKE + 2), {}, mb.MOL_E_ALIGN), ({}, {}, dict(lora=FAKE + 2), mb.MOL_E_ALIGN),
    ({}, None, dict(M=0, x=None, y=None, ids=None, weights=None, ws=None, bytes=0), mb.MOL_OK),
])
def test_layer_refuses(w, ad, kw, status):
    assert layer(w, ad, **kw) == status


def test_layer_refuses_without_weights():
    assert mb.lib().mol_moe_layer(None, None, FAKE, 64, FAKE, FAKE, None, 4, 2, FAKE, 64, FAKE,
                                  1 << 20, None) == mb.MOL_E_ARG


def test_layer_workspace_bytes():
    f = mb.lib().mol_moe_layer_workspace_bytes
    assert f(mb.MOL_BF16, 1, 8, 2048, 768, 0) >= 8 * 768 * 2
    assert f(mb.MOL_BF16, 0, 8, 2048, 768, 0) == 0
    # h, the weighted rows (many tokens), and both rank products
    assert f(mb.MOL_F32, 128, 8, 2048, 768, 32) >= 1024 * 4 * (768 + 2048 + 96)
    sizes = [f(mb.MOL_BF16, m, 8, 2048, 768, 32) for m in range(0, 513)]
    assert sizes == sorted(sizes)  # a workspace for M tokens serves fewer
    for args, status in (((2, 1, 8, 64, 32, 0), mb.MOL_E_DTYPE), ((1, -1, 8, 64, 32, 0), mb.MOL_E_ARG),
                         ((1, 1, 0, 64, 32, 0), mb.MOL_E_ARG), ((1, 1, 8, 0, 32, 0), mb.MOL_E_ARG),
                         ((1, 1, 8, 64, 0, 0), mb.MOL_E_ARG), ((1, 1, 8, 64, 32, -1), mb.MOL_E_ARG),
                         ((1, 513, 8, 64, 32, 0), mb.MOL_E_LIMIT), ((1, 1, 65, 64, 32, 0), mb.MOL_E_LIMIT),
                         ((1, 1, 8, 64, 32, 136), mb.MOL_E_LIMIT)):
        assert f(*args) == -status

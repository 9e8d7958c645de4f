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

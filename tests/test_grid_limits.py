"""Launches of 2^32 threads or more, which HIP does not take, are refused as a limit before anything is enqueued
(on the host: no call here touches a device)."""
import pytest

from tests.test_operators_abi import layer, q4, router
from virtual_expert_routed_amd import binding as mb


@pytest.mark.parametrize("kw", [dict(M=2**28, topk=1, E=8, ld=8, local=8), dict(M=2**27, topk=10, E=300, ld=300, local=300),
                                dict(M=2**26, topk=17, E=128)])
def test_router(kw):
    assert router(**kw) == mb.MOL_E_LIMIT


def test_q4():
    # 2^17 blocks of 128 or more items
    assert q4(N=2**13, ld_out=2**13, E=1, numel=2**21, block_m=16) == mb.MOL_E_LIMIT


def test_layer():
    # 4095 experts of 8192 items of 256 rows of down
    assert layer(dict(num_experts=4095, inter=8, hidden=2**21), M=2048, ld_x=2**21, ld_y=2**21,
                 bytes=2**40) == mb.MOL_E_LIMIT

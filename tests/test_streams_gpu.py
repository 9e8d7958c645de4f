"""Every form of the weight streams through the C ABI against the 64-bit definitions: the 4-bit product and both
stages of the layer over items of 64 rows and of several times 64, x in one stage and in several, passes of 4
to 64 columns and more than one pass, with and without adapters (cases and forms: stream_cases.py)."""
import functools

import numpy as np
import pytest
import torch

from tests import plain64, stream_cases as sc
from tests.test_moe_layer_gpu import Layer
from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("case", range(len(sc.PRODUCT)))
def test_product(case, group, dtype):
    E, N, block_m, K, _ = sc.PRODUCT[case]
    K, dt = K[group], DT[dtype]
    g = torch.Generator().manual_seed(100 * case + group)
    pairs = np.array(sc.product_pairs(E))
    numel = len(pairs)
    W = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    s = (torch.randn(E, N, K // group, generator=g) * 0.01).to(dt)
    z = torch.randint(0, 256, (E, N, K // group), generator=g, dtype=torch.uint8) if case % 2 else None
    x = torch.randn(numel, K, generator=g).to(dt)
    ids = torch.tensor(pairs, dtype=torch.int32).view(-1, 1).cuda()
    out = torch.full((numel, N), float("nan"), dtype=dt, device="cuda")
    r = mb.mol_align_block_size(ids, None, E, 1, block_m)
    mb.mol_moe_gemm_q4(x.cuda(), 1, W.cuda(), s.cuda(), *r, numel, block_m, out, zeros=None if z is None else z.cuda())
    got, x64, half = out.double().cpu().numpy(), x.double().numpy(), torch.finfo(dt).eps / 2
    assert np.all(np.isfinite(got))
    for e in list(range(len(sc.POPULAR))) + list(range(len(sc.POPULAR), E, max(1, E // 12))) + [E - 1]:
        p = np.nonzero(pairs == e)[0]
        w, mag = plain64.dequantise(W[e].numpy(), s[e].double().numpy(), None if z is None else z[e].numpy())
        ref, b = plain64.product(w, mag, x64[p])
        plain64.within(got[p], ref, b * (1 + half) + half * np.abs(ref) + 2.0 ** -134, f"expert {e}")


@pytest.mark.parametrize("adapters", [False, True])
@pytest.mark.parametrize("case", range(len(sc.LAYER)))
def test_layer(case, adapters):
    dtype, group, E, H, I, _, _ = sc.LAYER[case]
    r = 16 if dtype == "bf16" else 12
    la = Layer(dtype, H, I, E, 2 if adapters else 0, r if adapters else 0, group, ranks=(r, 7) if adapters else None,
               zeros=case % 2 == 1, seed=case)
    la.expert = (lambda f: lambda W: functools.lru_cache(None)(f(W)))(la.expert)
    pairs = sc.product_pairs(E)
    M = len(pairs)
    x, _, w, lora = la.step(M, 1, seed=case, sentinels=False)
    ids = torch.tensor(pairs, dtype=torch.int32).view(M, 1)
    got = la.call(x, ids, w, lora)
    assert torch.all(torch.isfinite(got))
    seen = torch.zeros(E, dtype=torch.int64)
    rows = []
    for m, e in enumerate(pairs):  # every popular expert's first, and every sixth of its pairs; some of the others
        if (e < len(sc.POPULAR) and seen[e] % 6 == 0) or (e >= len(sc.POPULAR) and e % 40 == 0) or e == E - 1:
            rows.append(m)
        seen[e] += 1
    rows = torch.tensor(rows)
    la.check(x[rows], ids[rows], w[rows], None if lora is None else lora[rows], got[rows.cuda()])


@pytest.mark.parametrize("dtype,group,H,I,_gu,_dn", sc.BY_PAIR)
@pytest.mark.parametrize("adapters", [False, True])
def test_layer_by_pair(dtype, group, H, I, _gu, _dn, adapters):
    """Fewer pairs than experts, in items of 64 rows and more: 96 pairs of 130 experts, some of them shared."""
    la = Layer(dtype, H, I, 130, 2 if adapters else 0, 8 if adapters else 0, group, seed=I)
    x, ids, w, lora = la.step(24, 4)
    ids[3:15, 1], ids[5:8, 2] = 9, 77
    la.check(x, ids, w, lora, la.call(x, ids, w, lora))

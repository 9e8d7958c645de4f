"""The 64-bit definitions of the routed operators catch wrong results: a plain computation in fp32
or with bf16 operands is inside their bounds, and each planted mistake is outside."""
import numpy as np
import pytest

from tests import plain64


def layer(seed=0, M=3, k=2, E=4, H=64, I=32, S=2, r=8):
    g = np.random.default_rng(seed)
    gu, dn = g.normal(0, 0.1, (E, 2 * I, H)), g.normal(0, 0.1, (E, H, I))
    ad = [g.normal(0, 0.1, s) for s in ((E * S, 2 * r, H), (E * S, 2 * I, r), (E * S, r, I),
                                        (E * S, H, r))]
    return dict(gu=gu, dn=dn, x=g.normal(0, 1, (M, H)), ids=np.array([[0, 3], [2, -1], [1, 1]]),
                w=g.uniform(0.2, 0.8, (M, k)), ad=(*ad, np.array([0.5, 2.0]), None),
                lora=np.array([1, -1, 0]))


def run(c, eps):
    def get(W):
        return lambda t: (W[t], np.abs(W[t]))
    return plain64.layer(c["x"], get(c["gu"]), get(c["dn"]), c["ids"], c["w"], eps, c["ad"],
                         c["lora"])


def swap_halves(c):
    return dict(c, gu=np.concatenate((c["gu"][:, 32:], c["gu"][:, :32]), axis=1))


def edit(key, f):
    return lambda c: dict(c, **{key: f(c[key])})


@pytest.mark.parametrize("eps", [2.0 ** -7, 2.0 ** -23])
@pytest.mark.parametrize("mistake", [
    swap_halves, edit("ids", lambda t: np.array([[0, 3], [2, 0], [1, 1]])),
    edit("lora", lambda t: np.array([0, -1, 0])), edit("lora", lambda t: np.array([1, 1, 0])),
    edit("w", lambda t: t[:, ::-1]), edit("ad", lambda t: (*t[:4], t[4] * 1.1, None)),
    edit("ad", lambda t: (*t[:5], (8, 7))), edit("dn", lambda t: np.roll(t, 1, axis=2)),
    edit("x", lambda t: t * 1.02)])
def test_a_mistake_in_a_layer_is_outside_the_bound(eps, mistake):
    c = layer()
    ref, bound = run(c, eps)
    plain64.within(ref.astype(np.float32), ref, bound)
    wrong, _ = run(mistake(c), eps)
    with pytest.raises(AssertionError):
        plain64.within(wrong, ref, bound)


def test_bf16_h_is_outside_the_bound_of_fp32():
    c = layer()
    ref, bound = run(c, 2.0 ** -23)
    with pytest.raises(AssertionError):
        plain64.within(ref * (1 + 2.0 ** -10), ref, bound)


def test_a_mistake_in_4bit_weights_is_outside_the_bound():
    g = np.random.default_rng(1)
    W = g.integers(0, 256, (8, 64), dtype=np.uint8)
    s, z = g.uniform(0.01, 0.02, (8, 4)), g.integers(0, 16, (8, 4), dtype=np.uint8)
    x = g.normal(0, 1, (1, 128))
    w, mag = plain64.dequantise(W, s, z)
    ref, bound = plain64.product(w, mag, x)
    for wrong in (((W << 4) | (W >> 4), s, z), (W, s, None), (W, s[:, ::-1], z),
                  (W, s, z ^ 1)):
        with pytest.raises(AssertionError):
            plain64.within(x @ plain64.dequantise(*wrong)[0].T, ref, bound)


def test_router_by_hand():
    ids, w = plain64.router([[0.0, 1.0, 1.0, -np.inf, np.nan]], 4)
    assert ids.tolist() == [[1, 2, 0, -1]]
    e = np.exp(1.0)
    assert np.allclose(w, [[e / (2 * e + 1), e / (2 * e + 1), 1 / (2 * e + 1), 0]])
    ids, w = plain64.router([[0.0, 2.0, 1.0]], 2, sigmoid=True, renorm=False, scale=3.0, first=1,
                            local=1)
    assert ids.tolist() == [[0, -1]] and np.allclose(w, [[3 / (1 + np.exp(-2.0)), 0]])

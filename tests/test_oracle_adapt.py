"""The fp64 forms of the gated projections and the low-rank adapters against
closed forms, differences and a dense weight."""
import numpy as np
import pytest

from oracle import adapt

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


def rnd(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("name,at", [("silu", 0.7310585786300049), ("gelu", 0.8413447460685429),
                                     ("gelu_tanh", 0.8411919906082768), ("relu", 1.0)])
def test_activation_values(name, at):
    a, s = adapt.act(name, np.array([1.0, 0.0, -40.0, 40.0]))
    assert abs(a[0] - at) < 1e-14 and a[1] == 0.0 and abs(a[2]) < 1e-14 and abs(a[3] - 40.0) < 1e-14
    assert s[1] == (0.0 if name == "relu" else 0.5) and abs(s[2]) < 1e-14 and abs(s[3] - 1.0) < 1e-14


@pytest.mark.parametrize("name", ACTS)
def test_activation_slopes_against_differences(name):
    g = np.linspace(-6.0, 6.0, 401) + 1e-3
    d = 1e-5
    diff = (adapt.act(name, g + d)[0] - adapt.act(name, g - d)[0]) / (2 * d)
    # truncation d^2 / 6 times the third derivative (below 2), rounding 2^-52 * 6 / d
    assert np.max(np.abs(diff - adapt.act(name, g)[1])) < 1e-9


@pytest.mark.parametrize("name", ACTS[:3])
def test_gated_gradient_against_differences(name):
    x, wg, wu, ga, ua, w = rnd(1, 5, 8), rnd(2, 6, 8), rnd(3, 6, 8), rnd(4, 5, 6), rnd(5, 5, 6), rnd(6, 5, 6)

    def loss(x, wg, wu, ga, ua):
        return float((w * adapt.gated(x, wg, wu, name, ga, ua)[0]).sum())

    _, g, u, _, _ = adapt.gated(x, wg, wu, name, ga, ua)
    dg, du = adapt.gated_slopes(w, g, u, name)
    (dx, dwg, dwu), _ = adapt.gated_grads(dg, du, x, wg, wu)
    args, grads = [x, wg, wu, ga, ua], [dx, dwg, dwu, dg, du]
    for i, grad in enumerate(grads):
        for at in np.ndindex(*grad.shape):
            d = 1e-5
            lo, hi = [v.copy() for v in args], [v.copy() for v in args]
            lo[i][at] -= d
            hi[i][at] += d
            assert abs((loss(*hi) - loss(*lo)) / (2 * d) - grad[at]) < 1e-6


def lora_case(seed, T=9, K=8, N=16, r=8, L=3):
    ids = np.random.default_rng(seed).integers(-1, L + 1, T)     # L: out of range, no adapter either
    return rnd(seed, T, K), ids, rnd(seed + 1, L, r, K), rnd(seed + 2, L, N, r), rnd(seed + 3, L), rnd(seed + 4, T, N)


def test_lora_is_the_dense_weight_that_it_stands_for():
    x, ids, a, b, s, base = lora_case(11)
    y, inner, outer = adapt.lora(x, ids, a, b, s, base)
    for t, e in enumerate(ids):
        want = base[t] + (x[t] @ (s[e] * b[e] @ a[e]).T if 0 <= e < 3 else 0.0)
        assert np.allclose(y[t], want, rtol=1e-13, atol=1e-13)
    assert (inner >= np.abs(y - base) - 1e-12).all() and (outer >= np.abs(y) - 1e-12).all()
    assert np.array_equal(adapt.lora(x, ids, a, b, None, None)[0], adapt.lora(x, ids, a, b, np.ones(3), None)[0])


def test_lora_gradient_against_differences():
    x, ids, a, b, s, base = lora_case(21)
    w = rnd(31, *base.shape)
    extra = rnd(32, *x.shape)
    (dx, da, db), _, _ = adapt.lora_grads(w, x, ids, a, b, s, extra)
    for i, grad in ((0, dx - extra), (2, da), (3, db)):
        for at in np.ndindex(*grad.shape):
            hi, lo = [x, ids, a, b, s, base], [x, ids, a, b, s, base]
            hi[i], lo[i] = hi[i].copy(), lo[i].copy()
            hi[i][at] += 0.5
            lo[i][at] -= 0.5
            diff = (w * (adapt.lora(*hi)[0] - adapt.lora(*lo)[0])).sum()      # linear in each: no truncation
            assert abs(diff - grad[at]) < 1e-11
    unused = [e for e in range(3) if e not in ids]
    assert all(not da[e].any() and not db[e].any() for e in unused)

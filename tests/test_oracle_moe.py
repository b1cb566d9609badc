"""The fp64 mixture-of-experts oracle against hand-worked cases, independent
formulations and central differences."""
import numpy as np
import pytest

from oracle import moe


def test_route_by_hand():
    l = np.array([[0.0, np.log(2.0), np.log(4.0), np.log(1.0)]])
    ids, w = moe.moe_route(l, 2)
    assert ids.tolist() == [[2, 1]]
    assert np.allclose(w, [[0.5, 0.25]], atol=1e-15)
    ids, w = moe.moe_route(l, 2, renormalize=True, scale=3.0)
    assert np.allclose(w, [[2.0, 1.0]], atol=1e-15)
    # a bias steers the choice, not the weight: softmax scores 1/8, 2/8, 4/8, 1/8
    ids, w = moe.moe_route(l, 2, bias=np.array([0.5, 0.0, 0.0, 0.0]))
    assert ids.tolist() == [[0, 2]] and np.allclose(w, [[0.125, 0.5]], atol=1e-15)


def test_route_groups_by_hand():
    s = np.array([0.9, 0.1, 0.6, 0.5, 0.2, 0.3])
    l = np.log(s / (1 - s))[None]
    kw = dict(score="sigmoid", n_group=3, topk_group=1)
    assert moe.moe_route(l, 2, group_score="max", **kw)[0].tolist() == [[0, 1]]
    assert moe.moe_route(l, 2, group_score="top2", **kw)[0].tolist() == [[2, 3]]


def test_route_ties_masks_and_empty_rows():
    inf = np.inf
    l = np.array([[1.0, 1.0, 1.0], [-inf, 2.0, -inf], [-inf, -inf, -inf], [0.0, np.nan, -0.0], [inf, 0.0, inf]])
    ids, w = moe.moe_route(l, 2)
    assert ids.tolist() == [[0, 1], [1, -1], [-1, -1], [0, 2], [0, 2]]
    assert np.allclose(w, [[1 / 3, 1 / 3], [1, 0], [0, 0], [0.5, 0.5], [0.5, 0.5]])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_equals_central_differences(score, renorm):
    rng = np.random.default_rng(3)
    l = rng.standard_normal((5, 7))
    l[1, 2] = -np.inf
    ids, _ = moe.moe_route(l, 3, score=score, renormalize=renorm, scale=1.7)
    ids[2, 1] = -1
    g = rng.standard_normal((5, 3))

    def loss(x):
        total = 0.0
        for t in range(5):
            s, _ = moe._scores(x[t], score)
            sel = [e for e in ids[t] if e >= 0]
            z = sum(s[e] for e in sel) if renorm else 1.0
            total += sum(1.7 * g[t, j] * s[e] / z for j, e in enumerate(ids[t]) if e >= 0)
        return total

    got, size = moe.moe_route_backward(g, l, ids, score=score, renormalize=renorm, scale=1.7)
    assert (np.abs(got) <= size + 1e-15).all()
    h = 1e-6
    for t in range(5):
        for e in range(7):
            if not np.isfinite(l[t, e]):
                assert got[t, e] == 0
                continue
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((loss(a) - loss(b)) / (2 * h) - got[t, e]) < 1e-8


def test_w4_dense_reads_twos_complement_nibbles():
    wq = np.array([[0x10, 0x8F]], np.uint8)     # codes 0, 1, -1, -8
    assert moe.w4_dense(wq, np.array([[2.0, 0.5]], np.float32), 2).tolist() == [[0.0, 2.0, -0.5, -4.0]]


def test_mlp_equals_a_dense_sum_over_experts():
    rng = np.random.default_rng(4)
    T, E, k, D, F, gc = 5, 4, 2, 64, 32, 32
    mk = lambda n, c: (rng.integers(0, 256, (E, n, c // 2), dtype=np.uint8),
                       rng.uniform(0.01, 0.1, (E, n, c // gc)).astype(np.float32))
    gate, up, down = mk(F, D), mk(F, D), mk(D, F)
    x = rng.standard_normal((T, D))
    ids = np.array([[0, 1], [3, 2], [-1, 1], [-1, -1], [2, 7]], np.int32)
    w = rng.uniform(0, 1, (T, k))
    full = np.zeros((T, E))
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                full[t, ids[t, j]] += w[t, j]
    want = np.zeros((T, D))
    for e in range(E):
        a = x @ moe.w4_dense(gate[0][e], gate[1][e], gc).T
        h = a * (0.5 * (1 + np.tanh(a / 2))) * (x @ moe.w4_dense(up[0][e], up[1][e], gc).T)
        want += full[:, e:e + 1] * (h @ moe.w4_dense(down[0][e], down[1][e], gc).T)
    got, bound = moe.moe_mlp(x, ids, w, gate, up, down, gc)
    assert np.allclose(got, want, rtol=1e-12, atol=1e-12)
    assert (got[3] == 0).all() and (bound >= 0).all() and (bound[3] == 0).all()

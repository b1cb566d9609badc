"""Gated projections and low-rank adapters in fp64, with their gradients, written
from their definitions.  Next to each value stands what its error bounds need: the
sum of the magnitudes of the terms it is a sum of."""

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(name, g):
    """(value, slope) of the activation at g."""
    with np.errstate(over="ignore"):
        if name == "silu":
            s = 1.0 / (1.0 + np.exp(-g))
            return g * s, s + g * s * (1.0 - s)
        if name == "gelu":
            phi = 0.5 * _erfc(-g * math.sqrt(0.5))
            return g * phi, phi + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
        if name == "gelu_tanh":
            c = math.sqrt(2.0 / math.pi)
            t = np.tanh(c * (g + 0.044715 * g ** 3))
            return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 0.134145 * g * g)
    assert name == "relu"
    return np.maximum(g, 0.0), (g > 0.0).astype(np.float64)


def product(x, w, add=None):
    """(x . w^T + add, the sum of its terms' magnitudes)."""
    y, size = x @ w.T, np.abs(x) @ np.abs(w).T
    return (y, size) if add is None else (y + add, size + np.abs(add))


def gated(x, gate, up, name="silu", gate_add=None, up_add=None):
    """(h, g, u, size of g, size of u)."""
    (g, sg), (u, su) = product(x, gate, gate_add), product(x, up, up_add)
    return act(name, g)[0] * u, g, u, sg, su


def gated_slopes(dh, g, u, name="silu"):
    """(dg, du): the gradients of the activation's argument and of its partner."""
    a, s = act(name, g)
    return dh * u * s, dh * a


def gated_grads(dg, du, x, gate, up):
    """(dx, dgate, dup) and their sizes."""
    dx = dg @ gate + du @ up
    sx = np.abs(dg) @ np.abs(gate) + np.abs(du) @ np.abs(up)
    return (dx, dg.T @ x, du.T @ x), (sx, np.abs(dg).T @ np.abs(x), np.abs(du).T @ np.abs(x))


def lora(x, ids, a, b, scale=None, base=None):
    """(y, size of the inner products carried through the outer one, size of the
    outer sum): y[t] = base[t] + scale[e] b[e] (a[e] x[t]), one token at a time."""
    T, (L, r, _), N = x.shape[0], a.shape, b.shape[1]
    y, inner, outer = np.zeros((T, N)), np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        e = int(ids[t])
        if 0 <= e < L:
            s = 1.0 if scale is None else float(scale[e])
            u = a[e] @ x[t]
            y[t] = s * (b[e] @ u)
            inner[t] = abs(s) * (np.abs(b[e]) @ (np.abs(a[e]) @ np.abs(x[t])))
            outer[t] = abs(s) * (np.abs(b[e]) @ np.abs(u))
    if base is not None:
        y, outer = y + base, outer + np.abs(base)
    return y, inner, outer


def lora_grads(dy, x, ids, a, b, scale=None, base=None):
    """(dx, da, db), and for each the two sizes as above."""
    T, (L, r, _) = x.shape[0], a.shape
    out = [np.zeros(x.shape), np.zeros(a.shape), np.zeros(b.shape)]
    inner, outer = [np.zeros_like(o) for o in out], [np.zeros_like(o) for o in out]
    for t in range(T):
        e = int(ids[t])
        if not 0 <= e < L:
            continue
        s = 1.0 if scale is None else float(scale[e])
        u, v = a[e] @ x[t], s * (b[e].T @ dy[t])
        su, sv = np.abs(a[e]) @ np.abs(x[t]), abs(s) * (np.abs(b[e]).T @ np.abs(dy[t]))
        for i, (value, p, q) in enumerate(((v @ a[e], sv @ np.abs(a[e]), np.abs(v) @ np.abs(a[e])),
                                           (np.outer(v, x[t]), np.outer(sv, np.abs(x[t])),
                                            np.outer(np.abs(v), np.abs(x[t]))),
                                           (s * np.outer(dy[t], u), abs(s) * np.outer(np.abs(dy[t]), su),
                                            abs(s) * np.outer(np.abs(dy[t]), np.abs(u))))):
            at = t if i == 0 else e
            out[i][at] += value
            inner[i][at] += p
            outer[i][at] += q
    if base is not None:
        out[0] += base
        outer[0] += np.abs(base)
    return out, inner, outer

"""Mixture-of-experts operators in fp64: routing and its gradient, linear layers
on 4-bit weights with group scales, the routed gated MLP.  Written from their
definitions, one token or expert at a time."""

import numpy as np


def _scores(row, score):
    """Scores of one token's logits; 0 where the logit is -inf or NaN."""
    live = row > -np.inf
    s = np.zeros_like(row)
    if score == "softmax":
        if live.any():
            e = np.exp(row[live] - row[live].max())
            s[live] = e / e.sum()
    else:
        with np.errstate(over="ignore"):
            s[live] = 1.0 / (1.0 + np.exp(-row[live]))
    return s, live


def moe_route(logits, k, score="softmax", bias=None, n_group=1, topk_group=1, group_score="max", renormalize=False,
              scale=1.0):
    """(ids int32 [T, k], weights float64 [T, k]); logits fp32 [T, E], bias fp32 [E]."""
    fmax = float(np.finfo(np.float32).max)
    x = np.minimum(logits.astype(np.float64), fmax)
    T, E = x.shape
    b = np.zeros(E) if bias is None else np.minimum(bias.astype(np.float64), fmax)
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    per = E // n_group
    for t in range(T):
        s, live = _scores(x[t], score)
        ok = live & (b > -np.inf)
        key = x[t] if bias is None else s + b
        left = [e for e in range(E) if ok[e]]
        if n_group > 1:
            value = []
            for g in range(n_group):
                mine = [e for e in left if e // per == g]
                if not mine:
                    value.append(-np.inf)
                elif group_score == "max":
                    value.append(max(key[e] for e in mine))
                else:
                    value.append(sum(sorted((s[e] + b[e] for e in mine), reverse=True)[:2]))
            keep = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
            left = [e for e in left if e // per in keep]
        best = sorted(left, key=lambda e: (-key[e], e))[:k]
        w = np.array([s[e] for e in best])
        if renormalize and len(best):
            w = w / max(w.sum(), 1e-300)
        ids[t, :len(best)] = best
        weights[t, :len(best)] = w * scale
    return ids, weights


def moe_route_backward(grad, logits, ids, score="softmax", renormalize=False, scale=1.0):
    """(dlogits [T, E], magnitude of the terms each is summed from)."""
    x = np.minimum(logits.astype(np.float64), float(np.finfo(np.float32).max))
    T, E = x.shape
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        sel = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < E]
        s, live = _scores(x[t], score)
        g = {e: float(grad[t, j]) for j, e in sel}
        if score == "softmax" and not renormalize:
            dot, mag = sum(g[e] * s[e] for e in g), sum(abs(g[e]) * s[e] for e in g)
            for e in range(E):
                out[t, e] = scale * s[e] * (g.get(e, 0.0) - dot)
                size[t, e] = scale * s[e] * (abs(g.get(e, 0.0)) + mag)
            continue
        if score == "softmax":
            top = max([x[t, e] for e in g if live[e]], default=0.0)
            r = {e: np.exp(x[t, e] - top) if live[e] else 0.0 for e in g}
            slope = {e: 1.0 for e in g}
        else:
            r = {e: s[e] for e in g}
            with np.errstate(over="ignore"):
                slope = {e: 1.0 / (1.0 + np.exp(x[t, e])) if live[e] else 0.0 for e in g}
        if renormalize:
            z = max(sum(r.values()), 1e-300)
            r = {e: r[e] / z for e in g}
            dot, mag = sum(g[e] * r[e] for e in g), sum(abs(g[e]) * r[e] for e in g)
        else:
            dot = mag = 0.0
        for e in g:
            out[t, e] = scale * r[e] * slope[e] * (g[e] - dot)
            size[t, e] = scale * r[e] * slope[e] * (abs(g[e]) + mag)
    return out, size


def w4_dense(wq, s, gc):
    """Packed nibbles [N, K/2] and scales [N, K/gc] -> the fp64 weight [N, K]."""
    n, half = wq.shape
    c = np.empty((n, 2 * half), np.int64)
    c[:, 0::2], c[:, 1::2] = wq & 15, wq >> 4
    c = np.where(c > 7, c - 16, c)
    return c * np.repeat(s.astype(np.float64), gc, axis=1)


def w4_linear(x, wq, s, gc, bias=None):
    """(Y, sum of the magnitudes of its terms), x fp64 [M, K]."""
    w = w4_dense(wq, s, gc)
    y, size = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        y, size = y + bias, size + np.abs(bias)
    return y, size


def sum_error(k, gc):
    """What a sum of k products may be off by relative to the sum of their
    magnitudes: at most gc additions inside a group, one product-and-add a
    group, the joining of 8 partial sums, a step of 2^-23 each (the matrix core
    may cut instead of rounding)."""
    return (gc + -(-k // gc) + 16) * 2.0 ** -23


def moe_mlp(x, ids, weights, gate, up, down, gc, h_step=2.0 ** -8):
    """(y, bound on a kernel's error before its last rounding); gate, up, down =
    (codes [E, ..], scales [E, ..]).  The kernel's own roundings: fp32 sums, h to
    h_step of its value."""
    T, D = x.shape
    E, F = gate[0].shape[0], gate[0].shape[1]
    y, bound = np.zeros((T, D)), np.zeros((T, D))
    eg, ef = sum_error(D, gc), sum_error(F, gc)
    for e in range(E):
        wd = None
        for t, j in zip(*np.nonzero(ids == e)):
            if wd is None:
                wg, wu, wd = (w4_dense(w[0][e], w[1][e], gc) for w in (gate, up, down))
            g, u = wg @ x[t], wu @ x[t]
            dg, du = eg * (np.abs(wg) @ np.abs(x[t])), eg * (np.abs(wu) @ np.abs(x[t]))
            si = g / (1.0 + np.exp(-g))
            h = si * u
            # silu's slope is below 1.1; its fp32 exponential and quotient within 2^-20
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(si) * du + (h_step + 2.0 ** -20) * np.abs(h)
            w = float(weights[t, j])
            y[t] += w * (wd @ h)
            bound[t] += abs(w) * (np.abs(wd) @ dh + ef * (np.abs(wd) @ (np.abs(h) + dh)))
    k = ids.shape[1]
    return y, bound + k * 2.0 ** -23 * (np.abs(y) + bound)

"""What is measured of the routing and 4-bit-weight operators: the cases, their
inputs, their plain forms and their values in 64 bits.

Four kinds of case:
  route       logits -> the experts of each token and their weights
  route_grad  the gradient of those weights with respect to the logits
  linear      Y = X . W^T, bf16 X and a 4-bit weight with group scales
  experts     the routed gated MLP on 4-bit expert weights

``own`` chooses between the library's calls (true) and elementary torch
operations (false).
"""

import math

import torch

own = False

DEV = "cuda:0"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token of a decoding step, the widest router: sigmoid scores, a balance bias, 4 of 8 groups
        dict(name="route_one_token", kind="route", T=1, E=256, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group_score="top2", renorm=True, scale=2.5, dtype="float32", masked=False),
        # a small ragged decoding batch over an odd number of experts, some of them switched off, one row with none left
        dict(name="route_batch_odd", kind="route", T=37, E=60, k=4, score="softmax", bias=False, n_group=1,
             topk_group=1, group_score="max", renorm=False, scale=1.0, dtype="bfloat16", masked=True),
        # a long prefill through the same router as the single token
        dict(name="route_prefill", kind="route", T=16384, E=256, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group_score="top2", renorm=True, scale=2.5, dtype="float32", masked=False),
        # fine-tuning the router: softmax weights kept as they are, so that the gradient reaches every logit
        dict(name="route_grad_softmax", kind="route_grad", T=4093, E=60, k=4, score="softmax", bias=False, n_group=1,
             topk_group=1, group_score="max", renorm=False, scale=1.0, dtype="bfloat16", masked=True),
        # the same for the wide sigmoid router with renormalised weights
        dict(name="route_grad_sigmoid", kind="route_grad", T=16384, E=256, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group_score="top2", renorm=True, scale=2.5, dtype="float32", masked=False),
        # one token through a square projection
        dict(name="linear_1x4096x4096", kind="linear", M=1, N=4096, K=4096, gc=128, out="bfloat16", bias=False),
        # one token through the widest up-projection, the finer scale groups
        dict(name="linear_1x14336x4096", kind="linear", M=1, N=14336, K=4096, gc=64, out="bfloat16", bias=False),
        # a ragged decoding batch through the down-projection, fp32 out (a partial sum that is reduced later)
        dict(name="linear_37x4096x14336", kind="linear", M=37, N=4096, K=14336, gc=128, out="float32", bias=True),
        # prefill
        dict(name="linear_2048x4096x4096", kind="linear", M=2048, N=4096, K=4096, gc=128, out="bfloat16", bias=False),
        # one token of a decoding step through its 8 experts
        dict(name="experts_one_token", kind="experts", T=1, E=64, k=8, D=4096, F=1024, gc=128, dropped=False),
        # a ragged decoding batch, an expert width that is no power of two, some pairs dropped
        dict(name="experts_batch_odd", kind="experts", T=29, E=60, k=4, D=2048, F=1408, gc=64, dropped=True),
        # prefill
        dict(name="experts_prefill", kind="experts", T=2048, E=64, k=8, D=4096, F=1024, gc=128, dropped=False),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "route_grad", "linear", "linear", "experts", "experts"])
    if kind in ("route", "route_grad"):
        n_group = rng.choice([1, 1, 2, 4, 8])
        per = _log(rng, 4, 256 // n_group)
        e = n_group * per
        topk_group = rng.randint(1, n_group)
        k = rng.randint(1, min(10, topk_group * per))
        return dict(kind=kind, T=_log(rng, 1 if kind == "route" else 64, 16384), E=e, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, n_group=n_group,
                    topk_group=topk_group, group_score=rng.choice(["max", "top2"]), renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["float32", "bfloat16"]),
                    masked=rng.random() < 0.3)
    gc = rng.choice([32, 64, 128])
    if kind == "linear":
        n, k = _log(rng, 500, 14336), gc * _log(rng, 512 // gc, 14336 // gc)
        # no more than the widest one-token weight, no more work than the prefill
        n = max(64, min(n, 14336 * 4096 // k))
        m = _log(rng, 1, 2048)
        m = max(1, min(m, 2048 * 4096 * 4096 // (n * k)))
        return dict(kind=kind, M=m, N=n, K=k, gc=gc, out=rng.choice(["float32", "bfloat16"]),
                    bias=rng.random() < 0.3)
    d, f = gc * _log(rng, 512 // gc, 4096 // gc), gc * _log(rng, 256 // gc, 2048 // gc)
    e = _log(rng, 4, 64)
    f = max(gc, min(f, gc * (4096 * 1024 // (d * gc))))
    k = rng.randint(1, min(8, e))
    return dict(kind=kind, T=_log(rng, 1, 2048), E=e, k=k, D=d, F=f, gc=gc, dropped=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs

def _quantise(gen, rows, cols, gc):
    """A weight N(0, 0.02) in 4 bits: codes two to a byte (element 2 j in the
    low half of byte j), one scale max|w| / 7 per row and group of gc."""
    w = torch.randn((rows, cols // gc, gc), generator=gen, device=DEV).mul_(0.02)
    s = w.abs().amax(-1).div_(7.0)
    c = torch.round(w / s[..., None]).clamp_(-7, 7).to(torch.int8).reshape(rows, cols // 2, 2)
    return ((c[..., 0] & 15) | ((c[..., 1] & 15) << 4)).view(torch.uint8), s


def _logits(case, gen):
    """Router outputs N(0, 1) with a popularity that differs between experts."""
    t, e = case["T"], case["E"]
    x = torch.randn((t, e), generator=gen, device=DEV) + 0.7 * torch.randn((e,), generator=gen, device=DEV)
    if case["masked"]:
        off = torch.rand((e,), generator=gen, device=DEV) < 0.1
        x[:, off] = float("-inf")
        x[t - 1] = float("-inf")          # a row that nothing is left of
        if t > 2:                          # padding held at the type's lowest value
            x[t // 2] = torch.finfo(getattr(torch, case["dtype"])).min
    return x.to(getattr(torch, case["dtype"])).contiguous()


def _inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    kind = case["kind"]
    if kind in ("route", "route_grad"):
        d = {"logits": _logits(case, gen), "bias": None}
        if case["bias"]:
            d["bias"] = 0.1 * torch.randn((case["E"],), generator=gen, device=DEV)
        if kind == "route_grad":
            d["ids"] = _select(case, d["logits"], d["bias"])[0]
            d["grad"] = torch.randn((case["T"], case["k"]), generator=gen, device=DEV)
        return d
    if kind == "linear":
        m, n, k = case["M"], case["N"], case["K"]
        d = {"x": torch.randn((m, k), generator=gen, device=DEV).to(torch.bfloat16), "bias": None}
        d["w"] = _quantise(gen, n, k, case["gc"])
        if case["bias"]:
            d["bias"] = torch.randn((n,), generator=gen, device=DEV)
        return d
    t, e, k, dm, f, gc = (case[v] for v in ("T", "E", "k", "D", "F", "gc"))
    d = {"x": torch.randn((t, dm), generator=gen, device=DEV).to(torch.bfloat16)}
    pop = torch.randn((t, e), generator=gen, device=DEV) + 0.7 * torch.randn((e,), generator=gen, device=DEV)
    top, ids = pop.topk(k, dim=1)
    d["ids"] = ids.to(torch.int32)
    d["weights"] = torch.softmax(top, dim=1).contiguous()
    if case["dropped"]:
        drop = torch.rand((t, k), generator=gen, device=DEV) < 0.1
        d["ids"] = torch.where(drop, -1, d["ids"])
        d["weights"] = torch.where(drop, 0.0, d["weights"])
    d["ids"] = d["ids"].contiguous()
    for name, rows, cols in (("gate", f, dm), ("up", f, dm), ("down", dm, f)):
        one = [_quantise(gen, rows, cols, gc) for _ in range(e)]
        d[name] = (torch.stack([c for c, _ in one]), torch.stack([s for _, s in one]))
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    if own:
        import sparse_gemm_layers_amd as sg
        for name in ("w", "gate", "up", "down"):      # a weight is packed once, when the model is loaded
            if name in d:
                d[name] = sg.w4_pack(*d[name], gc=case["gc"])
    return {"case": case, **d}


# ------------------------------------------------------------------ plain forms

def _select(case, logits, bias):
    """The routing in elementary operations.  Scores are taken in 64 bits: two
    experts whose keys lie next to each other must come out in the same order
    however the scores are computed."""
    t, e = logits.shape
    k, ng = case["k"], case["n_group"]
    x = logits.double()
    ok = logits > float("-inf")
    if bias is not None:
        ok = ok & (bias > float("-inf"))
    if case["score"] == "softmax":
        top = torch.where(logits > float("-inf"), x, torch.full_like(x, -1e300)).amax(1, keepdim=True)
        ex = torch.where(logits > float("-inf"), torch.exp(x - top), torch.zeros_like(x))
        s = ex / ex.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    low = torch.full_like(x, float("-inf"))
    key = torch.where(ok, x if bias is None else s + bias.double(), low)
    if ng > 1:
        per = e // ng
        val = key
        if case["group_score"] == "top2":
            val = torch.where(ok, s if bias is None else s + bias.double(), low)
        val = val.reshape(t, ng, per).sort(dim=2, descending=True).values
        if case["group_score"] == "top2" and per > 1:      # a group of one usable expert counts that one alone
            second = val[:, :, 1]
            val = val[:, :, 0] + torch.where(second > float("-inf"), second, torch.zeros_like(second))
        else:
            val = val[:, :, 0]
        best = val.sort(dim=1, descending=True, stable=True).indices[:, :case["topk_group"]]
        keep = torch.zeros((t, ng), dtype=torch.bool, device=logits.device).scatter_(1, best, True)
        key = torch.where(keep.repeat_interleave(per, 1), key, low)
    key, ids = key.sort(dim=1, descending=True, stable=True)
    key, ids = key[:, :k], ids[:, :k]
    some = key > float("-inf")
    w = torch.where(some, s.gather(1, ids), 0.0)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return torch.where(some, ids, -1).to(torch.int32), (w * case["scale"]).float()


def _route_grad(case, logits, ids, grad):
    sel = ids >= 0
    at = ids.clamp_min(0).long()
    x = logits.float()
    g = torch.where(sel, grad, 0.0)
    out = torch.zeros_like(x)
    c = case["scale"]
    if case["score"] == "softmax" and not case["renorm"]:
        top = x.amax(1, keepdim=True)
        ex = torch.exp(x - torch.where(top > float("-inf"), top, 0.0))
        p = ex / ex.sum(1, keepdim=True).clamp_min(1e-37)
        ps = torch.where(sel, p.gather(1, at), 0.0)
        out = -c * p * (g * ps).sum(1, keepdim=True)
        out.scatter_add_(1, at, c * ps * g)
        return out.to(logits.dtype)
    xs = torch.where(sel, x.gather(1, at), float("-inf"))
    s = torch.sigmoid(xs)
    if case["renorm"]:
        if case["score"] == "softmax":
            top = xs.amax(1, keepdim=True)
            r = torch.exp(xs - torch.where(top > float("-inf"), top, 0.0))
            slope = torch.ones_like(r)
        else:
            r, slope = s, 1.0 - s
        r = r / r.sum(1, keepdim=True).clamp_min(1e-37)
        d = c * r * slope * (g - (g * r).sum(1, keepdim=True))
    else:
        d = c * g * s * (1.0 - s)
    out.scatter_add_(1, at, torch.where(sel, d, 0.0))
    return out.to(logits.dtype)


def _codes(wq):
    """int4 codes of packed bytes, as whole numbers in a wider type."""
    lo, hi = (wq & 15).to(torch.int8), (wq >> 4).to(torch.int8)
    c = torch.stack((lo, hi), -1).flatten(-2)
    return torch.where(c > 7, c - 16, c)


def _dense(wq, s, gc, dtype):
    c = _codes(wq)
    return (c.reshape(c.shape[0], -1, gc).to(dtype) * s[..., None].to(dtype)).reshape(c.shape)


def _experts_plain(case, d):
    t, k = d["ids"].shape
    x = d["x"].float()
    pair = torch.zeros((t, k, case["D"]), device=x.device)
    for e in d["ids"].unique().tolist():
        if e < 0:
            continue
        rows, slots = (d["ids"] == e).nonzero(as_tuple=True)
        g = x[rows] @ _dense(d["gate"][0][e], d["gate"][1][e], case["gc"], torch.float32).t()
        u = x[rows] @ _dense(d["up"][0][e], d["up"][1][e], case["gc"], torch.float32).t()
        h = g * torch.sigmoid(g) * u
        pair[rows, slots] = h @ _dense(d["down"][0][e], d["down"][1][e], case["gc"], torch.float32).t()
    return (pair * d["weights"][..., None]).sum(1).to(torch.bfloat16)


def run(state):
    case, kind = state["case"], state["case"]["kind"]
    if own:
        import sparse_gemm_layers_amd as sg
        if kind == "route":
            return sg.moe_route(state["logits"], case["k"], score=case["score"], bias=state["bias"],
                                n_group=case["n_group"], topk_group=case["topk_group"],
                                group_score=case["group_score"], renormalize=case["renorm"], scale=case["scale"])
        if kind == "route_grad":
            return sg.moe_route_backward(state["grad"], state["logits"], state["ids"], score=case["score"],
                                         renormalize=case["renorm"], scale=case["scale"])
        if kind == "linear":
            return sg.w4a16_gemm_groupwise_packed(state["x"], state["w"], case["N"], gc=case["gc"],
                                                  out_dtype=getattr(torch, case["out"]), bias=state["bias"])
        return sg.w4a16_moe_mlp(state["x"], state["ids"], state["weights"], state["gate"], state["up"],
                                state["down"], case["F"], gc=case["gc"])
    if kind == "route":
        return _select(case, state["logits"], state["bias"])
    if kind == "route_grad":
        return _route_grad(case, state["logits"], state["ids"], state["grad"])
    if kind == "linear":
        y = state["x"].float() @ _dense(*state["w"], case["gc"], torch.float32).t()
        if state["bias"] is not None:
            y = y + state["bias"]
        return y.to(getattr(torch, case["out"]))
    return _experts_plain(case, state)


# ------------------------------------------------------------------ cost

def work(case):
    kind = case["kind"]
    if kind in ("route", "route_grad"):
        t, e, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "float32" else 2
        if kind == "route":      # logits and bias in; ids and weights out
            return {"bytes": t * e * size + (4 * e if case["bias"] else 0) + 8 * t * k, "flops": 8 * t * e}
        # ids and the weights' gradient in, the logits' gradient out; all logits are read where every
        # probability enters, else those of the chosen experts
        every = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": 8 * t * k + t * (e if every else k) * size + t * e * size,
                "flops": (8 * t * e if every else 12 * t * k)}
    if kind == "linear":
        m, n, k = case["M"], case["N"], case["K"]
        out = 4 if case["out"] == "float32" else 2
        return {"bytes": n * k // 2 + 4 * n * (k // case["gc"]) + 2 * m * k + out * m * n
                + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    t, e, k, d, f, gc = (case[v] for v in ("T", "E", "k", "D", "F", "gc"))
    # experts that t tokens reach when each takes k of e at even odds
    active = e * (1.0 - (1.0 - k / e) ** t)
    return {"bytes": int(active * 3 * d * f * (0.5 + 4.0 / gc)) + 4 * t * d + 8 * t * k, "flops": 6 * t * k * d * f}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    d = _inputs(case, seed)
    kind = case["kind"]
    if kind == "route":
        return _exact_route(case, d["logits"].double().cpu(), None if d["bias"] is None else d["bias"].double().cpu())
    if kind == "route_grad":
        return _exact_route_grad(case, d["logits"].double(), d["ids"].long(), d["grad"].double())
    if kind == "linear":
        wq, s = d["w"]
        y = torch.matmul(d["x"].double(), _exact_weight(wq, s, case["gc"]).T)
        return y if d["bias"] is None else y + d["bias"].double()
    x, out = d["x"].double(), torch.zeros((case["T"], case["D"]), dtype=torch.float64, device=DEV)
    ids, w = d["ids"], d["weights"].double()
    for e in range(case["E"]):
        hit = (ids == e)
        share = torch.where(hit, w, 0.0).sum(1)          # an expert appears once at most among a token's
        rows = torch.nonzero(hit.any(1)).flatten()
        if rows.numel() == 0:
            continue
        wg, wu, wd = (_exact_weight(d[v][0][e], d[v][1][e], case["gc"]) for v in ("gate", "up", "down"))
        a = torch.matmul(x[rows], wg.T)
        h = a / (1.0 + torch.exp(-a)) * torch.matmul(x[rows], wu.T)
        out[rows] += share[rows, None] * torch.matmul(h, wd.T)
    return out


def _exact_weight(wq, s, gc):
    n, half = wq.shape
    b = wq.to(torch.float64)
    hi = torch.floor(b / 16.0)
    c = torch.empty((n, 2 * half), dtype=torch.float64, device=wq.device)
    c[:, 0::2], c[:, 1::2] = b - 16.0 * hi, hi
    c -= 16.0 * (c >= 8.0)
    return c * torch.repeat_interleave(s.double(), gc, dim=1)


def _exact_route(case, x, bias):
    """On the host with numpy, ordered by (key descending, index ascending)."""
    import numpy as np
    x = x.numpy()
    t, e = x.shape
    b = np.zeros(e) if bias is None else bias.numpy()
    usable = np.isfinite(x) & np.isfinite(b)
    with np.errstate(over="ignore", invalid="ignore"):
        if case["score"] == "softmax":
            top = np.max(x, axis=1, keepdims=True)
            top[~np.isfinite(top)] = 0.0
            p = np.exp(x - top)
            s = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
        else:
            s = 1.0 / (1.0 + np.exp(-x))
    by_score = s + b
    rank = x if bias is None else by_score
    if case["n_group"] > 1:
        ng, per = case["n_group"], e // case["n_group"]
        if case["group_score"] == "top2":
            best = -np.sort(-np.where(usable, by_score, -np.inf).reshape(t, ng, per), axis=2)[:, :, :2]
            value = np.where(np.isfinite(best[:, :, 0]), np.where(np.isfinite(best), best, 0.0).sum(2), -np.inf)
        else:
            value = np.where(usable, rank, -np.inf).reshape(t, ng, per).max(2)
        order = np.argsort(-value, axis=1, kind="stable")[:, :case["topk_group"]]
        keep = np.zeros((t, ng), dtype=bool)
        np.put_along_axis(keep, order, True, axis=1)
        usable = usable & np.repeat(keep, per, axis=1)
    order = np.argsort(-np.where(usable, rank, -np.inf), axis=1, kind="stable")[:, :case["k"]]
    got = np.take_along_axis(usable, order, 1)
    w = np.where(got, np.take_along_axis(s, order, 1), 0.0)
    if case["renorm"]:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    ids = np.where(got, order, -1).astype(np.int32)
    return torch.from_numpy(ids).to(DEV), torch.from_numpy(w * case["scale"]).to(DEV)


def _exact_route_grad(case, x, ids, grad):
    """The Jacobian written out over all experts: d w_j / d l_i."""
    t, e = x.shape
    chosen = torch.zeros((t, e), dtype=torch.float64, device=x.device)
    g = torch.zeros_like(chosen)
    for j in range(ids.shape[1]):
        rows = torch.nonzero(ids[:, j] >= 0).flatten()
        chosen[rows, ids[rows, j]] = 1.0
        g[rows, ids[rows, j]] = grad[rows, j]
    live = torch.isfinite(x)
    if case["score"] == "softmax":
        m = torch.where(live, x, -1e308).amax(1, keepdim=True)
        s = torch.where(live, torch.exp(x - m), 0.0)
        s = s / s.sum(1, keepdim=True).clamp_min(1e-300)
        own_slope = None
    else:
        s = torch.where(live, 1.0 / (1.0 + torch.exp(-x)), 0.0)
        own_slope = torch.where(live, 1.0 / (1.0 + torch.exp(x)), 0.0)          # 1 - s
    if case["renorm"]:
        share = s * chosen
        share = share / share.sum(1, keepdim=True).clamp_min(1e-300)
        out = share * (g - (g * share).sum(1, keepdim=True))
        if own_slope is not None:
            out = out * own_slope
    elif case["score"] == "softmax":
        out = s * (g - (g * s).sum(1, keepdim=True))
    else:
        out = g * s * own_slope
    return case["scale"] * out

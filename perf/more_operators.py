"""What is measured of the gated projections and the low-rank adapters: the cases,
their inputs, their plain forms and their values in 64 bits.

Four kinds of case:
  gated       H = act(X . Wg^T) * (X . Wu^T), the first half of a gated feed-forward block
  gated_grad  its backward pass: the gradients of X, of both weights and of both products
  lora        Y = base + s_e (X . A_e^T) . B_e^T, every token with its own adapter e
  lora_grad   its backward pass: the gradients of X and of every adapter

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
        # one token of a decoding step through the widest block
        dict(name="gated_one_token", kind="gated", T=1, D=4096, F=14336, act="silu", add=False),
        # a ragged decoding batch, sizes that no tile divides, adapters on both projections
        dict(name="gated_batch_odd", kind="gated", T=37, D=2040, F=5512, act="gelu", add=True),
        # a large decoding batch, or a short prompt
        dict(name="gated_batch_256", kind="gated", T=256, D=4096, F=11008, act="silu", add=False),
        # prefill, or a training step's forward pass
        dict(name="gated_prefill", kind="gated", T=2048, D=4096, F=14336, act="silu", add=False),
        # fine-tuning on a short ragged batch with the products computed again instead of kept
        dict(name="gated_grad_odd", kind="gated_grad", T=333, D=1032, F=2760, act="gelu_tanh", add=True, kept=False),
        # a training step's backward pass, the products kept by the forward pass
        dict(name="gated_grad_train", kind="gated_grad", T=2048, D=4096, F=11008, act="silu", add=False, kept=True),
        # one token of one request beside a square projection
        dict(name="lora_one_token", kind="lora", T=1, K=4096, N=4096, r=16, L=8, order="mixed", none=0.0, base=True,
             out="bfloat16"),
        # a ragged decoding batch, each request with an adapter of its own or none, beside the up-projection
        dict(name="lora_batch_mixed", kind="lora", T=37, K=4096, N=14336, r=64, L=16, order="mixed", none=0.2,
             base=True, out="bfloat16"),
        # prompts of several requests one after the other
        dict(name="lora_prefill", kind="lora", T=2048, K=4096, N=4096, r=16, L=4, order="runs", none=0.0, base=True,
             out="bfloat16"),
        # odd sizes, a partial sum kept in fp32 that is reduced later
        dict(name="lora_prefill_odd", kind="lora", T=1003, K=1416, N=2056, r=40, L=5, order="runs", none=0.1,
             base=False, out="float32"),
        # several adapters trained at once on a shuffled ragged batch
        dict(name="lora_grad_odd", kind="lora_grad", T=333, K=1032, N=2760, r=24, L=5, order="mixed", none=0.1,
             base=True, out="bfloat16"),
        # one adapter trained on a long batch, its gradients in fp32
        dict(name="lora_grad_train", kind="lora_grad", T=4096, K=4096, N=4096, r=16, L=1, order="runs", none=0.0,
             base=True, out="float32"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["gated", "gated", "gated_grad", "lora", "lora", "lora_grad"])
    if kind.startswith("gated"):
        back = kind == "gated_grad"
        case = dict(kind=kind, T=_log(rng, 64 if back else 1, 2048), D=8 * _log(rng, 64, 512),
                    F=8 * _log(rng, 64, 1376 if back else 1792), act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]),
                    add=rng.random() < 0.3)
        if back:      # a product next to 0 has the slope of either side of relu's corner, unless it has been kept
            case["kept"] = case["act"] == "relu" or rng.random() < 0.5
        return case
    back = kind == "lora_grad"
    k = 8 * _log(rng, 64, 1792)
    n = 8 * _log(rng, 64, 1792)
    n = max(64, min(n, 8 * (4096 * 4096 // (8 * k)) if back else 8 * (14336 * 4096 // (8 * k))))
    return dict(kind=kind, T=_log(rng, 64, 4096) if back else _log(rng, 1, 2048), K=k, N=n, r=8 * _log(rng, 1, 16),
                L=_log(rng, 1, 32), order=rng.choice(["runs", "mixed"]), none=rng.choice([0.0, 0.1]),
                base=rng.random() < 0.7, out=rng.choice(["float32", "bfloat16"]))


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device=DEV).mul_(std).to(torch.bfloat16)


def _inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t = case["T"]
    if case["kind"].startswith("gated"):
        dm, f = case["D"], case["F"]
        d = {"x": _normal(gen, (t, dm)), "gate": _normal(gen, (f, dm), 0.02), "up": _normal(gen, (f, dm), 0.02)}
        d["gate_add"] = _normal(gen, (t, f), 0.2) if case["add"] else None
        d["up_add"] = _normal(gen, (t, f), 0.2) if case["add"] else None
        if case["kind"] == "gated_grad":
            d["dh"] = _normal(gen, (t, f))
            d["g"] = d["u"] = None
            if case["kept"]:      # what the forward pass has kept
                g, u = _products(d)
                d["g"], d["u"] = g.to(torch.bfloat16), u.to(torch.bfloat16)
        return d
    k, n, r, e = case["K"], case["N"], case["r"], case["L"]
    d = {"x": _normal(gen, (t, k)), "a": _normal(gen, (e, r, k), k ** -0.5), "b": _normal(gen, (e, n, r), 0.05),
         "scale": 0.5 + torch.rand((e,), generator=gen, device=DEV)}
    ids = torch.randint(0, e, (t,), generator=gen, device=DEV)
    if case["order"] == "runs":
        ids = ids.sort().values
    out = torch.rand((t,), generator=gen, device=DEV) < case["none"]
    d["ids"] = torch.where(out, -1, ids).to(torch.int32).contiguous()
    wide = getattr(torch, case["out"])
    if case["kind"] == "lora":
        d["base"] = torch.randn((t, n), generator=gen, device=DEV).to(wide) if case["base"] else None
    else:
        d["dy"] = _normal(gen, (t, n))
        d["base"] = _normal(gen, (t, k)) if case["base"] else None
    return d


def prepare(case, seed):
    return {"case": case, **_inputs(case, seed)}


# ------------------------------------------------------------------ plain forms

_ROOT2, _ROOT2PI = math.sqrt(0.5), math.sqrt(2.0 / math.pi)


def _act(name, g):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * _ROOT2))
    if name == "gelu_tanh":
        return 0.5 * g * (1.0 + torch.tanh(_ROOT2PI * (g + 0.044715 * g * g * g)))
    return torch.where(g > 0.0, g, torch.zeros_like(g))


def _slope(name, g):
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(g * _ROOT2)) + g * torch.exp(-0.5 * g * g) * (0.5 * _ROOT2 * 2.0 / math.sqrt(math.pi))
    if name == "gelu_tanh":
        t = torch.tanh(_ROOT2PI * (g + 0.044715 * g * g * g))
        return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * _ROOT2PI * (1.0 + 3.0 * 0.044715 * g * g)
    return torch.where(g > 0.0, torch.ones_like(g), torch.zeros_like(g))


def _products(d):
    x = d["x"].float()
    g, u = x @ d["gate"].float().t(), x @ d["up"].float().t()
    if d["gate_add"] is not None:
        g, u = g + d["gate_add"].float(), u + d["up_add"].float()
    return g, u


def _gated_grad(case, d):
    g, u = _products(d) if d["g"] is None else (d["g"].float(), d["u"].float())
    dh = d["dh"].float()
    dg, du = dh * u * _slope(case["act"], g), dh * _act(case["act"], g)
    x = d["x"].float()
    dx = dg @ d["gate"].float() + du @ d["up"].float()
    return [v.to(torch.bfloat16) for v in (dx, dg.t() @ x, du.t() @ x, dg, du)]


def _lora(case, d):
    x = d["x"].float()
    y = torch.zeros((case["T"], case["N"]), device=x.device)
    for e in d["ids"].unique().tolist():
        if e >= 0:
            rows = (d["ids"] == e).nonzero().flatten()
            y[rows] = (x[rows] @ d["a"][e].float().t()) @ d["b"][e].float().t() * d["scale"][e]
    if d["base"] is not None:
        y = y + d["base"].float()
    return y.to(getattr(torch, case["out"]))


def _lora_grad(case, d):
    x, dy = d["x"].float(), d["dy"].float()
    dx = torch.zeros_like(x)
    da, db = torch.zeros(d["a"].shape, device=x.device), torch.zeros(d["b"].shape, device=x.device)
    for e in d["ids"].unique().tolist():
        if e >= 0:
            rows = (d["ids"] == e).nonzero().flatten()
            a, b = d["a"][e].float(), d["b"][e].float()
            v = (dy[rows] @ b) * d["scale"][e]
            dx[rows] = v @ a
            da[e] = v.t() @ x[rows]
            db[e] = dy[rows].t() @ (x[rows] @ a.t()) * d["scale"][e]
    if d["base"] is not None:
        dx = dx + d["base"].float()
    wide = getattr(torch, case["out"])
    return [dx.to(torch.bfloat16), da.to(wide), db.to(wide)]


def run(state):
    case, kind = state["case"], state["case"]["kind"]
    if own:
        import sparse_gemm_layers_amd as sg
        if kind == "gated":
            return sg.gated_gemm(state["x"], state["gate"], state["up"], act=case["act"], gate_add=state["gate_add"],
                                 up_add=state["up_add"])
        if kind == "gated_grad":
            return list(sg.gated_gemm_backward(state["dh"], state["x"], state["gate"], state["up"], act=case["act"],
                                               g=state["g"], u=state["u"], gate_add=state["gate_add"],
                                               up_add=state["up_add"]))
        if kind == "lora":
            return sg.lora_gemm(state["x"], state["ids"], state["a"], state["b"], scale=state["scale"],
                                base=state["base"], out_dtype=getattr(torch, case["out"]))
        return list(sg.lora_gemm_backward(state["dy"], state["x"], state["ids"], state["a"], state["b"],
                                          scale=state["scale"], base=state["base"],
                                          grad_dtype=getattr(torch, case["out"])))
    if kind == "gated":
        g, u = _products(state)
        return (_act(case["act"], g) * u).to(torch.bfloat16)
    if kind == "gated_grad":
        return _gated_grad(case, state)
    if kind == "lora":
        return _lora(case, state)
    return _lora_grad(case, state)


# ------------------------------------------------------------------ cost

def work(case):
    t = case["T"]
    if case["kind"].startswith("gated"):
        d, f = case["D"], case["F"]
        if case["kind"] == "gated":      # x, both weights and what is added in; the hidden values out
            return {"bytes": 2 * (t * d + 2 * f * d + t * f + (2 * t * f if case["add"] else 0)),
                    "flops": 4 * t * d * f}
        # dh, x, both weights and the kept (or added) products in; all gradients out
        pairs = 2 * t * f if case["kept"] or case["add"] else 0
        return {"bytes": 2 * (t * f + t * d + 2 * f * d + pairs + t * d + 2 * f * d + 2 * t * f),
                "flops": (8 if case["kept"] else 12) * t * d * f}
    k, n, r, e = case["K"], case["N"], case["r"], case["L"]
    active = e * (1.0 - (1.0 - 1.0 / e) ** t)          # adapters that t tokens reach at even odds
    with_one = t * (1.0 - case["none"])
    wide = 4 if case["out"] == "float32" else 2
    if case["kind"] == "lora":
        return {"bytes": int(2 * with_one * k + 4 * t + 2 * active * r * (k + n)
                             + t * n * wide * (2 if case["base"] else 1)),
                "flops": int(2 * with_one * r * (k + n))}
    return {"bytes": int(2 * with_one * (k + n) + 4 * t + 2 * active * r * (k + n)
                         + 2 * t * k * (2 if case["base"] else 1) + wide * e * r * (k + n)),
            "flops": int(2 * with_one * r * 3 * (k + n))}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    d = {n: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for n, v in _inputs(case, seed).items()}
    kind = case["kind"]
    if kind == "gated":
        g, u = _exact_products(d)
        return _exact_act(case["act"], g)[0] * u
    if kind == "gated_grad":
        g, u = _exact_products(d) if d["g"] is None else (d["g"], d["u"])
        value, slope = _exact_act(case["act"], g)
        both = torch.cat((d["dh"] * slope * u, d["dh"] * value), dim=1)
        f = case["F"]
        dx = torch.matmul(both, torch.cat((d["gate"], d["up"])))
        dw = torch.matmul(both.T, d["x"])
        return [dx, dw[:f], dw[f:], both[:, :f], both[:, f:]]
    if kind == "lora":
        y = torch.zeros((case["T"], case["N"]), dtype=torch.float64, device=DEV)
        for e in range(case["L"]):
            mine = d["ids"] == e
            if mine.any():      # the weight that the adapter stands for, written out
                y[mine] = torch.matmul(d["x"][mine], torch.matmul(d["b"][e], d["a"][e]).T) * d["scale"][e]
        return y if d["base"] is None else y + d["base"]
    dx = torch.zeros((case["T"], case["K"]), dtype=torch.float64, device=DEV) if d["base"] is None else d["base"]
    da, db = torch.zeros_like(d["a"]), torch.zeros_like(d["b"])
    for e in range(case["L"]):
        mine = d["ids"] == e
        if mine.any():
            x, dy = d["x"][mine], d["dy"][mine] * d["scale"][e]
            full = torch.matmul(dy.T, x)                     # the gradient of that weight
            da[e] = torch.matmul(d["b"][e].T, full)
            db[e] = torch.matmul(full, d["a"][e].T)
            dx[mine] += torch.matmul(dy, torch.matmul(d["b"][e], d["a"][e]))
    return [dx, da, db]


def _exact_products(d):
    f = d["gate"].shape[0]
    both = torch.matmul(d["x"], torch.cat((d["gate"], d["up"])).T)
    if d["gate_add"] is not None:
        both += torch.cat((d["gate_add"], d["up_add"]), dim=1)
    return both[:, :f], both[:, f:]


def _exact_act(name, g):
    """The activation and its derivative."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if name == "gelu":
        phi = torch.special.ndtr(g)
        return g * phi, phi + g * torch.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":      # (1 + tanh z) / 2 = sigmoid(2 z)
        z2 = 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
        s = torch.sigmoid(z2)
        inner = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * g ** 2)
        return g * s, s + g * s * torch.sigmoid(-z2) * inner
    return g.clamp_min(0.0), (g > 0.0).double()

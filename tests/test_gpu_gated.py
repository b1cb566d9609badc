"""The gated projections on the GPU against the fp64 oracle, at the sizes where the
ways of computing them change and at odd ones.

Error allowed, from the arithmetic: a fp32 sum of n terms is off by at most (n + 4)
2^-24 times the sum of their magnitudes; the activation's value and slope are within
2^-18 (1 + |g|) (an exponential whose relative error is 2^-21 + |g| 2^-23, times g), have
slopes of at most 1.13 and 0.8, and carry the error of their argument with those; half
a step of the result's type comes last.  dx and the weights' gradients are checked
against the bf16 dg and du that the call returns, which are their operands."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, down, say
from oracle import adapt

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TINY = 2.0 ** -120


def bf(seed, *shape, std=1.0):
    return (std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(BF16)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def gpu(t):
    return None if t is None else t.to(DEV)


def within(what, got, ref, tol):
    err = np.abs(down(got).astype(np.float64) - ref)
    assert np.isfinite(err).all(), f"{what}: not finite"
    assert (err <= tol).all(), f"{what}: off by {np.max(err / tol):.3g} of what is allowed"
    say(f"  {what}: max |err| / allowed = {np.max(err / tol):.3g}")


def half(dtype, ref):
    return torch.finfo(dtype).eps / 2 * np.abs(ref) + TINY


def sum_tol(n, size):
    return (n + 4) * 2.0 ** -24 * size


def product_errors(D, g, u, size_g, size_u):
    """(allowed errors of G, of U, of a(G), of a'(G))."""
    eg, eu = sum_tol(D, size_g), sum_tol(D, size_u)
    own = 2.0 ** -18 * (1.0 + np.abs(g))
    return eg, eu, 1.13 * eg + own, 0.8 * eg + own


def make(T, F, D, add, seed=0):
    x, gate, up = bf(seed + 1, T, D), bf(seed + 2, F, D, std=D ** -0.5), bf(seed + 3, F, D, std=D ** -0.5)
    return x, gate, up, bf(seed + 4, T, F) if add else None, bf(seed + 5, T, F) if add else None


SHAPES = [
    # T, F, D, act, addends
    (1, 8, 8, "silu", False), (1, 16, 136, "gelu", True), (1, 1000, 4096, "silu", False), (3, 24, 40, "gelu_tanh", True),
    (16, 48, 128, "relu", False), (17, 264, 72, "silu", True), (37, 136, 264, "gelu", False), (48, 520, 1032, "silu", False),
    (64, 128, 256, "relu", True), (65, 64, 32, "silu", False), (129, 72, 200, "gelu_tanh", False),
    (300, 520, 96, "gelu", True), (257, 1032, 264, "silu", True), (128, 128, 64, "relu", False),
    (4093, 2056, 72, "silu", False), (4096, 2048, 40, "gelu_tanh", True),
]


@pytest.mark.parametrize("T,F,D,act,add", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward(T, F, D, act, add, dtype):
    say(f"gated {T}x{F}x{D} {act} {dtype}")
    x, gate, up, ga, ua = make(T, F, D, add)
    h, g, u = sg.gated_gemm(*map(gpu, (x, gate, up)), act=act, gate_add=gpu(ga), up_add=gpu(ua), out_dtype=dtype, keep=True)
    rh, rg, ru, size_g, size_u = adapt.gated(*map(f64, (x, gate, up)), act, f64(ga), f64(ua))
    eg, eu, ea, _ = product_errors(D, rg, ru, size_g, size_u)
    within("g", g, rg, eg + half(BF16, rg) * (1 + 2.0 ** -8))
    within("u", u, ru, eu + half(BF16, ru) * (1 + 2.0 ** -8))
    eh = ea * (np.abs(ru) + eu) + np.abs(adapt.act(act, rg)[0]) * eu + 2.0 ** -23 * np.abs(rh)
    within("h", h, rh, eh + half(dtype, np.abs(rh) + eh))
    alone = sg.gated_gemm(*map(gpu, (x, gate, up)), act=act, gate_add=gpu(ga), up_add=gpu(ua), out_dtype=dtype)
    assert torch.equal(alone, h)      # keeping G and U changes nothing


BACK = [
    (1, 8, 8, "silu", False), (2, 24, 136, "gelu", True), (16, 48, 128, "relu", False), (37, 136, 264, "gelu_tanh", True),
    (64, 264, 72, "silu", False), (65, 64, 32, "gelu", False), (129, 72, 200, "silu", True), (300, 520, 96, "gelu_tanh", False),
    (333, 1032, 264, "silu", False), (40, 4104, 2056, "silu", False), (2049, 72, 2048, "gelu", False),
    (1025, 2056, 520, "relu", True), (4093, 2056, 72, "silu", False),
]


@pytest.mark.parametrize("T,F,D,act,add", BACK)
@pytest.mark.parametrize("kept", [True, False])
def test_backward(T, F, D, act, add, kept):
    say(f"gated backward {T}x{F}x{D} {act} kept {kept}")
    x, gate, up, ga, ua = make(T, F, D, add, seed=10)
    dh = bf(16, T, F)
    args = [gpu(v) for v in (x, gate, up)]
    g = u = None
    if kept:
        _, g, u = sg.gated_gemm(*args, act=act, gate_add=gpu(ga), up_add=gpu(ua), keep=True)
    dx, dgate, dup, dg, du = sg.gated_gemm_backward(gpu(dh), *args, act=act, g=g, u=u, gate_add=gpu(ga), up_add=gpu(ua))
    if kept:
        rg, ru = f64(g), f64(u)
        zero = np.zeros_like(rg)
        eg, eu, ea, es = product_errors(D, rg, ru, zero, zero)
    else:
        _, rg, ru, size_g, size_u = adapt.gated(*map(f64, (x, gate, up)), act, f64(ga), f64(ua))
        eg, eu, ea, es = product_errors(D, rg, ru, size_g, size_u)
        if act == "relu":
            es = np.where(np.abs(rg) <= eg, 1.0, es)      # either side of the corner
    d = np.abs(f64(dh))
    a, s = adapt.act(act, rg)
    rdg, rdu = adapt.gated_slopes(f64(dh), rg, ru, act)
    edg = d * (es * (np.abs(ru) + eu) + np.abs(s) * eu) + 2.0 ** -22 * np.abs(rdg)
    edu = d * ea + 2.0 ** -23 * np.abs(rdu)
    within("dg", dg, rdg, edg + half(BF16, np.abs(rdg) + edg))
    within("du", du, rdu, edu + half(BF16, np.abs(rdu) + edu))
    refs, sizes = adapt.gated_grads(*map(f64, (dg, du, x, gate, up)))
    for what, got, ref, size, n in zip(("dx", "dgate", "dup"), (dx, dgate, dup), refs, sizes, (2 * F, T, T)):
        e = sum_tol(n + 64, size)      # parts of a sum are added too
        within(what, got, ref, e + half(BF16, np.abs(ref) + e))


@pytest.mark.parametrize("T", [5, 70, 300])
def test_slope_against_differences(T):
    """h moves with gate_add as dg says, and with up_add, in which it is linear, as du
    says.  A step of 2^-6 in bf16 values that are multiples of 2^-6: exact; d^2 / 6
    times a third derivative of at most 2 is left out; h's fp32 error is divided by d."""
    F, D, d = 72, 104, 2.0 ** -6
    x, gate, up = bf(1, T, D), bf(2, F, D, std=D ** -0.5), bf(3, F, D, std=D ** -0.5)
    ga = (torch.randint(-64, 64, (T, F), generator=torch.Generator().manual_seed(4)) / 64).to(BF16)
    zero = torch.zeros((T, F), dtype=BF16)
    args = [gpu(v) for v in (x, gate, up)]
    one = gpu(torch.ones((T, F), dtype=BF16))
    for act in ("silu", "gelu", "gelu_tanh"):
        def h(dg, du):
            # multiples of 2^-6 below 2 have at most 7 significant bits, as bf16 has
            return f64(sg.gated_gemm(*args, act=act, gate_add=gpu((ga + dg).to(BF16)), up_add=gpu((zero + du).to(BF16)),
                                     out_dtype=F32))

        _, _, _, dg, du = sg.gated_gemm_backward(one, *args, act=act, gate_add=gpu(ga), up_add=gpu(zero))
        _, rg, ru, size_g, size_u = adapt.gated(*map(f64, (x, gate, up)), act, f64(ga), f64(zero))
        eg, eu, ea, es = product_errors(D, rg, ru, size_g, size_u)
        eh = ea * (np.abs(ru) + 1) + np.abs(rg) * eu + 2.0 ** -22 * np.abs(rg * ru)
        by_g, by_u = (h(d, 0) - h(-d, 0)) / (2 * d), (h(0, d) - h(0, -d)) / (2 * d)
        within(f"{act} dg", dg, by_g, d * d / 3 * np.abs(ru) + eh / d + es * np.abs(ru) + eu * 1.13 + half(BF16, by_g) * 1.01)
        within(f"{act} du", du, by_u, eh / d + ea + half(BF16, by_u) * 1.01)

"""The gated projections' gradients against the formula itself, in fp64 from the inputs to the end:
what rounding dG and dU to bf16 before the products that follow may cost is bounded here, next to
half a step of the result's type.

dG is off by at most e_G = its own error (test_gpu_gated) and half a bf16 step of |dG|; so dx is off
by at most e_G |Wg| + e_U |Wu|, plus the fp32 sum's error, plus half a step; likewise the weights'.
Over all elements those roundings are independent: bf16 values step by 2^-7 of the power of two below
them, so an error's mean square is 2^-14 / 12 of that power's square, at most that of the value's.  With
terms of random signs the products carry dG's and dU's to the sum at that size, and the sum's own
rounding comes on top: over the whole output the relative error is under sqrt(2) * 2^-7 / sqrt(12)."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import down, say
from oracle import adapt
from test_gpu_gated import BF16, bf, f64, gpu, half, make, product_errors, sum_tol, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,F,D,act", [(9, 136, 264, "gelu"), (333, 1032, 520, "silu"), (387, 1552, 2216, "gelu_tanh")])
@pytest.mark.parametrize("kept", [True, False])
def test_gradients(T, F, D, act, kept):
    say(f"gated gradients {T}x{F}x{D} {act} kept {kept}")
    x, gate, up, _, _ = make(T, F, D, False, seed=280)
    dh = bf(286, T, F)
    args = [gpu(v) for v in (x, gate, up)]
    g = u = None
    if kept:
        g, u = bf(287, T, F), bf(288, T, F)
        rg, ru = f64(g), f64(u)
        size_g = size_u = np.zeros_like(rg)
    else:
        _, rg, ru, size_g, size_u = adapt.gated(*map(f64, (x, gate, up)), act)
    got = sg.gated_gemm_backward(gpu(dh), *args, act=act, g=gpu(g), u=gpu(u))[:3]
    eg, eu, ea, es = product_errors(D, rg, ru, size_g, size_u)
    d = np.abs(f64(dh))
    rdg, rdu = adapt.gated_slopes(f64(dh), rg, ru, act)
    edg = d * (es * (np.abs(ru) + eu) + np.abs(adapt.act(act, rg)[1]) * eu) + 2.0 ** -22 * np.abs(rdg)
    edu = d * ea + 2.0 ** -23 * np.abs(rdu)
    edg, edu = edg + half(BF16, np.abs(rdg) + edg), edu + half(BF16, np.abs(rdu) + edu)
    (X, G, U) = map(f64, (x, gate, up))
    refs, sizes = adapt.gated_grads(rdg, rdu, X, G, U)
    carried = (edg @ np.abs(G) + edu @ np.abs(U), edg.T @ np.abs(X), edu.T @ np.abs(X))
    for what, have, ref, size, e, n in zip(("dx", "dgate", "dup"), got, refs, sizes, carried, (2 * F, T, T)):
        e = e + sum_tol(n + 64, size + e)
        within(what, have, ref, e + half(BF16, np.abs(ref) + e))
        rel = np.linalg.norm(down(have).astype(np.float64) - ref) / np.linalg.norm(ref)
        say(f"  {what}: {rel:.5f} of the whole")
        assert rel < np.sqrt(2.0) * 2.0 ** -7 / np.sqrt(12.0)

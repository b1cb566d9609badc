"""Every way a gated projection and its backward pass go, by size, against the fp64 oracle: each
case says which it is meant for and fails if it goes another.  Sizes that no tile divides, and
sums long enough that each ring of blocks in LDS goes round."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
import test_gpu_gated as gated
from gpu_helpers import say
from oracle import adapt
from test_gpu_adapt_use import same, wide
from test_gpu_gated import BF16, F32, bf, f64, gpu, half, make, sum_tol, within

pytestmark = pytest.mark.gpu

# (T, F, D, act, addends), (tokens, hidden values) of a workgroup
FORWARD = [
    ((7, 520, 1032, "gelu", True), (16, 16)), ((70, 1032, 1032, "silu", False), (64, 32)),
    ((203, 4104, 552, "relu", False), (128, 64)), ((389, 4152, 552, "silu", True), (256, 64)),
    ((790, 4360, 552, "gelu_tanh", False), (256, 128)),
]
# T, F, D, with the weights' gradients, (rows and columns of a gradient, whether dx's sum has parts)
BACKWARD = [
    (345, 288, 264, True, (128, False)), (37, 440, 280, True, (128, True)), (455, 264, 552, False, (128, False)),
    (333, 1032, 520, False, (128, True)), (1066, 400, 4152, True, (256, False)), (387, 1552, 2216, True, (256, True)),
    (2389, 264, 3368, False, (256, False)), (661, 2656, 3592, False, (256, True)),
]


def backward_way(T, F, D, dw):
    tile, parts = sg.gated_gemm_backward_plan(T, F, D, dw)
    return tile, parts > 1


@pytest.mark.parametrize("size,way", FORWARD)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward(size, way, dtype):
    assert sg.gated_gemm_plan(*size[:3]) == way
    gated.test_forward(*size, dtype)


@pytest.mark.parametrize("size,way", FORWARD)
def test_products_computed_again(size, way):
    assert sg.gated_gemm_plan(*size[:3]) == way
    gated.test_backward(*size, False)


@pytest.mark.parametrize("T,F,D,dw,way", BACKWARD)
def test_backward(T, F, D, dw, way):
    assert backward_way(T, F, D, dw) == way
    say(f"gated backward {T}x{F}x{D} dw {dw} {way}")
    x, gate, up, _, _ = make(T, F, D, False, seed=120)
    g, u, dh = bf(126, T, F), bf(127, T, F), bf(128, T, F)
    args = [gpu(v) for v in (dh, x, gate, up)]
    kept = dict(g=gpu(g), u=gpu(u), need_dw=dw)
    dx, dgate, dup, dg, du = sg.gated_gemm_backward(*args, **kept)
    refs, sizes = adapt.gated_grads(*map(f64, (dg, du, x, gate, up)))
    for what, got, ref, size, n in zip(("dx", "dgate", "dup"), (dx, dgate, dup), refs, sizes, (2 * F, T, T)):
        if got is not None:
            e = sum_tol(n + 64, size)
            within(what, got, ref, e + half(BF16, np.abs(ref) + e))
    assert (dgate is None) == (dup is None) == (not dw)
    # rows further apart, NaN behind each; results of the caller's
    strided = [wide(v, 8 * (i + 1)) for i, v in enumerate(args)]
    out = dict(dx=wide(torch.zeros_like(dx), 8), dg=wide(torch.zeros_like(dg), 24), du=wide(torch.zeros_like(du), 24))
    if dw:
        out.update(dgate=wide(torch.zeros_like(dgate), 16), dup=wide(torch.zeros_like(dup), 16))
    got = sg.gated_gemm_backward(*strided, g=wide(kept["g"], 8), u=wide(kept["u"], 8), need_dw=dw, **out)
    for p, q in zip(got, (dx, dgate, dup, dg, du)):
        assert (p is None and q is None) or same(p, q)
    for t in out.values():
        assert torch.isnan(t.as_strided((T if t.shape[0] == T else F, t.stride(0)), (t.stride(0), 1))[:, t.shape[1]:]).all()
    if dw:
        only = sg.gated_gemm_backward(*args, **kept, need_dx=False)
        assert only[0] is None and all(same(p, q) for p, q in zip(only[1:], (dgate, dup, dg, du)))

"""Infinite elements of every operand of the low-rank adapters, in each way a call goes:
infinities and NaN stand where the formulas in fp64 put them, signs included.

A finite result has no infinite term, so its error is bounded as in test_gpu_lora."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import down, say
from oracle import adapt
from test_gpu_lora import BF16, F32, allowed, bf, f64, gpu, make

pytestmark = pytest.mark.gpu

INF = float("inf")


def like(what, got, ref, tol):
    got = down(got).astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN at {np.argwhere(np.isnan(got) != np.isnan(ref))[:4]}"
    far = np.isinf(ref)
    assert np.array_equal(np.isinf(got), far) and np.array_equal(got[far], ref[far]), f"{what}: infinities differ"
    at = np.isfinite(ref)
    assert (np.abs(got[at] - ref[at]) <= tol[at]).all(), what
    say(f"  {what}: {far.sum()} infinite, {np.isnan(ref).sum()} NaN")
    return far.any()


# T, K, N, r, L, order: one launch with 16, 32 and 64 ranks, two launches, 32-token items
FORWARD = [(3, 72, 136, 8, 2, "mixed"), (20, 136, 520, 16, 3, "mixed"), (9, 264, 72, 24, 2, "runs"), (33, 72, 264, 40, 2, "mixed"),
           (70, 72, 136, 16, 2, "mixed"), (90, 136, 264, 72, 3, "runs"), (600, 72, 136, 40, 3, "mixed")]


@pytest.mark.parametrize("T,K,N,r,L,order", FORWARD)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_infinite_b(T, K, N, r, L, order, dtype):
    say(f"lora {T}x{K}x{N} r {r} L {L} {order} {dtype}")
    x, ids, a, b, scale = make(T, K, N, r, L, order, seed=200)
    b[0, 3, 1], b[0, 17, r - 1], b[1, 5, 0], b[1, 40, 2] = INF, -INF, -INF, float("nan")
    b[0, 33, 0], b[0, 33, 3] = INF, INF             # of one sign or not, as the token has it
    # exactly one: its second bf16 part is nothing
    x[0], a[0, 1], ids[0], scale[0] = 0.0, 0.0, 0, 1.0
    x[0, 4], a[0, 1, 4] = 1.0, 1.0
    with np.errstate(invalid="ignore"):
        ref, inner, outer = adapt.lora(f64(x), ids.numpy(), f64(a), f64(b), f64(scale))
        tol = allowed(dtype, dtype == F32, ref, inner, outer, K, r)
    assert ref[0, 3] == INF
    assert like("y", sg.lora_gemm(gpu(x), gpu(ids), gpu(a), gpu(b), gpu(scale), out_dtype=dtype), ref, tol)


BACK = [(5, 72, 136, 8, 2, "mixed"), (90, 136, 264, 24, 3, "runs"), (300, 72, 136, 40, 2, "mixed"), (1100, 72, 136, 16, 1, "one"),
        (1100, 72, 136, 72, 1, "one")]


@pytest.mark.parametrize("T,K,N,r,L,order", BACK)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("where", ["x", "dy", "a", "b"])
def test_backward(T, K, N, r, L, order, dtype, where):
    say(f"lora backward {T}x{K}x{N} r {r} L {L} {order} {dtype}: infinite {where}")
    x, ids, a, b, scale = make(T, K, N, r, L, order, seed=220)
    dy = bf(226, T, N)
    ids[0], ids[T // 2] = 0, L - 1
    if where == "x":
        x[0, 3], x[T // 2, 20] = INF, -INF
    elif where == "dy":
        dy[0, 3], dy[T // 2, 20] = INF, -INF
    elif where == "a":
        a[0, 1, 3], a[L - 1, r - 1, 20] = INF, -INF
    else:
        b[0, 3, 1], b[L - 1, 20, r - 1] = INF, -INF
    with np.errstate(invalid="ignore"):
        refs, inner, outer = adapt.lora_grads(f64(dy), f64(x), ids.numpy(), f64(a), f64(b), f64(scale))
        sizes = [(n_in, n_out) for n_in, n_out in ((N, r), (N, T), (K, T))]
        tols = [allowed(BF16 if i == 0 else dtype, i > 0 and dtype == F32, refs[i], inner[i], outer[i], *sizes[i])
                for i in range(3)]
    got = sg.lora_gemm_backward(gpu(dy), gpu(x), gpu(ids), gpu(a), gpu(b), gpu(scale), grad_dtype=dtype)
    far = [like(what, *three) for what, *three in zip(("dx", "da", "db"), got, refs, tols)]
    assert any(far)
    alone = sg.lora_gemm_backward(gpu(dy), gpu(x), gpu(ids), gpu(a), gpu(b), gpu(scale), need_dab=False)[0]
    like("dx alone", alone, refs[0], tols[0])

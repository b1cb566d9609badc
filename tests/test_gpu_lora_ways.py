"""Every way the low-rank adapters' calls go, by size, against the fp64 oracle: each case says
which it is meant for and fails if it goes another."""
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import say
from oracle import adapt
from test_gpu_adapt_use import same, wide
from test_gpu_lora import BF16, F32, allowed, bf, f64, gpu, make, within

pytestmark = pytest.mark.gpu

# T, K, N, r, L, order; forward: launches, tokens, ranks, parts; backward: tokens, ranks, parts of both
# sums, ranks and token parts of the sums over tokens
CASES = [
    ((20, 72, 1032, 16, 3, "mixed"), (1, 16, 16, 1), (16, 16, 2, 1, 16, 1)),
    ((33, 136, 520, 24, 2, "mixed"), (1, 16, 32, 1), (16, 16, 1, 1, 32, 1)),
    ((50, 264, 328, 56, 3, "runs"), (1, 16, 64, 1), (16, 16, 1, 1, 64, 1)),
    ((90, 136, 72, 16, 3, "mixed"), (2, 16, 16, 1), (16, 16, 1, 1, 16, 1)),
    ((90, 1032, 2056, 40, 3, "runs"), (2, 16, 16, 2), (16, 16, 2, 2, 64, 1)),
    ((2100, 72, 136, 32, 2, "mixed"), (2, 16, 32, 1), (16, 32, 1, 1, 32, 4)),
    ((2500, 264, 72, 24, 3, "runs"), (2, 16, 32, 1), (16, 32, 1, 1, 32, 3)),
    ((1500, 1032, 72, 24, 1, "one"), (2, 16, 32, 2), (16, 16, 1, 2, 32, 5)),
    ((500, 72, 136, 256, 2, "mixed"), (2, 16, 32, 1), (16, 32, 1, 1, 64, 1)),
    ((500, 1032, 1040, 256, 2, "mixed"), (2, 16, 64, 2), (16, 64, 2, 2, 64, 1)),
    ((600, 136, 264, 48, 2, "mixed"), (2, 32, 32, 1), (32, 32, 1, 1, 64, 1)),
    ((600, 1032, 1040, 64, 1, "runs"), (2, 32, 32, 2), (32, 32, 2, 2, 64, 2)),
    ((2300, 264, 136, 72, 1, "mixed"), (2, 32, 64, 1), (32, 64, 1, 1, 64, 8)),
    ((2040, 1032, 1048, 72, 1, "one"), (2, 32, 64, 2), (32, 64, 2, 2, 64, 7)),
    ((4100, 72, 40, 8, 2, "runs"), (2, 16, 16, 1), (16, 16, 1, 1, 16, 8)),
]


def forward_way(T, K, N, r, L):
    return tuple(sg.lora_gemm_plan(T, K, N, r, L).values())


def backward_way(T, K, N, r, L):
    return tuple(sg.lora_gemm_backward_plan(T, K, N, r, L).values())


@pytest.mark.parametrize("size,way,_", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward(size, way, _, dtype):
    T, K, N, r, L, order = size
    assert forward_way(*size[:5]) == way
    say(f"lora {size} {dtype} {way}")
    x, ids, a, b, scale = make(*size, seed=140)
    base = bf(146, T, N)
    args = [gpu(v) for v in (ids, a, b, scale)]
    y = sg.lora_gemm(gpu(x), *args, gpu(base), out_dtype=dtype)
    ref, inner, outer = adapt.lora(f64(x), ids.numpy(), f64(a), f64(b), f64(scale), f64(base))
    within("y", y, ref, allowed(dtype, dtype == F32, ref, inner, outer, K, r))
    out = wide(torch.zeros_like(y), 24)
    assert same(sg.lora_gemm(wide(gpu(x), 8), *args, wide(gpu(base), 16), y=out), y)
    assert torch.isnan(out.as_strided((T, out.stride(0)), (out.stride(0), 1))[:, N:]).all()


@pytest.mark.parametrize("size,_,way", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward(size, _, way, dtype):
    T, K, N, r, L, order = size
    assert backward_way(*size[:5]) == way
    say(f"lora backward {size} {dtype} {way}")
    x, ids, a, b, scale = make(*size, seed=160)
    dy, base = bf(166, T, N), bf(167, T, K)
    args = [gpu(v) for v in (x, ids, a, b, scale)]
    got = sg.lora_gemm_backward(gpu(dy), *args, gpu(base), grad_dtype=dtype)
    refs, inner, outer = adapt.lora_grads(f64(dy), f64(x), ids.numpy(), f64(a), f64(b), f64(scale), f64(base))
    for i, (what, n_in, n_out) in enumerate((("dx", N, r), ("da", N, T), ("db", K, T))):
        t = BF16 if i == 0 else dtype
        within(what, got[i], refs[i], allowed(t, i > 0 and dtype == F32, refs[i], inner[i], outer[i], n_in, n_out))
    alone = sg.lora_gemm_backward(gpu(dy), *args, gpu(base), need_dab=False)
    assert same(alone[0], got[0])
    alone = sg.lora_gemm_backward(gpu(dy), *args, gpu(base), need_dx=False, grad_dtype=dtype)
    assert alone[0] is None and same(alone[1], got[1]) and same(alone[2], got[2])
    dx = wide(torch.zeros_like(got[0]), 8)
    args[0] = wide(args[0], 8)
    again = sg.lora_gemm_backward(wide(gpu(dy), 24), *args, wide(gpu(base), 16), dx=dx, grad_dtype=dtype)
    assert all(same(p, q) for p, q in zip(again, got))

"""Batches whose tokens are nearly all of one adapter among many, with the tokens of the
sums in parts: most parts and adapters have nothing to add."""
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import say
from oracle import adapt
from test_gpu_lora import BF16, F32, allowed, bf, f64, gpu, make, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N,r,L", [(11000, 72, 40, 16, 20), (8400, 40, 72, 72, 16)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("others", [False, True])
def test_nearly_all_of_one_adapter(T, K, N, r, L, dtype, others):
    say(f"lora {T}x{K}x{N} r {r} L {L} {dtype} others {others}")
    assert sg.lora_gemm_backward_plan(T, K, N, r, L)["token_parts"] > 1
    x, ids, a, b, scale = make(T, K, N, r, L, "one", seed=260)
    ids[:] = 7
    if others:      # in the first part alone, in the last alone, and none at all
        ids[5], ids[64:70], ids[T - 1], ids[T - 300:T - 290] = 0, 3, L - 1, -1
    dy, base = bf(266, T, N), bf(267, T, K)
    args = [gpu(v) for v in (x, ids, a, b, scale)]
    got = sg.lora_gemm_backward(gpu(dy), *args, gpu(base), grad_dtype=dtype)
    refs, inner, outer = adapt.lora_grads(f64(dy), f64(x), ids.numpy(), f64(a), f64(b), f64(scale), f64(base))
    for i, (what, n_in, n_out) in enumerate((("dx", N, r), ("da", N, T), ("db", K, T))):
        t = BF16 if i == 0 else dtype
        within(what, got[i], refs[i], allowed(t, i > 0 and dtype == F32, refs[i], inner[i], outer[i], n_in, n_out))
    for e in range(L):
        if not (ids == e).any():
            assert not got[1][e].any() and not got[2][e].any()
    y = sg.lora_gemm(*args)
    ref, inner, outer = adapt.lora(f64(x), ids.numpy(), f64(a), f64(b), f64(scale))
    within("y", y, ref, allowed(BF16, False, ref, inner, outer, K, r))

"""An infinite element of x with a rank that is no multiple of 16: the ranks that fill a
matrix instruction up are no part of the sum."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import say
from oracle import adapt
from test_gpu_lora import BF16, F32, allowed, f64, gpu, make
from test_gpu_lora_infinite import INF, like

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [2, 64, 90])
@pytest.mark.parametrize("r", [8, 16, 24, 40, 56, 64, 72])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward(T, r, dtype):
    say(f"lora {T} tokens, rank {r} {dtype}")
    K, N, L = 72, 136, 2
    x, ids, a, b, scale = make(T, K, N, r, L, "mixed", seed=240)
    a, b = a.abs() + 0.25, b.abs() + 0.25          # every term of one sign
    ids[0], ids[T - 1] = 0, 1
    x[0, 3], x[T - 1, 70] = INF, -INF
    with np.errstate(invalid="ignore"):
        ref, inner, outer = adapt.lora(f64(x), ids.numpy(), f64(a), f64(b), f64(scale))
        tol = allowed(dtype, dtype == F32, ref, inner, outer, K, r)
    assert (ref[0] == INF).all() and (ref[T - 1] == -INF).all()
    assert like("y", sg.lora_gemm(gpu(x), gpu(ids), gpu(a), gpu(b), gpu(scale), out_dtype=dtype), ref, tol)

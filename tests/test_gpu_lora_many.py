"""As many adapters as a call takes: 65535 beside 33024 columns, 35 GB of them, most of which
nothing reads (they are not even written here)."""
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV
from oracle import adapt
from test_gpu_lora import BF16, allowed, bf, f64, gpu, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [6, 70])
def test_forward(T):
    K, N, r, L = 8, 33024, 8, 65535
    a, b = (torch.empty(s, dtype=BF16, device=DEV) for s in ((L, r, K), (L, N, r)))
    used = [0, 1, 32767, L - 1]
    small_a, small_b = bf(1, 4, r, K, std=K ** -0.5), bf(2, 4, N, r, std=0.1)
    for i, e in enumerate(used):
        a[e].copy_(small_a[i])
        b[e].copy_(small_b[i])
    x = bf(3, T, K)
    local = torch.randint(-1, 4, (T,), generator=torch.Generator().manual_seed(4))
    local[0], local[1] = 3, -1
    ids = torch.tensor([used[i] if i >= 0 else L for i in local.tolist()], dtype=torch.int32)
    y = sg.lora_gemm(gpu(x), gpu(ids), a, b)
    ref, inner, outer = adapt.lora(f64(x), local.numpy(), f64(small_a), f64(small_b))
    within("y", y, ref, allowed(BF16, False, ref, inner, outer, K, r))
    with pytest.raises(sg.SgError, match="2\\^24"):
        sg.lora_gemm_backward(gpu(bf(5, T, N)), gpu(x), gpu(ids), a, b)

"""Sizes of the adapters' calls at the edge of what they take: the forward call has no limit
but those of its operands, the backward call that of its launch's workgroups (under
2^24 of 256 threads).  Fake addresses, never dereferenced; only where no GPU is visible."""
import pytest

import sparse_gemm_layers_amd as sg
from sparse_gemm_layers_amd import _lora
from test_adapt_abi import HIP, LORA, LORA_BACK, SHAPE, call, no_gpu

# T, K, N, r, L: each within the limits of the operands
WIDE = [(1, 65536, 65536, 16, 40000), (100, 4096, 16384, 256, 65535), (1 << 21, 4096, 131072, 16, 1), (5, 8, 33024, 8, 65535)]


def back_fits(T, K, N, r, L):
    return -(-max(K, N) // 256) * (2 * L * -(-r // 64) + -(-T // 64)) < (1 << 24) - 4096


@pytest.mark.parametrize("T,K,N,r,L", WIDE)
def test_workspaces(T, K, N, r, L):
    assert sg.lora_gemm_workspace(T, K, N, r, L) >= 0
    assert not back_fits(T, K, N, r, L) and sg.lora_gemm_backward_workspace(T, K, N, r, L) == -1


def test_edge_of_the_backward_call():
    # 128 column blocks: 2 * 65535 + ceil(T / 64) under 2^17 - 32, so no token fits; 127: all do
    edge = [(T, 8, 32768, 8, L) for T in (1, 64, 65, 4096) for L in (65500, 65519, 65520, 65521, 65535)]
    seen = set()
    for case in edge + [(T, 32512, 8, 64, 65535) for T in (1, 4096, 65536, 70000)]:
        assert (sg.lora_gemm_backward_workspace(*case) > 0) == back_fits(*case), case
        seen.add(back_fits(*case))
    assert seen == {True, False}


@no_gpu
@pytest.mark.parametrize("T,K,N,r,L", WIDE)
def test_calls(T, K, N, r, L):
    size = dict(T=T, K=K, N=N, r=r, L=L, ldx=K, ldy=N, ldb=N)
    assert call(_lora, "sg_lora_gemm", LORA, size) == HIP                 # launched (there is no GPU)
    assert call(_lora, "sg_lora_gemm_backward", LORA_BACK, dict(T=T, K=K, N=N, r=r, L=L, ldx=K, lddy=N, ldb=K, lddx=K)) == SHAPE


def test_the_error_names_what_is_wrong():
    for back, words in ((False, ["65535", "2^22"]), (True, ["65535", "2^22", "2^24"])):
        with pytest.raises(sg.SgError) as e:
            _lora._need(back, 1, 8, 8, 8, 70000)
        assert all(w in str(e.value) for w in words)

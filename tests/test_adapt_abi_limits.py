"""Sizes and workspaces at the edge of what the calls take: the adapters' forward call has no
limit but those of its operands, the backward call that of its launch's workgroups (under
2^24 of 256 threads); workspaces are taken at their size and refused a byte below it.  Fake
addresses, never dereferenced; only where no GPU is visible."""
import pytest

import sparse_gemm_layers_amd as sg
from sparse_gemm_layers_amd import _gated, _lora
from test_adapt_abi import GATED_BACK, HIP, LORA, LORA_BACK, SHAPE, call, no_gpu

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


GRADS = [(333, 2760, 1032), (500, 2056, 2056), (2049, 1032, 2056), (37, 440, 280), (661, 2656, 3592)]


@no_gpu
@pytest.mark.parametrize("dw", [True, False])
@pytest.mark.parametrize("T,F,D", GRADS)
def test_gated_backward_takes_the_workspace_of_its_own_plan_and_no_less(T, F, D, dw):
    parts = sg.gated_gemm_backward_plan(T, F, D, dw)[1]
    need = 4 * parts * T * D if parts > 1 else 0
    size = dict(T=T, F=F, D=D, lddh=F, ldx=D, ldg=D, ldu=D, ldgu=F, lda=F, lddgu=F, lddx=D, lddw=D)
    if not dw:
        size.update(dgate=None, dup=None)
    assert call(_gated, "sg_gated_gemm_backward", GATED_BACK, dict(size, wsb=need)) == HIP       # launched
    if need:
        assert call(_gated, "sg_gated_gemm_backward", GATED_BACK, dict(size, wsb=need - 1)) == SHAPE
    # without dx none is needed
    assert call(_gated, "sg_gated_gemm_backward", GATED_BACK, dict(size, dx=None, ws=None, wsb=0)) == HIP
    assert sg.gated_gemm_backward_workspace(T, F, D) >= need


@no_gpu
@pytest.mark.parametrize("T,K,N,r,L", [(65, 40, 48, 16, 5), (100, 1032, 2056, 40, 3), (1500, 4096, 72, 24, 1), (2040, 1032, 1048, 72, 1)])
def test_adapters_take_their_workspace_and_no_less(T, K, N, r, L):
    size = dict(T=T, K=K, N=N, r=r, L=L, ldx=K, ldy=N, ldb=N)
    need, plan = sg.lora_gemm_workspace(T, K, N, r, L), sg.lora_gemm_plan(T, K, N, r, L)
    assert need >= 4 * plan["parts"] * T * r
    assert call(_lora, "sg_lora_gemm", LORA, dict(size, wsb=need)) == HIP
    assert call(_lora, "sg_lora_gemm", LORA, dict(size, wsb=need - 1)) == SHAPE
    size = dict(T=T, K=K, N=N, r=r, L=L, ldx=K, lddy=N, ldb=K, lddx=K)
    need, plan = sg.lora_gemm_backward_workspace(T, K, N, r, L), sg.lora_gemm_backward_plan(T, K, N, r, L)
    parts = plan["token_parts"] if plan["token_parts"] > 1 else 0
    assert need >= 4 * (T * r * (plan["parts_u"] + plan["parts_v"]) + parts * L * r * (K + N))
    assert call(_lora, "sg_lora_gemm_backward", LORA_BACK, dict(size, wsb=need)) == HIP
    assert call(_lora, "sg_lora_gemm_backward", LORA_BACK, dict(size, wsb=need - 1)) == SHAPE

"""Sizes of the 4-bit operators past what one launch has threads for (2^32 along x):
refused on the host, since of such a grid only the remainder would run, without an
error.  Fake addresses, never dereferenced; only where no GPU is visible."""
import pytest

import sparse_gemm_layers_amd as sg
from test_moe_abi import GEMM, HIP, MLP, PACK, SHAPE, call, no_gpu


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(N=(1 << 27) - 15, K=32, gc=32, ldx=32, ldy=1 << 28), SHAPE),      # 2^23 workgroups of 512
    (dict(N=(1 << 27) - 16, K=32, gc=32, ldx=32, ldy=1 << 28), HIP),        # one fewer: launched (there is no GPU)
    (dict(M=(1 << 30) + 1, N=8, K=32, gc=32, ldx=32), SHAPE), (dict(M=1 << 29, N=8, K=32, gc=32, ldx=32), HIP),
])
def test_linear(kw, code):
    assert call("sg_w4a16_gemm_groupwise_packed", GEMM, list(GEMM), kw) == code


@no_gpu
def test_pack_takes_any_number_of_chunks():
    assert call("sg_w4_pack", PACK, list(PACK), dict(L=1 << 34)) == HIP
    assert call("sg_w4_pack", PACK, list(PACK), dict(L=1 << 40)) == SHAPE


@no_gpu
def test_mlp():
    big = dict(T=1 << 25, k=32, E=8, D=32, F=32, ldx=32, ldy=32, gc=32, wsb=1 << 40)
    assert call("sg_w4a16_moe_mlp", MLP, list(MLP), big) == SHAPE
    assert call("sg_w4a16_moe_mlp", MLP, list(MLP), dict(big, k=31)) == HIP


def test_mlp_workspace():
    ws = sg.w4a16_moe_mlp_workspace
    assert ws(1 << 25, 32, 8, 32, 32) == -1 and ws(1 << 25, 31, 8, 32, 32) > 0
    assert ws(1 << 20, 8, 8, 128, 128 * 128) == -1 and ws(1 << 20, 8, 8, 128, 127 * 128) > 0

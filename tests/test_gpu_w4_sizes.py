"""4-bit linear layers at the sizes that its launch rule tells apart: every split
of rows and columns, and the tiles, with one, two, three and odd K blocks, against
the fp64 oracle on some rows and columns and against themselves elsewhere."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, down, say
from oracle import moe
from test_gpu_w4 import BF16, F32, up, weight

pytestmark = pytest.mark.gpu

# (M, N): one per split, the last three in tiles
SIZES = [(1, 40), (7, 40), (12, 40), (12, 4100), (130, 500), (17, 4136), (25, 2076), (30, 4100), (30, 9000), (130, 1000),
         (40, 4100), (40, 9000), (2108, 65), (41, 4143), (41, 8218), (50, 4138), (49, 8444), (60, 4100), (60, 9000),
         (190, 16400), (1100, 3300), (2049, 1700)]
COLS = [(32, 32), (160, 32), (128, 128), (320, 64), (384, 128), (1056, 32), (2240, 64), (2048, 128)]


@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("K,gc", COLS)
def test_every_split(M, N, K, gc):
    say(f"w4 split {M}x{N}x{K} gc{gc}")
    wq, s = weight(M + N + K, N, K, gc)
    x = torch.randn((M, K), generator=torch.Generator().manual_seed(M)).to(BF16)
    wp = sg.w4_pack(up(wq), up(s), gc)
    y = sg.w4a16_gemm_groupwise_packed(x.to(DEV), wp, N, gc, out_dtype=F32)
    g = np.random.default_rng(K)
    rows = np.unique(np.r_[0, M - 1, g.integers(0, M, 20)])
    cols = np.unique(np.r_[0, N - 1, g.integers(0, N, 300)])
    ref, size = moe.w4_linear(x[rows].double().numpy(), wq[cols], s[cols], gc)
    err = np.abs(down(y)[np.ix_(rows, cols)] - ref)
    tol = moe.sum_error(K, gc) * size + 2.0 ** -24 * np.abs(ref) + 1e-30
    assert np.isfinite(err).all() and (err <= tol).all(), f"off by {np.max(err / tol):.3g} of what is allowed"
    # rows do not depend on each other: a row alone differs by its sum's order at most
    for m in rows[:3]:
        one = down(sg.w4a16_gemm_groupwise_packed(x[m:m + 1].to(DEV), wp, N, gc, out_dtype=F32))[0]
        ref1, size1 = np.abs(down(y)[m] - one), np.abs(x[m].float().numpy()).sum() * 8 * np.abs(s).max()
        assert ref1.max() <= 2 * moe.sum_error(K, gc) * size1
    b = sg.w4a16_gemm_groupwise_packed(x.to(DEV), wp, N, gc, out_dtype=BF16)
    assert torch.equal(b, y.to(BF16))


@pytest.mark.parametrize("M,N", [(130, 500), (60, 9000), (1100, 3300)])
def test_bias_strides_and_repeats(M, N):
    K, gc = 288, 32
    wq, s = weight(9, N, K, gc)
    wp = sg.w4_pack(up(wq), up(s), gc)
    big = torch.full((M + 200, K + 40), float("nan"), dtype=BF16, device=DEV)
    big[:M, :K] = torch.randn((M, K), generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(2)).to(DEV)
    out = torch.full((M + 3, N + 5), 7.0, device=DEV)
    say(f"w4 strided {M}x{N}")
    y = sg.w4a16_gemm_groupwise_packed(big[:M, :K], wp, N, gc, bias=bias, y=out[:M, :N]).clone()
    assert (out[M:] == 7).all() and (out[:, N:] == 7).all()
    plain = sg.w4a16_gemm_groupwise_packed(big[:M, :K].contiguous(), wp, N, gc, out_dtype=F32)
    # one rounding of the sum with the bias, and one of this difference
    assert ((y - plain - bias).abs() <= 2.0 ** -23 * (plain.abs() + bias.abs() + y.abs())).all()
    for _ in range(3):
        assert torch.equal(y, sg.w4a16_gemm_groupwise_packed(big[:M, :K], wp, N, gc, out_dtype=F32, bias=bias))

"""4-bit linear layers on the GPU against the fp64 oracle: the error allowed is
oracle.moe.sum_error (a step per addition of the kernel's fp32 sum) on the sum of
the terms' magnitudes, then half a step of the output type."""
import numpy as np
import pytest
import torch

import oracle
import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, down, say
from oracle import moe

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def weight(seed, n, k, gc, lead=()):
    g = np.random.default_rng(seed)
    wq = g.integers(0, 256, (*lead, n, k // 2), dtype=np.uint8)      # every code, -8 among them
    s = np.exp2(g.uniform(-9, -5, (*lead, n, k // gc))).astype(np.float32)
    return wq, s


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check(y, ref, size, k, gc, dtype):
    tol = moe.sum_error(k, gc) * size + torch.finfo(dtype).eps / 2 * np.abs(ref) + 1e-30
    err = np.abs(down(y) - ref)
    assert np.isfinite(err).all() and (err <= tol).all(), f"off by {np.max(err / tol):.3g} of what is allowed"
    say(f"  max |err| / allowed = {np.max(err / tol):.3g}")


SHAPES = [
    # M, N, K, gc
    (1, 1, 32, 32), (1, 16, 128, 128), (1, 500, 576, 64), (1, 4096, 1024, 128), (2, 100, 96, 32), (15, 130, 640, 128),
    (16, 64, 2048, 64), (17, 48, 1120, 32), (31, 257, 384, 128), (33, 1000, 512, 64), (37, 4096, 896, 128),
    (48, 33, 288, 32), (64, 600, 256, 64), (65, 600, 256, 64), (100, 90, 160, 32), (200, 300, 1152, 128),
    (257, 130, 320, 64), (300, 700, 1056, 32), (513, 1000, 640, 128), (1000, 129, 384, 128), (2048, 260, 192, 64),
]


@pytest.mark.parametrize("M,N,K,gc", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_linear(M, N, K, gc, dtype):
    say(f"w4 linear {M}x{N}x{K} gc{gc} {dtype}")
    wq, s = weight(M + N + K, N, K, gc)
    x = torch.randn((M, K), generator=torch.Generator().manual_seed(M)).to(BF16)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(N)) if (M + N) % 2 else None
    wp = sg.w4_pack(up(wq), up(s), gc)
    y = sg.w4a16_gemm_groupwise_packed(x.to(DEV), wp, N, gc, out_dtype=dtype,
                                       bias=None if bias is None else bias.to(DEV))
    ref, size = moe.w4_linear(x.double().numpy(), wq, s, gc, None if bias is None else bias.double().numpy())
    check(y, ref, size, K, gc, dtype)


@pytest.mark.parametrize("M,N,K,gc", [(1, 40, 256, 64), (33, 40, 288, 32), (64, 100, 384, 128), (300, 150, 448, 64)])
def test_linear_is_exact_where_fp32_is(M, N, K, gc):
    """Whole x and power-of-two scales: every sum fits 24 bits, so every bit has to be right."""
    say(f"w4 exact {M}x{N}x{K}")
    g = np.random.default_rng(7)
    wq, _ = weight(1, N, K, gc)
    s = np.exp2(g.integers(-2, 2, (N, K // gc))).astype(np.float32)
    x = g.integers(-4, 5, (M, K)).astype(np.float32)
    wp = sg.w4_pack(up(wq), up(s), gc)
    y = sg.w4a16_gemm_groupwise_packed(up(x).to(BF16), wp, N, gc, out_dtype=F32)
    ref, _ = moe.w4_linear(x.astype(np.float64), wq, s, gc)
    assert np.array_equal(down(y).astype(np.float64), ref)


@pytest.mark.parametrize("M", [3, 300])
def test_rows_and_columns_outside_are_not_read(M):
    """X in a wider buffer of NaN (columns past K, rows past M), y in a wider one that keeps its rest."""
    N, K, gc = 90, 160, 32
    wq, s = weight(2, N, K, gc)
    big = torch.full((M + 300, K + 64), float("nan"), dtype=BF16)
    big[:M, :K] = torch.randn((M, K), generator=torch.Generator().manual_seed(1)).to(BF16)
    wp = sg.w4_pack(up(wq), up(s), gc)
    y = torch.full((M + 5, N + 7), 3.0, device=DEV)
    sg.w4a16_gemm_groupwise_packed(big.to(DEV)[:M, :K], wp, N, gc, y=y[:M, :N])
    say(f"w4 strided M{M}")
    ref, size = moe.w4_linear(big[:M, :K].double().numpy(), wq, s, gc)
    check(y[:M, :N], ref, size, K, gc, F32)
    assert (y[M:] == 3).all() and (y[:, N:] == 3).all()


@pytest.mark.parametrize("M", [2, 40, 300])
def test_non_finite_rows_stay_in_their_rows(M):
    N, K, gc = 64, 256, 128
    wq, s = weight(3, N, K, gc)
    x = torch.randn((M, K), generator=torch.Generator().manual_seed(1)).to(BF16)
    clean = x.clone()
    x[1, 7] = float("nan")
    wp = sg.w4_pack(up(wq), up(s), gc)
    a = sg.w4a16_gemm_groupwise_packed(x.to(DEV), wp, N, gc)
    b = sg.w4a16_gemm_groupwise_packed(clean.to(DEV), wp, N, gc)
    assert torch.isnan(a[1]).all()
    keep = torch.arange(M) != 1
    assert torch.equal(a[keep.to(DEV)], b[keep.to(DEV)])


def test_pack_of_many_takes_strides():
    L, N, K, gc = 3, 50, 192, 64
    wq, s = weight(4, N, K, gc, (L,))
    big = torch.zeros((L, N + 4, K // 2 + 8), dtype=torch.uint8, device=DEV)
    big[:, :N, :K // 2] = up(wq)
    sm = up(s.transpose(0, 2, 1)).transpose(1, 2)       # contiguous along rows
    a = sg.w4_pack(big[:, :N, :K // 2], sm, gc)
    assert a.shape == (L, sg.w4_packed_bytes(N, K, gc))
    for i in range(L):
        assert torch.equal(a[i], sg.w4_pack(up(wq[i]), up(s[i]), gc))


def test_the_quantiser_feeds_the_pack():
    """int4_quant_groupwise -> w4_pack -> GEMM, against the oracle's quantiser."""
    g = torch.Generator().manual_seed(5)
    w, x = 0.02 * torch.randn((96, 384), generator=g), torch.randn((5, 384), generator=g).to(BF16)
    wq, s = sg.int4_quant_groupwise(w.to(DEV), gc=128)
    y = sg.w4a16_gemm_groupwise_packed(x.to(DEV), sg.w4_pack(wq, s, 128), 96, 128, out_dtype=F32)
    oq, os_ = oracle.int4_quant_groupwise(w.numpy(), 128)
    ref, size = moe.w4_linear(x.double().numpy(), oq, os_, 128)
    check(y, ref, size, 384, 128, F32)


def test_refusals():
    wp = sg.w4_pack(torch.zeros((16, 64), dtype=torch.uint8, device=DEV), torch.ones((16, 1), device=DEV))
    x = torch.zeros((2, 128), dtype=BF16, device=DEV)
    for bad in (lambda: sg.w4_pack(torch.zeros((16, 64), dtype=torch.int8, device=DEV), torch.ones((16, 1), device=DEV)),
                lambda: sg.w4_pack(torch.zeros((16, 64), dtype=torch.uint8, device=DEV), torch.ones((16, 2), device=DEV)),
                lambda: sg.w4_pack(torch.zeros((16, 50), dtype=torch.uint8, device=DEV), torch.ones((16, 1), device=DEV)),
                lambda: sg.w4a16_gemm_groupwise_packed(x.float(), wp, 16),
                lambda: sg.w4a16_gemm_groupwise_packed(x, wp, 17), lambda: sg.w4a16_gemm_groupwise_packed(x, wp, 16, gc=64),
                lambda: sg.w4a16_gemm_groupwise_packed(x, wp, 16, gc=100),
                lambda: sg.w4a16_gemm_groupwise_packed(x[:, ::2], wp, 16),
                lambda: sg.w4a16_gemm_groupwise_packed(x[:0], wp, 16),
                lambda: sg.w4a16_gemm_groupwise_packed(x, wp, 16, out_dtype=torch.float16),
                lambda: sg.w4a16_gemm_groupwise_packed(x, wp, 16, bias=torch.zeros(15, device=DEV)),
                lambda: sg.w4a16_gemm_groupwise_packed(x, wp, 16, y=torch.zeros((2, 15), device=DEV))):
        with pytest.raises(sg.SgError):
            bad()

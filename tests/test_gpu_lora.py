"""The low-rank adapters on the GPU against the fp64 oracle.

Error allowed, from the arithmetic: a fp32 sum of n terms is off by at most (n + 20)
2^-24 times the sum of their magnitudes (parts of it are added too); the inner
product's error goes through the outer one; splitting it into two bf16 parts leaves
out 2^-16 of it at most, three 2^-24; half a step of the result's type comes last."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, down, say
from oracle import adapt

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TINY = 2.0 ** -120


def bf(seed, *shape, std=1.0):
    return (std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(BF16)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def gpu(t):
    return None if t is None else t.to(DEV)


def within(what, got, ref, tol):
    err = np.abs(down(got).astype(np.float64) - ref)
    assert np.isfinite(err).all(), f"{what}: not finite"
    assert (err <= tol).all(), f"{what}: off by {np.max(err / tol):.3g} of what is allowed"
    say(f"  {what}: max |err| / allowed = {np.max(err / tol):.3g}")


def allowed(dtype, wide, ref, inner, outer, n_in, n_out):
    """wide: whether the [T, r] values enter in three parts."""
    e = (n_in + 20) * 2.0 ** -24 * inner + ((n_out + 20) * 2.0 ** -24 + 2.0 ** -(24 if wide else 16)) * outer
    return e + torch.finfo(dtype).eps / 2 * (np.abs(ref) + e) + TINY


def make(T, K, N, r, L, order, seed=0):
    gen = torch.Generator().manual_seed(seed + 99)
    ids = torch.randint(-1, L + 1, (T,), generator=gen, dtype=torch.int32)      # -1 and L: none
    if order == "runs":
        ids = ids.sort().values
    elif order == "one":
        ids = torch.full((T,), L - 1, dtype=torch.int32)
    elif order == "none":
        ids = torch.full((T,), -1, dtype=torch.int32)
    return (bf(seed + 1, T, K), ids, bf(seed + 2, L, r, K, std=K ** -0.5), bf(seed + 3, L, N, r, std=0.1),
            torch.rand(L, generator=gen) + 0.5)


SHAPES = [
    # T, K, N, r, L, order
    (1, 8, 8, 8, 1, "one"), (1, 4096, 520, 16, 3, "one"), (2, 72, 264, 8, 2, "mixed"), (15, 200, 64, 24, 20, "mixed"),
    (16, 264, 136, 16, 4, "runs"), (17, 136, 1032, 32, 40, "mixed"), (37, 1000, 520, 64, 16, "mixed"),
    (40, 72, 72, 72, 3, "none"), (64, 520, 264, 40, 5, "runs"), (100, 136, 264, 128, 2, "mixed"),
    (129, 64, 256, 256, 2, "runs"), (300, 1032, 72, 16, 7, "mixed"), (700, 264, 328, 8, 3, "runs"),
]


@pytest.mark.parametrize("T,K,N,r,L,order", SHAPES)
@pytest.mark.parametrize("dtype,base", [(F32, None), (BF16, BF16), (BF16, None), (F32, BF16), (BF16, F32)])
def test_forward(T, K, N, r, L, order, dtype, base):
    say(f"lora {T}x{K}x{N} r {r} L {L} {order} {dtype} base {base}")
    x, ids, a, b, scale = make(T, K, N, r, L, order)
    c = None if base is None else torch.randn((T, N), generator=torch.Generator().manual_seed(5)).to(base)
    if r == 8:
        scale = None
    y = sg.lora_gemm(gpu(x), gpu(ids), gpu(a), gpu(b), gpu(scale), gpu(c), out_dtype=dtype)
    ref, inner, outer = adapt.lora(f64(x), ids.numpy(), f64(a), f64(b), f64(scale), f64(c))
    within("y", y, ref, allowed(dtype, dtype == F32, ref, inner, outer, K, r))
    if base == dtype:
        inplace = gpu(c).clone()
        out = sg.lora_gemm(gpu(x), gpu(ids), gpu(a), gpu(b), gpu(scale), inplace, y=inplace)
        assert out is inplace and torch.equal(inplace, y)
        none = (ids < 0) | (ids >= L)
        assert torch.equal(inplace[none.to(DEV)].cpu(), c[none])      # as they were


@pytest.mark.parametrize("T,K,N,r,L,order", SHAPES)
@pytest.mark.parametrize("dtype,base", [(F32, True), (BF16, False)])
def test_backward(T, K, N, r, L, order, dtype, base):
    say(f"lora backward {T}x{K}x{N} r {r} L {L} {order} {dtype}")
    x, ids, a, b, scale = make(T, K, N, r, L, order, seed=20)
    dy, c = bf(26, T, N), bf(27, T, K) if base else None
    if r == 8:
        scale = None
    got = sg.lora_gemm_backward(gpu(dy), gpu(x), gpu(ids), gpu(a), gpu(b), gpu(scale), gpu(c), grad_dtype=dtype)
    refs, inner, outer = adapt.lora_grads(f64(dy), f64(x), ids.numpy(), f64(a), f64(b), f64(scale), f64(c))
    for i, (what, n_in, n_out) in enumerate((("dx", N, r), ("da", N, T), ("db", K, T))):
        t = BF16 if i == 0 else dtype
        assert got[i].dtype == t
        within(what, got[i], refs[i], allowed(t, i > 0 and dtype == F32, refs[i], inner[i], outer[i], n_in, n_out))
    for e in range(L):
        if not (ids == e).any():
            assert not got[1][e].any() and not got[2][e].any()
    if base:
        inplace = gpu(c).clone()
        sg.lora_gemm_backward(gpu(dy), gpu(x), gpu(ids), gpu(a), gpu(b), gpu(scale), inplace, dx=inplace, need_dab=False)
        assert torch.equal(inplace, got[0])


def test_one_adapter_without_ids():
    x, _, a, b, scale = make(50, 72, 136, 16, 2, "one")
    zeros = torch.zeros(50, dtype=torch.int32, device=DEV)
    args = gpu(a), gpu(b), gpu(scale)
    assert torch.equal(sg.lora_gemm(gpu(x), None, *args), sg.lora_gemm(gpu(x), zeros, *args))
    dy = gpu(bf(9, 50, 136))
    for p, q in zip(sg.lora_gemm_backward(dy, gpu(x), None, *args), sg.lora_gemm_backward(dy, gpu(x), zeros, *args)):
        assert torch.equal(p, q)


def test_gradient_against_differences():
    """y is linear in x, in a and in b: a difference of two calls over any step is the
    derivative, up to the rounding of both (fp32 out).  Steps in directions of small
    whole numbers, so that the shifted bf16 operands are exact."""
    T, K, N, r, L = 45, 72, 136, 16, 3
    gen = torch.Generator().manual_seed(3)

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=gen).to(BF16)

    x, a, b, w = whole(T, K), whole(L, r, K), whole(L, N, r), whole(T, N)
    ids = torch.randint(-1, L, (T,), generator=gen, dtype=torch.int32)
    grads = sg.lora_gemm_backward(gpu(w), gpu(x), gpu(ids), gpu(a), gpu(b), grad_dtype=F32)
    for i, at in enumerate((x, a, b)):
        d = whole(*at.shape)
        args = [x, a, b]
        y = []
        for s in (1, -1):
            args[i] = at + s * d
            y.append(f64(sg.lora_gemm(gpu(args[0]), gpu(ids), gpu(args[1]), gpu(args[2]), out_dtype=F32)))
        diff = (f64(w) * (y[0] - y[1])).sum() / 2
        # whole numbers below 2^24 everywhere: exact, but for dx's rounding to bf16
        want = (f64(grads[i]) * f64(d)).sum()
        slack = 2.0 ** -8 * (np.abs(f64(grads[i])) * np.abs(f64(d))).sum() if i == 0 else 0.0
        say(f"  {'x a b'.split()[i]}: {diff} {want}")
        assert abs(diff - want) <= slack

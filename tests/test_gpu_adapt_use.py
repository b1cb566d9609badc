"""The gated projections and the low-rank adapters as a program uses them: strided
and very long operands, masked tokens that hold NaN, other streams and graphs, results
of the caller's, and all of them together."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, say
from oracle import adapt
from sparse_gemm_layers_amd import _gated
from test_gpu_gated import BACK, half, product_errors, sum_tol
from test_gpu_gated import make as make_gated
from test_gpu_lora import allowed, bf, f64, gpu, within
from test_gpu_lora import make as make_lora

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int16 if a.dtype == BF16 else torch.int32),
                       b.contiguous().view(torch.int16 if b.dtype == BF16 else torch.int32))


def wide(t, pad, seed=0):
    """t as a view into rows that are pad longer and full of NaN behind it."""
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


# ------------------------------------------------------------------ adapters

LONG = [
    # T, K, N, r, L, order: parts of the tokens that are joined, 64-rank chunks, several 1024-token lists
    (1100, 72, 136, 16, 1, "one"), (2300, 264, 520, 40, 2, "runs"), (3000, 72, 72, 96, 1, "mixed"),
    (1500, 520, 264, 200, 3, "runs"), (4097, 40, 24, 8, 2, "mixed"),
]


@pytest.mark.parametrize("T,K,N,r,L,order", LONG)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lora_long(T, K, N, r, L, order, dtype):
    say(f"lora long {T}x{K}x{N} r {r} L {L} {order} {dtype}")
    x, ids, a, b, scale = make_lora(T, K, N, r, L, order, seed=40)
    dy, base = bf(46, T, N), bf(47, T, K)
    args = gpu(x), gpu(ids), gpu(a), gpu(b), gpu(scale)
    y = sg.lora_gemm(*args, out_dtype=dtype)
    ref, inner, outer = adapt.lora(f64(x), ids.numpy(), f64(a), f64(b), f64(scale))
    within("y", y, ref, allowed(dtype, dtype == F32, ref, inner, outer, K, r))
    got = sg.lora_gemm_backward(gpu(dy), *args, gpu(base), grad_dtype=dtype)
    refs, inner, outer = adapt.lora_grads(f64(dy), f64(x), ids.numpy(), f64(a), f64(b), f64(scale), f64(base))
    for i, (what, n_in, n_out) in enumerate((("dx", N, r), ("da", N, T), ("db", K, T))):
        t = BF16 if i == 0 else dtype
        within(what, got[i], refs[i], allowed(t, i > 0 and dtype == F32, refs[i], inner[i], outer[i], n_in, n_out))


@pytest.mark.parametrize("T,K,N,r,L", [(1, 8192, 520, 64, 2), (7, 14336, 264, 32, 9), (33, 4096, 1032, 64, 12),
                                       (64, 1024, 520, 128, 5)])
def test_lora_few_tokens_long_sums(T, K, N, r, L):
    say(f"lora {T}x{K}x{N} r {r} L {L}")
    x, ids, a, b, scale = make_lora(T, K, N, r, L, "mixed", seed=60)
    base = bf(66, T, N)
    y = sg.lora_gemm(gpu(x), gpu(ids), gpu(a), gpu(b), gpu(scale), gpu(base))
    ref, inner, outer = adapt.lora(f64(x), ids.numpy(), f64(a), f64(b), f64(scale), f64(base))
    within("y", y, ref, allowed(BF16, False, ref, inner, outer, K, r))


@pytest.mark.parametrize("T", [5, 90, 700])
def test_lora_masked_tokens_and_other_adapters_do_not_reach(T):
    """NaN and infinities in the rows of tokens without an adapter, and in adapters that
    no token has, change nothing; a NaN in one token stays with it and its adapter."""
    K, N, r, L = 136, 264, 24, 4
    x, ids, a, b, scale = make_lora(T, K, N, r, L, "mixed", seed=70)
    ids[ids == 2] = 1                                  # adapter 2 is nobody's
    dy = bf(76, T, N)
    args = [gpu(v) for v in (x, ids, a, b, scale)]
    dyg = gpu(dy)
    y, grads = sg.lora_gemm(*args), sg.lora_gemm_backward(dyg, *args, grad_dtype=F32)
    none = ((ids < 0) | (ids >= L)).to(DEV)
    dirty = [v.clone() for v in args]
    dirty_dy = dyg.clone()
    dirty[0][none] = float("nan")
    dirty_dy[none] = float("inf")
    dirty[2][2], dirty[3][2], dirty[4][2] = float("nan"), float("inf"), float("nan")
    y2, grads2 = sg.lora_gemm(*dirty), sg.lora_gemm_backward(dirty_dy, *dirty, grad_dtype=F32)
    assert same(y, y2) and all(same(p, q) for p, q in zip(grads, grads2))
    assert not grads2[1][2].any() and not grads2[2][2].any()
    mine = int((~none).nonzero()[0])
    e = int(ids[mine])
    one = [v.clone() for v in args]
    one[0][mine, 3] = float("nan")
    y3, (dx3, da3, db3) = sg.lora_gemm(*one), sg.lora_gemm_backward(dyg, *one, grad_dtype=F32)
    keep = torch.arange(T, device=DEV) != mine
    assert torch.isnan(y3[mine]).all() and same(y3[keep], y[keep])
    assert same(dx3, grads[0])                          # dx does not depend on x
    others = [i for i in range(L) if i != e]
    assert same(da3[others], grads[1][others]) and same(db3[others], grads[2][others])
    assert torch.isnan(da3[e][:, 3]).all() and not torch.isnan(da3[e][:, :3]).any() and torch.isnan(db3[e]).all()


def test_lora_infinite_inner_product():
    """An infinite x . A gives infinite results, not the NaN of taking a part from it."""
    x, a = torch.full((3, 8), 2.0 ** 120, dtype=BF16), torch.full((1, 8, 8), 2.0 ** 10, dtype=BF16)
    b = torch.full((1, 16, 8), 0.5, dtype=BF16)
    for T in (3, 70):
        y = sg.lora_gemm(gpu(x[:1].repeat(T, 1)), None, gpu(a), gpu(b), out_dtype=F32)
        assert torch.isposinf(y).all()


@pytest.mark.parametrize("T", [3, 40, 600])
def test_lora_strides_and_given_results(T):
    K, N, r, L = 72, 136, 40, 3
    x, ids, a, b, scale = make_lora(T, K, N, r, L, "mixed", seed=80)
    dy, base, dbase = bf(86, T, N), bf(87, T, N), bf(88, T, K)
    args = [gpu(v) for v in (ids, a, b, scale)]
    y = sg.lora_gemm(gpu(x), *args, gpu(base))
    grads = sg.lora_gemm_backward(gpu(dy), gpu(x), *args, gpu(dbase))
    xs, dys, bs, dbs = wide(gpu(x), 24), wide(gpu(dy), 8), wide(gpu(base), 40), wide(gpu(dbase), 16)
    out, dx = wide(torch.zeros_like(y), 56), wide(torch.zeros_like(grads[0]), 32)
    da, db = torch.empty_like(grads[1]), torch.empty_like(grads[2])
    need = sg.lora_gemm_backward_workspace(T, K, N, r, L)
    ws = torch.empty(need + 512, dtype=torch.uint8, device=DEV)
    assert sg.lora_gemm(xs, *args, bs, y=out, workspace=ws) is out and same(out, y)
    got = sg.lora_gemm_backward(dys, xs, *args, dbs, dx=dx, da=da, db=db, workspace=ws)
    assert all(same(p, q) for p, q in zip(got, grads)) and got[0] is dx and got[1] is da and got[2] is db
    for t in (out, dx):                                 # nothing behind the rows
        whole = t.as_strided((T, t.stride(0)), (t.stride(0), 1)) if T > 1 else t
        assert torch.isnan(whole[:, t.shape[1]:]).all()


def test_lora_offsets_past_32_bits():
    """Rows further apart than 2^31 bytes in all: 140000 rows of 16 KB."""
    T, K, N, r, L = 140000, 64, 64, 8, 3
    gen = torch.Generator(device=DEV).manual_seed(1)
    big = torch.zeros((T, 8192), dtype=BF16, device=DEV)
    x = big[:, :K]
    x.normal_(generator=gen)
    y, dx = big[:, 1024:1024 + N], big[:, 2048:2048 + K]
    dy = big[:, 4096:4096 + N]
    dy.normal_(generator=gen)
    ids = torch.randint(-1, L, (T,), generator=gen, device=DEV, dtype=torch.int32)
    a, b = (0.1 * torch.randn((L, r, K), generator=gen, device=DEV)).to(BF16), torch.randn((L, N, r), generator=gen, device=DEV).to(BF16)
    sg.lora_gemm(x, ids, a, b, y=y)
    _, da, db = sg.lora_gemm_backward(dy, x, ids, a, b, dx=dx, grad_dtype=F32)
    pick = torch.cat((torch.arange(50, device=DEV), torch.arange(T - 200, T, device=DEV)))
    ref, inner, outer = adapt.lora(f64(x[pick]), ids[pick].cpu().numpy(), f64(a), f64(b))
    within("y", y[pick], ref, allowed(BF16, False, ref, inner, outer, K, r))
    refs, ri, ro = adapt.lora_grads(f64(dy[pick]), f64(x[pick]), ids[pick].cpu().numpy(), f64(a), f64(b))
    within("dx", dx[pick], refs[0], allowed(BF16, False, refs[0], ri[0], ro[0], N, r))
    for e in range(L):
        m = ids == e
        xe, de, ae, be = (v.double() for v in (x[m], dy[m], a[e], b[e]))
        v, u = de @ be, xe @ ae.t()
        va, ua = de.abs() @ be.abs(), xe.abs() @ ae.abs().t()
        for what, got, ref, inn, out, n_in in (
                ("da", da[e], v.t() @ xe, va.t() @ xe.abs(), v.abs().t() @ xe.abs(), N),
                ("db", db[e], de.t() @ u, de.abs().t() @ ua, de.abs().t() @ u.abs(), K)):
            within(what, got, f64(ref), allowed(F32, True, f64(ref), f64(inn), f64(out), n_in, int(m.sum())))


# ------------------------------------------------------------------ gated projections

@pytest.mark.parametrize("T,F,D", [(1, 24, 40), (16, 264, 136), (30, 72, 264), (130, 200, 72), (300, 1032, 136)])
def test_gated_strides_and_given_results(T, F, D):
    x, gate, up, ga, ua = (gpu(v) for v in make_gated(T, F, D, True, seed=90))
    dh = gpu(bf(96, T, F))
    h, g, u = sg.gated_gemm(x, gate, up, gate_add=ga, up_add=ua, keep=True)
    grads = sg.gated_gemm_backward(dh, x, gate, up, g=g, u=u)
    again = sg.gated_gemm_backward(dh, x, gate, up, gate_add=ga, up_add=ua)
    xs, gs, us, dhs = wide(x, 8), wide(gate, 24), wide(up, 40), wide(dh, 16)      # gate's and up's rows differ
    gas, uas = wide(ga, 8), wide(ua, 8)
    hs, kg, ku = wide(torch.zeros_like(h), 8), wide(torch.zeros_like(g), 16), wide(torch.zeros_like(u), 16)
    out = sg.gated_gemm(xs, gs, us, gate_add=gas, up_add=uas, h=hs, g=kg, u=ku)
    assert out[0] is hs and all(same(p, q) for p, q in zip(out, (h, g, u)))
    dx, dg, du = wide(torch.zeros_like(x), 8), wide(torch.zeros_like(g), 8), wide(torch.zeros_like(g), 8)
    dgate, dup = wide(torch.zeros_like(gate), 8), wide(torch.zeros_like(up), 8)
    need = sg.gated_gemm_backward_workspace(T, F, D)
    ws = torch.empty(need + 256, dtype=torch.uint8, device=DEV)
    got = sg.gated_gemm_backward(dhs, xs, gs, us, g=kg, u=ku, dx=dx, dgate=dgate, dup=dup, dg=dg, du=du, workspace=ws)
    assert all(same(p, q) for p, q in zip(got, grads))
    assert all(same(p, q) for p, q in zip(sg.gated_gemm_backward(dhs, xs, gs, us, gate_add=gas, up_add=uas), again))
    got = sg.gated_gemm_backward(dh, x, gate, up, g=g, u=u, dg=g, du=u)           # in their place
    assert got[3] is g and all(same(p, q) for p, q in zip(got, grads))
    for t in (hs, kg, ku, dx, dg, du, dgate, dup):
        whole = t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1)) if t.shape[0] > 1 else t
        assert torch.isnan(whole[:, t.shape[1]:]).all()


@pytest.mark.parametrize("T,F,D", [(37, 72, 264), (333, 264, 136)])
def test_gated_parts_of_the_backward_pass(T, F, D):
    x, gate, up, _, _ = (gpu(v) for v in make_gated(T, F, D, False, seed=100))
    dh = gpu(bf(106, T, F))
    h, g, u = sg.gated_gemm(x, gate, up, keep=True)
    dx, dgate, dup, dg, du = sg.gated_gemm_backward(dh, x, gate, up, g=g, u=u)
    only = sg.gated_gemm_backward(dh, x, gate, up, g=g, u=u, need_dx=False)
    assert only[0] is None and all(same(p, q) for p, q in zip(only[1:], (dgate, dup, dg, du)))
    only = sg.gated_gemm_backward(dh, x, gate, up, g=g, u=u, need_dw=False)
    assert only[1] is None and only[2] is None and all(same(p, q) for p, q in zip(only[3:], (dg, du)))
    # fewer workgroups: dx's sum may be cut elsewhere
    ref, size = (m[0] for m in adapt.gated_grads(*map(f64, (dg, du, x, gate, up))))
    e = sum_tol(2 * F + 64, size)
    within("dx alone", only[0], ref, e + half(BF16, np.abs(ref) + e))
    only = sg.gated_gemm_backward(dh, x, gate, up, g=g, u=u, need_dx=False, need_dw=False)
    assert only[:3] == (None, None, None) and same(only[3], dg) and same(only[4], du)


@pytest.mark.parametrize("T", [3, 40, 300])
def test_gated_nan_stays_in_its_row(T):
    F, D = 264, 136
    x, gate, up, _, _ = (gpu(v) for v in make_gated(T, F, D, False, seed=110))
    h = sg.gated_gemm(x, gate, up)
    x2, gate2 = x.clone(), gate.clone()
    x2[T // 2, 5] = float("nan")
    gate2[17, 3] = float("inf")
    keep = torch.arange(T, device=DEV) != T // 2
    h2 = sg.gated_gemm(x2, gate, up)
    assert torch.isnan(h2[T // 2]).all() and same(h2[keep], h[keep])
    h3 = sg.gated_gemm(x, gate2, up)
    cols = torch.arange(F, device=DEV) != 17
    assert same(h3[:, cols], h[:, cols]) and not torch.isfinite(h3[:, 17]).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gated_far_values(act):
    """Sums whose exponentials and cubes overflow: the limits, not NaN."""
    for v, value, slope in ((2.0 ** 40, 2.0 ** 40, 1.0), (-(2.0 ** 40), 0.0, 0.0), (300.0, 300.0, 1.0), (-300.0, 0.0, 0.0)):
        x = torch.zeros((2, 8), dtype=BF16, device=DEV)
        x[:, 0] = v
        gate, up = torch.zeros((8, 8), dtype=BF16, device=DEV), torch.zeros((8, 8), dtype=BF16, device=DEV)
        gate[:, 0] = 1.0
        one = torch.ones((2, 8), dtype=BF16, device=DEV)
        h = sg.gated_gemm(x, gate, up, act=act, up_add=one, out_dtype=F32)
        want = torch.full_like(h, torch.tensor(v, dtype=BF16).item() if value else 0.0)
        assert torch.equal(h, want), (act, v, h[0, 0].item())
        dg, du = sg.gated_gemm_backward(one, x, gate, up, act=act, up_add=one, need_dx=False, need_dw=False)[3:]
        assert torch.equal(dg.float(), torch.full_like(h, slope)) and torch.equal(du.float(), want)


def test_gated_offsets_past_32_bits():
    """Rows of x, h and the gradients further apart than 2^31 bytes in all."""
    T, F, D = 140000, 64, 72
    gen = torch.Generator(device=DEV).manual_seed(2)
    big = torch.zeros((T, 8192), dtype=BF16, device=DEV)
    x, h, dh, dx = big[:, :D], big[:, 512:512 + F], big[:, 1024:1024 + F], big[:, 2048:2048 + D]
    g, u = big[:, 4096:4096 + F], big[:, 5120:5120 + F]
    x.normal_(generator=gen)
    dh.normal_(generator=gen)
    gate, up = ((0.1 * torch.randn((F, D), generator=gen, device=DEV)).to(BF16) for _ in range(2))
    sg.gated_gemm(x, gate, up, h=h, g=g, u=u)
    _, dgate, dup, dg, du = sg.gated_gemm_backward(dh, x, gate, up, g=g, u=u, dx=dx)
    pick = torch.cat((torch.arange(50, device=DEV), torch.arange(T - 300, T, device=DEV)))
    rh, rg, ru, sg_, su = adapt.gated(*map(f64, (x[pick], gate, up)))
    eg, eu, ea, _ = product_errors(D, rg, ru, sg_, su)
    eh = ea * (np.abs(ru) + eu) + np.abs(adapt.act("silu", rg)[0]) * eu + 2.0 ** -23 * np.abs(rh)
    within("h", h[pick], rh, eh + half(BF16, np.abs(rh) + eh))
    refs, sizes = adapt.gated_grads(*map(f64, (dg[pick], du[pick], x[pick], gate, up)))
    e = sum_tol(2 * F, sizes[0])
    within("dx", dx[pick], refs[0], e + half(BF16, np.abs(refs[0]) + e))
    for what, got, d in (("dgate", dgate, dg), ("dup", dup, du)):
        ref, size = f64(d.double().t() @ x.double()), f64(d.double().abs().t() @ x.double().abs())
        e = sum_tol(T, size)
        within(what, got, ref, e + half(BF16, np.abs(ref) + e))


def test_shapes_of_the_backward_pass_reach_every_way():
    """Both tile sizes, with and without parts, among the shapes of test_gpu_gated."""
    parts = [sg.gated_gemm_backward_workspace(T, F, D) for T, F, D, _, _ in BACK]
    assert any(p == 0 for p in parts) and any(p > 0 for p in parts)


# ------------------------------------------------------------------ refusals

@pytest.mark.parametrize("call", [
    lambda t: sg.gated_gemm(t(4, 12), t(8, 12), t(8, 12)),                                   # D no multiple of 8
    lambda t: sg.gated_gemm(t(4, 16), t(12, 16), t(12, 16)),                                 # F no multiple of 8
    lambda t: sg.gated_gemm(t(4, 16), t(8, 24), t(8, 24)),
    lambda t: sg.gated_gemm(t(4, 16), t(8, 16), t(16, 16)),
    lambda t: sg.gated_gemm(t(4, 16), t(8, 16), t(8, 16).float()),
    lambda t: sg.gated_gemm(t(4, 16).half(), t(8, 16).half(), t(8, 16).half()),
    lambda t: sg.gated_gemm(t(0, 16), t(8, 16), t(8, 16)),
    lambda t: sg.gated_gemm(t(4, 16), t(8, 16), t(8, 16), act="tanh"),
    lambda t: sg.gated_gemm(t(4, 16), t(8, 16), t(8, 16), g=t(4, 8)),
    lambda t: sg.gated_gemm(t(4, 16), t(8, 16), t(8, 16), out_dtype=torch.float16),
    lambda t: sg.gated_gemm(t(4, 17)[:, 1:], t(8, 16), t(8, 16)),                            # misaligned
    lambda t: sg.gated_gemm(t(4, 20)[:, :16], t(8, 16), t(8, 16)),                           # rows not 16-byte aligned
    lambda t: sg.gated_gemm(t(16, 4).t(), t(8, 16), t(8, 16)),                               # column stride
    lambda t: sg.gated_gemm(t(4, 16), t(8, 16), t(8, 16), gate_add=t(4, 16)[:, :8], up_add=t(4, 8)),
    lambda t: sg.gated_gemm_backward(t(4, 8), t(4, 16), t(8, 16), t(8, 16), g=t(4, 8)),
    lambda t: sg.gated_gemm_backward(t(4, 16), t(4, 16), t(8, 16), t(8, 16)),
    lambda t: sg.gated_gemm_backward(t(64, 2048), t(64, 16), t(2048, 16), t(2048, 16), need_dw=False,
                                     workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
    lambda t: sg.lora_gemm(t(4, 16), None, t(2, 8, 24), t(2, 16, 8)),
    lambda t: sg.lora_gemm(t(4, 16), None, t(2, 8, 16), t(3, 16, 8)),
    lambda t: sg.lora_gemm(t(4, 16), None, t(2, 12, 16), t(2, 16, 12)),
    lambda t: sg.lora_gemm(t(4, 16), None, t(1, 264, 16), t(1, 16, 264)),
    lambda t: sg.lora_gemm(t(4, 16), None, t(2, 8, 32)[:, :, :16], t(2, 16, 8)),              # not contiguous
    lambda t: sg.lora_gemm(t(4, 16), torch.zeros(4, dtype=torch.int64, device=DEV), t(2, 8, 16), t(2, 16, 8)),
    lambda t: sg.lora_gemm(t(4, 16), torch.zeros(5, dtype=torch.int32, device=DEV), t(2, 8, 16), t(2, 16, 8)),
    lambda t: sg.lora_gemm(t(4, 16), None, t(2, 8, 16), t(2, 16, 8), scale=torch.ones(3, device=DEV)),
    lambda t: sg.lora_gemm(t(4, 16), None, t(2, 8, 16), t(2, 16, 8), base=t(4, 8)),
    lambda t: sg.lora_gemm(t(4, 16), None, t(2, 8, 16), t(2, 16, 8), y=t(4, 16).half()),
    lambda t: sg.lora_gemm(t(0, 16), None, t(2, 8, 16), t(2, 16, 8)),
    lambda t: sg.lora_gemm(t(100, 16), None, t(2, 8, 16), t(2, 16, 8), workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
    lambda t: sg.lora_gemm_backward(t(4, 8), t(4, 16), None, t(2, 8, 16), t(2, 16, 8)),
    lambda t: sg.lora_gemm_backward(t(4, 16), t(4, 16), None, t(2, 8, 16), t(2, 16, 8), da=t(2, 8, 16)),
    lambda t: sg.lora_gemm_backward(t(4, 16), t(4, 16), None, t(2, 8, 16), t(2, 16, 8), grad_dtype=torch.float16),
    lambda t: sg.lora_gemm_backward(t(4, 16), t(4, 16), None, t(2, 8, 16), t(2, 16, 8), da=1, db=1),
    lambda t: sg.lora_gemm_backward(t(4, 16), t(4, 16), None, t(2, 8, 16), t(2, 16, 8), da=t(2, 8, 16), db=t(2, 16, 8).float()),
])
def test_refusals(call):
    with pytest.raises(sg.SgError):
        call(lambda *s: torch.zeros(s, dtype=BF16, device=DEV))


# ------------------------------------------------------------------ streams, graphs, together

class Block:
    """A gated feed-forward block on frozen weights with adapters on both projections and
    on the 4-bit down projection."""

    def __init__(self, T, D, F, r, L, seed=0):
        gen = torch.Generator(device=DEV).manual_seed(seed)

        def w(*shape, std=1.0):
            return (std * torch.randn(shape, generator=gen, device=DEV)).to(BF16)

        self.F, self.D = F, D
        self.gate, self.up = w(F, D, std=D ** -0.5), w(F, D, std=D ** -0.5)
        codes, scales = sg.int4_quant_groupwise(w(D, F, std=F ** -0.5), gc=64)
        self.down = sg.w4_pack(codes, scales, 64)
        self.pairs = [(w(L, r, i, std=i ** -0.5), w(L, o, r, std=0.1)) for i, o in ((D, F), (D, F), (F, D))]
        self.scale = torch.rand(L, generator=gen, device=DEV) + 0.5
        self.x, self.dy = w(T, D), w(T, D)
        self.ids = torch.randint(-1, L, (T,), generator=gen, device=DEV, dtype=torch.int32)

    def forward(self, keep=False):
        (ag, bg), (au, bu), (ad, bd) = self.pairs
        add_g = sg.lora_gemm(self.x, self.ids, ag, bg, self.scale)
        add_u = sg.lora_gemm(self.x, self.ids, au, bu, self.scale)
        out = sg.gated_gemm(self.x, self.gate, self.up, gate_add=add_g, up_add=add_u, keep=keep)
        h = out[0] if keep else out
        y = sg.w4a16_gemm_groupwise_packed(h, self.down, self.D, 64)
        sg.lora_gemm(h, self.ids, ad, bd, self.scale, base=y, y=y)
        return (y, add_g, add_u, *out) if keep else y

    def backward(self, h, g, u, dh_base):
        (ag, bg), (au, bu), (ad, bd) = self.pairs
        dh, dad, dbd = sg.lora_gemm_backward(self.dy, h, self.ids, ad, bd, self.scale, base=dh_base)
        dx, _, _, dg, du = sg.gated_gemm_backward(dh, self.x, self.gate, self.up, g=g, u=u, need_dw=False)
        dx, dag, dbg = sg.lora_gemm_backward(dg, self.x, self.ids, ag, bg, self.scale, base=dx, dx=dx)
        dx, dau, dbu = sg.lora_gemm_backward(du, self.x, self.ids, au, bu, self.scale, base=dx, dx=dx)
        return dh, dx, dag, dbg, dau, dbu, dad, dbd


@pytest.mark.parametrize("T,D,F,r,L", [(1, 256, 512, 16, 3), (24, 256, 384, 8, 5), (200, 128, 256, 40, 3)])
def test_block_together(T, D, F, r, L):
    """Each step against fp64 on the operands it was given."""
    say(f"block {T} {D} {F} r {r} L {L}")
    m = Block(T, D, F, r, L)
    y, add_g, add_u, h, g, u = m.forward(keep=True)
    assert same(m.forward(), y)
    (ag, bg), (au, bu), (ad, bd) = m.pairs
    n = m.ids.cpu().numpy()
    for add, a, b in ((add_g, ag, bg), (add_u, au, bu)):
        ref, inner, outer = adapt.lora(f64(m.x), n, f64(a), f64(b), f64(m.scale))
        within("addend", add, ref, allowed(BF16, False, ref, inner, outer, D, r))
    rh, rg, ru, size_g, size_u = adapt.gated(*map(f64, (m.x, m.gate, m.up)), "silu", f64(add_g), f64(add_u))
    eg, eu, ea, _ = product_errors(D, rg, ru, size_g, size_u)
    eh = ea * (np.abs(ru) + eu) + np.abs(adapt.act("silu", rg)[0]) * eu + 2.0 ** -23 * np.abs(rh)
    within("h", h, rh, eh + half(BF16, np.abs(rh) + eh))
    alone = sg.w4a16_gemm_groupwise_packed(h, m.down, D, 64)
    ref, inner, outer = adapt.lora(f64(h), n, f64(ad), f64(bd), f64(m.scale), f64(alone))
    within("y", y, ref, allowed(BF16, False, ref, inner, outer, F, r))
    dh, dx, dag, dbg, dau, dbu, dad, dbd = m.backward(h, g, u, None)
    refs, ri, ro = adapt.lora_grads(f64(m.dy), f64(h), n, f64(ad), f64(bd), f64(m.scale))
    for got, i, n_in, n_out in ((dh, 0, D, r), (dad, 1, D, T), (dbd, 2, F, T)):
        within("down", got, refs[i], allowed(BF16, False, refs[i], ri[i], ro[i], n_in, n_out))
    dx0, _, _, dg, du = sg.gated_gemm_backward(dh, m.x, m.gate, m.up, g=g, u=u, need_dw=False)
    base = dx0
    for d, a, b, got_a, got_b in ((dg, ag, bg, dag, dbg), (du, au, bu, dau, dbu)):
        refs, ri, ro = adapt.lora_grads(f64(d), f64(m.x), n, f64(a), f64(b), f64(m.scale), f64(base))
        step = sg.lora_gemm_backward(d, m.x, m.ids, a, b, m.scale, base=base)
        within("dx", step[0], refs[0], allowed(BF16, False, refs[0], ri[0], ro[0], F, r))
        assert same(step[1], got_a) and same(step[2], got_b)
        for got, i, n_in in ((got_a, 1, F), (got_b, 2, D)):
            within("up", got, refs[i], allowed(BF16, False, refs[i], ri[i], ro[i], n_in, T))
        base = step[0]
    assert same(base, dx)


@pytest.mark.parametrize("T", [1, 20, 300])
def test_graph_replays_equal_eager(T):
    m = Block(T, 256, 512, 16, 3, seed=1)

    def step():
        y, _, _, h, g, u = m.forward(keep=True)
        return (y, *m.backward(h, g, u, None))

    def load(seed):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        m.x.normal_(generator=gen)
        m.dy.normal_(generator=gen)
        m.ids.random_(-1, 3, generator=gen)

    wants = []
    for seed in (1, 2, 3):
        load(seed)
        wants.append([t.clone() for t in step()])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        out = step()
    torch.cuda.current_stream().wait_stream(s)
    for seed in (1, 2, 3, 2):
        load(seed)                                      # the same addresses, other values
        for t in out:
            t.fill_(7.0)
        junk = torch.randn(1 << 18, device=DEV).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(p, q) for p, q in zip(out, wants[seed - 1])), seed
        assert all(same(p, q) for p, q in zip(step(), wants[seed - 1]))      # eager work between
        del junk


def test_two_streams_at_once():
    blocks = [Block(150, 256, 512, 16, 3, seed=s) for s in (5, 6)]
    wants = [b.forward() for b in blocks]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                got.append(b.forward())
    torch.cuda.synchronize()
    assert all(same(y, wants[i % 2]) for i, y in enumerate(got))


def test_same_bits_every_time():
    m = Block(500, 256, 512, 40, 2, seed=7)
    y, _, _, h, g, u = m.forward(keep=True)
    first = m.backward(h, g, u, None)
    w = sg.gated_gemm_backward(h, m.x, m.gate, m.up, g=g, u=u)
    for _ in range(3):
        assert all(same(p, q) for p, q in zip(m.backward(h, g, u, None), first))
        assert all(same(p, q) for p, q in zip(sg.gated_gemm_backward(h, m.x, m.gate, m.up, g=g, u=u), w))


def test_called_with_another_device_current(monkeypatch):
    """The launch goes to the tensors' device: with another current one it is made current."""
    m = Block(9, 128, 256, 8, 2, seed=8)
    want = m.forward()
    entered = []

    class Device:
        def __init__(self, d):
            entered.append(d)

        def __enter__(self):
            return self

        def __exit__(self, *a):
            return False

    with monkeypatch.context() as p:
        p.setattr(_gated.torch._C, "_cuda_getDevice", lambda: 1)
        p.setattr(_gated.torch.cuda, "device", Device)
        (ag, bg), _, _ = m.pairs
        add = sg.lora_gemm(m.x, m.ids, ag, bg, m.scale)
        sg.gated_gemm(m.x, m.gate, m.up, gate_add=add)
    assert entered == [0, 0]
    assert same(m.forward(), want)

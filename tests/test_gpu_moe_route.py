"""Routing to experts and its gradient on the GPU against the fp64 oracle.

Weights: fp32 of a value computed in fp64, except softmax without a bias, whose
sum is fp32: each term's exponential is within 2 steps of 2^-24 plus d 2^-24 for
the rounding of its argument's distance d to the largest logit (sum p d <= ln E
< 7), and at most 22 additions follow: 32 * 2^-24 bounds all of it.
Gradients: the same per factor, at most 4 of them, on the magnitude of the terms
a value is summed from, then half a step of the result's type."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, say
from oracle import moe

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def logits_of(seed, T, E, dtype, masked=False):
    g = torch.Generator().manual_seed(seed)
    x = 1.5 * torch.randn((T, E), generator=g)
    if masked and T > 4:
        x[:, torch.rand(E, generator=g) < 0.2] = -float("inf")
        x[0] = -float("inf")
        x[1] = torch.finfo(dtype).min
        x[2, ::2] = float("nan")
        x[3, 0] = float("inf")
        x[4] = 0.0
        x[4, ::3] = -0.0
    return x.to(dtype)


def check_route(l, k, **kw):
    bias = kw.get("bias")
    dev = dict(kw, bias=None if bias is None else bias.to(DEV))
    ids, w = sg.moe_route(l.to(DEV), k, **dev)
    torch.cuda.synchronize()
    oid, ow = moe.moe_route(l.float().numpy(), k, **dict(kw, bias=None if bias is None else bias.numpy()))
    ids, w = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    bad = np.argwhere(ids != oid)
    assert len(bad) == 0, f"{len(bad)} ids differ, first at {bad[0]}: {ids[bad[0][0]]} for {oid[bad[0][0]]}"
    err = np.abs(w - ow)
    assert (err <= 32 * 2.0 ** -24 * ow + 1e-38).all(), f"weights off by {np.max(err / (ow + 1e-38)):.3g}"
    return oid


CASES = [
    # T, E, k, n_group, topk_group
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (37, 60, 4, 1, 1), (5, 64, 64, 1, 1), (7, 65, 10, 5, 2), (66, 128, 6, 4, 3),
    (13, 200, 8, 8, 3), (130, 256, 8, 8, 4), (9, 512, 16, 64, 9), (6, 1000, 7, 40, 4), (6, 1024, 64, 1, 1),
    (33, 24, 3, 24, 5), (40, 96, 5, 3, 1),
]


@pytest.mark.parametrize("T,E,k,ng,tg", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(T, E, k, ng, tg, dtype, score):
    say(f"route T{T} E{E} k{k} groups {tg}/{ng} {dtype} {score}")
    g = torch.Generator().manual_seed(E)
    for n, (bias, gs, renorm) in enumerate([(False, "max", False), (True, "top2", True), (False, "top2", True),
                                            (True, "max", False)]):
        b = 0.2 * torch.randn(E, generator=g) if bias else None
        if bias and E > 8:
            b[3], b[5] = -float("inf"), float("nan")
        check_route(logits_of(10 * E + n, T, E, dtype, masked=n < 3), k, score=score, bias=b, n_group=ng, topk_group=tg,
                    group_score=gs, renormalize=renorm, scale=1.0 if n == 0 else 2.5)


@pytest.mark.parametrize("E", [48, 256])
def test_keys_that_fp32_cannot_tell_apart(E):
    """Pairs of experts whose score + bias differ in the fp64 value alone, in both orders."""
    T = 64
    l = logits_of(5, T, E, F32)
    # experts 2 i and 2 i + 1: logits one fp32 step apart and the same bias
    l[:, 1::2] = torch.nextafter(l[:, 0::2], torch.where(torch.arange(T)[:, None] % 2 == 0, 1e9, -1e9).expand(T, E // 2))
    b = torch.zeros(E)
    b[::2] = b[1::2] = torch.randn(E // 2, generator=torch.Generator().manual_seed(1))
    say(f"near ties E{E}")
    for score in ("softmax", "sigmoid"):
        check_route(l, 8, score=score, bias=b)
        check_route(l, 8, score=score, bias=b, n_group=4, topk_group=2, group_score="top2")


def test_all_equal_goes_to_the_lowest():
    for E in (5, 64, 300):
        l = torch.full((3, E), 0.25)
        say(f"equal E{E}")
        for bias in (None, torch.full((E,), 0.125)):
            oid = check_route(l, min(E, 5), bias=bias)
            assert (oid == np.arange(5)).all()


def test_strided_logits_and_given_outputs():
    big = torch.randn((9, 100), generator=torch.Generator().manual_seed(2)).to(DEV)
    l = big[:, 17:77]
    ids, w = torch.empty((9, 4), dtype=torch.int32, device=DEV), torch.empty((9, 4), device=DEV)
    r = sg.moe_route(l, 4, ids=ids, weights=w)
    assert r[0] is ids and r[1] is w
    i2, w2 = sg.moe_route(l.contiguous(), 4)
    assert torch.equal(ids, i2) and torch.equal(w, w2)
    g = torch.randn((9, 4), generator=torch.Generator().manual_seed(3)).to(DEV)
    out = torch.full((9, 100), 7.0, device=DEV)
    sg.moe_route_backward(g, l, ids, dlogits=out[:, 17:77])
    assert torch.equal(out[:, 17:77], sg.moe_route_backward(g, l.contiguous(), ids))
    assert (out[:, :17] == 7).all() and (out[:, 77:] == 7).all()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (37, 60, 4), (5, 64, 64), (66, 130, 6), (9, 512, 16), (6, 1024, 64)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward(T, E, k, dtype, score, renorm):
    say(f"grad T{T} E{E} k{k} {dtype} {score} {renorm}")
    l = logits_of(E + 1, T, E, dtype, masked=True)
    l[l == float("inf")] = 3.0
    ids, _ = moe.moe_route(l.float().numpy(), k, score=score)
    if T > 5:
        ids[5, 0] = E + 3          # out of range: empty slots
        ids[4, -1] = -1
    g = torch.randn((T, k), generator=torch.Generator().manual_seed(T))
    got = sg.moe_route_backward(g.to(DEV), l.to(DEV), torch.from_numpy(ids).to(DEV), score=score, renormalize=renorm,
                                scale=1.5)
    assert got.dtype == dtype
    got = got.double().cpu().numpy()
    want, size = moe.moe_route_backward(g.numpy(), l.float().numpy(), ids, score=score, renormalize=renorm, scale=1.5)
    half = torch.finfo(dtype).eps / 2
    tol = 4 * 32 * 2.0 ** -24 * size + half * np.abs(want) + 1e-37
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert len(bad) == 0, f"{len(bad)} off, first at {bad[0]}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}"


def test_gradient_equals_differences_of_the_forward():
    """Central differences of moe_route's own weights (fp32, so a wide step)."""
    T, E, k, h = 8, 16, 3, 2.0 ** -6
    l = logits_of(9, T, E, F32).to(DEV)
    g = torch.randn((T, k), generator=torch.Generator().manual_seed(1)).to(DEV)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, _ = sg.moe_route(l, k, score=score, renormalize=renorm)
            got = sg.moe_route_backward(g, l, ids, score=score, renormalize=renorm)
            for e in range(E):
                side = []
                for s in (h, -h):
                    p = l.clone()
                    p[:, e] += s
                    i2, w2 = sg.moe_route(p, E, score=score)       # every score, put back in the first choice's order
                    full = torch.zeros((T, E), device=DEV).scatter_(1, i2.long(), w2)
                    w = full.gather(1, ids.long())
                    side.append(((w / w.sum(1, keepdim=True) if renorm else w) * g).sum(1))
                diff = (side[0] - side[1]) / (2 * h)
                # third derivatives of these weights are below 2, sum |g| below 8; fp32 rounding 2^-22 / h
                assert (diff - got[:, e]).abs().max() <= 16 * h * h / 6 + 16 * 2.0 ** -22 / h


def test_refusals():
    l = torch.zeros((4, 16), device=DEV)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    for bad in (lambda: sg.moe_route(l, 0), lambda: sg.moe_route(l, 17), lambda: sg.moe_route(l, 2, score="relu"),
                lambda: sg.moe_route(l, 2, group_score="sum"), lambda: sg.moe_route(l, 2, n_group=3),
                lambda: sg.moe_route(l, 5, n_group=4, topk_group=1), lambda: sg.moe_route(l.half(), 2),
                lambda: sg.moe_route(l.t(), 2), lambda: sg.moe_route(l[:0], 2),
                lambda: sg.moe_route(l, 2, bias=torch.zeros(15, device=DEV)),
                lambda: sg.moe_route(l, 2, bias=torch.zeros(16)),
                lambda: sg.moe_route(l, 2, ids=ids.long()), lambda: sg.moe_route(l, 2, weights=l[:, :2]),
                lambda: sg.moe_route_backward(l[:, :2], l, ids), lambda: sg.moe_route_backward(l, l, ids),
                lambda: sg.moe_route_backward(l[:, :2].contiguous(), l, ids.long())):
        with pytest.raises(sg.SgError):
            bad()

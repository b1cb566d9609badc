"""Routing and its gradient over more tokens than one pass of the kernels' loops
takes (their grids are bounded): what a later pass gives equals the same tokens in
small batches, and sampled rows equal the oracle's."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, say
from oracle import moe

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
STEP = 2.0 ** -24


def logits(seed, T, E, dtype):
    g = torch.Generator().manual_seed(seed)
    x = 1.5 * torch.randn((T, E), generator=g)
    x[:, torch.rand(E, generator=g) < 0.1] = -float("inf")
    for t in (3, T // 2, T - 2):
        x[t] = -float("inf")
    x[T - 3, ::2] = float("nan")
    return x.to(dtype)


ROUTE = [
    # T, E, k, n_group, topk_group
    (16384 + 5, 256, 8, 8, 4), (2 * 16384 + 3, 60, 4, 1, 1), (16384 + 9, 240, 8, 16, 5),
    (8192 + 5, 300, 8, 4, 2), (8192 + 5, 64, 20, 1, 1), (8192 + 7, 96, 5, 32, 9), (3 * 8192 + 1, 1024, 6, 64, 9),
]


@pytest.mark.parametrize("T,E,k,ng,tg", ROUTE)
@pytest.mark.parametrize("score,dtype", [("sigmoid", F32), ("softmax", BF16)])
def test_route(T, E, k, ng, tg, score, dtype):
    l = logits(E, T, E, dtype)
    x = l.to(DEV)
    for bias, gs in ((True, "top2"), (False, "max")):
        b = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E)) if bias else None
        kw = dict(score=score, n_group=ng, topk_group=tg, group_score=gs, renormalize=bias, scale=2.5)
        say(f"route passes T{T} E{E} k{k} groups {tg}/{ng} {score} {dtype} bias {bias}")
        dev = dict(kw, bias=None if b is None else b.to(DEV))
        ids, w = sg.moe_route(x, k, **dev)
        parts = [sg.moe_route(x[i:i + 2048], k, **dev) for i in range(0, T, 2048)]
        want, ww = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
        bad = (ids != want).any(1).nonzero().flatten()
        assert len(bad) == 0, f"{len(bad)} tokens differ, the first {bad[0]}"
        # each within 32 steps of its value (test_gpu_moe_route.py counts them)
        assert ((w - ww).abs() <= 64 * STEP * ww + 1e-38).all()
        pick = np.unique(np.r_[0:4, T // 2, T - 4:T, np.random.default_rng(1).integers(T // 2, T, 12)])
        oid, ow = moe.moe_route(l[pick].float().numpy(), k, **dict(kw, bias=None if b is None else b.numpy()))
        assert np.array_equal(ids.cpu().numpy()[pick], oid)
        assert (np.abs(w.double().cpu().numpy()[pick] - ow) <= 32 * STEP * ow + 1e-38).all()


GRAD = [
    # T, E, k, score, renormalize
    (8192 + 5, 60, 4, "softmax", False), (8192 + 5, 300, 8, "softmax", False), (2 * 8192 + 3, 1000, 3, "softmax", False),
    (8192 + 5, 64, 20, "softmax", True), (8192 + 7, 600, 4, "sigmoid", True), (8192 + 7, 64, 17, "sigmoid", False),
    (32768 + 5, 60, 4, "sigmoid", True), (32768 + 5, 130, 8, "softmax", True), (2 * 32768 + 9, 61, 3, "sigmoid", False),
]


@pytest.mark.parametrize("T,E,k,score,renorm", GRAD)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_backward(T, E, k, score, renorm, dtype):
    say(f"grad passes T{T} E{E} k{k} {score} {renorm} {dtype}")
    l = logits(E + 1, T, E, dtype)
    x = l.to(DEV)
    ids, _ = sg.moe_route(x, k, score=score)
    ids[5, 0], ids[T - 1, k - 1] = E + 3, -1           # empty slots
    g = torch.randn((T, k), generator=torch.Generator().manual_seed(T))
    gd = g.to(DEV)
    kw = dict(score=score, renormalize=renorm, scale=1.5)
    got = sg.moe_route_backward(gd, x, ids, **kw)
    want = torch.cat([sg.moe_route_backward(gd[i:i + 2048], x[i:i + 2048], ids[i:i + 2048], **kw)
                      for i in range(0, T, 2048)])
    assert torch.equal(got, want)                      # one token's arithmetic is the same in every pass
    pick = np.unique(np.r_[0:6, T // 2, T - 4:T, np.random.default_rng(1).integers(T // 2, T, 12)])
    ref, size = moe.moe_route_backward(g.numpy()[pick], l[pick].float().numpy(), ids.cpu().numpy()[pick], **kw)
    tol = 4 * 32 * STEP * size + torch.finfo(dtype).eps / 2 * np.abs(ref) + 1e-37
    assert (np.abs(got.double().cpu().numpy()[pick] - ref) <= tol).all()

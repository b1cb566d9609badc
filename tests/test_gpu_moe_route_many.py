"""Routing of many tokens (another kernel from 8192 on): the ids equal those of
the same tokens routed a few at a time, which test_gpu_moe_route.py holds to the
oracle, and some rows are held to it here; weights within 32 steps of 2^-24 each."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, say
from oracle import moe

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
T = 8192 + 5
STEP = 2.0 ** -24


def compare(l, k, rows=24, **kw):
    T, bias = l.shape[0], kw.get("bias")
    dev = dict(kw, bias=None if bias is None else bias.to(DEV))
    x = l.to(DEV)
    ids, w = sg.moe_route(x, k, **dev)
    parts = [sg.moe_route(x[i:i + 2048], k, **dev) for i in range(0, T, 2048)]
    want, ww = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    bad = (ids != want).any(1).nonzero().flatten()
    assert len(bad) == 0, f"{len(bad)} tokens differ, {bad[0]}: {ids[bad[0]].tolist()} for {want[bad[0]].tolist()}"
    assert ((w - ww).abs() <= 64 * STEP * ww + 1e-38).all()
    pick = np.unique(np.r_[0:6, np.random.default_rng(1).integers(0, T, rows), T - 3:T])
    oid, ow = moe.moe_route(l[pick].float().numpy(), k, **dict(kw, bias=None if bias is None else bias.numpy()))
    assert np.array_equal(ids.cpu().numpy()[pick], oid)
    assert (np.abs(w.double().cpu().numpy()[pick] - ow) <= 32 * STEP * ow + 1e-38).all()


def logits(seed, E, dtype, masked):
    g = torch.Generator().manual_seed(seed)
    x = 1.5 * torch.randn((T, E), generator=g)
    if masked:
        x[:, torch.rand(E, generator=g) < 0.2] = -float("inf")
        x[0] = -float("inf")
        x[1] = torch.finfo(dtype).min
        x[2, ::2] = float("nan")
        x[3, 0] = float("inf")
        x[4] = 0.0
        x[4, ::3] = -0.0
        x[5, 1 % E] = torch.finfo(dtype).max
        x[5, 2 % E] = float("inf")
        x[T - 1] = -float("inf")
    return x.to(dtype)


CASES = [
    # E, k, n_group, topk_group
    (1, 1, 1, 1), (5, 3, 1, 1), (60, 4, 1, 1), (64, 16, 4, 2), (65, 10, 5, 2), (96, 5, 3, 1), (128, 6, 4, 3), (200, 8, 8, 3),
    (240, 8, 16, 5), (256, 8, 8, 4), (256, 16, 1, 1), (13, 2, 13, 4),
]


@pytest.mark.parametrize("E,k,ng,tg", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many(E, k, ng, tg, dtype, score):
    say(f"route many E{E} k{k} groups {tg}/{ng} {dtype} {score}")
    g = torch.Generator().manual_seed(E)
    for n, (bias, gs, renorm) in enumerate([(False, "max", False), (True, "top2", True), (False, "top2", True),
                                            (True, "max", False)]):
        b = 0.2 * torch.randn(E, generator=g) if bias else None
        if bias and E > 8:
            b[3], b[5] = -float("inf"), float("nan")
        compare(logits(10 * E + n, E, dtype, masked=n < 3), k, score=score, bias=b, n_group=ng, topk_group=tg,
                group_score=gs, renormalize=renorm, scale=1.0 if n == 0 else 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift", [0.0, 1000.0, -3e7, 1e30])
def test_biases_of_every_size(score, shift):
    """Spans and offsets that 24-bit keys cannot hold: the choice is still the fp64 one."""
    E = 96
    l = logits(3, E, F32, False)
    b = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(2)) + shift
    say(f"bias shift {shift} {score}")
    compare(l, 6, score=score, bias=b, n_group=4, topk_group=2, group_score="top2")
    b[::7] = 1e34
    compare(l, 6, score=score, bias=b)


def test_keys_that_fp32_cannot_tell_apart():
    E = 128
    l = logits(5, E, F32, False)
    l[:, 1::2] = torch.nextafter(l[:, 0::2], torch.where(torch.arange(T)[:, None] % 2 == 0, 1e9, -1e9).expand(T, E // 2))
    b = torch.zeros(E)
    b[::2] = b[1::2] = torch.randn(E // 2, generator=torch.Generator().manual_seed(1))
    for score in ("softmax", "sigmoid"):
        say(f"near ties {score}")
        compare(l, 8, score=score, bias=b)
        compare(l, 8, score=score, bias=b, n_group=4, topk_group=2, group_score="top2")
    compare(l, 8)
    compare(l, 8, n_group=8, topk_group=3)


def test_equal_logits_and_strides():
    l = torch.full((T, 100), 0.25)
    compare(l, 5)
    compare(l, 5, bias=torch.full((100,), 0.125), n_group=4, topk_group=2, group_score="top2")
    big = torch.randn((T, 131), generator=torch.Generator().manual_seed(2)).to(DEV)
    for lo, hi in ((3, 103), (1, 64), (0, 131)):
        say(f"strided {lo} {hi}")
        a = sg.moe_route(big[:, lo:hi], 4)
        b = sg.moe_route(big[:, lo:hi].contiguous(), 4)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])

"""Routing of many tokens with experts masked by a finite bias (-1e4, -1e9, the
lowest fp32): the masked ones lie far below every key of the others, and still have
their order, since they are chosen where nothing else is left."""
import pytest
import torch

from gpu_helpers import say
from test_gpu_moe_route_many import F32, BF16, T, compare, logits

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min


def bias_of(E, mask, share, seed=3):
    g = torch.Generator().manual_seed(seed)
    b = 0.1 * torch.randn(E, generator=g)
    off = torch.rand(E, generator=g) < share
    off[0] = True
    b[off] = mask
    return b


@pytest.mark.parametrize("score,dtype", [("softmax", BF16), ("sigmoid", F32)])
@pytest.mark.parametrize("mask", [-1000.0, -1e4, -1e9, LOWEST])
@pytest.mark.parametrize("E,k,ng,tg,gs", [
    (256, 8, 8, 4, "top2"), (256, 8, 8, 4, "max"), (256, 8, 1, 1, "max"), (60, 4, 1, 1, "max"), (64, 6, 16, 4, "top2"),
    (96, 6, 4, 2, "max"),
])
@pytest.mark.parametrize("share", [0.1, 0.6, 0.97])
def test_finite_masks(E, k, ng, tg, gs, mask, score, dtype, share):
    say(f"finite mask {mask} on {share} of {E}, k{k} groups {tg}/{ng} {gs} {score}")
    compare(logits(E, E, dtype, False), k, rows=8, score=score, bias=bias_of(E, mask, share), n_group=ng, topk_group=tg,
            group_score=gs, renormalize=True, scale=2.5)


@pytest.mark.parametrize("gs", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_whole_groups_and_steps_of_masks(gs, score):
    """Groups masked whole, masks of several depths that score or logit order decides between, one key far above."""
    E = 96
    l = logits(1, E, F32, True)
    b = bias_of(E, -1e4, 0.1)
    b[:24] = -1e4
    say(f"masked groups {gs} {score}")
    compare(l, 5, score=score, bias=b, n_group=4, topk_group=3, group_score=gs)
    compare(l, 5, score=score, bias=b, n_group=4, topk_group=4, group_score=gs)
    b = -1000.0 * torch.arange(E)
    compare(l, 8, score=score, bias=b, n_group=8, topk_group=3, group_score=gs)
    b = bias_of(E, -1e4, 0.5)
    b[7] = 2000.0
    compare(l, 8, score=score, bias=b, n_group=8, topk_group=5, group_score=gs)
    b = torch.linspace(-80.0, 0.0, E)
    b[::5] -= 2000.0
    compare(l, 8, score=score, bias=b, n_group=12, topk_group=5, group_score=gs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_group_of_one_masked_expert(score):
    """Its value is the one key, -1e4; groups of two keys each 60 below the best sum up to about -120."""
    E = 48
    b = torch.full((E,), -60.0)
    b[:12] = -float("inf")
    b[3] = -1e4
    b[12:24] = -float("inf")
    b[14] = b[20] = 0.0                  # two of the four that are chosen
    say(f"one masked expert {score}")
    for tg in (1, 2, 3, 4):
        compare(logits(2, E, F32, False), 4, score=score, bias=b, n_group=4, topk_group=tg, group_score="top2")


def test_tokens():
    assert T >= 8192      # from where many tokens have their own kernel

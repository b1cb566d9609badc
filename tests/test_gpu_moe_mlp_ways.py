"""The routed 4-bit MLP at the sizes that its launch rule tells apart: a handful of
pairs, streamed row blocks (with several passes over an expert), tiles of every
size class, long rows, and more pairs than the sorting launch keeps in registers."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, down, say
from oracle import moe
from test_gpu_moe_mlp import BF16, F32, layer, routing, run_and_check, up

pytestmark = pytest.mark.gpu

CASES = [
    # T, E, k, D, F, gc, dropped, hot
    (16, 40, 1, 128, 96, 32, 0.2, None), (2, 8, 8, 160, 64, 32, 0.0, None), (5, 9, 3, 288, 32, 32, 0.5, None),
    (24, 64, 3, 128, 96, 32, 0.1, None), (40, 200, 2, 128, 64, 64, 0.0, 7), (12, 64, 3, 160, 96, 32, 0.0, 3),
    (9, 40, 3, 4096, 64, 32, 0.0, 5), (6, 40, 3, 8192, 32, 32, 0.0, 2), (6, 40, 3, 64, 8192, 64, 0.0, 2),
    (5, 12, 4, 10240, 64, 64, 0.0, None), (33, 16, 2, 128, 4096, 128, 0.0, None),
    (33, 1, 1, 256, 128, 128, 0.0, None), (65, 1, 1, 160, 96, 32, 0.0, None), (97, 1, 1, 192, 128, 64, 0.0, None),
    (129, 2, 2, 384, 160, 32, 0.0, None), (300, 5, 3, 640, 320, 64, 0.1, 0),
]


@pytest.mark.parametrize("T,E,k,D,F,gc,drop,hot", CASES)
def test_ways(T, E, k, D, F, gc, drop, hot):
    say(f"moe ways T{T} E{E} k{k} D{D} F{F} gc{gc} hot {hot}")
    ids, w = routing(T + E, T, E, k, drop, hot)
    run_and_check(T, E, k, D, F, gc, F32, ids, w)


@pytest.mark.parametrize("T,E,k", [(9000, 8, 2), (4100, 1000, 5)])
def test_many_pairs(T, E, k):
    """More pairs than 16 a thread of the sorting launch; the oracle on some tokens."""
    D, F, gc = 64, 32, 32
    host, dev = layer(3, E, D, F, gc)
    ids, w = routing(1, T, E, k, 0.05)
    x = torch.randn((T, D), generator=torch.Generator().manual_seed(T)).to(BF16)
    say(f"many pairs {T * k}")
    y = sg.w4a16_moe_mlp(x.to(DEV), up(ids), up(w), *dev, F, gc, out_dtype=F32)
    pick = np.unique(np.r_[0, T - 1, np.random.default_rng(2).integers(0, T, 40)])
    ref, bound = moe.moe_mlp(x[pick].double().numpy(), ids[pick], w[pick], *host, gc)
    err = np.abs(down(y)[pick] - ref)
    assert (err <= bound + 2.0 ** -24 * (np.abs(ref) + bound) + 1e-30).all()


@pytest.mark.parametrize("T", [3, 30, 400])
def test_rows_of_nan_stay_in_their_tokens(T):
    E, k, D, F, gc = 32, 2, 160, 96, 32
    _, dev = layer(4, E, D, F, gc)
    ids, w = routing(7, T, E, k)
    x = torch.randn((T, D), generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    want = sg.w4a16_moe_mlp(x, up(ids), up(w), *dev, F, gc, out_dtype=F32)
    x[1] = float("nan")
    got = sg.w4a16_moe_mlp(x, up(ids), up(w), *dev, F, gc, out_dtype=F32)
    keep = torch.arange(T, device=DEV) != 1
    assert torch.isnan(got[1]).all() and torch.equal(got[keep], want[keep])

"""The routed 4-bit MLP's large tiles over several blocks of K: experts whose pairs
fill a tile to a quarter, half, three quarters, whole or more, either product in
turn over 2, 3 and an odd number of K blocks, each group size.  Sampled tokens
against the fp64 oracle, within its bound; the rest by repeating the call."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, down, say
from oracle import moe
from test_gpu_moe_mlp import BF16, F32, layer, up

pytestmark = pytest.mark.gpu

COUNTS = (20, 50, 80, 120, 200, 128, 129, 1, 0, 33, 96, 64)   # pairs of experts 0, 1, ..., again and again


def pairs(E, k, seed):
    """ids [T, k] with COUNTS pairs an expert, in any order; the slots left over are empty."""
    g = np.random.default_rng(seed)
    flat = np.concatenate([np.full(COUNTS[e % len(COUNTS)], e) for e in range(E)])
    flat = np.concatenate([flat, np.full(-len(flat) % k, -1)]).astype(np.int32)
    ids = g.permutation(flat).reshape(-1, k)
    w = g.uniform(0.05, 1.0, ids.shape).astype(np.float32)
    w[ids < 0] = np.nan                      # never read
    return ids, w


def tiles_about(P, E):
    """Tiles there are, about: the larger tiles are taken where these times the tiles of a row pass 256."""
    return -(-P // 128) + min(P, E) // 2


CASES = [
    # E, k, D, F, gc, which product has the larger tiles
    (48, 4, 256, 896, 128, "gate_up"), (48, 2, 288, 1152, 32, "gate_up"), (48, 3, 320, 896, 64, "gate_up"),
    (48, 1, 384, 896, 128, "gate_up"), (48, 4, 640, 896, 128, "gate_up"),
    (48, 4, 1792, 256, 128, "down"), (48, 2, 1824, 288, 32, "down"), (48, 3, 1792, 320, 64, "down"),
    (48, 1, 1792, 384, 128, "down"), (48, 4, 1792, 640, 128, "both"),
    (48, 2, 1792, 896, 64, "both"), (60, 5, 2048, 1408, 32, "both"),
]


@pytest.mark.parametrize("E,k,D,F,gc,which", CASES)
def test_large_tiles(E, k, D, F, gc, which):
    ids, w = pairs(E, k, E + D)
    T = len(ids)
    n = tiles_about(ids.size, E)
    large = (n * -(-F // 128) > 256, n * -(-D // 256) > 256)
    assert large == {"gate_up": (True, False), "down": (False, True), "both": (True, True)}[which]
    say(f"moe large tiles T{T} E{E} k{k} D{D} F{F} gc{gc} {which}")
    host, dev = layer(D + F, E, D, F, gc)
    x = torch.randn((T, D), generator=torch.Generator().manual_seed(T)).to(BF16)
    y = sg.w4a16_moe_mlp(x.to(DEV), up(ids), up(w), *dev, F, gc, out_dtype=F32)
    pick = np.unique(np.r_[0, T - 1, np.random.default_rng(1).integers(0, T, 60)])
    ref, bound = moe.moe_mlp(x[pick].double().numpy(), ids[pick], w[pick], *host, gc)
    tol = bound + 2.0 ** -24 * (np.abs(ref) + bound) + 1e-30
    err = np.abs(down(y)[pick] - ref)
    assert np.isfinite(err).all() and (err <= tol).all(), f"off by {np.max(err / tol):.3g} of what is allowed"
    say(f"  max |err| / allowed = {np.max(err / tol):.3g}")
    # a token's result does not depend on which pairs share its tiles
    order = torch.from_numpy(np.random.default_rng(2).permutation(T)).to(DEV)
    again = sg.w4a16_moe_mlp(x.to(DEV)[order], up(ids)[order], up(w)[order], *dev, F, gc, out_dtype=F32)
    assert torch.equal(again, y[order])

"""The routed gated MLP on the GPU against the fp64 oracle, within the bound that
oracle.moe.moe_mlp derives from the kernel's roundings, then half a step of the
output type; its use on other streams, in graphs, and after the router."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, down, say
from oracle import moe

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def layer(seed, E, D, F, gc):
    g = np.random.default_rng(seed)

    def one(n, k):
        return (g.integers(0, 256, (E, n, k // 2), dtype=np.uint8),
                np.exp2(g.uniform(-9, -6, (E, n, k // gc))).astype(np.float32))

    host = [one(F, D), one(F, D), one(D, F)]
    return host, [sg.w4_pack(up(c), up(s), gc) for c, s in host]


def routing(seed, T, E, k, drop=0.0, hot=None):
    g = np.random.default_rng(seed)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    if hot is not None:
        ids[:, 0] = hot
        for t in range(T):
            rest = [e for e in g.permutation(E) if e != hot]
            ids[t, 1:] = rest[:k - 1]
    w = g.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    out = g.random((T, k)) < drop
    ids[out] = np.where(g.random(out.sum()) < 0.5, -1, E + 2)
    w[out] = np.nan                       # never read
    return ids, w


def run_and_check(T, E, k, D, F, gc, dtype, ids, w, seed=0):
    host, dev = layer(seed, E, D, F, gc)
    x = torch.randn((T, D), generator=torch.Generator().manual_seed(T)).to(BF16)
    y = sg.w4a16_moe_mlp(x.to(DEV), up(ids), up(w), *dev, F, gc, out_dtype=dtype)
    ref, bound = moe.moe_mlp(x.double().numpy(), ids, w, *host, gc)
    tol = bound + torch.finfo(dtype).eps / 2 * (np.abs(ref) + bound) + 1e-30
    err = np.abs(down(y) - ref)
    assert np.isfinite(err).all() and (err <= tol).all(), f"off by {np.max(err / tol):.3g} of what is allowed"
    say(f"  max |err| / allowed = {np.max(err / tol):.3g}")


CASES = [
    # T, E, k, D, F, gc, dropped
    (1, 1, 1, 32, 32, 32, 0.0), (1, 8, 4, 256, 128, 128, 0.0), (1, 64, 8, 512, 320, 64, 0.0), (3, 5, 2, 96, 160, 32, 0.3),
    (17, 8, 8, 128, 64, 64, 0.0), (29, 60, 4, 256, 192, 64, 0.1), (40, 3, 2, 288, 96, 32, 0.2), (70, 4, 1, 128, 384, 128, 0.0),
    (90, 2, 2, 192, 192, 64, 0.0), (130, 4, 4, 160, 224, 32, 0.1), (200, 3, 3, 256, 256, 128, 0.0),
    (260, 2, 1, 640, 128, 128, 0.5), (150, 16, 6, 128, 128, 128, 0.0),
]


@pytest.mark.parametrize("T,E,k,D,F,gc,drop", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_mlp(T, E, k, D, F, gc, drop, dtype):
    say(f"moe mlp T{T} E{E} k{k} D{D} F{F} gc{gc} {dtype}")
    ids, w = routing(T + E, T, E, k, drop)
    run_and_check(T, E, k, D, F, gc, dtype, ids, w)


@pytest.mark.parametrize("T", [6, 50, 300])
def test_one_expert_takes_all(T):
    say(f"hot expert T{T}")
    ids, w = routing(3, T, 24, 3, hot=7)
    run_and_check(T, 24, 3, 128, 96, 32, F32, ids, w)


@pytest.mark.parametrize("T", [2, 64, 300])
def test_nothing_routed_gives_zeros(T):
    E, D, F, gc = 4, 128, 64, 64
    _, dev = layer(1, E, D, F, gc)
    ids = torch.full((T, 2), -1, dtype=torch.int32, device=DEV)
    w = torch.full((T, 2), float("nan"), device=DEV)
    y = sg.w4a16_moe_mlp(torch.ones((T, D), dtype=BF16, device=DEV), ids, w, *dev, F, gc)
    assert (y == 0).all()


@pytest.mark.parametrize("T", [3, 40, 300])
def test_strides_workspace_and_repeats(T):
    """Rows of wider buffers, a given (dirty) workspace; the same bits every time."""
    E, k, D, F, gc = 6, 2, 160, 96, 32
    _, dev = layer(2, E, D, F, gc)
    ids, w = routing(5, T, E, k)
    big = torch.full((T, D + 32), float("nan"), dtype=BF16, device=DEV)
    big[:, :D] = torch.randn((T, D), generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    need = sg.w4a16_moe_mlp_workspace(T, k, E, D, F)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((T, D + 8), 5.0, device=DEV)
    say(f"moe strides T{T}")
    y = sg.w4a16_moe_mlp(big[:, :D], up(ids), up(w), *dev, F, gc, y=out[:, :D], workspace=ws).clone()
    assert (out[:, D:] == 5).all() and (ws[need:] == 255).all()
    for _ in range(3):
        again = sg.w4a16_moe_mlp(big[:, :D].contiguous(), up(ids), up(w), *dev, F, gc, out_dtype=F32)
        assert torch.equal(y, again)


def test_another_stream():
    E, k, D, F, gc, T = 8, 2, 128, 64, 64, 20
    _, dev = layer(3, E, D, F, gc)
    ids, w = routing(6, T, E, k)
    ids, w = up(ids), up(w)
    x = torch.randn((T, D), generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    want = sg.w4a16_moe_mlp(x, ids, w, *dev, F, gc)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [sg.w4a16_moe_mlp(x, ids, w, *dev, F, gc) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(s)
    for g in got:
        g.record_stream(torch.cuda.current_stream())
        assert torch.equal(g, want)


@pytest.mark.parametrize("T", [1, 30, 300])
def test_route_then_mlp_in_a_graph(T):
    """Router, MLP, a 4-bit linear layer and the router's gradient captured once;
    replays on new inputs equal the eager calls."""
    E, k, D, F, gc = 16, 2, 128, 96, 32
    _, dev = layer(4, E, D, F, gc)
    g = np.random.default_rng(1)
    wl = sg.w4_pack(up(g.integers(0, 256, (64, D // 2), dtype=np.uint8)), torch.full((64, D // gc), 0.01, device=DEV), gc)
    x = torch.zeros((T, D), dtype=BF16, device=DEV)
    logits = torch.zeros((T, E), device=DEV)
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(1)).to(DEV)
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(2)).to(DEV)

    def step():
        ids, w = sg.moe_route(logits, k, score="sigmoid", bias=bias, renormalize=True)
        y = sg.w4a16_moe_mlp(x, ids, w, *dev, F, gc)
        z = sg.w4a16_gemm_groupwise_packed(y, wl, 64, gc)
        return ids, w, y, z, sg.moe_route_backward(dw, logits, ids, score="sigmoid", renormalize=True)

    step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            out = step()
    torch.cuda.current_stream().wait_stream(s)
    for r in range(4):
        gen = torch.Generator().manual_seed(100 + r)
        x.copy_(torch.randn((T, D), generator=gen).to(BF16))
        logits.copy_(torch.randn((T, E), generator=gen))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), f"replay {r}"


def test_refusals():
    E, D, F = 4, 128, 64
    _, (gate, upw, dn) = layer(5, E, D, F, 64)
    x = torch.zeros((2, D), dtype=BF16, device=DEV)
    ids, w = torch.zeros((2, 2), dtype=torch.int32, device=DEV), torch.zeros((2, 2), device=DEV)

    def call(x=x, ids=ids, w=w, gate=gate, upw=upw, dn=dn, F=F, gc=64, **kw):
        return sg.w4a16_moe_mlp(x, ids, w, gate, upw, dn, F, gc, **kw)

    call()
    for bad in (dict(x=x.float()), dict(x=x[:0]), dict(ids=ids.long()), dict(ids=ids[:1]), dict(w=w[:, :1]),
                dict(w=w.double()), dict(gate=gate[:3]), dict(upw=upw[0]), dict(dn=dn[:, :-64].contiguous()), dict(F=128),
                dict(gc=32), dict(gc=48), dict(out_dtype=torch.float16), dict(y=torch.zeros((2, 64), device=DEV)),
                dict(workspace=torch.zeros(16, dtype=torch.uint8, device=DEV)), dict(gate=gate.cpu()),
                dict(x=x.cpu())):
        with pytest.raises(sg.SgError):
            call(**bad)


@pytest.mark.parametrize("T,k", [(1, 8), (3, 4), (4, 4), (7, 2), (16, 1), (12, 5), (100, 6)])
def test_an_expert_twice_in_a_token(T, k):
    """Slots of one token may name the same expert: each contributes."""
    E, D, F, gc = 6, 128, 96, 32
    g = np.random.default_rng(T)
    ids = g.integers(-1, 3, (T, k)).astype(np.int32)
    w = g.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    say(f"duplicates T{T} k{k}")
    run_and_check(T, E, k, D, F, gc, F32, ids, w)


@pytest.mark.parametrize("T", [2, 9, 60])
def test_an_expert_of_infinities_stays_with_its_tokens(T):
    """Scales of one expert's weights that are inf or NaN: tokens of others keep their bits."""
    E, D, F, gc, k = 8, 128, 64, 64, 2
    host, dev = layer(7, E, D, F, gc)
    ids = np.stack([np.array([t % 4, 4 + t % 3]) for t in range(T)]).astype(np.int32)     # expert 7 unused
    ids[0] = (7, 1)
    w = np.full((T, k), 0.5, np.float32)
    x = torch.randn((T, D), generator=torch.Generator().manual_seed(T)).to(BF16).to(DEV)
    want = sg.w4a16_moe_mlp(x, up(ids), up(w), *dev, F, gc, out_dtype=F32)
    for c, s in host:
        s[7] = np.inf
    host[2][1][7] = np.nan
    bad = [sg.w4_pack(up(c), up(s), gc) for c, s in host]
    got = sg.w4a16_moe_mlp(x, up(ids), up(w), *bad, F, gc, out_dtype=F32)
    assert torch.isnan(got[0]).all()
    assert torch.equal(got[1:], want[1:])

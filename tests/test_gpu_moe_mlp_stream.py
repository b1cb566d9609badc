"""The routed 4-bit MLP where few pairs meet many experts (row blocks streamed past
the pairs' rows): rows of wider buffers, dirty workspaces, repeated calls, other
streams, graphs, and experts that a token names twice."""
import numpy as np
import pytest
import torch

import sparse_gemm_layers_amd as sg
from gpu_helpers import DEV, say
from test_gpu_moe_mlp import BF16, F32, layer, routing, run_and_check, up

pytestmark = pytest.mark.gpu

SIZES = [
    # T, E, k, D, F, gc: 16 < T k <= rows / 4 * E, rows of LDS 16, 8 and 4
    (40, 32, 2, 160, 96, 32), (12, 40, 3, 4096, 64, 32), (6, 40, 3, 8192, 32, 32),
]


def streamed(T, E, k, D, F):
    row = -(-max(D, F) // 128) * 256
    rows = next(r for r in (16, 8, 4) if r * row <= 79 * 1024)
    return 16 < T * k and 4 * T * k <= rows * E


@pytest.mark.parametrize("T,E,k,D,F,gc", SIZES)
def test_strides_workspace_and_repeats(T, E, k, D, F, gc):
    assert streamed(T, E, k, D, F)
    _, dev = layer(2, E, D, F, gc)
    ids, w = routing(5, T, E, k, 0.1)
    big = torch.full((T, D + 32), float("nan"), dtype=BF16, device=DEV)
    big[:, :D] = torch.randn((T, D), generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    need = sg.w4a16_moe_mlp_workspace(T, k, E, D, F)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((T, D + 8), 5.0, device=DEV)
    say(f"moe stream strides T{T} D{D}")
    y = sg.w4a16_moe_mlp(big[:, :D], up(ids), up(w), *dev, F, gc, y=out[:, :D], workspace=ws).clone()
    assert (out[:, D:] == 5).all() and (ws[need:] == 255).all()
    for _ in range(3):
        again = sg.w4a16_moe_mlp(big[:, :D].contiguous(), up(ids), up(w), *dev, F, gc, out_dtype=F32)
        assert torch.equal(y, again)


@pytest.mark.parametrize("T,E,k,D,F,gc", SIZES)
def test_padded_rows_against_the_oracle(T, E, k, D, F, gc):
    ids, w = routing(8, T, E, k, 0.1)
    say(f"moe stream oracle T{T} D{D}")
    for dtype in (F32, BF16):
        run_and_check(T, E, k, D, F, gc, dtype, ids, w)


@pytest.mark.parametrize("T,E,k", [(12, 40, 5), (40, 32, 3), (17, 64, 6)])
def test_an_expert_twice_in_a_token(T, E, k):
    D, F, gc = 128, 96, 32
    assert streamed(T, E, k, D, F)
    g = np.random.default_rng(T)
    ids = g.integers(-1, 3, (T, k)).astype(np.int32)
    w = g.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    say(f"moe stream duplicates T{T} k{k}")
    run_and_check(T, E, k, D, F, gc, F32, ids, w)


def test_another_stream_and_a_graph():
    T, E, k, D, F, gc = SIZES[0]
    _, dev = layer(3, E, D, F, gc)
    ids, w = (up(a) for a in routing(6, T, E, k))
    x = torch.zeros((T, D), dtype=BF16, device=DEV)
    gen = torch.Generator().manual_seed(4)
    x.copy_(torch.randn((T, D), generator=gen).to(BF16))
    want = sg.w4a16_moe_mlp(x, ids, w, *dev, F, gc)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        got = [sg.w4a16_moe_mlp(x, ids, w, *dev, F, gc) for _ in range(4)]
        with torch.cuda.graph(graph, stream=s):
            out = sg.w4a16_moe_mlp(x, ids, w, *dev, F, gc)
    torch.cuda.current_stream().wait_stream(s)
    for g in got:
        g.record_stream(torch.cuda.current_stream())
        assert torch.equal(g, want)
    for r in range(4):
        x.copy_(torch.randn((T, D), generator=gen).to(BF16))
        want = sg.w4a16_moe_mlp(x, ids, w, *dev, F, gc)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {r}"

"""examples/adapter_layer.py end to end, and its gradients."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def example(monkeypatch):
    monkeypatch.syspath_prepend(os.path.join(ROOT, "examples"))
    monkeypatch.setattr(sys, "argv", ["adapter_layer.py", "--tokens", "96"])
    import adapter_layer
    return adapter_layer


def test_adapter_layer_example(example):
    _, worst, losses = example.main()
    # three roundings to bf16 in a row (addends, h, y before its adapter) and y's own, on
    # each side: 8 half steps of 2^-8
    assert worst < 8 * 2.0 ** -8
    assert all(math.isfinite(v) for v in losses)


def plain(block, x, ids, deltas):
    """The block in 64 bits on the same weights, its adapters moved by deltas."""
    out = []
    for ad, (da, db) in zip(block.adapters(), deltas):
        a, b = ad.a.double() + da, ad.b.double() + db
        which = ids.long().clamp(min=0)
        on = ((ids >= 0) * ad.scale[which]).double()
        out.append((a[which], b[which], on))

    def add(v, i):
        a, b, on = out[i]
        return on[:, None] * (b @ (a @ v[:, :, None]))[..., 0]

    x = x.double()
    g = x @ block.gate.double().t() + add(x, 0)
    u = x @ block.up.double().t() + add(x, 1)
    h = torch.nn.functional.silu(g) * u
    return h @ block.down_t.double() + add(h, 2)


def test_adapter_layer_gradients(example):
    """The directional derivative of the loss along the adapters, against central
    differences of the block in 64 bits."""
    gen = torch.Generator(device=example.DEV).manual_seed(3)
    block = example.Block(128, 256, 3, 8, gen)
    x = torch.randn((40, 128), generator=gen, device=example.DEV).to(torch.bfloat16)
    ids = torch.randint(-1, 3, (40,), generator=gen, device=example.DEV, dtype=torch.int32)
    target = torch.randn((40, 128), generator=gen, device=example.DEV)
    _, _, grads = example.loss_and_grads(block, x, ids, target)

    def loss(t, ways):
        y = plain(block, x, ids, [(t * p, t * q) for p, q in ways])
        return 0.5 * (y - target.double()).square().sum().item()

    for i in range(3):
        # along the gradient itself: no cancellation between its elements
        ways = [(da.double() * (i == j), db.double() * (i == j)) for j, (da, db) in enumerate(grads)]
        size = math.sqrt(sum(p.square().sum().item() + q.square().sum().item() for p, q in ways))
        t = 1e-5 / size
        slope = (loss(t, ways) - loss(-t, ways)) / (2 * t)
        # |grad|^2 against grad . exact: at most ten roundings to bf16 (addends, h, y, err, base and dh,
        # dg, du, the inner factors) stand between, each off by 2^-8 of its value
        assert abs(slope - size ** 2) < 10 * 2.0 ** -8 * size ** 2

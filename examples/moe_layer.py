"""A mixture-of-experts layer on 4-bit weights, served and fine-tuned.

    python examples/moe_layer.py [--tokens T] [--experts E]

One layer as a model holds it: a 4-bit projection in front (a weight quantised by
``int4_quant_groupwise`` and packed once), the router's logits in fp32, the choice
of experts, and the routed gated MLP on 4-bit experts.  A prefill of T tokens and
then single tokens run through the same calls; the single-token step is captured
in a graph and replayed.  Then the router alone is fine-tuned for a few steps: the
experts' outputs enter the gradient of the routing weights, and
``moe_route_backward`` takes it to the logits.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import sparse_gemm_layers_amd as sg  # noqa: E402

DEV = "cuda:0"
GC = 128


class Linear4:
    """y = x . W^T on a packed 4-bit weight."""

    def __init__(self, w):
        self.n = w.shape[0]
        codes, scales = sg.int4_quant_groupwise(w, gc=GC)
        self.packed = sg.w4_pack(codes, scales, GC)

    def __call__(self, x, **kw):
        return sg.w4a16_gemm_groupwise_packed(x, self.packed, self.n, GC, **kw)


class Experts4:
    """E gated MLPs, each Wd (silu(Wg x) * (Wu x)), packed one after the other."""

    def __init__(self, gate, up, down):
        self.f = gate.shape[1]
        self.gate, self.up, self.down = (self._pack(w) for w in (gate, up, down))

    @staticmethod
    def _pack(w):
        each = [sg.int4_quant_groupwise(one, gc=GC) for one in w]
        return sg.w4_pack(torch.stack([c for c, _ in each]), torch.stack([s for _, s in each]), GC)

    def __call__(self, x, ids, weights, **kw):
        return sg.w4a16_moe_mlp(x, ids, weights, self.gate, self.up, self.down, self.f, GC, **kw)


class Layer:
    def __init__(self, d, f, e, k, gen):
        def w(*shape):
            return 0.02 * torch.randn(shape, generator=gen, device=DEV)

        self.k = k
        self.route = dict(score="sigmoid", renormalize=True, scale=2.5)
        self.groups = dict(n_group=4, topk_group=2, group_score="top2")
        self.proj = Linear4(w(d, d))
        self.router = w(e, d)                            # fp32: it is fine-tuned below
        self.balance = torch.zeros(e, device=DEV)
        self.experts = Experts4(w(e, f, d), w(e, f, d), w(e, d, f))

    def choose(self, h):
        logits = h.float() @ self.router.t()
        return (logits, *sg.moe_route(logits, self.k, bias=self.balance, **self.groups, **self.route))

    def __call__(self, x):
        h = x + self.proj(x)
        _, ids, weights = self.choose(h)
        return h + self.experts(h, ids, weights)


def tune_router(layer, x, target, steps, rate):
    """Gradient descent on the router for 1/2 |y - target|^2; the losses."""
    h = x + layer.proj(x)
    t, k = h.shape[0], layer.k
    one = torch.ones((t * k, 1), device=DEV)
    losses = []
    for _ in range(steps):
        logits, ids, weights = layer.choose(h)
        # each slot's expert by itself: the derivative of y with respect to its weight
        parts = layer.experts(h.repeat_interleave(k, 0), ids.reshape(-1, 1), one, out_dtype=torch.float32)
        parts = parts.reshape(t, k, -1)
        err = h.float() + (weights[:, :, None] * parts).sum(1) - target
        losses.append(0.5 * err.square().mean().item())
        dweights = (parts * err[:, None]).sum(-1) / err.numel()
        dlogits = sg.moe_route_backward(dweights, logits, ids, **layer.route)
        layer.router -= rate * (dlogits.t() @ h.float())
    return losses


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--experts", type=int, default=32)
    a = ap.parse_args()
    gen = torch.Generator(device=DEV).manual_seed(0)
    d, f, k = 1024, 512, 4
    layer = Layer(d, f, a.experts, k, gen)
    x = torch.randn((a.tokens, d), generator=gen, device=DEV).to(torch.bfloat16)

    y = layer(x)
    print(f"prefill of {a.tokens} tokens: |y| = {y.float().norm().item():.3f}")

    # a token at a time gives the prefill's rows up to the order of its sums
    token = x[:1].clone()
    layer(token)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        out = layer(token)
    torch.cuda.current_stream().wait_stream(side)
    worst = 0.0
    for t in range(min(4, a.tokens)):
        token.copy_(x[t:t + 1])
        graph.replay()
        worst = max(worst, ((out - y[t]).float().norm() / y[t].float().norm()).item())
    print(f"decoded from a graph: rows within {worst:.1e} of the prefill's")

    small = x[:64]
    target = layer(small).float()
    layer.router += 0.02 * torch.randn(layer.router.shape, generator=gen, device=DEV)
    losses = tune_router(layer, small, target, steps=20, rate=200.0)
    print(f"router fine-tuned: loss {losses[0]:.3e} -> {losses[-1]:.3e}")
    return worst, losses


if __name__ == "__main__":
    main()

"""A feed-forward block with low-rank adapters of many requests, served and fine-tuned.

    python examples/adapter_layer.py [--tokens T] [--adapters L]

The block is frozen: gate and up projections in bf16 (``gated_gemm``), the down
projection on a packed 4-bit weight.  Every request may bring its own adapter for each of
the three, and a batch mixes them: ``lora_gemm`` adds each token's.  A prefill of T
tokens and then single tokens run through the same calls; the single-token step is
captured in a graph and replayed, with another adapter each time.  Then the adapters
are fine-tuned for a few steps through ``gated_gemm_backward`` and
``lora_gemm_backward``; the frozen weights get no gradient, and tokens without an
adapter contribute none.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import sparse_gemm_layers_amd as sg  # noqa: E402

DEV = "cuda:0"
BF16 = torch.bfloat16
GC = 128


class Adapters:
    """L low-rank pairs of one projection: fp32 master weights and their bf16 copies."""

    def __init__(self, count, n, k, rank, gen):
        self.wa = torch.randn((count, rank, k), generator=gen, device=DEV) * k ** -0.5
        self.wb = torch.randn((count, n, rank), generator=gen, device=DEV) * 0.02
        self.scale = torch.full((count,), 2.0, device=DEV)
        self.refresh()

    def refresh(self):
        self.a, self.b = self.wa.to(BF16), self.wb.to(BF16)

    def __call__(self, x, ids, **kw):
        return sg.lora_gemm(x, ids, self.a, self.b, scale=self.scale, **kw)

    def backward(self, dy, x, ids, **kw):
        """dx on top of ``base``, and the pair's gradients in fp32."""
        return sg.lora_gemm_backward(dy, x, ids, self.a, self.b, scale=self.scale, grad_dtype=torch.float32, **kw)

    def step(self, da, db, rate):
        self.wa -= rate * da
        self.wb -= rate * db
        self.refresh()


class Block:
    """x -> Wd (silu(Wg x) * (Wu x)), with adapters on all three."""

    def __init__(self, d, f, count, rank, gen):
        def w(n, k):
            return torch.randn((n, k), generator=gen, device=DEV) * k ** -0.5

        self.d, self.gate, self.up = d, w(f, d).to(BF16), w(f, d).to(BF16)
        codes, scales = sg.int4_quant_groupwise(w(d, f), gc=GC)
        self.down = sg.w4_pack(codes, scales, GC)
        # what the packed weight stands for, for the input gradient of fine-tuning: the library has no
        # product with a packed weight's columns, so this costs the memory that 4 bits save
        eye = torch.eye(f, dtype=BF16, device=DEV)
        self.down_t = sg.w4a16_gemm_groupwise_packed(eye, self.down, d, GC)        # [F, D]
        self.on_gate, self.on_up, self.on_down = (Adapters(count, n, k, rank, gen) for n, k in ((f, d), (f, d), (d, f)))

    def adapters(self):
        return self.on_gate, self.on_up, self.on_down

    def __call__(self, x, ids, keep=False):
        out = sg.gated_gemm(x, self.gate, self.up, gate_add=self.on_gate(x, ids), up_add=self.on_up(x, ids), keep=keep)
        h = out[0] if keep else out
        y = sg.w4a16_gemm_groupwise_packed(h, self.down, self.d, GC)
        self.on_down(h, ids, base=y, y=y)                                           # in place
        return (y, *out) if keep else y

    def backward(self, dy, x, ids, h, g, u):
        """dx and [(da, db) of each projection's adapters]."""
        dh, *ddown = self.on_down.backward(dy, h, ids, base=dy @ self.down_t.t())
        dx, _, _, dg, du = sg.gated_gemm_backward(dh, x, self.gate, self.up, g=g, u=u, need_dw=False)
        dx, *dgate = self.on_gate.backward(dg, x, ids, base=dx, dx=dx)
        dx, *dup = self.on_up.backward(du, x, ids, base=dx, dx=dx)
        return dx, [dgate, dup, ddown]


def loss_and_grads(block, x, ids, target):
    """1/2 |y - target|^2 over the tokens, and the adapters' gradients."""
    y, h, g, u = block(x, ids, keep=True)
    err = y.float() - target
    dx, grads = block.backward(err.to(BF16), x, ids, h, g, u)
    return 0.5 * err.double().square().sum().item(), dx, grads


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--adapters", type=int, default=6)
    a = ap.parse_args()
    gen = torch.Generator(device=DEV).manual_seed(0)
    d, f, rank = 1024, 2048, 16
    block = Block(d, f, a.adapters, rank, gen)
    x = torch.randn((a.tokens, d), generator=gen, device=DEV).to(BF16)
    ids = torch.randint(-1, a.adapters, (a.tokens,), generator=gen, device=DEV, dtype=torch.int32)

    y = block(x, ids)
    print(f"prefill of {a.tokens} tokens over {a.adapters} adapters: |y| = {y.float().norm().item():.3f}")

    # a token at a time gives the prefill's rows up to the order of its sums
    token, mine = x[:1].clone(), ids[:1].clone()
    block(token, mine)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        out = block(token, mine)
    torch.cuda.current_stream().wait_stream(side)
    worst = 0.0
    for t in range(min(6, a.tokens)):
        token.copy_(x[t:t + 1])
        mine.copy_(ids[t:t + 1])
        graph.replay()
        worst = max(worst, ((out - y[t]).float().norm() / y[t].float().norm()).item())
    print(f"decoded from a graph: rows within {worst:.1e} of the prefill's")

    small, owner = x[:128], ids[:128]
    target = block(small, owner).float() + 0.3 * torch.randn((small.shape[0], d), generator=gen, device=DEV)
    losses = []
    for _ in range(5):
        loss, _, grads = loss_and_grads(block, small, owner, target)
        losses.append(loss)
        for ad, (da, db) in zip(block.adapters(), grads):
            ad.step(da, db, 1e-4)
    print(f"adapters fine-tuned: loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    return block, worst, losses


if __name__ == "__main__":
    main()

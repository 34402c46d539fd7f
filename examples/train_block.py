"""One gated transformer MLP block trained with activations kept in 8 bits and
compressed gradients, all through the library's calls.

    x -> layer norm -> up, gate (linear) -> silu(up) * gate -> down (linear) -> + x

Forward, per step: the norm's input, the linear layers' inputs and the gated
activation's inputs are saved as 8-bit checkpoints (1 1/32 bytes per value of a
row of 512 columns, instead of 2 in bf16).  Backward: every call reads those checkpoints and writes
its parameters' gradients in fp32 at their places of one flat gradient, which
the bucketed compressor (error feedback, Top-K 1 %, 8-bit QSGD) takes as it
lies.  The plain matrix products of the forward pass and of the input gradients
are torch.matmul.

    python examples/train_block.py [--steps N] [--tokens T] [--width D] [--hidden F]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from gradient_compression_ef_gb300 import gc  # noqa: E402

EPS = 1e-5


class Kept:
    """The 8-bit checkpoint of a [rows, cols] activation."""

    def __init__(self, rows, cols):
        self.codes = torch.empty(gc.ckpt_codes_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(gc.ckpt_scales_bytes(rows, cols), dtype=torch.uint8,
                                  device="cuda")

    def nbytes(self):
        return self.codes.numel() + self.scales.numel()


class Block:
    """Weights (fp32 masters, bf16 copies), one flat gradient, its compressor."""

    def __init__(self, tokens, width, hidden, seed=0, ratio=100):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        shapes = {"gamma": (width,), "beta": (width,), "up": (hidden, width),
                  "up_b": (hidden,), "gate": (hidden, width), "gate_b": (hidden,),
                  "down": (width, hidden), "down_b": (width,)}
        sizes = [int(torch.Size(s).numel()) for s in shapes.values()]
        total = sum(sizes)
        self.tokens, self.width, self.hidden = tokens, width, hidden
        self.master = torch.zeros(total, device="cuda")
        self.grad = torch.zeros(total, device="cuda")
        self.err = torch.zeros(total, device="cuda")
        self.dense = torch.zeros(total, device="cuda")
        self.weight, self.dweight, at = {}, {}, 0
        for (name, shape), n in zip(shapes.items(), sizes):
            w = self.master[at:at + n].view(shape)
            if len(shape) == 2:
                w.copy_(torch.randn(shape, generator=gen, device="cuda") * shape[1] ** -0.5)
            self.weight[name], self.dweight[name] = w, self.grad[at:at + n].view(shape)
            at += n
        self.weight["gamma"].fill_(1.0)

        # the compressor's plan: a bucket for each parameter tensor
        self.sizes, self.ks = sizes, [max(1, n // ratio) for n in sizes]
        self.ctx = gc.Context(max(sizes))
        self.ctx.set_buckets(self.sizes, self.ks)
        self.oi, self.oc, self.os = gc.bucket_offsets(self.ks, 8, 64)
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.idx = torch.empty(self.oi[-1], dtype=torch.int32, device="cuda")
        self.codes, self.scales = torch.empty(self.oc[-1], **u8), torch.empty(
            self.os[-1], device="cuda")
        self.ctx.reserve_scratch(max(
            gc.layernorm_scratch_bytes(tokens, width),
            gc.linear_wgrad_scratch_bytes(tokens, hidden, width, torch.bfloat16),
            gc.linear_wgrad_scratch_bytes(tokens, width, hidden, torch.bfloat16)))

        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.kept = {"x": Kept(tokens, width), "h": Kept(tokens, width),
                     "up": Kept(tokens, hidden), "gate": Kept(tokens, hidden),
                     "act": Kept(tokens, hidden)}
        self.h, self.act = torch.empty(tokens, width, **bf), torch.empty(tokens, hidden, **bf)
        self.mean, self.rstd = torch.empty(tokens, device="cuda"), torch.empty(tokens,
                                                                             device="cuda")
        self.dup, self.dgate = torch.empty(tokens, hidden, **bf), torch.empty(tokens, hidden, **bf)
        self.dx = torch.empty(tokens, width, **bf)

    def forward(self, x):
        w, k, ctx = self.weight, self.kept, self.ctx
        gc.layernorm_forward(ctx, x, w["gamma"], w["beta"], EPS, self.h, self.mean, self.rstd,
                             k["x"].codes, k["x"].scales)
        gc.ckpt_save(ctx, self.h, k["h"].codes, k["h"].scales)
        up = torch.addmm(w["up_b"].bfloat16(), self.h, w["up"].bfloat16().t())
        gate = torch.addmm(w["gate_b"].bfloat16(), self.h, w["gate"].bfloat16().t())
        gc.act_forward(ctx, "silu", up, self.act, k["up"].codes, k["up"].scales, gate,
                       k["gate"].codes, k["gate"].scales)
        gc.ckpt_save(ctx, self.act, k["act"].codes, k["act"].scales)
        return torch.addmm(w["down_b"].bfloat16(), self.act, w["down"].bfloat16().t()) + x

    def backward(self, dy, accumulate=False):
        """Fills (or adds to) the flat gradient; returns the input's."""
        w, d, k, ctx = self.weight, self.dweight, self.kept, self.ctx
        gc.linear_wgrad(ctx, dy, k["act"].codes, k["act"].scales, d["down"], d["down_b"],
                        accumulate)
        dact = dy @ w["down"].bfloat16()
        gc.act_backward(ctx, "silu", dact, self.dup, k["up"].codes, k["up"].scales, self.dgate,
                        k["gate"].codes, k["gate"].scales)
        gc.linear_wgrad(ctx, self.dup, k["h"].codes, k["h"].scales, d["up"], d["up_b"], accumulate)
        gc.linear_wgrad(ctx, self.dgate, k["h"].codes, k["h"].scales, d["gate"], d["gate_b"],
                        accumulate)
        dh = self.dup @ w["up"].bfloat16() + self.dgate @ w["gate"].bfloat16()
        gc.layernorm_backward(ctx, dh, None, w["gamma"], self.mean, self.rstd, self.dx,
                              d["gamma"], d["beta"], k["x"].codes, k["x"].scales, accumulate)
        return self.dx + dy

    def update(self, lr, step):
        """Compresses the flat gradient, rebuilds what a receiver would, steps."""
        gc.ef_topk_quant_buckets(self.ctx, self.grad, self.err, 8, 64, "stochastic", 1000, step,
                                 self.idx, self.codes, self.scales)
        at = 0
        for b, (n, k) in enumerate(zip(self.sizes, self.ks)):
            gc.topk_quant_aggregate(self.ctx, 1, k, self.idx[self.oi[b]:], self.codes[self.oc[b]:],
                                    self.scales[self.os[b]:], 8, 64, n, self.dense[at:at + n])
            at += n
        self.master.sub_(self.dense, alpha=lr)

    def kept_bytes(self):
        return sum(c.nbytes() for c in self.kept.values())


def train(steps=20, tokens=2048, width=512, hidden=1408, lr=20.0, seed=0, show=print):
    """Fits the block to a fixed random target; returns the losses."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)
    x = torch.randn(tokens, width, generator=gen, device="cuda").bfloat16()
    mix = torch.randn(width, width, generator=gen, device="cuda") * width ** -0.5
    target = torch.tanh(x.float() @ mix)
    block, losses = Block(tokens, width, hidden, seed), []
    bf16 = 2 * tokens * (2 * width + 3 * hidden)
    show("activations kept: %.1f MB in 8 bits, %.1f MB in bf16" % (block.kept_bytes() / 1e6,
                                                                  bf16 / 1e6))
    for step in range(steps):
        diff = block.forward(x).float() - target
        losses.append(float(diff.square().mean()))
        block.backward((2.0 * diff / diff.numel()).bfloat16())
        block.update(lr, step)
        if step % 5 == 0 or step == steps - 1:
            show("step %3d  loss %.5f" % (step, losses[-1]))
    block.ctx.check()
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--width", type=int, default=512)
    p.add_argument("--hidden", type=int, default=1408)
    a = p.parse_args()
    train(a.steps, a.tokens, a.width, a.hidden)

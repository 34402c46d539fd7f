"""One step of a small language model's layers through the library: embedding,
two RMS norms along a residual stream, a linear layer's weight gradient from 8
bits, the flat gradient they fill together, its compression with error
feedback, and the orthogonalised update; against 64-bit autograd on the same
numbers, and captured."""
import math

import pytest

from tests.gpu_helpers import torch_cuda

pytestmark = pytest.mark.gpu

EPS, PAD = 1e-5, -1


@pytest.fixture(scope="module")
def gc():
    torch_cuda()
    from gradient_compression_ef_gb300 import gc as binding
    return binding


class Step:
    """emb -> h1 -> norm -> linear -> + h1 = h2 -> norm; the loss is sum(r y2) + sum(q h2)."""

    def __init__(self, gc, ctx, tokens, vocab, width, seed=0):
        import torch
        self.gc, self.ctx = gc, ctx
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def rand(*shape, size=1.0):
            return size * torch.randn(*shape, generator=gen, device="cuda")

        def half(*shape):
            return torch.empty(*shape, dtype=torch.bfloat16, device="cuda")

        self.sizes = tokens, vocab, width
        self.scale = math.sqrt(width)
        self.ids = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
        self.ids[::9] = PAD
        self.ids[1::4] = 5  # one id more often than the others
        self.table = rand(vocab, width, size=0.02).bfloat16()
        self.w = rand(width, width, size=width ** -0.5).bfloat16()
        self.g1, self.g2 = 1 + rand(width, size=0.1), 1 + rand(width, size=0.1)
        self.r, self.q = rand(tokens, width, size=0.1).bfloat16(), rand(tokens, width, size=0.1).bfloat16()
        sizes = [vocab * width, width * width, width, width]
        self.flat = torch.zeros(sum(sizes), device="cuda")
        parts = torch.split(self.flat, sizes)
        self.dtable, self.dw = parts[0].view(vocab, width), parts[1].view(width, width)
        self.dg1, self.dg2 = parts[2], parts[3]
        self.err = torch.zeros_like(self.flat)
        self.k = self.flat.numel() // 50
        self.idx = torch.empty(self.k, dtype=torch.int32, device="cuda")
        self.val = torch.empty(self.k, device="cuda")
        self.total = torch.empty_like(self.flat)
        self.update = half(width, width)
        self.x, self.h1, self.y1, self.z, self.h2, self.y2, self.dh2, self.dy1, self.dx = (half(tokens, width) for _ in range(9))
        self.rstd1, self.rstd2 = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")

        def ckpt():
            return [torch.empty(gc.ckpt_codes_bytes(tokens, width), dtype=torch.uint8, device="cuda"),
                    torch.empty(gc.ckpt_scales_bytes(tokens, width), dtype=torch.uint8, device="cuda")]

        self.h1c, self.y1c, self.h2c = ckpt(), ckpt(), ckpt()
        ctx.reserve_scratch(max(gc.rmsnorm_scratch_bytes(tokens, width), gc.embedding_scratch_bytes(tokens, vocab, width),
                                gc.linear_wgrad_scratch_bytes(tokens, width, width, "bf16"),
                                gc.orthogonalize_scratch_bytes(width, width)))

    def gradient(self, accumulate=False):
        import torch
        gc, ctx = self.gc, self.ctx
        gc.embedding_forward(ctx, self.ids, self.table, self.scale, self.x, pad=PAD)
        gc.rmsnorm_forward(ctx, self.x, None, self.g1, EPS, self.h1, self.y1, self.rstd1, *self.h1c, *self.y1c)
        torch.matmul(self.y1, self.w.t(), out=self.z)
        gc.rmsnorm_forward(ctx, self.z, self.h1, self.g2, EPS, self.h2, self.y2, self.rstd2, *self.h2c)
        gc.rmsnorm_backward(ctx, self.r, self.q, None, self.g2, self.rstd2, self.dh2, self.dg2, *self.h2c,
                            accumulate=accumulate)
        gc.linear_wgrad(ctx, self.dh2, *self.y1c, self.dw, accumulate=accumulate)
        torch.matmul(self.dh2, self.w, out=self.dy1)
        gc.rmsnorm_backward(ctx, self.dy1, self.dh2, None, self.g1, self.rstd1, self.dx, self.dg1, *self.h1c,
                            accumulate=accumulate)
        gc.embedding_wgrad(ctx, self.dx, self.ids, self.scale, self.dtable, pad=PAD, accumulate=accumulate)

    def compress_and_update(self):
        gc, ctx = self.gc, self.ctx
        gc.ef_topk(ctx, self.flat, self.err, self.k, self.idx, self.val)
        gc.topk_aggregate(ctx, 1, self.k, self.idx, self.val, self.flat.numel(), self.total)
        first = self.dtable.numel()
        w = self.total[first:first + self.dw.numel()].view_as(self.dw)
        gc.orthogonalize(ctx, w, self.update, scale=0.2)
        return w


@pytest.mark.parametrize("tokens,vocab,width", [(600, 211, 256), (97, 40, 160), (2600, 900, 264)])
def test_step_against_autograd(gc, tokens, vocab, width):
    """8-bit checkpoints cost a relative error of up to 1/128 of a group's largest element, bf16 intermediates 2^-8
    each: a few percent of each gradient's norm, as for the block of layers."""
    import torch
    with gc.Context(1 << 20) as ctx:
        s = Step(gc, ctx, tokens, vocab, width)
        s.gradient()
        t, w, g1, g2 = (v.double().requires_grad_() for v in (s.table, s.w, s.g1, s.g2))
        some = (s.ids != PAD)[:, None]
        x = t[s.ids.clamp(min=0)] * s.scale * some

        def norm(h, g):
            return h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * g

        h2 = norm(x, g1) @ w.t() + x
        ((norm(h2, g2) * s.r.double()).sum() + (h2 * s.q.double()).sum()).backward()

        def rel(a, b):
            return float((a.double() - b).norm() / b.norm())

        for name, got, want in (("table", s.dtable, t.grad), ("w", s.dw, w.grad), ("g1", s.dg1, g1.grad), ("g2", s.dg2, g2.grad)):
            assert rel(got, want) < 0.04, name
        # a second micro-batch of the same tokens doubles it
        once = s.flat.clone()
        s.gradient(accumulate=True)
        assert float((s.flat - 2 * once).abs().max()) <= 1e-5 * float(once.abs().max())
        s.flat.copy_(once)

        # what is sent and what stays behind add up; the update is that of what was sent
        sent = s.compress_and_update()
        assert torch.equal(s.total + s.err, once)
        assert int((s.total != 0).sum()) <= s.k
        o = sent.double()
        o = o / (o.norm() + 1e-7)
        a, b, c = gc.QUINTIC
        for _ in range(5):
            m = o @ o.t()
            o = a * o + (b * m + c * (m @ m)) @ o
        # bf16: half a step of 2^-8 relative, and 2^-9.4 from the last step's operands
        assert float((s.update.double() - 0.2 * o).norm()) <= (2.0 ** -8 + 2.0 ** -9) * float((0.2 * o).norm())
        ctx.check()


def test_captured_step(gc):
    """The whole step as one graph gives the bits of the calls one by one."""
    import torch
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        with gc.Context(1 << 20, stream) as ctx:
            s = Step(gc, ctx, 300, 70, 192)
            s.gradient()
            s.compress_and_update()
            ctx.check()
            want = [v.clone() for v in (s.flat, s.total, s.update)]
            s.err.zero_()
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                s.gradient()
                s.compress_and_update()
            for _ in range(2):
                s.err.zero_()
                s.flat.fill_(7.0)
                s.update.zero_()
                graph.replay()
                torch.cuda.synchronize()
                for v, w in zip((s.flat, s.total, s.update), want):
                    assert torch.equal(v, w)
            ctx.check()

"""Orthogonalisation by Newton-Schulz products against its 64-bit reference:
single steps and whole runs, element types, tall, wide and odd sizes, strides,
slices at any element, in place, zeros, infinities, the ends of the range,
determinism, streams, capture, refusals.

Tolerances.  A product of 22-bit operands with fp32 sums is within
UNIT * |P| |Q| of P Q, element by element, with UNIT = 2^-18: 24 roundings
towards zero (2^-23 each) of a running sum between two read-outs, the rest
(the operands' 2^-22, the part lo lo that is left out, sums in registers) below
that.  Those bounds are carried through one step as they stand.  From step to
step an error grows at most by the largest slope of the polynomial, L (the
Lipschitz constant of X -> p(X) in the Frobenius norm).
"""
import numpy as np
import pytest

from oracle import stream as ref
from tests.gpu_helpers import torch_cuda

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -18
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
QUINTIC = (3.4445, -4.7750, 2.0315)
F32_QUINTIC = [float(np.float32(v)) for v in QUINTIC]


@pytest.fixture(scope="module")
def gc():
    torch_cuda()
    from gradient_compression_ef_gb300 import gc as binding
    return binding


@pytest.fixture(scope="module")
def ctx(gc):
    with gc.Context(0) as c:
        c.reserve_scratch(gc.orthogonalize_scratch_bytes(4200, 4200))
        yield c


def dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def slope(coefs, top=1.3):
    a, b, c = coefs
    x = np.linspace(0.0, top, 2001)
    return np.abs(a + 3 * b * x ** 2 + 5 * c * x ** 4).max()


def reference(g, coefs, eps, scale):
    """(result, Frobenius bound of its error) in binary64 on the GPU."""
    import torch
    x = g.double()
    x = x / (torch.linalg.norm(x) + eps)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t()
    err = 2.0 ** -21 * float(torch.linalg.norm(x))
    for a, b, c in coefs:
        gram = x @ x.t()
        ax, ag = x.abs(), gram.abs()
        eg = UNIT * (ax @ ax.t())
        poly = b * gram + c * (gram @ gram)
        poly.diagonal().add_(a)
        ep = abs(b) * eg + abs(c) * (eg @ ag + ag @ eg + UNIT * (ag @ ag)) + 2.0 ** -21 * poly.abs()
        ex = UNIT * (poly.abs() @ ax) + ep @ ax
        x = poly @ x
        err = slope((a, b, c)) * err + float(torch.linalg.norm(ex + 2.0 ** -21 * x.abs()))
    return scale * (x.t() if tall else x), abs(scale) * err


def check(got, want, err, out):
    import torch
    assert not bool(got.isnan().any())
    # the rounding to the output's type, and of the smallest fp16 numbers
    room = err + float(torch.linalg.norm(U[out] * want)) + 2.0 ** -25 * want.numel() ** 0.5
    off = float(torch.linalg.norm(got.double() - want))
    assert off <= room, "off %g, bound %g, norm %g" % (off, room, float(torch.linalg.norm(want)))


def update(seed, m, n, dtype="f32", size=1e-3):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    g = torch.randn(m, n, generator=gen, device="cuda")
    k = max(1, min(m, n) // 8)
    g += torch.randn(m, k, generator=gen, device="cuda") @ torch.randn(k, n, generator=gen,
                                                                       device="cuda")
    return (g * size).to(dt(dtype))


SIZES = [(1, 1), (1, 7), (5, 3), (8, 8), (16, 64), (64, 64), (65, 130), (130, 65), (128, 64), (255, 256),
         (257, 511), (1000, 300), (300, 1000), (513, 513), (700, 2051), (2051, 700), (1, 5000), (5000, 1),
         (1025, 1537), (64, 6000)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("steps", [1, 2, 5])
def test_against_the_reference(gc, ctx, m, n, steps):
    import torch
    g = update(m + n, m, n)
    out = torch.full((m, n), 7.0, device="cuda")
    gc.orthogonalize(ctx, g, out, steps=steps, coefs=QUINTIC, eps=1e-7, scale=0.7)
    want, err = reference(g, [F32_QUINTIC] * steps, 1e-7, 0.7)
    check(out, want, err, "f32")
    ctx.check()


def test_the_reference_agrees_with_the_oracle(gc, ctx):
    g = update(1, 40, 70)
    want, _ = reference(g, [F32_QUINTIC] * 3, 1e-7, 2.0)
    o = ref.orthogonalize(g.double().cpu().numpy(), [F32_QUINTIC] * 3, 1e-7, 2.0)
    assert np.allclose(want.cpu().numpy(), o, rtol=0, atol=1e-12)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n", [(96, 200), (333, 150)])
@pytest.mark.parametrize("pad", [0, 3, 16])
def test_types_and_strides(gc, ctx, dtype, out, m, n, pad):
    import torch
    buf = torch.full((m, n + pad), float("nan"), dtype=dt(dtype), device="cuda")
    g = buf[:, :n]
    g.copy_(update(7, m, n, dtype, 1.0))
    obuf = torch.full((m, n + pad), 7.0, dtype=dt(out), device="cuda")
    gc.orthogonalize(ctx, g, obuf[:, :n], steps=3)
    want, err = reference(g, [F32_QUINTIC] * 3, 1e-7, 1.0)
    check(obuf[:, :n], want, err, out)
    assert bool((obuf[:, n:] == 7.0).all())


@pytest.mark.parametrize("m,n", [(60, 77), (77, 60), (300, 512), (520, 264)])
def test_permuted_diagonal_keeps_its_digits(gc, ctx, m, n):
    """With one value per row and column every sum has one term: what is left
    is the roundings of the operands (2^-22 each) and of a few fp32 steps, at
    most 2^-19 of the terms of a step's polynomial, 10 |x| together."""
    import torch
    k = min(m, n)
    r = np.random.default_rng(m)
    d = r.uniform(0.1, 1.0, k) * r.choice([-1.0, 1.0], k)
    rows, cols = r.permutation(m)[:k], r.permutation(n)[:k]
    g = torch.zeros(m, n, device="cuda")
    g[torch.from_numpy(rows), torch.from_numpy(cols)] = torch.from_numpy(d).float().cuda()
    for steps in (1, 5):
        out = torch.empty(m, n, device="cuda")
        gc.orthogonalize(ctx, g, out, steps=steps, eps=0.0)
        x = g.double()[torch.from_numpy(rows), torch.from_numpy(cols)].cpu().numpy()
        x = x / np.linalg.norm(x)
        err = 2.0 ** -21 * np.abs(x)
        a, b, c = F32_QUINTIC
        for _ in range(steps):
            err = np.abs(a + 3 * b * x ** 2 + 5 * c * x ** 4) * err * 1.01 + 10.0 * 2.0 ** -19 * np.abs(x)
            x = a * x + b * x ** 3 + c * x ** 5
        got = out[torch.from_numpy(rows), torch.from_numpy(cols)].double().cpu().numpy()
        assert (np.abs(got - x) <= err + 2.0 ** -34).all(), (np.abs(got - x) / err).max()
        off = out.clone()
        off[torch.from_numpy(rows), torch.from_numpy(cols)] = 0.0
        assert not bool(off.any())


def test_slices_at_any_element_and_in_place(gc, ctx):
    import torch
    m, n = 75, 131
    g = update(3, m, n)
    want = torch.empty(m, n, device="cuda")
    gc.orthogonalize(ctx, g, want)
    for at in range(4):
        flat = torch.full((m * n + 8,), 3.0, device="cuda")
        view = flat[at:at + m * n].view(m, n)
        view.copy_(g)
        gc.orthogonalize(ctx, view, view)
        assert torch.equal(view, want)
        assert bool((flat[:at] == 3.0).all()) and bool((flat[at + m * n:] == 3.0).all())
    half = torch.zeros(m * n + 8, dtype=torch.bfloat16, device="cuda")
    for at in (0, 1, 5):
        view = half[at:at + m * n].view(m, n)
        gc.orthogonalize(ctx, g, view)
        assert torch.equal(view, want.bfloat16())


def test_coefficients_for_each_step(gc, ctx):
    import torch
    coefs = [(3.4445, -4.7750, 2.0315), (2.5, -2.0, 0.5), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)]
    g = update(5, 120, 333)
    out = torch.empty_like(g)
    gc.orthogonalize(ctx, g, out, steps=4, coefs=coefs, eps=1e-7)
    want, err = reference(g, [[float(np.float32(v)) for v in c] for c in coefs], 1e-7, 1.0)
    check(out, want, err, "f32")


@pytest.mark.parametrize("m,n", [(50, 90), (90, 50)])
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-12, 1e12, 1e30, 3e36])
def test_magnitudes(gc, ctx, m, n, size):
    """X_0 does not depend on g's size but for roundings (1e-38: of g itself)."""
    import torch
    g = update(9, m, n, size=1.0) * size
    out = torch.empty_like(g)
    gc.orthogonalize(ctx, g, out, steps=3, eps=0.0)
    want, err = reference(g, [F32_QUINTIC] * 3, 0.0, 1.0)
    check(out, want, err, "f32")


@pytest.mark.parametrize("m,n", [(40, 300), (300, 40), (1, 1)])
def test_zeros_and_non_finite(gc, ctx, m, n):
    import torch
    for eps in (0.0, 1e-7):
        out = torch.full((m, n), 7.0, device="cuda")
        gc.orthogonalize(ctx, torch.zeros(m, n, device="cuda"), out, eps=eps)
        assert bool((out == 0).all())
    for bad in (float("inf"), -float("inf"), float("nan")):
        for steps in (1, 5):
            g = update(2, m, n)
            g[m // 2, n // 3] = bad
            gc.orthogonalize(ctx, g, out, steps=steps)
            assert bool(out.isnan().all())
    ctx.check()


def test_empty(gc, ctx):
    import torch
    for m, n in ((0, 5), (5, 0), (0, 0)):
        t = torch.empty(m, n, device="cuda")
        gc.orthogonalize(ctx, t, t)
    ctx.check()


@pytest.mark.parametrize("m,n", [(4096, 4096), (4200, 1500), (1000, 20000)])
def test_many_tiles(gc, m, n):
    """More tiles than pairs of SMs, and ragged ones among them."""
    import torch
    with gc.Context(0) as c:
        c.reserve_scratch(gc.orthogonalize_scratch_bytes(m, n))
        g = update(11, m, n)
        out = torch.empty_like(g)
        gc.orthogonalize(c, g, out, steps=2)
        want, err = reference(g, [F32_QUINTIC] * 2, 1e-7, 1.0)
        check(out, want, err, "f32")
        again = torch.empty_like(g)
        gc.orthogonalize(c, g, again, steps=2)
        assert torch.equal(out, again)
        c.check()


@pytest.mark.parametrize("m,n", [(120, 250), (900, 600)])
def test_same_bits_other_stream_and_capture(gc, m, n):
    import torch
    g = update(4, m, n)
    stream = torch.cuda.Stream()
    with gc.Context(0, stream) as c:
        c.reserve_scratch(gc.orthogonalize_scratch_bytes(m, n))
        one, two = torch.empty_like(g), torch.empty_like(g)
        stream.wait_stream(torch.cuda.current_stream())
        gc.orthogonalize(c, g, one)
        c.check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            gc.orthogonalize(c, g, two)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(one, two)


def test_back_to_back(gc, ctx):
    """Calls in a row on one context, of two sizes in turn: each gives what it gives alone."""
    import torch
    gs = [update(1, 200, 300), update(2, 600, 120)]
    alone = []
    for g in gs:
        o = torch.empty_like(g)
        gc.orthogonalize(ctx, g, o)
        ctx.check()
        alone.append(o)
    outs = [[torch.empty_like(g) for g in gs] for _ in range(20)]
    for pair in outs:
        for g, o in zip(gs, pair):
            gc.orthogonalize(ctx, g, o)
    ctx.check()
    for pair in outs:
        assert all(torch.equal(o, a) for o, a in zip(pair, alone))


def test_refusals(gc, ctx):
    import torch
    g = torch.zeros(6, 8, device="cuda")
    for kw in (dict(steps=0), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(gc.GCError) as e:
            gc.orthogonalize(ctx, g, g, **kw)
        assert e.value.status == gc.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        gc.orthogonalize(ctx, g, g[:5])
    with pytest.raises(ValueError):
        gc.orthogonalize(ctx, g, g, steps=3, coefs=[(1.0, 2.0, 3.0)] * 2)
    with pytest.raises(ValueError):
        gc.orthogonalize(ctx, g.t(), g.t())
    with pytest.raises(TypeError):
        gc.orthogonalize(ctx, g.double(), g)
    with gc.Context(0) as bare:
        with pytest.raises(gc.GCError) as e:
            gc.orthogonalize(bare, g, g)
        assert e.value.status == gc.ERR_WORKSPACE


@pytest.mark.parametrize("m,n,steps", [(128, 38912, 2), (128, 38913, 2), (129, 257, 2), (20, 90, 32), (20, 90, 33)])
def test_both_sides_of_the_narrow_kernel(gc, m, n, steps):
    """Narrow matrices run in one kernel up to a width, a length and a number of steps."""
    import torch
    coefs = [(1.5, -0.5, 0.0)] * steps
    with gc.Context(0) as c:
        c.reserve_scratch(gc.orthogonalize_scratch_bytes(m, n))
        g = update(13, m, n)
        for x in (g, g.t().contiguous()):
            out = torch.empty_like(x)
            gc.orthogonalize(c, x, out, steps=steps, coefs=coefs)
            want, err = reference(x, coefs, 1e-7, 1.0)
            check(out, want, err, "f32")
        c.check()


@pytest.mark.parametrize("m,n", [(150, 400), (400, 150), (700, 700)])
@pytest.mark.parametrize("dtype,size", [("bf16", 1e-38), ("bf16", 1e-20), ("bf16", 1e36), ("f16", 1e-5), ("f16", 1e4),
                                        ("f32", 1e-38), ("f32", 1e36)])
@pytest.mark.parametrize("steps", [1, 3])
def test_magnitudes_of_wider_matrices(gc, ctx, m, n, dtype, size, steps):
    """Two orders of magnitude between the elements, at the ends of the types' ranges."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(m)
    spread = 10.0 ** (-2.0 * torch.rand(m, n, generator=gen, device="cuda"))
    g = (torch.randn(m, n, generator=gen, device="cuda").clamp(-4, 4) * spread * size).to(dt(dtype))
    for out in ("f32", "bf16"):
        o = torch.empty(m, n, dtype=dt(out), device="cuda")
        gc.orthogonalize(ctx, g, o, steps=steps, eps=0.0, scale=1.3)
        want, err = reference(g, [F32_QUINTIC] * steps, 0.0, 1.3)
        # a bf16 result's last step takes X and B with 11 bits: 2^-12 of each entry, grown by the largest slope of the
        # polynomial or, from B, as it is; 2^-11 + 4 2^-12 = 2^-9.4 of the norm at most
        check(o, want, err + (2.0 ** -9.4 * float(torch.linalg.norm(want)) if out == "bf16" else 0.0), out)
    ctx.check()


@pytest.mark.parametrize("m,n", [(150, 400), (400, 150)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_zeros_and_non_finite_of_wider_matrices(gc, ctx, m, n, dtype):
    import torch
    out = torch.full((m, n), 7.0, dtype=dt(dtype), device="cuda")
    for eps in (0.0, 1e-7):
        gc.orthogonalize(ctx, torch.zeros(m, n, dtype=dt(dtype), device="cuda"), out, eps=eps)
        assert bool((out == 0).all())
    for bad in (float("inf"), -float("inf"), float("nan")):
        g = update(2, m, n, dtype, 1.0)
        g[m // 2, n // 3] = bad
        gc.orthogonalize(ctx, g, out)
        assert bool(out.isnan().all())
    # far below eps: X_0 is 0 to all its bits
    gc.orthogonalize(ctx, update(2, m, n, dtype, 1e-4 if dtype == "f16" else 1e-30), out, eps=1e30)
    assert bool((out == 0).all())
    ctx.check()


@pytest.mark.parametrize("m,n,dtype", [(64, 3000, "f32"), (3000, 100, "bf16"), (700, 1300, "bf16"), (1300, 260, "f16")])
def test_capture_of_every_kernel(gc, m, n, dtype):
    """The kernels whose blocks wait for one another, and tiles in parts, captured and replayed."""
    import torch
    stream = torch.cuda.Stream()
    g = update(4, m, n, dtype, 1.0)
    with gc.Context(0, stream) as c:
        c.reserve_scratch(gc.orthogonalize_scratch_bytes(m, n))
        one, two = torch.empty_like(g), torch.empty_like(g)
        stream.wait_stream(torch.cuda.current_stream())
        gc.orthogonalize(c, g, one)
        c.check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            gc.orthogonalize(c, g, two)
        for _ in range(3):
            two.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(one, two)
        c.check()


def test_two_streams_at_once(gc):
    """Contexts of their own on streams of their own, every kernel in flight next to another's."""
    import torch
    sizes = [(64, 6000), (128, 20000), (500, 900), (100, 9000)]
    gs = [update(k, m, n) for k, (m, n) in enumerate(sizes)]
    streams = [torch.cuda.Stream() for _ in sizes]
    ctxs = [gc.Context(0, s) for s in streams]
    try:
        for c, (m, n) in zip(ctxs, sizes):
            c.reserve_scratch(gc.orthogonalize_scratch_bytes(m, n))
        alone = []
        torch.cuda.synchronize()
        for c, g in zip(ctxs, gs):
            o = torch.empty_like(g)
            gc.orthogonalize(c, g, o)
            c.check()
            alone.append(o)
        outs = [torch.empty_like(g) for g in gs]
        torch.cuda.synchronize()
        for _ in range(30):
            for c, g, o in zip(ctxs, gs, outs):
                gc.orthogonalize(c, g, o)
        for c, o, a in zip(ctxs, outs, alone):
            c.check()
            assert torch.equal(o, a)
    finally:
        for c in ctxs:
            c.close()

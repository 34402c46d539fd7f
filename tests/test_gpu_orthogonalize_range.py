"""Orthogonalisation at the ends of what its iterates hold: results in bf16
against those in fp32, updates of few directions or far below eps, elements of very
different sizes.

Tolerances.  A result in bf16 is the fp32 one rounded once: the same bits.  Of
few directions: the bounds of the products.
Where the polynomial is a X (coefficients (a, 0, 0), or singular values so small
that b A X is below every rounding), each sum has one term: its roundings are the
operands' (2^-22 each: B's diagonal, X), at most 12 of the running sum towards
zero (2^-23 each), what is put back for them (3 2^-25), and a few in registers:
STEP = 2^-18 of the value for each step, together with the rounding of X_0.  Below
that the second plane ends, at 2^-48 of the power of two that holds the largest
singular value: fp16's smallest step is 2^-24; the planes hold X_0 2^12, the second
one 2^11 more; half a step.
"""
import numpy as np
import pytest

from tests.gpu_helpers import torch_cuda
from tests.test_gpu_orthogonalize import F32_QUINTIC, check, dt, reference, update

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -18


@pytest.fixture(scope="module")
def gc():
    torch_cuda()
    from gradient_compression_ef_gb300 import gc as binding
    return binding


@pytest.fixture(scope="module")
def ctx(gc):
    with gc.Context(0) as c:
        c.reserve_scratch(gc.orthogonalize_scratch_bytes(1300, 1300))
        yield c


def rank(m, n, k, dtype):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(m + k)
    g = torch.randn(m, k, generator=gen, device="cuda") @ torch.randn(k, n, generator=gen, device="cuda")
    return (1e-2 * g).to(dt(dtype))


@pytest.mark.parametrize("m,n", [(100, 300), (150, 400), (800, 1300), (1300, 260)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("k", [1, 4, None])
def test_a_bf16_result_is_the_fp32_one_rounded(gc, ctx, m, n, dtype, k):
    import torch
    g = update(m, m, n, dtype, 1e-2) if k is None else rank(m, n, k, dtype)
    for steps in (1, 5):
        whole = torch.empty(m, n, device="cuda")
        half = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        gc.orthogonalize(ctx, g, whole, steps=steps, scale=0.3)
        gc.orthogonalize(ctx, g, half, steps=steps, scale=0.3)
        assert torch.equal(half, whole.bfloat16())
    ctx.check()


@pytest.mark.parametrize("m,n", [(90, 300), (300, 512), (520, 264)])
@pytest.mark.parametrize("k", [1, 4])
def test_few_directions(gc, ctx, m, n, k):
    g = rank(m, n, k, "f32")
    out = g.clone()
    for steps in (1, 2, 5):
        gc.orthogonalize(ctx, g, out, steps=steps)
        want, err = reference(g, [F32_QUINTIC] * steps, 1e-7, 1.0)
        check(out, want, err, "f32")


@pytest.mark.parametrize("m,n", [(60, 77), (77, 60), (128, 2000), (300, 512), (520, 264), (1024, 1024)])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "f32"), ("f16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("ratio", [1e-2, 1e-4, 1e-6, 1e-13, 1e-25])
def test_far_below_eps(gc, ctx, m, n, dtype, out, ratio):
    import torch
    g = update(m, m, n, dtype, 1e-2)
    eps = float(np.float32(float(torch.linalg.norm(g.double())) / ratio))
    for steps in (1, 3, 5):
        o = torch.empty(m, n, dtype=dt(out), device="cuda")
        gc.orthogonalize(ctx, g, o, steps=steps, eps=eps, scale=0.5 / ratio)
        want, _ = reference(g, [F32_QUINTIC] * steps, eps, float(np.float32(0.5 / ratio)))
        off = float(torch.linalg.norm(o.double() - want) / torch.linalg.norm(want))
        assert off <= (steps + 1) * STEP + (2.0 ** -8 if out == "bf16" else 0.0), off
    ctx.check()


@pytest.mark.parametrize("m,n", [(64, 90), (300, 512), (520, 264)])
def test_growing_out_of_the_depths(gc, ctx, m, n):
    """From 1e-9 of eps to singular values of order one: the iterates' power of two follows them.  While they are
    small an error stays what it is of them; above, the slopes (at most |a| where the values grow by |a|) hold it."""
    import torch
    g = update(m, m, n, size=1e-2)
    eps = float(np.float32(float(torch.linalg.norm(g.double())) * 1e9))
    steps = 20
    o = torch.empty_like(g)
    gc.orthogonalize(ctx, g, o, steps=steps, eps=eps)
    want, _ = reference(g, [F32_QUINTIC] * steps, eps, 1.0)
    off = float(torch.linalg.norm(o.double() - want) / torch.linalg.norm(want))
    assert float(torch.linalg.norm(want)) > 0.3 * min(m, n) ** 0.5
    x, _ = reference(g, [F32_QUINTIC] * 14, eps, 1.0)
    x14 = float(torch.linalg.norm(x))
    assert x14 < 0.2
    # 14 steps of STEP each in front, grown by |a| at most in each of the last six; these as the reference bounds
    # them for such an X (divided by a norm of 1: |X| + 1 - |X|)
    _, bound = reference(x, [F32_QUINTIC] * 6, 1.0 - x14, 1.0)
    assert off <= (15 * STEP * x14 * 3.4445 ** 6 + bound) / float(torch.linalg.norm(want)) + 2.0 ** -24, off


@pytest.mark.parametrize("m,n", [(64, 90), (120, 1000), (300, 512), (520, 264)])
@pytest.mark.parametrize("what", ["row", "column", "element"])
def test_beside_something_dominant(gc, ctx, m, n, what):
    """One row, column or element 10^8 times the others: these keep their digits.  The terms of a step are at most
    |a| + 2 |b| + 3 |c| = 19 times X, each within STEP, where the small ones grow by |a|: 6 STEP of them.  What the
    large ones are off after a step (19 STEP) comes into the small ones through A and A A in the next: (2 |b| + 4 |c|)
    19 / |a| = 97 STEP."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    g = torch.randn(m, n, generator=gen, device="cuda")
    rest = torch.ones(m, n, dtype=torch.bool, device="cuda")
    if what == "row":
        g[m // 3] *= 1e8
        rest[m // 3] = False
    elif what == "column":
        g[:, n // 3] *= 1e8
        rest[:, n // 3] = False
    else:
        g[m // 3, n // 3] = 1e9
        rest[m // 3] = False
        rest[:, n // 3] = False
    for steps, room in ((1, 6 * STEP), (2, 110 * STEP)):
        o = torch.empty_like(g)
        gc.orthogonalize(ctx, g, o, steps=steps)
        want, _ = reference(g, [F32_QUINTIC] * steps, 1e-7, 1.0)
        off = float(torch.linalg.norm((o.double() - want)[rest]) / torch.linalg.norm(want[rest]))
        x0 = g.double() / torch.linalg.norm(g.double())
        floor = 2.0 ** -48 / float(x0[rest].square().mean().sqrt())
        assert off <= room + steps * floor, (off, floor)
    ctx.check()


@pytest.mark.parametrize("m,n", [(64, 90), (120, 1000), (300, 512), (520, 264)])
@pytest.mark.parametrize("dtype,bits", [("f32", 46), ("bf16", 36), ("f16", 24)])
def test_every_element_by_itself(gc, ctx, m, n, dtype, bits):
    """With the polynomial 1 X the result is X_0, element by element: of elements down to 2^-bits of the largest.
    A 16-bit matrix is held in one plane, to 2^-39 of its largest element; an fp32 one in two, to 2^-48."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(m)
    spread = torch.exp2(-bits * torch.rand(m, n, generator=gen, device="cuda", dtype=torch.float64))
    g = (spread * torch.sign(torch.randn(m, n, generator=gen, device="cuda"))).to(dt(dtype))
    o = torch.empty(m, n, device="cuda")
    x0 = g.double() / torch.linalg.norm(g.double())
    top = float(x0.abs().max())
    for steps in (1, 4):
        gc.orthogonalize(ctx, g, o, steps=steps, coefs=(1.0, 0.0, 0.0), eps=0.0)
        room = (steps + 1) * STEP * x0.abs() + steps * 2.0 ** -48
        if dtype != "f32" and min(m, n) > 128:
            room += 2.0 ** -39 * top
        assert bool(((o.double() - x0).abs() <= room).all()), float(((o.double() - x0).abs() / room).max())
    ctx.check()

"""Results of an orthogonalisation in bf16 against those in fp32, of updates of
full rank and of few directions.

A result in bf16 is the fp32 one rounded once: the same bits.  The fp32 one is
compared with the 64-bit reference within the bounds of its products.
"""
import pytest

from tests.gpu_helpers import torch_cuda
from tests.test_gpu_orthogonalize import F32_QUINTIC, check, dt, reference, update

pytestmark = pytest.mark.gpu


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

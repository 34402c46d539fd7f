"""Embedding and RMS norm at the ends of the range: subnormal sums added to a
table, tables without rows, infinite parameters.

Sums of a few equal values and one addition to what is there are compared with
the same fp32 operations on the host, bit for bit (subnormals kept).
"""
import numpy as np
import pytest

from tests.gpu_helpers import torch_cuda
from tests.test_gpu_backward import ckpt, f64, matrix, out_matrix, pad_untouched
from tests.test_gpu_rmsnorm import EPS, same_ckpt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gc():
    torch_cuda()
    from gradient_compression_ef_gb300 import gc as binding
    return binding


@pytest.fixture(scope="module")
def ctx(gc):
    with gc.Context(0) as c:
        c.reserve_scratch(64 << 20)
        yield c


@pytest.mark.parametrize("tokens,vocab", [(3, 5), (200, 40), (1000, 7), (1000, 900), (9000, 3000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols,pad", [(64, 0), (33, 0), (300, 4), (4096, 0)])
def test_added_subnormals(gc, ctx, tokens, vocab, dtype, cols, pad):
    """Subnormal sums, and subnormal values in the rows that they are added to."""
    import torch
    r = np.random.default_rng(tokens + cols)
    scale = 2.0 ** -120 if dtype == "f16" else 1.0
    dy, _, _ = matrix(r.integers(-8, 9, (tokens, cols)) * (2.0 ** -20 if dtype == "f16" else 2.0 ** -133), dtype, pad)
    ids = torch.from_numpy(r.integers(0, vocab, tokens)).cuda()
    first, _ = out_matrix(vocab, cols, "f32", pad)
    gc.embedding_wgrad(ctx, dy, ids, scale, first)
    sums = first.cpu().numpy()
    assert ((sums != 0) & (np.abs(sums) < 2.0 ** -126)).any()
    base = (r.integers(-2 ** 20, 2 ** 20, (vocab, cols)) * 2.0 ** -149).astype(np.float32)
    base[:, ::3] = r.integers(-3, 4, base[:, ::3].shape) * np.float32(2.0 ** -126)
    d, buf = out_matrix(vocab, cols, "f32", pad)
    d.copy_(torch.from_numpy(base))
    gc.embedding_wgrad(ctx, dy, ids, scale, d, accumulate=True)
    used = np.zeros((vocab, 1), bool)
    used[ids.cpu().numpy()] = True
    want = np.where(used, base + sums, base)
    got = d.cpu().numpy()
    assert np.array_equal(got, want), "%d differ" % int((got != want).sum())
    pad_untouched(buf, cols)
    ctx.check()


@pytest.mark.parametrize("tokens", [3, 300, 9000])
def test_ids_of_a_table_without_rows(gc, ctx, tokens):
    """Every id that is not padding is outside it: the gradient's call says so too."""
    import torch
    ids = torch.full((tokens,), 4, device="cuda")
    table = torch.empty(0, 8, device="cuda")
    y = torch.ones(tokens, 8, device="cuda")
    for accumulate in (False, True):
        gc.embedding_wgrad(ctx, y, ids, 1.0, table, accumulate=accumulate)
        with pytest.raises(gc.GCError) as e:
            ctx.check()
        assert e.value.status == gc.ERR_DEVICE_CHECK
        gc.embedding_wgrad(ctx, y, ids, 1.0, table, pad=4, accumulate=accumulate)
        ctx.check()
    gc.embedding_forward(ctx, ids, table, 1.0, y)
    assert bool((y == 0).all())
    with pytest.raises(gc.GCError):
        ctx.check()


@pytest.mark.parametrize("rows,cols", [(3, 40), (300, 200), (5, 700), (5, 4100), (300, 4099), (300, 4096), (200, 11008),
                                       (4, 20001)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ptype", ["f32", "bf16", "f16"])
def test_infinite_parameters(gc, ctx, rows, cols, dtype, ptype):
    """y is infinite, with h's sign times gamma's, where gamma is; NaN where h is 0 or gamma NaN; elsewhere what it is
    without such parameters."""
    import torch
    r = np.random.default_rng(cols)
    v = r.standard_normal((rows, cols))
    v[:, 0] = 0.0
    x, _, _ = matrix(v, dtype, 3 if cols % 2 else 0)
    pt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[ptype]
    gamma = torch.from_numpy(1.0 + 0.3 * r.standard_normal(cols)).to(pt).cuda()
    plain, _ = out_matrix(rows, cols, dtype)
    rstd = torch.empty(rows, device="cuda")
    gc.rmsnorm_forward(ctx, x, None, gamma, EPS, None, plain, rstd)
    inf = float("inf")
    bad = {0: inf, 1: inf, cols // 2: -inf, cols - 2: inf, cols - 1: float("nan"), cols // 3: -inf}
    for c, b in bad.items():
        gamma[c] = b
    y, _ = out_matrix(rows, cols, dtype)
    yc = ckpt(rows, cols)
    gc.rmsnorm_forward(ctx, x, None, gamma, EPS, None, y, rstd, None, None, *yc)
    want = plain.clone()
    for c, b in bad.items():
        want[:, c] = x[:, c] * b
    assert bool(want[:, 0].isnan().all()) and bool(want[:, 1].isinf().all())
    assert torch.equal(y.isnan(), want.isnan())
    assert torch.equal(y.nan_to_num(0.0, inf, -inf), want.nan_to_num(0.0, inf, -inf))
    same_ckpt(yc, f64(y))
    ctx.check()

"""RMS norm behind the residual's addition against its 64-bit reference: sums
and outputs in 8 bits bit for bit, strides, odd sizes, every kernel's widths,
empty and non-finite rows, offsets past 32 bits, accumulation, determinism,
streams, capture, refusals.

Tolerances are bounds on rounding, not fits: u is half an ulp of the output
type; fp32 work in front of it is bounded by counting its roundings (at most
128 in a chain everywhere below, so 2^-17 of the terms that are added).
"""
import numpy as np
import pytest

from oracle import backward as ckpt_ref
from oracle import stream as ref
from tests.gpu_helpers import torch_cuda
from tests.test_gpu_backward import (CHAIN, TINY, U, acts, ckpt, close, f64, matrix, out_matrix,
                                     pad_untouched)

pytestmark = pytest.mark.gpu

EPS = 1e-5
# one lane to several units per lane, a warp per row, a block per row, two and
# four units per thread, rows wider than a block holds
SHAPES = [(1, 1), (3, 8), (2, 33), (9, 255), (17, 513), (5, 1000), (33, 1024), (40, 1027), (2, 4096),
          (21, 4099), (3, 8195), (2, 11008), (5, 16385), (1, 16384), (3, 20001)]


@pytest.fixture(scope="module")
def gc():
    torch_cuda()
    from gradient_compression_ef_gb300 import gc as binding
    return binding


@pytest.fixture(scope="module")
def ctx(gc):
    with gc.Context(0) as c:
        c.reserve_scratch(gc.rmsnorm_scratch_bytes(4096, 20001))
        yield c


def params(r, cols, dtype):
    import torch
    if dtype is None:
        return None, None
    g = torch.from_numpy((1.0 + 0.3 * r.standard_normal(cols)).astype(np.float32)).cuda()
    g = g.to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype])
    return g, f64(g)


def forward(gc, ctx, x, res, gamma, pad, whole=True):
    import torch
    rows, cols = x.shape
    dtype = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[x.dtype]
    h, hbuf = out_matrix(rows, cols, dtype, pad)
    y, ybuf = out_matrix(rows, cols, dtype, pad)
    rstd = torch.full((rows,), 7.0, device="cuda")
    hc, yc = ckpt(rows, cols), ckpt(rows, cols)
    gc.rmsnorm_forward(ctx, x, res, gamma, EPS, h, y if whole else None, rstd, *hc, *yc)
    pad_untouched(hbuf, cols)
    pad_untouched(ybuf, cols)
    return h, y, rstd, hc, yc


def same_ckpt(got, values):
    codes, b = ckpt_ref.encode(values)
    assert np.array_equal(got[0].cpu().numpy(), codes)
    assert np.array_equal(got[1].cpu().numpy()[:, :b.shape[1]], b)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("pad,ptype,with_res", [(0, "f32", True), (3, "bf16", True),
                                                (16, None, True), (0, "f16", False)])
def test_forward_and_backward(gc, ctx, dtype, rows, cols, pad, ptype, with_res):
    import torch
    r = np.random.default_rng(rows * 31 + cols + pad)
    x, _, _ = matrix(acts(r, rows, cols), dtype, pad)
    res = matrix(acts(r, rows, cols), dtype, 0 if pad == 16 else pad)[0] if with_res else None
    gamma, gv = params(r, cols, ptype)
    h, y, rstd, hc, yc = forward(gc, ctx, x, res, gamma, pad)
    want = (x.float() + res.float()).to(x.dtype) if with_res else x
    assert torch.equal(h, want)
    hv = f64(want)
    want_y, want_rstd = ref.rmsnorm_forward(hv, gv, EPS)
    close(f64(rstd), want_rstd, CHAIN * want_rstd, "rstd")
    close(f64(y), want_y, (CHAIN + U[dtype]) * np.abs(want_y) + TINY[dtype], "y")
    same_ckpt(hc, hv)
    same_ckpt(yc, f64(y))

    # 8 bits alone: the same bytes
    _, _, rstd2, _, yc2 = forward(gc, ctx, x, res, gamma, pad, whole=False)
    assert torch.equal(rstd, rstd2)
    groups = -(-cols // 32)
    assert torch.equal(yc[0], yc2[0]) and torch.equal(yc[1][:, :groups], yc2[1][:, :groups])

    dy, dyv, _ = matrix(1e-2 * r.standard_normal((rows, cols)), dtype, pad)
    dres, drv, _ = matrix(1e-2 * r.standard_normal((rows, cols)), dtype, 5 if pad else 0)
    for whole in (True, False):
        kept = hv if whole else ckpt_ref.restored(hv)
        for with_dres in (True, False):
            dx, dxbuf = out_matrix(rows, cols, dtype, pad)
            dgamma = torch.full((cols,), 7.0, device="cuda")
            gc.rmsnorm_backward(ctx, dy, dres if with_dres else None, h if whole else None, gamma,
                                rstd, dx, dgamma, *((None, None) if whole else hc))
            wdx, wdg, sdx, sdg = ref.rmsnorm_backward(dyv, drv if with_dres else None, kept, gv,
                                                      f64(rstd))
            close(f64(dx), wdx, CHAIN * sdx + U[dtype] * np.abs(wdx) + TINY[dtype], "dx")
            close(f64(dgamma), wdg, CHAIN * sdg + TINY["f32"], "dgamma")
            pad_untouched(dxbuf, cols)
    ctx.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(2500, 96), (1300, 700), (900, 4096), (700, 9000)])
def test_many_rows(gc, ctx, dtype, rows, cols):
    """Several rows per team of threads: what is loaded ahead, the column sums of many blocks."""
    import torch
    r = np.random.default_rng(rows)
    x, _, _ = matrix(acts(r, rows, cols), dtype)
    res, _, _ = matrix(acts(r, rows, cols), dtype)
    gamma, gv = params(r, cols, "f32")
    h, y, rstd, hc, yc = forward(gc, ctx, x, res, gamma, 0)
    hv = f64(h)
    want_y, want_rstd = ref.rmsnorm_forward(hv, gv, EPS)
    close(f64(rstd), want_rstd, CHAIN * want_rstd, "rstd")
    close(f64(y), want_y, (CHAIN + U[dtype]) * np.abs(want_y) + TINY[dtype], "y")
    same_ckpt(hc, hv)
    same_ckpt(yc, f64(y))
    dy, dyv, _ = matrix(1e-2 * r.standard_normal((rows, cols)), dtype)
    flat = torch.full((cols + 9,), 3.0, device="cuda")
    got = []
    for accumulate in (False, True):
        dx, _ = out_matrix(rows, cols, dtype)
        gc.rmsnorm_backward(ctx, dy, dy, None, gamma, rstd, dx, flat[5:5 + cols], *hc,
                            accumulate=accumulate)
        got.append((dx.clone(), flat[5:5 + cols].clone()))
    wdx, wdg, sdx, sdg = ref.rmsnorm_backward(dyv, dyv, ckpt_ref.restored(hv), gv, f64(rstd))
    close(f64(got[0][0]), wdx, CHAIN * sdx + U[dtype] * np.abs(wdx) + TINY[dtype], "dx")
    close(f64(got[0][1]), wdg, CHAIN * sdg, "dgamma")
    assert torch.equal(got[0][0], got[1][0])
    assert torch.equal(got[1][1], got[0][1] + got[0][1])  # the same sum, added once
    assert bool((flat[:5] == 3.0).all()) and bool((flat[5 + cols:] == 3.0).all())
    ctx.check()


def test_gradient_by_differences(gc, ctx):
    """dx is the slope of sum(dy * y) + sum(dres * h) along a direction: the
    forward call's outputs at h +- t v, in fp32.  The difference's own error: the
    outputs' rounding at either end, CHAIN of the sum of |dy y|, and the third
    derivative's t^3 / 3 of a few times that sum."""
    import torch
    r = np.random.default_rng(5)
    rows, cols, t = 4, 300, 2.0 ** -6
    x = r.standard_normal((rows, cols)).astype(np.float32)
    v = r.standard_normal((rows, cols)).astype(np.float32)
    dyn, drn = r.standard_normal((rows, cols)), r.standard_normal((rows, cols))
    gamma, gv = params(r, cols, "f32")
    dy, dyv, _ = matrix(dyn, "f32")
    dres, drv, _ = matrix(drn, "f32")
    hm, h0, _ = matrix(x, "f32")
    _, y, rstd, _, _ = forward(gc, ctx, hm, None, gamma, 0)
    dx, _ = out_matrix(rows, cols, "f32")
    gc.rmsnorm_backward(ctx, dy, dres, hm, gamma, rstd, dx)
    ends = []
    for s in (t, -t):
        h, hv, _ = matrix(x + np.float32(s) * v, "f32")
        ends.append(((dyv * f64(forward(gc, ctx, h, None, gamma, 0)[1])).sum(axis=1)
                     + (drv * hv).sum(axis=1), hv))
    step = ends[0][1] - ends[1][1]  # as rounded
    slope = (f64(dx) * step).sum(axis=1)
    size = (np.abs(dyv * f64(y)).sum(axis=1))
    tol = 2 * CHAIN * size + 16.0 * t ** 3 * size
    close(slope, ends[0][0] - ends[1][0], tol, "slope")


@pytest.mark.parametrize("cols", [40, 4100, 20001])
def test_empty_and_non_finite_rows(gc, ctx, cols):
    import torch
    rows = 6
    x = np.random.default_rng(1).standard_normal((rows, cols)).astype(np.float32)
    x[0] = 0.0
    x[1, 3], x[2, cols - 1], x[3, 0] = np.inf, np.nan, -np.inf
    m, v, _ = matrix(x, "f32", 1)
    h, y, rstd, hc, yc = forward(gc, ctx, m, None, None, 1)
    assert float(rstd[0]) == pytest.approx(EPS ** -0.5, rel=1e-6) and bool((y[0] == 0).all())
    assert bool(torch.isfinite(y[4:]).all())
    assert float(rstd[1]) == 0.0 and bool(y[1, 3].isnan()) and bool((y[1, :3] == 0).all())
    assert bool(y[2].isnan().all()) and bool(rstd[2].isnan())
    same_ckpt(hc, v)
    same_ckpt(yc, f64(y))
    dx, _ = out_matrix(rows, cols, "f32")
    dgamma = torch.empty(cols, device="cuda")
    dy, dyv, _ = matrix(np.ones((rows, cols)), "f32")
    gc.rmsnorm_backward(ctx, dy, None, None, None, rstd, dx, dgamma, *hc)
    assert bool(torch.isfinite(dx[4:]).all()) and bool(dx[2].isnan().all())
    assert bool(torch.isfinite(dx[0]).all()) and bool(dgamma.isnan().any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_sizes(gc, ctx, dtype):
    import torch
    for rows, cols in ((0, 8), (3, 0), (0, 0)):
        m, _ = out_matrix(rows, cols, dtype)
        c = ckpt(rows, cols)
        gc.rmsnorm_forward(ctx, m, m, None, EPS, None, m, torch.empty(rows, device="cuda"), *c, *c)
        for accumulate, want in ((True, 7.0), (False, 0.0 if rows == 0 else 7.0)):
            dgamma = torch.full((cols,), 7.0, device="cuda")
            gc.rmsnorm_backward(ctx, m, None, m, None, torch.empty(rows, device="cuda"), m, dgamma,
                                accumulate=accumulate)
            assert bool((dgamma == want).all())
    ctx.check()


def test_offsets_past_32_bits(gc, ctx):
    """More than 2^32 bytes from the first row to the last, checkpoints past 2^31."""
    import torch
    rows, cols, ld = 70001, 40, 32776
    buf = torch.zeros(rows, ld, dtype=torch.bfloat16, device="cuda")
    x = buf[:, :cols]
    x.copy_(torch.randn(rows, cols, device="cuda"))
    y = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    gc.rmsnorm_forward(ctx, x, x, None, EPS, None, y, rstd)
    want = (x.float() * 2).bfloat16().float()
    want = want * torch.rsqrt(want.square().mean(1, keepdim=True) + EPS)
    assert float((y.float() - want).abs().max()) <= 2.0 ** -7 * float(want.abs().max())
    dx = buf[:, 48:48 + cols]
    gc.rmsnorm_backward(ctx, y, None, x, None, rstd, dx)
    n = x.double() * rstd.double()[:, None]
    d = y.double()
    w = rstd.double()[:, None] * (d - n * (d * n).mean(1, keepdim=True))
    size = (rstd.double()[:, None] * (d.abs() + n.abs() * (d * n).abs().mean(1, keepdim=True)))
    assert bool(((dx.double() - w).abs() <= (CHAIN + U["bf16"]) * size + TINY["bf16"]).all())
    del buf, x, dx
    torch.cuda.empty_cache()


def test_same_bits_other_stream_and_capture(gc):
    import torch
    r = np.random.default_rng(2)
    rows, cols = 700, 4099
    x, _, _ = matrix(acts(r, rows, cols), "bf16", 1)
    res, _, _ = matrix(acts(r, rows, cols), "bf16")
    gamma, _ = params(r, cols, "bf16")
    dy, _, _ = matrix(r.standard_normal((rows, cols)), "bf16", 3)
    stream = torch.cuda.Stream()
    with gc.Context(0, stream) as c:
        c.reserve_scratch(gc.rmsnorm_scratch_bytes(rows, cols))

        def call(o):
            gc.rmsnorm_forward(c, x, res, gamma, EPS, o["h"], o["y"], o["rstd"], *o["hc"], *o["yc"])
            gc.rmsnorm_backward(c, dy, res, None, gamma, o["rstd"], o["dx"], o["dgamma"], *o["hc"])

        def outputs():
            return {"h": out_matrix(rows, cols, "bf16")[0], "y": out_matrix(rows, cols, "bf16")[0],
                    "rstd": torch.empty(rows, device="cuda"), "hc": ckpt(rows, cols),
                    "yc": ckpt(rows, cols), "dx": out_matrix(rows, cols, "bf16")[0],
                    "dgamma": torch.empty(cols, device="cuda")}

        one, two = outputs(), outputs()
        stream.wait_stream(torch.cuda.current_stream())
        call(one)
        c.check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call(two)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        for k in ("h", "y", "rstd", "dx", "dgamma"):
            assert torch.equal(one[k], two[k]), k
        assert torch.equal(one["yc"][0], two["yc"][0]) and torch.equal(one["hc"][0], two["hc"][0])


def test_refusals(gc, ctx):
    import torch
    x, _ = out_matrix(4, 64, "bf16")
    rstd, g = torch.empty(4, device="cuda"), torch.empty(64, device="cuda")
    c = ckpt(4, 64)
    ok = dict(x=x, res=x, gamma=g, eps=EPS, h=None, y=x, rstd=rstd)

    def status(exc=gc.GCError, fn=gc.rmsnorm_forward, base=ok, extra=(), **kw):
        with pytest.raises(exc) as e:
            fn(ctx, *{**base, **kw}.values(), *extra)
        return getattr(e.value, "status", None)

    assert status(y=None) == gc.ERR_INVALID_ARG                      # no output of y
    assert status(eps=-1.0) == gc.ERR_INVALID_ARG
    assert status(eps=float("nan")) == gc.ERR_INVALID_ARG
    assert status(extra=(c[0], None)) == gc.ERR_INVALID_ARG          # half a checkpoint
    odd = torch.empty(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 64)
    assert status(res=odd) == gc.ERR_ALIGNMENT
    status(ValueError, res=out_matrix(4, 65, "bf16")[0])
    status(ValueError, y=out_matrix(4, 64, "f16")[0])
    status(ValueError, gamma=g[:63])
    status(ValueError, rstd=rstd[:3])
    status(TypeError, x=x.double(), res=None, y=x.double())
    back = dict(dy=x, dres=None, h=x, gamma=g, rstd=rstd, dx=x, dgamma=g)
    assert status(fn=gc.rmsnorm_backward, base=back, extra=c) == gc.ERR_INVALID_ARG  # both
    assert status(fn=gc.rmsnorm_backward, base=back, h=None) == gc.ERR_INVALID_ARG   # neither
    assert status(fn=gc.rmsnorm_backward, base=back, dres=odd) == gc.ERR_ALIGNMENT
    with gc.Context(0) as bare:
        with pytest.raises(gc.GCError) as e:
            gc.rmsnorm_backward(bare, *back.values())
        assert e.value.status == gc.ERR_WORKSPACE
        gc.rmsnorm_backward(bare, x, None, x, g, rstd, out_matrix(4, 64, "bf16")[0])  # no dgamma
        bare.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(200, 600), (153, 1056), (311, 4099), (460, 4096), (170, 11008), (155, 13800),
                                       (155, 15800)])
@pytest.mark.parametrize("pad,ptype,with_res", [(0, "f32", True), (3, "bf16", False), (1, None, True)])
def test_more_rows_than_multiprocessors(gc, ctx, dtype, rows, cols, pad, ptype, with_res):
    """Rows through the ring of stages: the same checks as above."""
    test_forward_and_backward(gc, ctx, dtype, rows, cols, pad, ptype, with_res)


@pytest.mark.parametrize("cols", [40, 700, 4100])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_non_finite_rows_stay_alone(gc, ctx, cols, dtype):
    """Among many rows: an infinity, a NaN and zeros change no other row."""
    import torch
    rows = 400
    r = np.random.default_rng(cols)
    x = r.standard_normal((rows, cols)).astype(np.float32)
    clean, _, _ = matrix(x, dtype, 1)
    x[7] = 0.0
    x[190, 3], x[191, cols - 1], x[399, 0] = np.inf, np.nan, -np.inf
    bad = [190, 191, 399]
    m, _, _ = matrix(x, dtype, 1)
    outs = [forward(gc, ctx, a, None, None, 1) for a in (clean, m)]
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[bad + [7]] = False
    assert torch.equal(outs[0][1][keep], outs[1][1][keep])
    assert bool((outs[1][1][7] == 0).all())
    for b in bad:
        assert bool(outs[1][1][b].isnan().any())
    dy, _, _ = matrix(r.standard_normal((rows, cols)), dtype)
    dxs = []
    for h, _, rstd, hc, _ in outs:
        for whole in (True, False):
            dx, _ = out_matrix(rows, cols, dtype)
            gc.rmsnorm_backward(ctx, dy, dy, h if whole else None, None, rstd, dx, None, *((None, None) if whole else hc))
            dxs.append(dx)
    for a, b in ((dxs[0], dxs[2]), (dxs[1], dxs[3])):
        assert torch.equal(a[keep], b[keep])
        assert bool(b[191].isnan().all()) and bool(torch.isfinite(b[7]).all())
    ctx.check()

"""The calls that fill the flat gradient against their 64-bit reference:
8-bit checkpoints (bit for bit), activation functions, layer norm, linear
weight gradients; strides, odd sizes, empty and non-finite rows, sizes past
32-bit offsets, accumulation, determinism, streams, capture, refusals.

Tolerances are bounds on rounding, not fits: u is half an ulp of the output
type; fp32 work in front of it is bounded by counting its roundings (at most
128 in a chain everywhere below, so 2^-17 of the terms that are added).
"""
import numpy as np
import pytest

from oracle import backward as ref
from tests.gpu_helpers import torch_cuda

pytestmark = pytest.mark.gpu

U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}
CHAIN = 2.0 ** -17
EPS = 1e-5


@pytest.fixture(scope="module")
def gc():
    torch_cuda()
    from gradient_compression_ef_gb300 import gc as binding
    return binding


@pytest.fixture(scope="module")
def ctx(gc):
    with gc.Context(0) as c:
        c.reserve_scratch(256 << 20)
        yield c


def _dt(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def matrix(a, dtype, pad=0, fill=float("nan")):
    """A device matrix [rows, cols] inside a buffer whose extra columns hold
    `fill`; also its exact values as float64."""
    import torch
    a = np.asarray(a, np.float32)
    rows, cols = a.shape
    buf = torch.full((rows, cols + pad), fill, dtype=_dt(torch, dtype), device="cuda")
    m = buf[:, :cols]
    m.copy_(torch.from_numpy(a))
    return m, m.double().cpu().numpy(), buf


def out_matrix(rows, cols, dtype, pad=0):
    import torch
    buf = torch.full((rows, cols + pad), 7.0, dtype=_dt(torch, dtype), device="cuda")
    return buf[:, :cols], buf


def ckpt(rows, cols):
    import torch
    return (torch.full((rows, ref.codes_pitch(cols)), 0xEE, dtype=torch.uint8, device="cuda"),
            torch.full((rows, ref.scales_pitch(cols)), 0xEE, dtype=torch.uint8, device="cuda"))


def device_ckpt(codes, b):
    """Device copies of reference codes and scale bytes; the scale rows'
    padding holds 255 (NaN), which no call may use."""
    import torch
    rows, ng = b.shape
    s = np.full((rows, -(-ng // 16) * 16), 255, np.uint8)
    s[:, :ng] = b
    return torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda()


def f64(t):
    return t.double().cpu().numpy()


def close(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(want)), what + ": NaN at other places"
    fine = ~np.isnan(want)
    bad = np.abs(got - want) > np.broadcast_to(tol, want.shape)
    bad &= fine
    assert not bad.any(), "%s: %d outside, first %s got %r want %r tol %r" % (
        what, bad.sum(), np.argwhere(bad)[0], got[bad][0], want[bad][0],
        np.broadcast_to(tol, want.shape)[bad][0])


def pad_untouched(buf, cols):
    assert bool((buf[:, cols:] == 7.0).all())


def acts(r, rows, cols, scale=1.0):
    x = r.standard_normal((rows, cols)) * np.exp(r.standard_normal((1, cols)))
    x[r.random(rows) < 0.1] = 0.0
    return (x * scale).astype(np.float32)


SHAPES = [(1, 1), (1, 33), (3, 32), (5, 31), (7, 100), (2, 513), (64, 4096), (17, 4099),
          (300, 65), (2, 11008)]


# --- checkpoint ----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("pad", [0, 3, 16])
def test_checkpoint_bit_for_bit(gc, ctx, dtype, rows, cols, pad):
    r = np.random.default_rng(rows * 7 + cols + pad)
    x, xv, _ = matrix(acts(r, rows, cols), dtype, pad)
    codes, scales = ckpt(rows, cols)
    gc.ckpt_save(ctx, x, codes, scales)
    want, b = ref.encode(xv)
    assert np.array_equal(codes.cpu().numpy(), want)
    assert np.array_equal(scales.cpu().numpy()[:, :b.shape[1]], b)
    out, buf = out_matrix(rows, cols, dtype, pad)
    gc.ckpt_restore(ctx, codes, scales, out)
    assert np.array_equal(f64(out), ref.decode(want, b, cols))
    pad_untouched(buf, cols)


def test_checkpoint_edges_of_the_format(gc, ctx):
    rows = [np.zeros(40), np.full(40, 127.5), np.linspace(-127.9, 127.9, 40),
            np.arange(40) / 2.0 - 10, np.full(40, 2.0 ** -120), np.full(40, 2.0 ** -121),
            np.full(40, 1e-42), np.full(40, 2.0 ** 126 * 1.99), np.full(40, -2.0 ** 127)]
    special = np.ones((6, 40))
    special[0, 3], special[1, 35], special[2, 0] = np.inf, -np.inf, np.nan
    special[3, 39], special[4, 32] = -np.nan, 3.4e38
    special[5, 1] = -0.0
    x, xv, _ = matrix(np.concatenate([np.array(rows), special]), "f32")
    codes, scales = ckpt(*x.shape)
    gc.ckpt_save(ctx, x, codes, scales)
    want, b = ref.encode(xv)
    assert np.array_equal(codes.cpu().numpy(), want)
    assert np.array_equal(scales.cpu().numpy()[:, :2], b)
    for dtype in ("f32", "bf16"):
        out, _ = out_matrix(*x.shape, dtype)
        gc.ckpt_restore(ctx, codes, scales, out)
        close(f64(out), ref.decode(want, b, 40), 0.0, dtype)


def test_checkpoint_every_finite_half(gc, ctx):
    bits = np.arange(0x7C00, dtype=np.uint16).view(np.float16).astype(np.float32)
    x = np.stack([bits, np.roll(bits, 1), -np.roll(bits, 700)], axis=1)
    x = np.concatenate([x, np.zeros((x.shape[0], 29), np.float32)], axis=1)
    d, xv, _ = matrix(x, "f16")
    codes, scales = ckpt(*d.shape)
    gc.ckpt_save(ctx, d, codes, scales)
    out, _ = out_matrix(*d.shape, "f16")
    gc.ckpt_restore(ctx, codes, scales, out)
    assert np.array_equal(f64(out), ref.restored(xv))


def test_offsets_past_32_bits(gc, ctx):
    """Rows 2^24 elements apart: the last ones lie past 2^32 bytes and 2^31
    elements."""
    import torch
    rows, cols, ld = 160, 65, 1 << 24
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.view(rows, ld)[:, :cols]
    r = np.random.default_rng(0)
    x.copy_(torch.from_numpy(acts(r, rows, cols)))
    xv = f64(x)
    codes, scales = ckpt(rows, cols)
    gc.ckpt_save(ctx, x, codes, scales)
    assert np.array_equal(codes.cpu().numpy(), ref.encode(xv)[0])
    gamma = torch.ones(cols, device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    y = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    gc.layernorm_forward(ctx, x, gamma, None, EPS, y, mean, rstd)
    want, m, _ = ref.layernorm(xv, None, None, EPS)
    close(f64(y), want, U["bf16"] * np.abs(want) + 1e-4, "y")
    dw = torch.empty(cols, cols, device="cuda")
    gc.linear_wgrad(ctx, x, codes, scales, dw)
    xs = ref.restored(xv)
    close(f64(dw), xv.T @ xs, (rows / 8 + 64) * 2.0 ** -23 * (np.abs(xv).T @ np.abs(xs)), "dw")
    del buf


# --- activation functions ------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["gelu", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (5, 31, 1), (7, 100, 0), (3, 513, 5),
                                           (64, 4096, 0), (33, 4097, 0), (9, 1024, 8)])
def test_activation(gc, ctx, dtype, kind, gated, rows, cols, pad):
    r = np.random.default_rng(rows + cols)
    x, xv, _ = matrix(acts(r, rows, cols), dtype, pad)
    y, ybuf = out_matrix(rows, cols, dtype, pad)
    codes, scales = ckpt(rows, cols)
    gate = gv = gcodes = gscales = None
    if gated:
        gate, gv, _ = matrix(acts(r, rows, cols), dtype, pad)
        gcodes, gscales = ckpt(rows, cols)
    gc.act_forward(ctx, kind, x, y, codes, scales, gate, gcodes, gscales)
    f, _ = ref.act(kind, xv)
    g = gv if gated else np.ones_like(xv)
    # f: at most 8 roundings relative to |x| (2^-21 |x|)
    close(f64(y), f * g, U[dtype] * np.abs(f * g) + 2.0 ** -21 * np.abs(xv * g) + TINY[dtype], "y")
    pad_untouched(ybuf, cols)
    assert np.array_equal(codes.cpu().numpy(), ref.encode(xv)[0])
    if gated:
        assert np.array_equal(gcodes.cpu().numpy(), ref.encode(gv)[0])
    # the same without a checkpoint
    y2, _ = out_matrix(rows, cols, dtype, pad)
    gc.act_forward(ctx, kind, x, y2, gate=gate)
    assert bool((y2 == y).all())

    dy, dyv, _ = matrix(r.standard_normal((rows, cols)), dtype, pad)
    dx, dxbuf = out_matrix(rows, cols, dtype, pad)
    dgate, dgbuf = out_matrix(rows, cols, dtype, pad) if gated else (None, None)
    gc.act_backward(ctx, kind, dy, dx, codes, scales, dgate, gcodes, gscales)
    xs = ref.restored(xv)
    fs, ds = ref.act(kind, xs)
    gs = ref.restored(gv) if gated else np.ones_like(xs)
    want = dyv * gs * ds
    # f': at most 16 roundings of terms up to 1 + |x| phi(x) < 1.25 (2^-19 in all)
    close(f64(dx), want, U[dtype] * np.abs(want) + 2.0 ** -19 * np.abs(dyv * gs) + TINY[dtype],
          "dx")
    pad_untouched(dxbuf, cols)
    if gated:
        close(f64(dgate), dyv * fs,
              U[dtype] * np.abs(dyv * fs) + 2.0 ** -21 * np.abs(dyv * xs) + TINY[dtype], "dgate")
        pad_untouched(dgbuf, cols)


@pytest.mark.parametrize("kind", ["gelu", "silu"])
def test_activation_over_the_whole_range(gc, ctx, kind):
    x = np.concatenate([np.linspace(-40, 40, 8001), -np.exp(np.linspace(-80, 80, 500)),
                        np.exp(np.linspace(-80, 80, 500)), [0.0, -0.0]])
    x = np.pad(x, (0, -x.size % 32)).reshape(-1, 32)
    d, xv, _ = matrix(x, "f32")
    y, _ = out_matrix(*x.shape, "f32")
    gc.act_forward(ctx, kind, d, y)
    f, _ = ref.act(kind, xv)
    close(f64(y), f, U["f32"] * np.abs(f) + 2.0 ** -21 * np.abs(xv) + TINY["f32"], "y")
    # far left both functions go to zero: no more than 1e-6 there
    assert np.abs(f64(y))[(xv < -20) & (xv > -1e4)].max() <= 1e-6


@pytest.mark.parametrize("kind", ["gelu", "silu"])
def test_activation_lets_non_finite_values_through(gc, ctx, kind):
    import torch
    x = np.ones((3, 40), np.float32)
    x[0, 3], x[1, 36], x[2, 0] = np.inf, np.nan, -np.inf
    d, _, _ = matrix(x, "bf16")
    y, _ = out_matrix(3, 40, "bf16")
    codes, scales = ckpt(3, 40)
    gc.act_forward(ctx, kind, d, y, codes, scales)
    yv = f64(y)
    assert yv[0, 3] == np.inf and np.isnan(yv[1, 36]) and not np.isfinite(yv[2, 0])
    assert np.isfinite(np.delete(yv[0], 3)).all()
    dy, _, _ = matrix(np.ones((3, 40)), "bf16")
    dx, _ = out_matrix(3, 40, "bf16")
    gc.act_backward(ctx, kind, dy, dx, codes, scales)
    dxv = f64(dx)
    assert np.isnan(dxv[0, :32]).all() and np.isfinite(dxv[0, 32:]).all()
    assert np.isfinite(dxv[1, :32]).all() and np.isnan(dxv[1, 32:]).all()
    torch.cuda.synchronize()


# --- layer norm ----------------------------------------------------------------------------------

NORM_SHAPES = [(1, 1, 0), (1, 4096, 0), (3, 33, 2), (40, 100, 0), (700, 1024, 0), (33, 1025, 0),
               (5, 2049, 7), (350, 4096, 0), (19, 4099, 0), (320, 5000, 8), (9, 11008, 0),
               (7, 16384, 0), (310, 16385, 0), (5, 40000, 0), (1, 70001, 0)]


def _norm_case(rows, cols, dtype, pad, offset=0.0):
    r = np.random.default_rng(rows * 31 + cols)
    return r, matrix(acts(r, rows, cols) + np.float32(offset), dtype, pad)


def _norm_tol(xv, mean, rstd, gamma, y, dtype):
    a = np.abs(xv).mean(axis=1, keepdims=True)
    n = np.abs((xv - mean[:, None]) * rstd[:, None])
    # the mean's error shifts the row and enters the variance squared
    return U[dtype] * np.abs(y) + CHAIN * (np.abs(gamma) * (rstd[:, None] * (a + np.abs(xv)) + n)
                                           + 1e-3) + TINY[dtype]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols,pad", NORM_SHAPES)
@pytest.mark.parametrize("keep", [True, False])
def test_layernorm(gc, ctx, dtype, rows, cols, pad, keep):
    import torch
    r, (x, xv, _) = _norm_case(rows, cols, dtype, pad)
    gamma = (1 + 0.2 * r.standard_normal(cols)).astype(np.float32)
    beta = (0.2 * r.standard_normal(cols)).astype(np.float32)
    gd, bd = torch.from_numpy(gamma).cuda(), torch.from_numpy(beta).cuda()
    y, ybuf = out_matrix(rows, cols, dtype, pad)
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
    codes, scales = ckpt(rows, cols) if keep else (None, None)
    gc.layernorm_forward(ctx, x, gd, bd, EPS, y, mean, rstd, codes, scales)
    yw, mw, rw = ref.layernorm(xv, gamma, beta, EPS)
    a = np.abs(xv).mean(axis=1)
    close(f64(mean), mw, CHAIN * a + 1e-30, "mean")
    spread = 1 / rw
    close(f64(rstd), rw, CHAIN * rw * (1 + (a / spread) ** 2 * CHAIN), "rstd")
    close(f64(y), yw, _norm_tol(xv, mw, rw, gamma, yw, dtype), "y")
    pad_untouched(ybuf, cols)
    xs = xv
    if keep:
        want, b = ref.encode(xv)
        assert np.array_equal(codes.cpu().numpy(), want)
        assert np.array_equal(scales.cpu().numpy()[:, :b.shape[1]], b)
        codes, scales = device_ckpt(want, b)
        xs = ref.decode(want, b, cols)

    dy, dyv, _ = matrix(r.standard_normal((rows, cols)) * 0.01, dtype, pad)
    dx, dxbuf = out_matrix(rows, cols, dtype, pad)
    dg, db = (torch.full((cols,), 5.0, device="cuda") for _ in range(2))
    m32, r32 = mw.astype(np.float32), rw.astype(np.float32)
    md, rd = torch.from_numpy(m32).cuda(), torch.from_numpy(r32).cuda()
    args = (ctx, dy, None if keep else x, gd, md, rd, dx, dg, db, codes, scales)
    gc.layernorm_backward(*args)
    m64, r64 = m32.astype(np.float64), r32.astype(np.float64)
    dxw, dgw, dbw = ref.layernorm_backward(dyv, xs, gamma, m64, r64)
    big = r64[:, None] * (np.abs(xs) + np.abs(m64[:, None]))  # bounds n and its rounding
    d = np.abs(dyv * gamma)
    tol = r64[:, None] * (d + d.mean(axis=1, keepdims=True)
                          + big * (d * big).mean(axis=1, keepdims=True))
    close(f64(dx), dxw, U[dtype] * np.abs(dxw) + CHAIN * tol + TINY[dtype], "dx")
    pad_untouched(dxbuf, cols)
    gtol, btol = CHAIN * (np.abs(dyv) * big).sum(axis=0), CHAIN * np.abs(dyv).sum(axis=0)
    close(f64(dg), dgw, gtol, "dgamma")
    close(f64(db), dbw, btol, "dbeta")
    # again: equal bits; then added to what is there
    dg2, db2, dx2 = torch.empty_like(dg), torch.empty_like(db), torch.empty_like(dx)
    gc.layernorm_backward(ctx, dy, args[2], gd, md, rd, dx2, dg2, db2, codes, scales)
    assert bool((dg2 == dg).all()) and bool((db2 == db).all()) and bool((dx2 == dx).all())
    gc.layernorm_backward(ctx, dy, args[2], gd, md, rd, dx2, dg2, db2, codes, scales,
                          accumulate=True)
    assert bool((dg2 == dg + dg).all()) and bool((db2 == db + db).all())


def test_layernorm_parameters_of_other_types_and_none(gc, ctx):
    import torch
    rows, cols = 12, 260
    r, (x, xv, _) = _norm_case(rows, cols, "bf16", 0)
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
    dy, dyv, _ = matrix(r.standard_normal((rows, cols)), "bf16")
    for dtype in (torch.bfloat16, torch.float16, None):
        gamma = beta = g64 = None
        if dtype is not None:
            gamma = torch.from_numpy(1 + 0.2 * r.standard_normal(cols)).to(dtype).cuda()
            beta = torch.from_numpy(r.standard_normal(cols)).to(dtype).cuda()
            g64 = f64(gamma)
        y, _ = out_matrix(rows, cols, "bf16")
        gc.layernorm_forward(ctx, x, gamma, beta, EPS, y, mean, rstd)
        yw, mw, rw = ref.layernorm(xv, g64, None if beta is None else f64(beta), EPS)
        close(f64(y), yw, _norm_tol(xv, mw, rw, 1.0 if g64 is None else g64, yw, "bf16"), "y")
        dx, _ = out_matrix(rows, cols, "bf16")
        dg = torch.empty(cols, device="cuda")
        gc.layernorm_backward(ctx, dy, x, gamma, mean, rstd, dx, dg, None)
        dxw, dgw, _ = ref.layernorm_backward(dyv, xv, g64, f64(mean), f64(rstd))
        close(f64(dx), dxw, U["bf16"] * np.abs(dxw) + 1e-3, "dx")
        close(f64(dg), dgw, 1e-3, "dgamma")
        db = torch.empty(cols, device="cuda")
        gc.layernorm_backward(ctx, dy, x, gamma, mean, rstd, dx, None, db)
        close(f64(db), dyv.sum(axis=0), 1e-3, "dbeta")
        gc.layernorm_backward(ctx, dy, x, gamma, mean, rstd, dx)


@pytest.mark.parametrize("cols", [100, 4096, 20000])
def test_layernorm_far_from_zero(gc, ctx, cols):
    """A mean a thousand times the spread: no cancellation in the variance."""
    import torch
    r = np.random.default_rng(cols)
    x, xv, _ = matrix(1000.0 + r.standard_normal((6, cols)), "f32")
    y, _ = out_matrix(6, cols, "f32")
    mean, rstd = (torch.empty(6, device="cuda") for _ in range(2))
    gc.layernorm_forward(ctx, x, None, None, EPS, y, mean, rstd)
    yw, mw, rw = ref.layernorm(xv, None, None, EPS)
    assert np.abs(f64(rstd) / rw - 1).max() < 1e-4
    # the mean within 2^-17 of 1000
    close(f64(y), yw, 1000 * CHAIN * 1.1, "y")


def test_layernorm_non_finite_and_empty_rows(gc, ctx):
    import torch
    x = np.random.default_rng(1).standard_normal((5, 700))
    x[1, 5], x[3, 600] = np.inf, np.nan
    x[4] = 0.0
    d, xv, _ = matrix(x, "bf16")
    y, _ = out_matrix(5, 700, "bf16")
    mean, rstd = (torch.empty(5, device="cuda") for _ in range(2))
    codes, scales = ckpt(5, 700)
    gc.layernorm_forward(ctx, d, None, None, EPS, y, mean, rstd, codes, scales)
    yv = f64(y)
    assert np.isnan(yv[1]).any() and np.isnan(yv[3]).all()
    assert (yv[4] == 0).all() and np.isfinite(yv[[0, 2, 4]]).all()
    dy, _, _ = matrix(np.ones((5, 700)), "bf16")
    dx, _ = out_matrix(5, 700, "bf16")
    dg, db = torch.empty(700, device="cuda"), torch.empty(700, device="cuda")
    gc.layernorm_backward(ctx, dy, None, None, mean, rstd, dx, dg, db, codes, scales)
    dxv = f64(dx)
    assert np.isnan(dxv[1]).any() and np.isnan(dxv[3]).all()
    assert np.isfinite(dxv[[0, 2, 4]]).all() and (f64(db) == 5).all()
    assert not np.isfinite(f64(dg)).all()
    # no rows: zero gradients, or what was there
    e, none = torch.empty(0, 700, dtype=torch.bfloat16, device="cuda"), torch.empty(0, device="cuda")
    gc.layernorm_forward(ctx, e, None, None, EPS, e.clone(), none, none)
    gc.layernorm_backward(ctx, e, e, None, none, none, e.clone(), dg, db)
    assert (f64(dg) == 0).all() and (f64(db) == 0).all()
    db.fill_(3.0)
    gc.layernorm_backward(ctx, e, e, None, none, none, e.clone(), None, db, accumulate=True)
    assert (f64(db) == 3).all()


# --- linear weight gradients ---------------------------------------------------------------------

LINEAR_SHAPES = [(1, 1, 1, 0), (1, 64, 64, 0), (3, 33, 35, 0), (16, 128, 128, 0),
                 (100, 512, 512, 0), (63, 129, 257, 0), (65, 127, 255, 3), (200, 1001, 300, 0),
                 (513, 96, 1100, 8), (1000, 600, 72, 0), (4099, 130, 140, 0), (20000, 64, 32, 0),
                 (2048, 1024, 1536, 0), (333, 2560, 520, 0)]


def _linear_tol(rows, dyv, xs):
    return (rows / 8 + 64) * 2.0 ** -23 * (np.abs(dyv).T @ np.abs(xs))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,out,pad", LINEAR_SHAPES)
def test_linear_wgrad(gc, ctx, dtype, rows, cols, out, pad):
    import torch
    r = np.random.default_rng(rows + 3 * cols + out)
    xcodes, b = ref.encode(acts(r, rows, cols))
    xs = ref.decode(xcodes, b, cols)
    codes, scales = device_ckpt(xcodes, b)
    dy, dyv, _ = matrix(r.standard_normal((rows, out)) * np.exp(r.standard_normal((rows, 1))),
                        dtype, pad)
    assert gc.linear_wgrad_scratch_bytes(rows, out, cols, dtype) <= 256 << 20
    for wpad in (0, 5):
        dw, buf = out_matrix(out, cols, "f32", wpad)
        db = torch.full((out,), 9.0, device="cuda")
        gc.linear_wgrad(ctx, dy, codes, scales, dw, db)
        want, wantb = ref.linear_wgrad(dyv, xs)
        close(f64(dw), want, _linear_tol(rows, dyv, xs), "dw")
        close(f64(db), wantb, (rows / 8 + 64) * 2.0 ** -23 * np.abs(dyv).sum(axis=0), "db")
        pad_untouched(buf, cols)
        norm = np.linalg.norm(want)
        assert np.linalg.norm(f64(dw) - want) <= 1e-5 * norm
    dw2, _ = out_matrix(out, cols, "f32")
    gc.linear_wgrad(ctx, dy, codes, scales, dw2)
    assert bool((dw2 == dw).all())  # equal bits, with and without db
    gc.linear_wgrad(ctx, dy, codes, scales, dw2, db, accumulate=True)
    assert bool((dw2 == dw + dw).all())
    close(f64(db), 2 * wantb, (rows / 4 + 128) * 2.0 ** -23 * np.abs(dyv).sum(axis=0), "2 db")


def test_linear_wgrad_exact_integers(gc, ctx):
    """Small whole numbers: every product and sum is exact, so is the result,
    whatever the order (places, masks and edges of every tile)."""
    import torch
    r = np.random.default_rng(8)
    for rows, cols, out in ((70, 200, 270), (129, 513, 129), (1000, 257, 511)):
        x = r.integers(-8, 9, (rows, cols)).astype(np.float32)
        x[:, ::32] = 64.0  # the step is 1 everywhere
        xcodes, b = ref.encode(x)
        assert np.array_equal(ref.decode(xcodes, b, cols), x)
        codes, scales = device_ckpt(xcodes, b)
        d = r.integers(-4, 5, (rows, out)).astype(np.float32)
        for dtype in ("bf16", "f16", "f32"):
            dy, _, _ = matrix(d, dtype)
            dw, db = torch.empty(out, cols, device="cuda"), torch.empty(out, device="cuda")
            gc.linear_wgrad(ctx, dy, codes, scales, dw, db)
            assert np.array_equal(f64(dw), d.T.astype(np.float64) @ x)
            assert np.array_equal(f64(db), d.sum(axis=0, dtype=np.float64))


def test_linear_wgrad_non_finite_values_stay_in_their_columns(gc, ctx):
    import torch
    rows, cols, out = 50, 100, 70
    r = np.random.default_rng(2)
    x = acts(r, rows, cols)
    x[7, 40] = np.nan  # columns 32..63 of the checkpoint's row 7 restore as NaN
    codes, scales = device_ckpt(*ref.encode(x))
    d = r.standard_normal((rows, out)).astype(np.float32)
    d[3, 11] = np.inf
    for dtype in ("bf16", "f16", "f32"):
        dy, _, _ = matrix(d, dtype)
        dw, db = torch.empty(out, cols, device="cuda"), torch.empty(out, device="cuda")
        gc.linear_wgrad(ctx, dy, codes, scales, dw, db)
        w, bv = f64(dw), f64(db)
        assert np.isnan(w[:, 32:64]).all() and not np.isfinite(w[11]).any()
        rest = np.delete(np.delete(w, np.arange(32, 64), axis=1), 11, axis=0)
        assert np.isfinite(rest).all()
        assert not np.isfinite(bv[11]) and np.isfinite(np.delete(bv, 11)).all()


def test_linear_wgrad_without_rows(gc, ctx):
    import torch
    dy = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    codes, scales = ckpt(0, 50)
    dw, db = torch.full((40, 50), 2.0, device="cuda"), torch.full((40,), 2.0, device="cuda")
    gc.linear_wgrad(ctx, dy, codes, scales, dw, db, accumulate=True)
    assert bool((dw == 2).all()) and bool((db == 2).all())
    gc.linear_wgrad(ctx, dy, codes, scales, dw, db)
    assert bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [0, 3, 1000])
def test_linear_wgrad_without_input_features(gc, ctx, rows, dtype):
    """A layer that is only a bias: db is written all the same."""
    import torch
    out = 40
    r = np.random.default_rng(rows)
    dy, dyv, _ = matrix(r.standard_normal((rows, out)), dtype)
    codes, scales = ckpt(rows, 0)
    dw, db = torch.empty(out, 0, device="cuda"), torch.full((out,), 2.0, device="cuda")
    tol = (rows / 8 + 64) * 2.0 ** -23 * np.abs(dyv).sum(axis=0)
    gc.linear_wgrad(ctx, dy, codes, scales, dw, db, accumulate=True)
    close(f64(db), 2 + dyv.sum(axis=0), tol + 2.0 ** -20, "db on top")
    gc.linear_wgrad(ctx, dy, codes, scales, dw, db)
    close(f64(db), dyv.sum(axis=0), tol, "db")


@pytest.mark.parametrize("dtype,rows,cols,out", [("f32", 2501, 1001, 2051), ("bf16", 4096, 2048, 5504)])
def test_linear_wgrad_back_to_back(gc, ctx, dtype, rows, cols, out):
    """Hundreds of calls in a row on rotating inputs (codes and dy come from
    memory in any order): every result keeps its bits, no wait runs out."""
    import torch
    r = np.random.default_rng(rows)
    sets = []
    for _ in range(3):
        x = torch.randn(rows, cols, device="cuda") + float(r.standard_normal())
        codes, scales = ckpt(rows, cols)
        gc.ckpt_save(ctx, x, codes, scales)
        sets.append((torch.randn(rows, out, device="cuda").to(_dt(torch, dtype)), codes, scales,
                     torch.empty(out, cols, device="cuda"), torch.empty(out, device="cuda")))
    with gc.Context(0) as own:
        own.reserve_scratch(gc.linear_wgrad_scratch_bytes(rows, out, cols, dtype))
        first = []
        for dy, codes, scales, dw, db in sets:
            gc.linear_wgrad(own, dy, codes, scales, dw, db)
            first.append((dw.clone(), db.clone()))
        for i in range(1500):
            dy, codes, scales, dw, db = sets[i % 3]
            gc.linear_wgrad(own, dy, codes, scales, dw, db if i % 2 else None)
        own.check()
        for (dw0, db0), (_, _, _, dw, db) in zip(first, sets):
            assert bool((dw == dw0).all()) and bool((db == db0).all())


# --- all together --------------------------------------------------------------------------------

def test_another_stream_and_capture(gc):
    """The calls run on the context's stream and can be captured; replays
    repeat them on new inputs."""
    import torch
    rows, cols, out = 200, 256, 192
    r = np.random.default_rng(6)
    x, xv, _ = matrix(acts(r, rows, cols), "bf16")
    dy, dyv, _ = matrix(r.standard_normal((rows, out)), "bf16")
    dn, _, _ = matrix(r.standard_normal((rows, cols)), "bf16")
    y, dx, a, da = (torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
    dw, db = torch.empty(out, cols, device="cuda"), torch.empty(out, device="cuda")
    dg, dbt = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    codes, scales = ckpt(rows, cols)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with gc.Context(0, stream) as c:
        c.reserve_scratch(max(gc.layernorm_scratch_bytes(rows, cols),
                              gc.linear_wgrad_scratch_bytes(rows, out, cols, "bf16")))

        def step():
            gc.layernorm_forward(c, x, None, None, EPS, y, mean, rstd, codes, scales)
            gc.act_forward(c, "gelu", x, a, codes, scales)
            gc.act_backward(c, "gelu", dn, da, codes, scales)
            gc.linear_wgrad(c, dy, codes, scales, dw, db)
            gc.layernorm_backward(c, dn, None, None, mean, rstd, dx, dg, dbt, codes, scales)

        with torch.cuda.stream(stream):
            step()
        stream.synchronize()
        first = [t.clone() for t in (y, a, da, dw, db, dx, dg, dbt)]
        close(f64(dw), dyv.T @ ref.restored(xv), _linear_tol(rows, dyv, ref.restored(xv)), "dw")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        x.mul_(-2.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert bool((dw == -2.0 * first[3]).all()) and bool((db == first[4]).all())
        assert c.launch_count() > 0
        c.check()


def test_refusals(gc, ctx):
    import torch
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, y = torch.zeros(4, 64, **bf), torch.zeros(4, 64, **bf)
    codes, scales = ckpt(4, 64)
    mean, rstd = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    for bad in (lambda: gc.ckpt_save(ctx, x[:, ::2], codes, scales),
                lambda: gc.ckpt_save(ctx, x, codes[:3], scales),
                lambda: gc.ckpt_save(ctx, x, codes, scales[:3]),
                lambda: gc.ckpt_save(ctx, x[0], codes, scales),
                lambda: gc.act_forward(ctx, "gelu", x, y[:3], codes, scales),
                lambda: gc.act_forward(ctx, "gelu", x, y.float(), codes, scales),
                lambda: gc.layernorm_forward(ctx, x, mean, None, EPS, y, mean, rstd),
                lambda: gc.layernorm_forward(ctx, x, None, None, EPS, y, mean[:2], rstd),
                lambda: gc.linear_wgrad(ctx, x, codes, scales, torch.zeros(64, 64, **bf)),
                lambda: gc.linear_wgrad(ctx, x, codes, scales, torch.zeros(5, 64, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        gc.ckpt_save(ctx, torch.zeros(4, 64, dtype=torch.float64, device="cuda"), codes, scales)
    with pytest.raises(KeyError):
        gc.act_forward(ctx, "relu", x, y)

    def status(call):
        with pytest.raises(gc.GCError) as e:
            call()
        return e.value.status

    assert status(lambda: gc.act_forward(ctx, 7, x, y)) == gc.ERR_INVALID_ARG
    assert status(lambda: gc.act_forward(ctx, "gelu", x, y, codes)) == gc.ERR_INVALID_ARG
    assert status(lambda: gc.act_forward(ctx, "gelu", x, y, codes, scales, x)) == \
        gc.ERR_INVALID_ARG
    assert status(lambda: gc.act_backward(ctx, "gelu", x, y, codes, scales, None, codes,
                                          scales)) == gc.ERR_INVALID_ARG
    assert status(lambda: gc.ckpt_save(ctx, x[:, 1:], codes, scales)) == gc.ERR_ALIGNMENT
    assert status(lambda: gc.layernorm_forward(ctx, x, None, None, -1.0, y, mean, rstd)) == \
        gc.ERR_INVALID_ARG
    assert status(lambda: gc.layernorm_forward(ctx, x, None, None, float("nan"), y, mean,
                                               rstd)) == gc.ERR_INVALID_ARG
    assert status(lambda: gc.layernorm_backward(ctx, x, x, None, mean, rstd, y, None, None, codes,
                                                scales)) == gc.ERR_INVALID_ARG
    assert status(lambda: gc.layernorm_backward(ctx, x, None, None, mean, rstd, y)) == \
        gc.ERR_INVALID_ARG
    with gc.Context(0) as small:
        dg = torch.zeros(64, device="cuda")
        assert status(lambda: gc.layernorm_backward(small, x, x, None, mean, rstd, y, dg)) == \
            gc.ERR_WORKSPACE
        gc.layernorm_backward(small, x, x, None, mean, rstd, y)  # needs none without dgamma, dbeta
        small.check()
    L, bad = gc.lib, gc.ERR_INVALID_ARG
    h, p = ctx.handle, x.data_ptr()
    c, s = codes.data_ptr(), scales.data_ptr()
    assert L.gc_ckpt_save(h, p, 3, 4, 64, 64, c, s) == bad
    assert L.gc_ckpt_save(h, p, 1, 4, 64, 63, c, s) == bad
    assert L.gc_ckpt_save(h, p, 1, -1, 64, 64, c, s) == bad
    assert L.gc_ckpt_save(h, None, 1, 4, 64, 64, c, s) == bad
    assert L.gc_ckpt_save(h, p, 1, 4, 64, 64, c, None) == bad
    assert L.gc_ctx_reserve_scratch(h, -1) == bad
    torch.cuda.synchronize()

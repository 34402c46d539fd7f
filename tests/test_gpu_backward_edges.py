"""The calls that fill the flat gradient where the tests of
test_gpu_backward.py do not reach: the negative tails of the activation
functions, kernels that only large matrices are given to, long-running calls,
parameter gradients that start anywhere, the scratch's growth.

Tolerances are bounds on rounding, as there: U is half an ulp of the output
type, relative; the rest is stated where it is used.
"""
import numpy as np
import pytest

from oracle import backward as ref
from tests.gpu_helpers import torch_cuda
from tests.test_gpu_backward import (CHAIN, EPS, TINY, U, _dt, acts, ckpt, close, device_ckpt, f64,
                                     matrix, out_matrix, pad_untouched)

pytestmark = pytest.mark.gpu

SMALLEST = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}


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


# --- the negative tails of the activation functions ----------------------------------------------
#
# GELU there is x times exp(-x^2 / 2) R: three roundings of the exponent, each
# 2^-24 of x^2 / 2 at most, are x^2 2^-23 of the value, and 2^-18 covers the
# rest for fp32 (the fit of R 7.3e-7 = 2^-20.4, eight steps of Horner's rule at
# 2^-24, exponential and reciprocal 2^-22 each); 16-bit types take a fit of
# 2^-14.4, in all 2^-14.  SiLU's exponent has two roundings of 2^-24 |x|, the
# rest is below 2^-20.

TAIL = {"gelu": -13.1, "silu": -91.0}


def _part(kind, x, dtype):
    """The part of itself that f may be off by at x < 0."""
    if kind == "silu":
        return 2.0 ** -20 - x * 2.0 ** -23
    return (2.0 ** -18 if dtype == "f32" else 2.0 ** -14) + x * x * 2.0 ** -23


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["gelu", "silu"])
def test_negative_tail_forward(gc, ctx, kind, dtype):
    x = np.concatenate([np.linspace(TAIL[kind], -1e-3, 20000 - 2048), -np.geomspace(1e-6, 1, 2048)])
    d, xv, _ = matrix(np.maximum(x, TAIL[kind]).reshape(-1, 32), dtype)
    y, _ = out_matrix(*d.shape, dtype)
    gc.act_forward(ctx, kind, d, y)
    f, _ = ref.act(kind, xv)
    tol = (U[dtype] + _part(kind, xv, dtype)) * np.abs(f)
    if dtype == "f16":
        tol += SMALLEST["f16"] / 2  # subnormal outputs
    close(f64(y), f, tol, "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["gelu", "silu"])
def test_negative_tail_backward(gc, ctx, kind, dtype):
    """Columns hold one value each that the checkpoint keeps as it is: 64 to
    127 times a power of two."""
    import torch
    x = np.concatenate([-np.arange(64, 128) * 2.0 ** -k for k in range(0, 12)])
    x = x[x >= TAIL[kind]]
    x = np.repeat(x[:, None], 32, axis=1)
    d, xv, _ = matrix(x, "f32")
    rows, cols = x.shape
    codes, scales = (torch.zeros(n, dtype=torch.uint8, device="cuda")
                     for n in (gc.ckpt_codes_bytes(rows, cols), gc.ckpt_scales_bytes(rows, cols)))
    gc.ckpt_save(ctx, d, codes, scales)
    assert np.array_equal(ref.restored(xv), xv)
    dy, dyv, _ = matrix(np.full(x.shape, 1.5), dtype)
    dx, _ = out_matrix(rows, cols, dtype)
    dgate, _ = out_matrix(rows, cols, dtype)
    gc.act_backward(ctx, kind, dy, dx, codes, scales, dgate, codes, scales)
    f, df = ref.act(kind, xv)
    if kind == "gelu":
        terms = f / xv + np.abs(xv) * np.exp(-xv * xv / 2) / np.sqrt(2 * np.pi)
    else:
        terms = f / xv * (1 + np.abs(xv))
    small = SMALLEST["f16"] / 2 if dtype == "f16" else 0.0
    part = _part(kind, xv, dtype)
    # where Phi(x) or s(x) itself is subnormal it has a spacing of 2^-149
    close(f64(dx), dyv * xv * df, U[dtype] * np.abs(dyv * xv * df)
          + np.abs(dyv * xv) * (2 * part * terms + np.abs(xv) * 2.0 ** -148) + small, "dx")
    close(f64(dgate), dyv * f,
          (U[dtype] + part) * np.abs(dyv * f) + np.abs(xv) * 2.0 ** -148 + small, "dgate")


@pytest.mark.parametrize("kind", ["gelu", "silu"])
def test_ends_of_the_range(gc, ctx, kind):
    """Largest and smallest magnitudes, fp32: the identity on the right, half
    of it near zero, nothing on the left."""
    x = np.array([[3.4e38, 1e30, 200.0, 2.0 ** -126, -2.0 ** -126, 1e-30, -1e-30, 0.0, -0.0,
                   -100.0, -1e10, -3.4e38]], np.float32)
    d, xv, _ = matrix(x, "f32")
    y, _ = out_matrix(1, x.shape[1], "f32")
    gc.act_forward(ctx, kind, d, y)
    got = f64(y)[0]
    assert np.array_equal(got[:3], xv[0, :3])
    assert np.abs(got[3:7] - xv[0, 3:7] / 2).max() <= 2.0 ** -149 + 2.0 ** -21 * 1e-30
    assert (got[7:] == 0).all()


# --- calls that run long -------------------------------------------------------------------------

def test_linear_wgrad_of_seconds(gc):
    """A product of 4.2e15 operations runs for more cycles than any single wait
    in it may take (4e9): no wait may be one for the whole kernel.  Operands of
    two values each (dy and the codes lie in one buffer, both only read), so
    that every sum is exact."""
    import torch
    rows, cols, out = 163840, 131072, 98304
    torch.cuda.empty_cache()
    scratch = gc.linear_wgrad_scratch_bytes(rows, out, cols, "f16")
    need = 2 * rows * out + 4 * out * cols + gc.ckpt_scales_bytes(rows, cols) + scratch
    if torch.cuda.mem_get_info()[0] < need + (16 << 30):
        pytest.skip("needs %d GB of device memory" % (need >> 30))
    dy = torch.ones(rows, out, dtype=torch.float16, device="cuda")  # bytes 0x00, 0x3C
    codes = dy.view(torch.uint8).view(-1)[:gc.ckpt_codes_bytes(rows, cols)]  # 0, 60, 0, 60, ...
    scales = torch.full((gc.ckpt_scales_bytes(rows, cols),), 134, dtype=torch.uint8, device="cuda")
    dw = torch.full((out, cols), 7.0, device="cuda")
    with gc.Context(0) as own:
        own.reserve_scratch(scratch)
        gc.linear_wgrad(own, dy, codes, scales, dw)
        own.check()
    for part in dw.split(8192):
        assert bool((part[:, 0::2] == 0).all()) and bool((part[:, 1::2] == 60.0 * rows).all())
    del dy, codes, scales, dw, part
    torch.cuda.empty_cache()


# --- parameter gradients that start anywhere -----------------------------------------------------

def _flat(sizes, at):
    """A buffer of sevens, and views of the given sizes back to back from
    float `at` on."""
    import torch
    buf = torch.full((at + sum(sizes) + 9,), 7.0, device="cuda")
    views = []
    for n in sizes:
        views.append(buf[at:at + n])
        at += n
    return buf, views


@pytest.mark.parametrize("at", [1, 2, 3])
@pytest.mark.parametrize("rows,cols", [(1, 4097), (50, 99), (400, 701), (20, 9001)])
def test_norm_gradients_at_any_float(gc, ctx, rows, cols, at):
    """dgamma, dbeta, mean and rstd off 16-byte boundaries: the bits that they
    have on one, and nothing beside them."""
    import torch
    r = np.random.default_rng(cols)
    x, _, _ = matrix(acts(r, rows, cols), "bf16")
    dy, _, _ = matrix(r.standard_normal((rows, cols)), "bf16")
    y, dx = (torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    got = []
    for place in (0, at):
        sbuf, (mean, rstd) = _flat((rows, rows), place) if place else _flat((rows + -rows % 4, rows),
                                                                            0)
        gbuf, (dg, db) = _flat((cols, cols), place) if place else _flat((cols + -cols % 4, cols), 0)
        mean, rstd, dg, db = mean[:rows], rstd[:rows], dg[:cols], db[:cols]
        gc.layernorm_forward(ctx, x, None, None, EPS, y, mean, rstd)
        gc.layernorm_backward(ctx, dy, x, None, mean, rstd, dx, dg, db)
        gc.layernorm_backward(ctx, dy, x, None, mean, rstd, dx, dg, db, accumulate=True)
        got.append([t.clone() for t in (y, dx, mean, rstd, dg, db)])
        if place:
            for buf, n in ((sbuf, 2 * rows), (gbuf, 2 * cols)):
                assert bool((buf[:at] == 7).all()) and bool((buf[at + n:] == 7).all())
    for a, b in zip(*got):
        assert bool((a == b).all())


@pytest.mark.parametrize("at", [1, 2, 3])
@pytest.mark.parametrize("rows,cols,out", [(0, 35, 21), (3, 33, 35), (1000, 257, 511)])
def test_linear_gradients_at_any_float(gc, ctx, rows, cols, out, at):
    """The same for dw and db, back to back: a layer with an odd number of
    outputs leaves the next parameter's gradient off every boundary."""
    import torch
    r = np.random.default_rng(rows)
    codes, scales = device_ckpt(*ref.encode(acts(r, rows, cols)))
    dy, _, _ = matrix(r.standard_normal((rows, out)), "bf16")
    dw0, db0 = torch.empty(out, cols, device="cuda"), torch.empty(out, device="cuda")
    gc.linear_wgrad(ctx, dy, codes, scales, dw0, db0)
    buf, (db, dw) = _flat((out, out * cols), at)
    dw = dw.view(out, cols)
    gc.linear_wgrad(ctx, dy, codes, scales, dw, db)
    assert bool((dw == dw0).all()) and bool((db == db0).all())
    gc.linear_wgrad(ctx, dy, codes, scales, dw, db, accumulate=True)
    assert bool((dw == 2 * dw0).all()) and bool((db == 2 * db0).all())
    assert bool((buf[:at] == 7).all()) and bool((buf[-9:] == 7).all())


def test_addresses_between_floats_are_refused(gc, ctx):
    import torch
    rows, cols = 4, 64
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    codes, scales = ckpt(rows, cols)
    f = torch.zeros(cols * cols, device="cuda").data_ptr()
    L, h, p = gc.lib, ctx.handle, x.data_ptr()
    c, s = codes.data_ptr(), scales.data_ptr()
    bad = gc.ERR_ALIGNMENT
    for off in (1, 2, 6):
        assert L.gc_layernorm_forward(h, p, cols, gc.BF16, rows, cols, None, None, 0, EPS,
                                      y.data_ptr(), cols, f + off, f, None, None) == bad
        assert L.gc_layernorm_forward(h, p, cols, gc.BF16, rows, cols, None, None, 0, EPS,
                                      y.data_ptr(), cols, f, f + off, None, None) == bad
        for dg, db in ((f + off, f), (f, f + off)):
            assert L.gc_layernorm_backward(h, p, cols, p, cols, None, None, gc.BF16, rows, cols,
                                           None, 0, f, f, y.data_ptr(), cols, dg, db, 0) == bad
        for dw, db in ((f + off, f), (f, f + off)):
            assert L.gc_linear_wgrad(h, p, gc.BF16, cols, c, s, rows, cols, cols, dw, cols, db,
                                     0) == bad
    torch.cuda.synchronize()


# --- the scratch's growth ------------------------------------------------------------------------

class _Step:
    """A weight gradient of cut tiles (partials in the scratch) and a norm's
    column sums, on one context."""

    rows, cols, out = 1000, 640, 130

    def __init__(self, gc, c, seed):
        import torch
        r = np.random.default_rng(seed)
        rows, cols, out = self.rows, self.cols, self.out
        self.gc, self.c = gc, c
        self.codes, self.scales = device_ckpt(*ref.encode(acts(r, rows, cols)))
        self.dy = matrix(r.standard_normal((rows, out)), "f32")[0]
        self.dn = matrix(r.standard_normal((rows, cols)), "f32")[0]
        self.mean, self.rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
        self.dx = torch.empty(rows, cols, device="cuda")
        self.outs = [torch.empty(out, cols, device="cuda")] + [
            torch.empty(n, device="cuda") for n in (out, cols, cols)]

    @classmethod
    def need(cls, gc):
        return max(gc.layernorm_scratch_bytes(cls.rows, cls.cols),
                   gc.linear_wgrad_scratch_bytes(cls.rows, cls.out, cls.cols, "f32"))

    def run(self):
        dw, db, dg, dbt = self.outs
        self.gc.linear_wgrad(self.c, self.dy, self.codes, self.scales, dw, db)
        self.gc.layernorm_backward(self.c, self.dn, None, None, self.mean, self.rstd, self.dx, dg,
                                   dbt, self.codes, self.scales)

    def results(self):
        return [t.clone() for t in self.outs]


def test_scratch_that_cannot_grow_stays(gc):
    with gc.Context(0) as c:
        c.reserve_scratch(_Step.need(gc))
        step = _Step(gc, c, 1)
        step.run()
        first = step.results()
        with pytest.raises(gc.GCError) as e:
            c.reserve_scratch(1 << 56)
        assert e.value.status == gc.ERR_NO_MEMORY
        step.run()
        for a, b in zip(first, step.results()):
            assert bool((a == b).all())
        c.check()


def test_scratch_growth_leaves_captured_graphs_valid(gc):
    """A graph holds the address that the scratch had: after a growth it still
    writes to memory of the context, and to no one else's."""
    import torch
    stream = torch.cuda.Stream()
    with gc.Context(0, stream) as c:
        c.reserve_scratch(_Step.need(gc))
        step = _Step(gc, c, 2)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            step.run()
        stream.synchronize()
        first = step.results()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step.run()
        c.reserve_scratch(2 * _Step.need(gc))
        others = [torch.full((_Step.need(gc) // 4,), 3.0, device="cuda") for _ in range(4)]
        for t in step.outs:
            t.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, step.results()):
            assert bool((a == b).all())
        assert all(bool((t == 3).all()) for t in others)
        c.check()


def test_scratch_growth_while_calls_are_under_way(gc):
    import torch
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    with gc.Context(0, one) as c:
        c.reserve_scratch(_Step.need(gc))
        a, b = _Step(gc, c, 3), _Step(gc, c, 4)
        torch.cuda.synchronize()
        want = []
        for s in (a, b):
            s.run()
            one.synchronize()
            want.append(s.results())
            for t in s.outs:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            a.run()
        c.set_stream(two)
        c.reserve_scratch(3 * _Step.need(gc))  # the first stream's calls are under way
        two.wait_stream(one)
        for _ in range(20):
            b.run()
        torch.cuda.synchronize()
        for s, w in zip((a, b), want):
            for x, y in zip(s.results(), w):
                assert bool((x == y).all())
        c.check()


# --- kernels that only large matrices are given to -----------------------------------------------
#
# Rows well above what the blocks of a launch have at a time and not a multiple
# of it; the references in 64 bits by torch on the GPU, written from the
# formulas.

def _encode64(x):
    """Codes [rows, pitch] and scale bytes [rows, groups] of x (float64)."""
    import torch
    rows, cols = x.shape
    groups = -(-cols // 32)
    g = torch.zeros(rows, groups * 32, dtype=torch.float64, device="cuda")
    g[:, :cols] = x
    g = g.view(rows, groups, 32)
    top = g.abs().amax(dim=2)
    e = torch.frexp(top).exponent
    small = top < 2.0 ** -120
    m = torch.clamp(torch.round(g.abs() * torch.exp2(7.0 - e.double())[..., None]), max=127)
    m = torch.where(small[..., None], torch.zeros_like(m), m).long()
    codes = m + 128 * ((g < 0) & (m > 0))
    return (codes.to(torch.uint8).view(rows, groups * 32),
            torch.where(small, torch.zeros_like(e), e + 127).to(torch.uint8))


def _decode64(codes, b, cols):
    import torch
    rows, groups = b.shape
    c = codes.view(rows, groups, 32).long()
    v = (c & 127).double() * torch.exp2(b.double() - 134.0)[..., None]
    return torch.where(c > 127, -v, v).view(rows, groups * 32)[:, :cols]


def _random(rows, cols, dtype, pad, seed, scale=1.0):
    """A device matrix of activations with a few empty rows, its pad NaN, and
    its values in float64."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(torch.randn(1, cols, generator=gen, device="cuda")) * scale
    x *= torch.rand(rows, 1, generator=gen, device="cuda") > 0.05
    buf = torch.full((rows, cols + pad), float("nan"), dtype=_dt(torch, dtype), device="cuda")
    buf[:, :cols] = x
    return buf[:, :cols], buf[:, :cols].double()


def _near(got, want, tol, what):
    bad = (got.double() - want).abs() > tol
    bad |= got.isnan()
    n = int(bad.sum())
    assert n == 0, "%s: %d outside, first at %s" % (what, n, bad.nonzero()[0].tolist())


def _same_codes(codes, scales, want, b):
    assert bool((codes == want).all()), "codes"
    assert bool((scales[:, :b.shape[1]] == b).all()), "scale bytes"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols,pad", [(2500, 1024, 0), (2500, 1025, 1), (700, 4100, 3),
                                           (900, 4097, 0), (801, 6016, 8)])
def test_checkpoint_of_many_rows(gc, ctx, dtype, rows, cols, pad):
    x, xv = _random(rows, cols, dtype, pad, cols)
    codes, scales = ckpt(rows, cols)
    gc.ckpt_save(ctx, x, codes, scales)
    want, b = _encode64(xv)
    _same_codes(codes, scales, want, b)
    out, buf = out_matrix(rows, cols, dtype, pad)
    gc.ckpt_restore(ctx, codes, scales, out)
    assert bool((out.double() == _decode64(want, b, cols)).all())
    pad_untouched(buf, cols)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["gelu", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,cols,pad", [(2500, 1024, 0), (2500, 1025, 1), (700, 4100, 3)])
def test_activation_of_many_rows(gc, ctx, dtype, kind, gated, rows, cols, pad):
    import torch

    def act(v):
        if kind == "gelu":
            p = torch.special.ndtr(v)
            return v * p, p + v * torch.exp(-v * v / 2) / np.sqrt(2 * np.pi)
        p = torch.sigmoid(v)
        return v * p, p * (1 + v * torch.sigmoid(-v))

    x, xv = _random(rows, cols, dtype, pad, cols)
    y, ybuf = out_matrix(rows, cols, dtype, pad)
    codes, scales = ckpt(rows, cols)
    gate = gcodes = gscales = None
    gv = torch.ones_like(xv)
    if gated:
        gate, gv = _random(rows, cols, dtype, pad, cols + 1)
        gcodes, gscales = ckpt(rows, cols)
    gc.act_forward(ctx, kind, x, y, codes, scales, gate, gcodes, gscales)
    f = act(xv)[0]
    # bounds as for the small shapes
    _near(y, f * gv, U[dtype] * (f * gv).abs() + 2.0 ** -21 * (xv * gv).abs() + TINY[dtype], "y")
    pad_untouched(ybuf, cols)
    want, b = _encode64(xv)
    _same_codes(codes, scales, want, b)
    xs, gs = _decode64(want, b, cols), gv
    if gated:
        want, b = _encode64(gv)
        _same_codes(gcodes, gscales, want, b)
        gs = _decode64(want, b, cols)

    dy, dyv = _random(rows, cols, dtype, pad, cols + 2, 0.1)
    dx, dxbuf = out_matrix(rows, cols, dtype, pad)
    dgate, dgbuf = out_matrix(rows, cols, dtype, pad) if gated else (None, None)
    gc.act_backward(ctx, kind, dy, dx, codes, scales, dgate, gcodes, gscales)
    fs, ds = act(xs)
    full = dyv * gs * ds
    _near(dx, full, U[dtype] * full.abs() + 2.0 ** -19 * (dyv * gs).abs() + TINY[dtype], "dx")
    pad_untouched(dxbuf, cols)
    if gated:
        _near(dgate, dyv * fs,
              U[dtype] * (dyv * fs).abs() + 2.0 ** -21 * (dyv * xs).abs() + TINY[dtype], "dgate")
        pad_untouched(dgbuf, cols)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("rows,cols,pad", [(20001, 100, 0), (12001, 333, 1), (9001, 640, 0),
                                           (9001, 1025, 3), (6001, 4096, 0), (5001, 4099, 2),
                                           (3001, 8192, 0), (2003, 16384, 0)])
def test_layernorm_of_many_rows(gc, ctx, dtype, keep, rows, cols, pad):
    """Rows per block far above the ring's stages: every stage is filled
    again, several times; the warp kernels take row after row."""
    import torch
    x, xv = _random(rows, cols, dtype, pad, cols)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    gamma = 1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")
    beta = 0.2 * torch.randn(cols, generator=gen, device="cuda")
    g64, b64 = gamma.double(), beta.double()
    y, ybuf = out_matrix(rows, cols, dtype, pad)
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
    codes, scales = ckpt(rows, cols) if keep else (None, None)
    gc.layernorm_forward(ctx, x, gamma, beta, EPS, y, mean, rstd, codes, scales)
    m = xv.mean(dim=1, keepdim=True)
    s = 1 / torch.sqrt((xv - m).square().mean(dim=1, keepdim=True) + EPS)
    want = (xv - m) * s * g64 + b64
    # bounds as for the small shapes
    a = xv.abs().mean(dim=1, keepdim=True)
    _near(mean[:, None], m, CHAIN * a + 1e-30, "mean")
    _near(rstd[:, None], s, CHAIN * s * (1 + (a * s) ** 2 * CHAIN), "rstd")
    n = ((xv - m) * s).abs()
    _near(y, want, U[dtype] * want.abs() + CHAIN * (g64.abs() * (s * (a + xv.abs()) + n) + 1e-3)
          + TINY[dtype], "y")
    pad_untouched(ybuf, cols)
    xs = xv
    if keep:
        wc, wb = _encode64(xv)
        _same_codes(codes, scales, wc, wb)
        xs = _decode64(wc, wb, cols)

    dy, dyv = _random(rows, cols, dtype, pad, cols + 1, 0.01)
    dx, dxbuf = out_matrix(rows, cols, dtype, pad)
    dg, db = (torch.full((cols,), 5.0, device="cuda") for _ in range(2))
    args = (dy, None if keep else x, gamma, mean, rstd)
    gc.layernorm_backward(ctx, *args, dx, dg, db, codes, scales)
    m, s = mean.double()[:, None], rstd.double()[:, None]
    n, d = (xs - m) * s, dyv * g64
    full = s * (d - d.mean(dim=1, keepdim=True) - n * (d * n).mean(dim=1, keepdim=True))
    big = s * (xs.abs() + m.abs())
    tol = s * (d.abs() + d.abs().mean(dim=1, keepdim=True)
               + big * (d.abs() * big).mean(dim=1, keepdim=True))
    _near(dx, full, U[dtype] * full.abs() + CHAIN * tol + TINY[dtype], "dx")
    pad_untouched(dxbuf, cols)
    _near(dg, (dyv * n).sum(dim=0), CHAIN * (dyv.abs() * big).sum(dim=0), "dgamma")
    _near(db, dyv.sum(dim=0), CHAIN * dyv.abs().sum(dim=0), "dbeta")
    dg2, db2, dx2 = torch.empty_like(dg), torch.empty_like(db), torch.empty_like(dx)
    gc.layernorm_backward(ctx, *args, dx2, dg2, db2, codes, scales)
    assert bool((dg2 == dg).all()) and bool((db2 == db).all()) and bool((dx2 == dx).all())
    ctx.check()


@pytest.mark.parametrize("ptype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(900, 64), (900, 500), (400, 777), (400, 4096), (100, 4099),
                                       (200, 9001), (200, 17000)])
def test_layernorm_with_16_bit_parameters(gc, ctx, ptype, rows, cols):
    """gamma and beta of the 16-bit types through every kernel: the bits that
    the same values in fp32 give."""
    import torch
    x, _ = _random(rows, cols, "bf16", 0, cols)
    dy, _ = _random(rows, cols, "bf16", 0, cols + 1, 0.01)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    gamma = (1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")).to(_dt(torch, ptype))
    beta = torch.randn(cols, generator=gen, device="cuda").to(_dt(torch, ptype))
    ctx.reserve_scratch(gc.layernorm_scratch_bytes(rows, cols))
    got = []
    for g, b in ((gamma, beta), (gamma.float(), beta.float())):
        y, dx = (torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
        dg, db = (torch.empty(cols, device="cuda") for _ in range(2))
        gc.layernorm_forward(ctx, x, g, b, EPS, y, mean, rstd)
        gc.layernorm_backward(ctx, dy, x, g, mean, rstd, dx, dg, db)
        got.append((y, mean, rstd, dx, dg, db))
    for a, b in zip(*got):
        assert bool((a == b).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,out", [(600, 2100, 2300), (600, 2100, 5000), (70, 4100, 9000)])
def test_linear_wgrad_of_whole_rounds_of_tiles(gc, ctx, dtype, rows, cols, out):
    """81, 180 and 612 tiles: rounds of whole tiles for every pair of SMs, then
    cut ones.  Whole numbers, so that every sum is exact."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(out)

    def whole(top, *shape):
        return torch.randint(-top, top + 1, shape, generator=gen, device="cuda").float()

    x = whole(8, rows, cols)
    x[:, ::32] = 64.0  # the step is 1 everywhere
    codes, scales = ckpt(rows, cols)
    gc.ckpt_save(ctx, x, codes, scales)
    _same_codes(codes, scales, *_encode64(x.double()))
    dy = whole(4, rows, out).to(_dt(torch, dtype))
    dw, db = torch.empty(out, cols, device="cuda"), torch.empty(out, device="cuda")
    with gc.Context(0) as own:
        own.reserve_scratch(gc.linear_wgrad_scratch_bytes(rows, out, cols, dtype))
        gc.linear_wgrad(own, dy, codes, scales, dw, db)
        want, wantb = dy.double().t() @ x.double(), dy.double().sum(dim=0)
        assert bool((dw == want).all()) and bool((db == wantb).all())
        gc.linear_wgrad(own, dy, codes, scales, dw, db, accumulate=True)
        assert bool((dw == 2 * want).all()) and bool((db == 2 * wantb).all())
        # not whole numbers
        codes2, scales2 = ckpt(rows, cols)
        x2, x2v = _random(rows, cols, "f16" if dtype == "f16" else "f32", 0, rows)
        gc.ckpt_save(own, x2, codes2, scales2)
        xs = _decode64(*_encode64(x2v), cols)
        dy2, dy2v = _random(rows, out, dtype, 0, cols)
        gc.linear_wgrad(own, dy2, codes2, scales2, dw, db)
        _near(dw, dy2v.t() @ xs, (rows / 8 + 64) * 2.0 ** -23 * (dy2v.abs().t() @ xs.abs()), "dw")
        _near(db, dy2v.sum(dim=0), (rows / 8 + 64) * 2.0 ** -23 * dy2v.abs().sum(dim=0), "db")
        own.check()


def test_linear_wgrad_of_the_smallest_values(gc, ctx):
    """fp16 operands in the subnormal range, bf16 ones at the end of the normal
    range: whole multiples of the smallest, every sum exact."""
    import torch
    rows, cols, out = 130, 64, 40
    r = np.random.default_rng(11)
    x = r.integers(-127, 128, (rows, cols)).astype(np.float64)
    x[:, ::32] = 127.0
    d = r.integers(-4, 5, (rows, out)).astype(np.float64)
    for dtype, unit, dunit in (("f16", 2.0 ** -24, 2.0 ** -24), ("f16", 2.0 ** -24, 1.0),
                               ("bf16", 2.0 ** -126, 1.0), ("f32", 2.0 ** -126, 1.0)):
        xm, xv, _ = matrix(x * unit, "f16" if dtype == "f16" else "f32")
        assert np.array_equal(xv, x * unit)
        codes, scales = ckpt(rows, cols)
        gc.ckpt_save(ctx, xm, codes, scales)
        dy, dyv, _ = matrix(d * dunit, dtype)
        dw, db = torch.empty(out, cols, device="cuda"), torch.empty(out, device="cuda")
        gc.linear_wgrad(ctx, dy, codes, scales, dw, db)
        assert np.array_equal(f64(dw), dyv.T @ xv)
        assert np.array_equal(f64(db), dyv.sum(axis=0))

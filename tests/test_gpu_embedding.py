"""Embedding lookup and the table's gradient against the 64-bit reference:
id and element types, strides, one token to many, one id to all, rows without
tokens, padding, ids outside the table, accumulation, offsets past 32 bits,
determinism, streams, capture, refusals.

The lookup is bit for bit (one fp32 product, one rounding).  A gradient of n
tokens is n additions in fp32 and one product: (n + 2) * 2^-24 of the sum of
magnitudes.
"""
import numpy as np
import pytest

from oracle import stream as ref
from tests.gpu_helpers import torch_cuda
from tests.test_gpu_backward import close, f64, matrix, out_matrix, pad_untouched

pytestmark = pytest.mark.gpu


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


def tensor_ids(ids, itype):
    import torch
    return torch.from_numpy(np.asarray(ids, np.int32 if itype == "i32" else np.int64)).cuda()


def some_ids(r, tokens, vocab, kind):
    if kind == "one":
        return np.full(tokens, vocab - 1)
    if kind == "few":
        return r.integers(0, min(vocab, 3), tokens)
    if kind == "skew":
        return np.minimum((r.pareto(0.7, tokens) * 2).astype(np.int64), vocab - 1)
    return r.integers(0, vocab, tokens)


@pytest.mark.parametrize("ptype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols,pad", [(1, 0), (128, 0), (333, 0), (512, 3), (1000, 8), (4099, 1)])
def test_lookup_bit_for_bit(gc, ctx, ptype, dtype, cols, pad):
    import torch
    r = np.random.default_rng(cols)
    vocab, tokens = 37, 50
    table, tv, _ = matrix(r.standard_normal((vocab, cols)), ptype, pad)
    for itype in ("i32", "i64"):
        ids = r.integers(0, vocab, tokens)
        ids[[0, 7, 49]] = 5
        t = tensor_ids(ids, itype)
        y, buf = out_matrix(tokens, cols, dtype, 16 if pad else 0)
        gc.embedding_forward(ctx, t, table, 3.7, y, pad=5)
        keep = (t != 5)[:, None]
        want = torch.where(keep, (table[t.long()].float() * 3.7), 0.0).to(y.dtype)
        assert torch.equal(y, want)
        pad_untouched(buf, cols)
        # against the definition: the scale's rounding, the product's and the output's
        wv = ref.embedding_forward(ids, tv, 3.7, 5)
        u = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
        close(f64(y), wv, np.abs(wv) * (u + 2.0 ** -22) + 2.0 ** -25, "y")
    ctx.check()


@pytest.mark.parametrize("tokens", [1, 2, 63, 64, 65, 129, 1000, 8192, 8193, 20011])
@pytest.mark.parametrize("vocab,kind", [(1, "one"), (7, "few"), (300, "any"), (1000, "skew"),
                                        (70001, "any")])
def test_gradient(gc, ctx, tokens, vocab, kind):
    import torch
    r = np.random.default_rng(tokens + vocab)
    cols = 40 if vocab > 1000 else 77
    dtype = ("f32", "bf16", "f16")[(tokens + vocab) % 3]
    ids = some_ids(r, tokens, vocab, kind)
    ids[r.random(tokens) < 0.05] = -100
    dy, dyv, _ = matrix(r.standard_normal((tokens, cols)), dtype, tokens % 2)
    want, size, n = ref.embedding_wgrad(dyv, ids, vocab, 1.5, -100)
    tol = (n[:, None] + 2) * 2.0 ** -24 * size
    itype = "i32" if tokens % 2 else "i64"
    flat = torch.full((vocab * cols + 8,), 7.0, device="cuda")
    d = flat[3:3 + vocab * cols].view(vocab, cols)
    gc.embedding_wgrad(ctx, dy, tensor_ids(ids, itype), 1.5, d, pad=-100)
    first = d.clone()
    close(f64(first), want, tol, "dtable")
    assert bool((flat[:3] == 7.0).all()) and bool((flat[3 + vocab * cols:] == 7.0).all())
    # added to what is there: untouched rows keep their bits
    base = torch.randn(vocab, cols, device="cuda")
    wide = torch.full((vocab, cols + 5), 7.0, device="cuda")
    wide[:, :cols] = base
    gc.embedding_wgrad(ctx, dy, tensor_ids(ids, itype), 1.5, wide[:, :cols], pad=-100,
                       accumulate=True)
    used = torch.from_numpy(n > 0).cuda()[:, None]
    assert torch.equal(wide[:, :cols], torch.where(used, base + first, base))
    pad_untouched(wide, cols)
    ctx.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols,pad", [(1, 0), (256, 0), (300, 5), (4096, 0), (5000, 8)])
def test_gradient_widths(gc, ctx, dtype, cols, pad):
    import torch
    r = np.random.default_rng(cols)
    tokens, vocab = 150, 40
    ids = some_ids(r, tokens, vocab, "skew")
    dy, dyv, _ = matrix(r.standard_normal((tokens, cols)), dtype, pad)
    want, size, n = ref.embedding_wgrad(dyv, ids, vocab, 0.25)
    d, buf = out_matrix(vocab, cols, "f32", pad)
    gc.embedding_wgrad(ctx, dy, tensor_ids(ids, "i64"), 0.25, d)
    close(f64(d), want, (n[:, None] + 2) * 2.0 ** -24 * size, "dtable")
    pad_untouched(buf, cols)
    ctx.check()


def test_gradient_by_differences(gc, ctx):
    """The lookup is linear in the table: sum(dy * y) changes along v by
    exactly sum(dtable * v), but for roundings (2^-20 of the magnitudes)."""
    import torch
    r = np.random.default_rng(3)
    tokens, vocab, cols = 300, 50, 60
    ids = tensor_ids(some_ids(r, tokens, vocab, "skew"), "i64")
    dy, dyv, _ = matrix(r.standard_normal((tokens, cols)), "f32")
    d, _ = out_matrix(vocab, cols, "f32")
    gc.embedding_wgrad(ctx, dy, ids, 2.5, d)
    v, vv, _ = matrix(r.standard_normal((vocab, cols)), "f32")
    y, _ = out_matrix(tokens, cols, "f32")
    gc.embedding_forward(ctx, ids, v, 2.5, y)
    size = np.abs(dyv * f64(y)).sum()
    assert abs((dyv * f64(y)).sum() - (f64(d) * vv).sum()) <= 2.0 ** -20 * size


def test_ids_outside_the_table(gc, ctx):
    import torch
    vocab, cols = 10, 33
    table = torch.ones(vocab, cols, device="cuda")
    ids = torch.tensor([0, 10, -1, 2 ** 40, 9, -2 ** 63], device="cuda")
    y, _ = out_matrix(6, cols, "f32")
    gc.embedding_forward(ctx, ids, table, 1.0, y)
    with pytest.raises(gc.GCError) as e:
        ctx.check()
    assert e.value.status == gc.ERR_DEVICE_CHECK
    assert y[:, 0].tolist() == [1.0, 0.0, 0.0, 0.0, 1.0, 0.0]
    d, _ = out_matrix(vocab, cols, "f32")
    gc.embedding_wgrad(ctx, torch.ones(6, cols, device="cuda"), ids, 1.0, d)
    with pytest.raises(gc.GCError):
        ctx.check()
    assert d[:, 5].tolist() == [1.0] + [0.0] * 8 + [1.0]
    # as padding one of them is none of these
    gc.embedding_forward(ctx, ids[2:3], table, 1.0, y[:1], pad=-1)
    ctx.check()


def test_non_finite_gradients_stay_in_their_rows(gc, ctx):
    import torch
    ids = torch.tensor([3, 1, 3, 0, 5, 5], device="cuda")
    dy = torch.ones(6, 70, device="cuda")
    dy[0, 4], dy[1, 5], dy[4, 6], dy[5, 6] = float("nan"), float("inf"), float("inf"), -float("inf")
    d, _ = out_matrix(7, 70, "f32")
    gc.embedding_wgrad(ctx, dy, ids, 1.0, d)
    bad = ~torch.isfinite(d)
    assert bad.sum() == 3 and bool(d[3, 4].isnan()) and float(d[1, 5]) == float("inf")
    assert bool(d[5, 6].isnan())


def test_empty_sizes(gc, ctx):
    import torch
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    for tokens, vocab, cols in ((0, 5, 8), (3, 0, 8), (3, 5, 0), (0, 0, 0)):
        ids = torch.full((tokens,), -1, dtype=torch.int64, device="cuda") if tokens else none
        table, d = out_matrix(vocab, cols, "f32")[0], out_matrix(vocab, cols, "f32")[0]
        y, _ = out_matrix(tokens, cols, "f32")
        gc.embedding_forward(ctx, ids, table, 1.0, y, pad=-1)
        assert bool((y == 0).all())
        gc.embedding_wgrad(ctx, y, ids, 1.0, d, pad=-1, accumulate=True)
        assert bool((d == 7.0).all())
        gc.embedding_wgrad(ctx, y, ids, 1.0, d, pad=-1)
        assert bool((d == 0.0).all())
    ctx.check()


def test_offsets_past_32_bits(gc, ctx):
    import torch
    vocab, cols, tokens = 70000, 20000, 300  # 5.6 GB of fp32, 1.4e9 elements
    ids = torch.randint(0, vocab, (tokens,), device="cuda")
    ids[0], ids[1] = vocab - 1, vocab - 1
    d = torch.full((vocab, cols), 7.0, device="cuda")
    dy = torch.randn(tokens, cols, device="cuda").bfloat16()
    ctx.reserve_scratch(gc.embedding_scratch_bytes(tokens, vocab, cols))
    gc.embedding_wgrad(ctx, dy, ids, 1.0, d)
    want = torch.zeros(tokens, cols, dtype=torch.float64, device="cuda")
    u, inv = ids.unique(return_inverse=True)
    want.index_add_(0, inv, dy.double())
    assert float((d[u].double() - want[:len(u)]).abs().max()) <= 2.0 ** -20
    assert int((d != 0).any(1).sum()) == len(u)
    y = torch.empty(tokens, cols, device="cuda")
    gc.embedding_forward(ctx, ids, d, 1.0, y)
    assert torch.equal(y, d[ids])
    ctx.check()
    del d, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tokens", [700, 9001])
def test_same_bits_other_stream_and_capture(gc, tokens):
    import torch
    r = np.random.default_rng(2)
    vocab, cols = 500, 333
    ids = tensor_ids(some_ids(r, tokens, vocab, "skew"), "i64")
    dy, _, _ = matrix(r.standard_normal((tokens, cols)), "bf16")
    table = torch.randn(vocab, cols, device="cuda")
    stream = torch.cuda.Stream()
    with gc.Context(0, stream) as c:
        c.reserve_scratch(gc.embedding_scratch_bytes(tokens, vocab, cols))
        y = [out_matrix(tokens, cols, "bf16")[0] for _ in range(2)]
        d = [out_matrix(vocab, cols, "f32")[0] for _ in range(2)]

        def call(i):
            gc.embedding_forward(c, ids, table, 2.0, y[i])
            gc.embedding_wgrad(c, dy, ids, 2.0, d[i])

        stream.wait_stream(torch.cuda.current_stream())
        call(0)
        c.check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call(1)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d[0], d[1]) and torch.equal(y[0], y[1])


def test_refusals(gc, ctx):
    import torch
    table, y = torch.zeros(5, 8, device="cuda"), torch.zeros(3, 8, device="cuda")
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (ids[:2], ids[::2]):
        with pytest.raises(ValueError):
            gc.embedding_forward(ctx, bad, table, 1.0, y)
    with pytest.raises(TypeError):
        gc.embedding_forward(ctx, ids.float(), table, 1.0, y)
    with pytest.raises(ValueError):
        gc.embedding_forward(ctx, ids, table[:, :7], 1.0, y)
    with pytest.raises(ValueError):
        gc.embedding_wgrad(ctx, y, ids, 1.0, table.half())
    with pytest.raises(gc.GCError) as e:
        gc.embedding_forward(ctx, ids, torch.zeros(41, device="cuda")[1:].view(5, 8), 1.0, y)
    assert e.value.status == gc.ERR_ALIGNMENT
    with gc.Context(0) as bare:
        with pytest.raises(gc.GCError) as e:
            gc.embedding_wgrad(bare, y, ids, 1.0, table)
        assert e.value.status == gc.ERR_WORKSPACE
    L = gc.lib
    p = table.data_ptr()
    args = [ctx.handle, y.data_ptr(), 8, 0, ids.data_ptr(), 1, 3, -1, 5, 8, 1.0, p, 8, 0]
    for at, value, want in ((2, 7, gc.ERR_INVALID_ARG), (3, 9, gc.ERR_INVALID_ARG),
                            (4, None, gc.ERR_INVALID_ARG), (4, ids.data_ptr() + 4, gc.ERR_ALIGNMENT),
                            (5, 2, gc.ERR_INVALID_ARG), (6, -1, gc.ERR_INVALID_ARG),
                            (8, 2 ** 31, gc.ERR_INVALID_ARG), (11, None, gc.ERR_INVALID_ARG),
                            (11, p + 2, gc.ERR_ALIGNMENT), (12, 7, gc.ERR_INVALID_ARG)):
        call = list(args)
        call[at] = value
        assert L.gc_embedding_wgrad(*call) == want, (at, value)


@pytest.mark.parametrize("vocab,tokens", [(2 ** 18, 3000), (2 ** 20 + 7, 70000), (511, 70000), (512, 2049)])
def test_sorting_passes(gc, ctx, vocab, tokens):
    """One to three radix passes, more than one round of tokens per block, digits of every width."""
    import torch
    r = np.random.default_rng(vocab)
    cols = 8
    ids = np.where(r.random(tokens) < 0.5, r.integers(0, vocab, tokens), r.integers(0, 40, tokens) * (vocab // 40))
    ids[0], ids[1] = 0, vocab - 1
    dy, dyv, _ = matrix(r.standard_normal((tokens, cols)), "f32")
    want, size, n = ref.embedding_wgrad(dyv, ids, vocab, 1.0)
    d, _ = out_matrix(vocab, cols, "f32")
    gc.embedding_wgrad(ctx, dy, tensor_ids(ids, "i32"), 1.0, d)
    close(f64(d), want, (n[:, None] + 2) * 2.0 ** -24 * size, "dtable")
    ctx.check()


@pytest.mark.parametrize("at", [0, 1, 2, 4])
def test_accumulation_at_any_float(gc, ctx, at):
    """Rows that start on and off 16-byte boundaries: the same bits."""
    import torch
    r = np.random.default_rng(at)
    tokens, vocab, cols = 500, 60, 132
    ids = tensor_ids(some_ids(r, tokens, vocab, "skew"), "i64")
    dy, _, _ = matrix(r.standard_normal((tokens, cols)), "f16")
    first = torch.empty(vocab, cols, device="cuda")
    gc.embedding_wgrad(ctx, dy, ids, 1.25, first)
    flat = torch.randn(vocab * cols + 8, device="cuda")
    before = flat.clone()
    view = flat[at:at + vocab * cols].view(vocab, cols)
    gc.embedding_wgrad(ctx, dy, ids, 1.25, view, accumulate=True)
    used = torch.zeros(vocab, 1, dtype=torch.bool, device="cuda")
    used[ids] = True
    old = before[at:at + vocab * cols].view(vocab, cols)
    assert torch.equal(view, torch.where(used, old + first, old))
    assert torch.equal(flat[:at], before[:at]) and torch.equal(flat[at + vocab * cols:], before[at + vocab * cols:])


@pytest.mark.parametrize("tokens", [255, 256, 257])
@pytest.mark.parametrize("kind,vocab", [("one", 3), ("any", 1000), ("skew", 77)])
@pytest.mark.parametrize("dtype,pad", [("f32", 3), ("bf16", 0), ("f16", 1)])
def test_with_and_without_sorting(gc, ctx, tokens, kind, vocab, dtype, pad):
    """Both sides of the number of tokens from which they are sorted."""
    r = np.random.default_rng(tokens)
    cols = 391
    ids = some_ids(r, tokens, vocab, kind)
    ids[::17] = -1
    dy, dyv, _ = matrix(r.standard_normal((tokens, cols)), dtype, pad)
    want, size, n = ref.embedding_wgrad(dyv, ids, vocab, 0.5, -1)
    d, buf = out_matrix(vocab, cols, "f32", pad)
    gc.embedding_wgrad(ctx, dy, tensor_ids(ids, "i32"), 0.5, d, pad=-1)
    close(f64(d), want, (n[:, None] + 2) * 2.0 ** -24 * size, "dtable")
    pad_untouched(buf, cols)
    gc.embedding_wgrad(ctx, dy, tensor_ids(ids, "i32"), 0.5, d, pad=-1, accumulate=True)
    close(f64(d), 2.0 * want, (2 * n[:, None] + 6) * 2.0 ** -24 * size, "dtable, twice")
    pad_untouched(buf, cols)
    ctx.check()

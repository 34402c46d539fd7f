"""The reference of the residual stream's calls against differences and
against properties, the host-only sizes, and refusals (no GPU)."""
import ctypes

import numpy as np
import pytest

from oracle import stream as ref


@pytest.fixture(scope="module")
def gc():
    import __graft_entry__
    __graft_entry__.build()
    from gradient_compression_ef_gb300 import gc as binding
    return binding


def test_rmsnorm_backward_is_the_forward_slope():
    r = np.random.default_rng(0)
    h, dy, dres = (r.standard_normal((3, 7)) for _ in range(3))
    gamma = r.standard_normal(7)
    _, rstd = ref.rmsnorm_forward(h, gamma, 0.1)
    dx, dgamma, _, _ = ref.rmsnorm_backward(dy, dres, h, gamma, rstd)

    def loss(h, g):
        return (dy * ref.rmsnorm_forward(h, g, 0.1)[0]).sum() + (dres * h).sum()

    t = 1e-5
    for i in range(3):
        for j in range(7):
            e = np.zeros((3, 7))
            e[i, j] = t
            assert abs((loss(h + e, gamma) - loss(h - e, gamma)) / (2 * t) - dx[i, j]) < 1e-8
    for j in range(7):
        e = np.zeros(7)
        e[j] = t
        assert abs((loss(h, gamma + e) - loss(h, gamma - e)) / (2 * t) - dgamma[j]) < 1e-8


def test_embedding_gradient_is_the_lookup_transposed():
    r = np.random.default_rng(1)
    ids = np.array([4, 0, 4, -1, 2, 9, 4])
    table, dy = r.standard_normal((5, 3)), r.standard_normal((7, 3))
    y = ref.embedding_forward(ids, table, 2.0, pad=-1)
    d, size, n = ref.embedding_wgrad(dy, ids, 5, 2.0, pad=-1)
    assert np.isclose((dy * y).sum(), (d * table).sum())
    assert n.tolist() == [1, 0, 1, 0, 3] and (size >= np.abs(d) - 1e-12).all()
    assert not y[3].any() and not y[5].any()


def fake(gc):
    """A zeroed context: only for calls that are refused before they look at a device."""
    return ctypes.create_string_buffer(4096)


def test_refusals_before_any_device_work(gc):
    L, c = gc.lib, fake(gc)
    buf = ctypes.create_string_buffer(4096)
    p = (ctypes.addressof(buf) + 255) // 256 * 256
    bad = gc.ERR_INVALID_ARG
    fwd = [c, p, 8, p, 8, 0, 4, 8, p, 0, 1e-5, p, 8, p, 8, p, None, None, None, None]
    for at, value, want in ((0, None, bad), (1, None, bad), (1, p + 4, gc.ERR_ALIGNMENT),
                            (2, 7, bad), (3, p + 8, gc.ERR_ALIGNMENT), (4, 7, bad), (5, 3, bad),
                            (6, -1, bad), (7, 2 ** 31, bad), (8, p + 4, gc.ERR_ALIGNMENT),
                            (9, 5, bad), (10, -1.0, bad), (11, p + 2, gc.ERR_ALIGNMENT),
                            (12, 7, bad), (13, None, bad), (14, 7, bad), (15, None, bad),
                            (15, p + 2, gc.ERR_ALIGNMENT), (16, p, bad), (19, p, bad)):
        call = list(fwd)
        call[at] = value
        assert L.gc_rmsnorm_forward(*call) == want, (at, value)
    back = [c, p, 8, p, 8, p, 8, None, None, 0, 4, 8, p, 0, p, p, 8, p, 0]
    for at, value, want in ((0, None, bad), (1, None, bad), (2, 7, bad), (3, p + 4, gc.ERR_ALIGNMENT),
                            (5, None, bad), (7, p, bad), (9, 7, bad), (13, 3, bad), (14, None, bad),
                            (15, None, bad), (16, 7, bad), (17, p + 1, gc.ERR_ALIGNMENT),
                            (18, 0, gc.ERR_WORKSPACE)):
        call = list(back)
        call[at] = value
        assert L.gc_rmsnorm_backward(*call) == want, (at, value)
    look = [c, p, 1, 4, -1, p, 8, 0, 5, 8, 1.0, p, 8, 1]
    for at, value, want in ((0, None, bad), (1, None, bad), (1, p + 4, gc.ERR_ALIGNMENT), (2, 2, bad),
                            (3, -1, bad), (5, None, bad), (6, 7, bad), (7, 9, bad), (8, -1, bad),
                            (9, -1, bad), (11, None, bad), (12, 7, bad), (13, 3, bad)):
        call = list(look)
        call[at] = value
        assert L.gc_embedding_forward(*call) == want, (at, value)
    grad = [c, p, 8, 0, p, 1, 4, -1, 5, 8, 1.0, p, 8, 0]
    for at, value, want in ((0, None, bad), (1, None, bad), (2, 7, bad), (4, None, bad), (5, 7, bad),
                            (6, 2 ** 31, bad), (8, 2 ** 31, bad), (11, None, bad), (12, 7, bad),
                            (13, 0, gc.ERR_WORKSPACE)):
        call = list(grad)
        call[at] = value
        assert L.gc_embedding_wgrad(*call) == want, (at, value)


def test_orthogonalize_maps_singular_values():
    r = np.random.default_rng(2)
    for m, n in ((6, 9), (9, 6)):
        g = r.standard_normal((m, n))
        coefs = [(3.4445, -4.775, 2.0315)] * 2 + [(1.5, -0.5, 0.0)] * 12
        u, s, vt = np.linalg.svd(g, full_matrices=False)
        x = s / np.sqrt((s ** 2).sum())
        for a, b, c in coefs:
            x = a * x + b * x ** 3 + c * x ** 5
        got = ref.orthogonalize(g, coefs, 0.0, 2.0)
        assert np.allclose(got, 2.0 * (u * x) @ vt, atol=1e-12)
        assert np.allclose(np.linalg.svd(got)[1], 2.0, atol=1e-6)


def test_orthogonalize_refusals_before_any_device_work(gc):
    L, c = gc.lib, fake(gc)
    buf = ctypes.create_string_buffer(4096)
    p = (ctypes.addressof(buf) + 255) // 256 * 256
    bad = gc.ERR_INVALID_ARG
    coefs = (ctypes.c_float * 3)(1.5, -0.5, 0.0)
    good = [c, p, 0, 4, 8, 8, 1, coefs, 1e-7, 1.0, p, 1, 8]
    for at, value, want in ((0, None, bad), (1, None, bad), (1, p + 2, gc.ERR_ALIGNMENT), (2, 3, bad),
                            (3, -1, bad), (3, 2 ** 30 + 1, bad), (4, -1, bad), (5, 7, bad), (6, 0, bad),
                            (7, None, bad), (8, -1.0, bad), (10, None, bad),
                            (10, p + 1, gc.ERR_ALIGNMENT), (11, 5, bad), (12, 7, bad),
                            (6, 1, gc.ERR_WORKSPACE)):
        call = list(good)
        call[at] = value
        assert L.gc_orthogonalize(*call) == want, (at, value)


def test_scratch_sizes(gc):
    assert gc.orthogonalize_scratch_bytes(-1, 4) == -1
    assert gc.orthogonalize_scratch_bytes(0, 4) == 0
    assert gc.orthogonalize_scratch_bytes(64, 128) == gc.orthogonalize_scratch_bytes(128, 64) > 0
    assert gc.rmsnorm_scratch_bytes(-1, 4) == -1 and gc.rmsnorm_scratch_bytes(4, -1) == -1
    assert gc.rmsnorm_scratch_bytes(0, 4096) == 0
    assert gc.rmsnorm_scratch_bytes(10 ** 6, 4096) < 16 << 20  # partial rows, whatever the rows
    assert gc.embedding_scratch_bytes(-1, 4, 4) == -1 and gc.embedding_scratch_bytes(4, 2 ** 31, 4) == -1
    assert gc.embedding_scratch_bytes(0, 10, 10) == 0
    assert gc.embedding_scratch_bytes(8192, 10, 64) >= 8192 * 8 + 128 * 2 * 64 * 4

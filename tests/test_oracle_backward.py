"""Pins of the 64-bit reference of the backward-pass calls: hand cases of the
checkpoint format, gradients against central differences."""
import numpy as np
import pytest

from oracle import backward as ref


def test_format_hand_cases():
    x = np.zeros((1, 70))
    x[0, :6] = [1.0, -1.0, 0.5, 1.5, -0.0078125, 0.0]  # max 1.5: exponent 0, step 2^-6
    x[0, 32:35] = [127.5, 126.5, -0.5]                 # max 127.5: step 1; a clamp, two ties
    x[0, 64] = 2.0 ** -121                             # below the smallest scale
    codes, b = ref.encode(x)
    assert codes.shape == (1, 96) and list(b[0]) == [128, 134, 0]
    assert list(codes[0, :6]) == [64, 128 + 64, 32, 96, 0, 0]  # -2^-7 is half a step: to 0, no sign
    assert list(codes[0, 32:35]) == [127, 126, 0]
    assert not codes[0, 64:].any()
    back = ref.decode(codes, b, 70)
    assert list(back[0, :4]) == [1.0, -1.0, 0.5, 1.5]
    assert list(back[0, 32:35]) == [127.0, 126.0, 0.0]


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan, 2.0 ** 127, -3.0e38])
def test_out_of_range_groups_restore_as_nan(value):
    x = np.ones((2, 40))
    x[1, 33] = value
    codes, b = ref.encode(x)
    assert list(b[0]) == [128, 128] and list(b[1]) == [128, 255]
    back = ref.decode(codes, b, 40)
    assert np.isnan(back[1, 32:]).all() and (back[1, :32] == 1.0).all() and (back[0] == 1.0).all()


def test_error_is_half_a_step_and_values_fit_bf16():
    r = np.random.default_rng(1)
    x = r.standard_normal((50, 96)) * np.exp(3 * r.standard_normal((50, 1)))
    v = ref.restored(x)
    top = np.repeat(np.abs(x.reshape(50, 3, 32)).max(axis=2), 32, axis=1)
    step = np.exp2(np.floor(np.log2(top)) - 6)
    clamped = np.abs(x) > 127 * step
    assert (np.abs(v - x)[~clamped] <= step[~clamped] / 2).all()
    assert (np.abs(v - x) <= step).all()
    bits = v.astype(np.float32).view(np.uint32)
    assert not (bits & 0xFFFF).any() and (v.astype(np.float32) == v).all()


def test_restored_fp16_values_are_exact_in_fp16():
    bits = np.arange(0x7C00, dtype=np.uint16)  # every finite magnitude, as a group of its own
    x = np.zeros((bits.size, 32), np.float16)
    x[:, 0] = bits.view(np.float16)
    x[:, 1] = np.roll(bits, 1).view(np.float16)
    v = ref.restored(x)
    assert (v.astype(np.float16).astype(np.float64) == v).all()


@pytest.mark.parametrize("kind", ["gelu", "silu"])
def test_act_derivative_against_differences(kind):
    x = np.linspace(-9, 9, 181)
    h = 1e-5
    num = (ref.act(kind, x + h)[0] - ref.act(kind, x - h)[0]) / (2 * h)
    assert np.abs(num - ref.act(kind, x)[1]).max() < 1e-8


def test_layernorm_gradient_against_differences():
    r = np.random.default_rng(3)
    x, dy = r.standard_normal((3, 7)), r.standard_normal((3, 7))
    gamma, beta, eps, h = r.standard_normal(7), r.standard_normal(7), 1e-5, 1e-6
    _, mean, rstd = ref.layernorm(x, gamma, beta, eps)
    dx, dg, db = ref.layernorm_backward(dy, x, gamma, mean, rstd)

    def loss(x_, g_, b_):
        return (ref.layernorm(x_, g_, b_, eps)[0] * dy).sum()

    for i in range(3):
        for j in range(7):
            e = np.zeros_like(x)
            e[i, j] = h
            assert abs((loss(x + e, gamma, beta) - loss(x - e, gamma, beta)) / (2 * h)
                       - dx[i, j]) < 1e-7
    for j in range(7):
        e = np.zeros(7)
        e[j] = h
        assert abs((loss(x, gamma + e, beta) - loss(x, gamma - e, beta)) / (2 * h) - dg[j]) < 1e-7
        assert abs((loss(x, gamma, beta + e) - loss(x, gamma, beta - e)) / (2 * h) - db[j]) < 1e-7


def test_linear_gradient_against_differences():
    r = np.random.default_rng(4)
    x, w, dy = r.standard_normal((5, 3)), r.standard_normal((4, 3)), r.standard_normal((5, 4))
    dw, db = ref.linear_wgrad(dy, x)
    h = 1e-6
    for o in range(4):
        for i in range(3):
            e = np.zeros_like(w)
            e[o, i] = h
            num = ((x @ (w + e).T * dy).sum() - (x @ (w - e).T * dy).sum()) / (2 * h)
            assert abs(num - dw[o, i]) < 1e-7
    assert np.allclose(db, dy.sum(axis=0))


def test_sizes_and_refusals_on_the_host():
    import __graft_entry__
    __graft_entry__.build()
    from gradient_compression_ef_gb300 import gc
    for rows in (0, 1, 3, 1000):
        for cols in (0, 1, 31, 32, 33, 512, 513, 4096, 11008):
            assert gc.ckpt_codes_bytes(rows, cols) == rows * ref.codes_pitch(cols)
            assert gc.ckpt_scales_bytes(rows, cols) == rows * ref.scales_pitch(cols)
    assert gc.ckpt_codes_bytes(-1, 4) == gc.ckpt_scales_bytes(4, -1) == -1
    assert gc.layernorm_scratch_bytes(-1, 4) == -1
    assert gc.layernorm_scratch_bytes(100, 64) >= 0
    assert gc.linear_wgrad_scratch_bytes(5, 5, -1, "bf16") == -1
    L, bad = gc.lib, gc.ERR_INVALID_ARG
    assert L.gc_ctx_reserve_scratch(None, 10) == bad
    assert L.gc_ckpt_save(None, None, 0, 1, 1, 1, None, None) == bad
    assert L.gc_ckpt_restore(None, None, None, 0, 1, 1, None, 1) == bad
    assert L.gc_act_forward(None, 0, None, 1, None, 0, 0, 1, 1, None, 1, None, None, None,
                            None) == bad
    assert L.gc_act_backward(None, 0, None, 1, None, None, None, None, 0, 1, 1, None, 1, None,
                             0) == bad
    assert L.gc_layernorm_forward(None, None, 1, 0, 1, 1, None, None, 0, 1e-5, None, 1, None, None,
                                  None, None) == bad
    assert L.gc_layernorm_backward(None, None, 1, None, 0, None, None, 0, 1, 1, None, 0, None,
                                   None, None, 1, None, None, 0) == bad
    assert L.gc_linear_wgrad(None, None, 0, 1, None, None, 1, 1, 1, None, 1, None, 0) == bad
    names = [gc.phase_name(p) for p in range(gc.PHASE_COUNT)]
    assert len(set(names)) == gc.PHASE_COUNT and "?" not in names

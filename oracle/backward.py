"""64-bit NumPy reference of the calls that fill the flat gradient: the 8-bit
activation checkpoint, the activation functions, layer norm and the linear
layer's weight gradient.  Written from the definitions in include/gc.h; it
shares no code with the CUDA library.
"""
import numpy as np

GROUP = 32


def codes_pitch(cols):
    return -(-cols // 32) * 32


def scales_pitch(cols):
    return -(-(-(-cols // 32)) // 16) * 16


def encode(x):
    """(codes, scale bytes, groups' scale bytes only) of x [rows, cols]; the
    scale rows come without their padding."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    ng = -(-cols // GROUP)
    g = np.zeros((rows, ng * GROUP))
    g[:, :cols] = x
    g = g.reshape(rows, ng, GROUP)
    with np.errstate(invalid="ignore"):
        top = np.abs(g).max(axis=2)  # NaN if any is NaN
    bad = ~np.isfinite(top) | (top >= 2.0 ** 127)
    small = top < 2.0 ** -120
    safe = np.where(bad | small, 1.0, top)
    _, e = np.frexp(safe)            # safe = f * 2^e, 1/2 <= f < 1
    b = np.where(bad, 255, np.where(small, 0, e + 127)).astype(np.int64)
    with np.errstate(invalid="ignore"):
        m = np.rint(np.abs(g) * np.exp2(134.0 - (e + 127))[..., None])
    m = np.minimum(m, 127.0)
    m = np.where((bad | small)[..., None], 0.0, m)
    code = m.astype(np.int64) + np.where((g < 0) & (m > 0), 128, 0)
    return (code.astype(np.uint8).reshape(rows, ng * GROUP), b.astype(np.uint8))


def decode(codes, b, cols):
    rows, width = codes.shape
    c = codes.reshape(rows, width // GROUP, GROUP).astype(np.int64)
    v = (c & 127) * np.exp2(b.astype(np.float64) - 134.0)[..., None]
    v = np.where(c > 127, -v, v)
    v = np.where((b == 255)[..., None], np.nan, v)
    return v.reshape(rows, width)[:, :cols]


def restored(x):
    x = np.asarray(x, np.float64)
    return decode(*encode(x), x.shape[1])


def act(kind, x):
    """f(x), f'(x)."""
    from scipy.special import expit, ndtr
    x = np.asarray(x, np.float64)
    if kind == "gelu":
        phi = np.exp(-0.5 * x * x) / np.sqrt(2.0 * np.pi)
        return x * ndtr(x), ndtr(x) + x * phi
    s = expit(x)
    return x * s, s * (1.0 + x * expit(-x))


def layernorm(x, gamma, beta, eps):
    """y, mean, rstd."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mean, rstd


def layernorm_backward(dy, x, gamma, mean, rstd):
    """dx, dgamma, dbeta of the given row statistics (x: the input, or what
    its checkpoint stands for)."""
    dy = np.asarray(dy, np.float64)
    n = (np.asarray(x, np.float64) - mean[:, None]) * rstd[:, None]
    d = dy if gamma is None else dy * gamma
    dx = rstd[:, None] * (d - d.mean(axis=1, keepdims=True)
                          - n * (d * n).mean(axis=1, keepdims=True))
    return dx, (dy * n).sum(axis=0), dy.sum(axis=0)


def linear_wgrad(dy, x):
    """dw [out, in], db [out]."""
    dy = np.asarray(dy, np.float64)
    return dy.T @ np.asarray(x, np.float64), dy.sum(axis=0)

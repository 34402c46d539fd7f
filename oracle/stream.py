"""64-bit NumPy reference of the calls around the residual stream and the
update: RMS norm behind the residual's addition, embedding lookup and the
table's gradient, orthogonalisation by Newton-Schulz products.  Written from
the definitions in include/gc.h; it shares no code with the CUDA library.
"""
import numpy as np


def rmsnorm_forward(h, gamma, eps):
    """(y, rstd) of h as it is stored."""
    h = np.asarray(h, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        rstd = 1.0 / np.sqrt(np.square(h).sum(axis=1) / h.shape[1] + eps)
        return h * rstd[:, None] * (1.0 if gamma is None else gamma), rstd


def rmsnorm_backward(dy, dres, h, gamma, rstd):
    """(dx, dgamma, size of the terms of dx, of dgamma): the sizes are what a
    rounding's part is taken of."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    n = h * np.asarray(rstd, np.float64)[:, None]
    d = dy * (1.0 if gamma is None else gamma)
    with np.errstate(invalid="ignore", over="ignore"):
        mean = (d * n).sum(axis=1, keepdims=True) / h.shape[1]
        size = (np.abs(d * n)).sum(axis=1, keepdims=True) / h.shape[1]
        dx = np.asarray(rstd)[:, None] * (d - n * mean)
        dx_size = np.asarray(rstd)[:, None] * (np.abs(d) + np.abs(n) * size)
        if dres is not None:
            dx = dx + dres
            dx_size = dx_size + np.abs(dres)
        return dx, (dy * n).sum(axis=0), dx_size, np.abs(dy * n).sum(axis=0)


def embedding_forward(ids, table, scale, pad=None):
    ids = np.asarray(ids)
    y = np.zeros((ids.size, table.shape[1]))
    for t, v in enumerate(ids):
        if v != pad and 0 <= v < table.shape[0]:
            y[t] = scale * np.asarray(table[v], np.float64)
    return y


def embedding_wgrad(dy, ids, vocab, scale, pad=None):
    """(dtable, sum of magnitudes, tokens of each id)."""
    dy, ids = np.asarray(dy, np.float64), np.asarray(ids)
    ok = (ids >= 0) & (ids < vocab)
    if pad is not None:
        ok &= ids != pad
    d, size = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1]))
    np.add.at(d, ids[ok], dy[ok])
    np.add.at(size, ids[ok], np.abs(dy[ok]))
    return scale * d, abs(scale) * size, np.bincount(ids[ok].astype(np.int64), minlength=vocab)


def orthogonalize(g, coefs, eps, scale):
    """scale * X_k with X_0 = g / (|g|_F + eps) and, for each (a, b, c),
    X <- a X + (b A + c A A) X, A = X X^T."""
    g = np.asarray(g, np.float64)
    if not np.isfinite(g).all():
        return np.full(g.shape, np.nan)
    x = g / (np.linalg.norm(g) + eps)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    for a, b, c in coefs:
        gram = x @ x.T
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return scale * (x.T if tall else x)

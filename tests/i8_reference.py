"""The 8-bit operators in plain float64 numpy, for the tests.

Where the contract rounds on the way (the residual sum to the tensors' type, the norm's product with
its weight to float32), the reference rounds there too and is otherwise in 64 bits.
"""
import numpy as np
import torch


def f64(t):
    return t.detach().double().cpu().numpy()


def levels(v):
    """(q, A) of float32 rows held in float64: 127 v / A to the nearest integer, ties to even. 127 v has at
    most 31 significant bits and A 24, so a quotient that is not a half keeps 2^-33 away from one
    and the division's rounding (2^-53) cannot bring it there."""
    a = np.abs(v).max(axis=1)
    ok = np.isfinite(v).all(axis=1) & (a > 0)
    q = np.zeros(v.shape, np.int64)
    q[ok] = np.rint(v[ok] * 127.0 / a[ok, None])
    return q, a


def rows(v):
    """(q, scale) of quant_rows for rows v of float32 values."""
    q, a = levels(v)
    return q, np.where(np.isfinite(v).all(axis=1), a / 127.0, np.nan)


def rmsnorm(x, weight, residual=None, eps=1e-6):
    """(q, scale, h) of the norm; h in the tensors' type."""
    if residual is None:
        h = x.cpu()
    else:
        h = (x.cpu().float() + residual.cpu().float()).to(x.dtype)   # one float32 sum, rounded to the type
    hd = f64(h)
    with np.errstate(all="ignore"):
        t = (h.float().numpy() * weight.cpu().numpy()).astype(np.float64)   # float32 product
        q, a = levels(t)
        ss = (hd * hd).sum(axis=1)
        scale = a / np.sqrt(ss / hd.shape[1] + np.float64(np.float32(eps))) / 127.0
        bad = ~np.isfinite(t).all(axis=1) | ~np.isfinite(hd).all(axis=1) | (ss > np.finfo(np.float32).max)
    q[bad] = 0
    return q, np.where(bad, np.nan, scale), h


def glu(x):
    """silu(gate) * up in float64."""
    v = f64(x)
    c = v.shape[1] // 2
    with np.errstate(over="ignore"):
        return v[:, :c] / (1.0 + np.exp(-v[:, :c])) * v[:, c:]


def product(q, qs, wq, ws, bias):
    """(y, the sum of the magnitudes that are rounded) of the product in float64; the sum itself is exact."""
    acc = q.cpu().numpy().astype(np.float64) @ wq.cpu().numpy().astype(np.float64).T   # |sum| < 2^31: exact
    y = acc * f64(qs)[:, None] * f64(ws)[None, :]
    mag = np.abs(y)
    if bias is not None:
        y = y + f64(bias)
        mag = mag + np.abs(f64(bias))
    return y, mag


def round_half(dtype):
    """Half a step of a type, relative to the value."""
    return torch.finfo(dtype).eps / 2

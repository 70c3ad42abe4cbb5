"""Float64 oracle of the residual RMS norm, its 8-bit form, its gradients, row quantisation and the 8-bit
product, with the elementwise error bounds that fp32 arithmetic and one final rounding allow.

Values are NumPy arrays; ``T`` names a storage type ("bf16" or "f32").  Storage roundings that belong to the
definitions (the stored sum, the fp32 product under the 8-bit code) are taken here too; everything else is
float64.  Unit roundoffs: fp32 2^-24, bf16 2^-8 (half a step, relative to the value).
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24
ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f32": 2.0 ** -149}     # smallest steps
# Longest chain of fp32 additions that a row sum may run through (elements of one thread, then a tree), and the
# handful of further roundings of a value (weight, rstd, products).
CHAIN = 64 + 12
OPS = 8


def store(v: np.ndarray, T: str) -> np.ndarray:
    """v rounded once (nearest even) to T, as float64."""
    v = np.asarray(v, dtype=np.float64)
    if T == "f32":
        with np.errstate(over="ignore"):
            return v.astype(np.float32).astype(np.float64)
    m, e = np.frexp(v)                               # |m| in [1/2, 1): 8 significant bits from 2^e
    e = np.maximum(e, -125)                          # subnormals share the step of the smallest normals
    q = np.ldexp(np.rint(np.ldexp(v, 8 - e)), e - 8)
    q = np.where(np.abs(q) >= 2.0 ** 128, np.copysign(np.inf, v), q)
    return np.where(np.isfinite(v), q, v)


def residual_sum(x: np.ndarray, r, T: str) -> np.ndarray:
    """s = T(fp32(x + r)): the addition is fp32, the storage rounding follows."""
    if r is None:
        return x
    with np.errstate(over="ignore", invalid="ignore"):
        return store((x.astype(np.float32) + r.astype(np.float32)).astype(np.float64), T)


def rstd_of(s: np.ndarray, eps: float) -> np.ndarray:
    eps = float(np.float32(eps))
    return 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)


def rms_norm(s: np.ndarray, w, eps: float):
    y = s * rstd_of(s, eps)
    return y if w is None else y * w


def rms_norm_bound(y: np.ndarray, T: str) -> np.ndarray:
    """A row sum off by CHAIN roundings moves rstd by half of that; OPS more; one storage rounding."""
    return np.abs(y) * ((CHAIN / 2 + OPS) * U32 + ROUND[T]) + TINY[T]


def codes(p: np.ndarray):
    """(q, m) of p (fp32 values): rint(127 p / m); zero rows give zeros."""
    m = np.abs(p).max(-1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.rint(p * 127.0 / m)
    return np.where(m > 0, q, 0.0).astype(np.int64), m


def rms_norm_i8(s: np.ndarray, w, eps: float):
    p = s if w is None else (s.astype(np.float32) * w.astype(np.float32)).astype(np.float64)
    q, m = codes(p)
    return q, (m * rstd_of(s, eps) / 127.0)[..., 0]


def quantize_rows_i8(x: np.ndarray):
    q, m = codes(x)
    return q, m[..., 0] / 127.0


def rms_norm_backward(dy: np.ndarray, s: np.ndarray, w, eps: float, ds):
    """(dx, dw, bound factors): see backward_bounds."""
    rs = rstd_of(s, eps)
    xh = s * rs
    g = dy if w is None else dy * w
    dx = rs * (g - xh * (g * xh).mean(-1, keepdims=True))
    return (dx if ds is None else dx + ds), (dy * xh).sum(0)


def backward_bounds(dy, s, w, eps, ds, T):
    """(bound of dx, bound of dw).  The mean is off by CHAIN roundings of its terms' magnitudes and rstd^2 by
    CHAIN more; the rest are OPS roundings of each term.  A column of dw is N products added in fp32 chains of
    at most 16 additions, which fp64 sums join and one rounding follows."""
    rs = rstd_of(s, eps)
    xh = s * rs
    g = dy if w is None else dy * w
    dx, _ = rms_norm_backward(dy, s, w, eps, ds)
    mag = rs * (np.abs(g) + np.abs(xh) * np.abs(g * xh).mean(-1, keepdims=True))
    b = mag * (2 * CHAIN + OPS) * U32 + np.abs(dx) * (ROUND[T] + U32) + TINY[T]
    if ds is not None:
        b = b + np.abs(ds) * U32
    chain = 16 + 1
    return b, np.abs(dy * xh).sum(0) * (CHAIN / 2 + OPS + chain) * U32 + TINY["f32"]


def matmul_i8(a, a_scale, b, b_scale, bias):
    out = (a.astype(np.float64) @ b.astype(np.float64).T) * a_scale[:, None] * b_scale[None, :]
    return out if bias is None else out + bias


def matmul_i8_bound(out, bias, T):
    """Integer sums are exact; their conversion, two scalings and the bias's addition round once each."""
    prod = out if bias is None else out - bias
    return np.abs(prod) * 4 * U32 + np.abs(out) * (ROUND[T] + 2 * U32) + TINY[T]

"""Layer norm, its gradient and the row quantiser from their formulas, in float64 numpy, with the bounds on
what float32 arithmetic may add to them.  Shares no code with the library."""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24                                # half a unit in the last place, relative, of float32
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # one rounding to the layer's dtype
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def norm(s, w, b, eps):
    """y, mean, rstd of the rows of s (float64)."""
    mean = s.mean(1)
    d = s - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    return d * rstd[:, None] * w + b, mean, rstd


def norm_bound(s, w, b, eps, dtype):
    """Elementwise bound on |y - norm()|.

    A thread adds at most 16 values of a row, a wave 6 partial sums, a workgroup 16: a sum over a row is off by fewer
    than 54 roundings of the mean magnitude M (the division and the eps addition: two more), so
      |mean'| error <= 56 u M,
      d = s - mean' carries that plus one rounding of |d|,
      the sum of squares 54 + 2 roundings and twice d's error (relative to the row's spread 1/rstd); the square root
      halves it; the square root and the reciprocal add one rounding each,
    and y = (d rstd) w + b adds three."""
    _, mean, rstd = norm(s, w, b, eps)
    m = np.abs(s).mean(1, keepdims=True) + np.abs(mean)[:, None]
    r = rstd[:, None]
    xh = np.abs(s - mean[:, None]) * r
    off = 56 * U32 * m * r                       # the mean's error in units of the spread
    rel = 30 * U32 + 2 * U32 + 2 * off           # relative error of rstd
    err = (off + U32 * xh + xh * (rel + 3 * U32)) * np.abs(w) + 3 * U32 * np.abs(b)
    y = np.abs((s - mean[:, None]) * r * w + b)
    return err + HALF_STEP[dtype] * (y + err)


def norm_grad(gy, s, w, mean, rstd, gs):
    xh = (s - mean[:, None]) * rstd[:, None]
    h = gy * w
    m1, m2 = h.mean(1, keepdims=True), (h * xh).mean(1, keepdims=True)
    dx = rstd[:, None] * (h - m1 - xh * m2)
    if gs is not None:
        dx = dx + gs
    return dx, (gy * xh).sum(0), gy.sum(0)


def norm_grad_bounds(gy, s, w, mean, rstd, gs, dtype):
    """Elementwise bounds for (grad_x, grad_weight, grad_bias).

    xh carries two roundings, h one.  Row means: at most 16 values in a thread, 6 + 16 partial sums, two roundings of
    scaling: fewer than 56 of the mean magnitude.  Column sums: a thread adds its rows one after the other (at most
    ceil(T / 256) of them, each product with three roundings), a workgroup up to 16 groups, then 16 partials of the 256
    and the 16 sums of those."""
    T = s.shape[0]
    xh = np.abs((s - mean[:, None]) * rstd[:, None])
    h = np.abs(gy * w)
    r = np.abs(rstd)[:, None]
    m1, m2 = h.mean(1, keepdims=True), (h * xh).mean(1, keepdims=True)
    err = r * U32 * (4 * h + 58 * m1 + xh * 66 * m2)
    if gs is not None:
        err = err + U32 * (np.abs(gs) + r * (h + m1 + xh * m2))
    dx = np.abs(norm_grad(gy, s, w, mean, rstd, gs)[0])
    n = -(-T // 256) + 16 + 16 + 16
    return (err + HALF_STEP[dtype] * (dx + err), (n + 4) * U32 * np.abs(gy * xh).sum(0) + 1e-30,
            n * U32 * np.abs(gy).sum(0) + 1e-30)


def quantize(x):
    """(q, scale): the exact quotient rounded to nearest, ties to even.  127 x is exact in float64 for float32 x, and a
    quotient that is no tie is further from one than float64's rounding."""
    big = np.abs(x).max(1)
    bad = ~np.isfinite(x).all(1)
    den = np.where(bad | (big == 0), 1.0, big)[:, None]
    q = np.rint(127.0 * np.where(bad[:, None], 0.0, x) / den)
    return q.astype(np.int8), np.where(bad, np.nan, (big.astype(np.float32) / np.float32(127.0)))

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


def norm_bound_about_mean(s, w, b, eps, dtype):
    """Elementwise bounds on |y - norm()|, |mean - norm()| and |rstd / norm() - 1| that do not grow with a row's common
    offset.  f32: for a mean that is summed in float64 and subtracted as two float32 parts; bf16: for rows whose values
    lie in one binade, so that float32 holds their sums (8 + 14 bits) and only the mean is rounded, to c = U |mean| where
    neighbouring values of a row are 2^-8 |mean| apart.

    Fewer than 54 additions and a division in float64 leave the mean within v = 56 2^-53 M, M = mean|s| + |mean|; its
    second part is at most U |mean| and rounded once, so
      d = (s - high) - low is off by 2 U |d| (two subtractions) and at most c = 3 U^2 |mean| + v.
    The sum of squares adds 54 roundings and two more for the division and eps, d's error twice 2 U and 2 c rstd; the
    square root halves them, it and the reciprocal add one each; y = (d rstd) w + b adds two."""
    _, mean, rstd = norm(s, w, b, eps)
    r, m = rstd[:, None], np.abs(mean)[:, None]
    v = 56 * 2.0 ** -53 * (np.abs(s).mean(1, keepdims=True) + m)
    c = 3 * U32 ** 2 * m + v if dtype == "f32" else U32 * m
    d = np.abs(s - mean[:, None])
    rel = (30 + 2) * U32 + c * r
    err = (r * (2 * U32 * d + c) + r * d * (rel + 2 * U32)) * np.abs(w) + 2 * U32 * np.abs(b)
    y = np.abs((s - mean[:, None]) * r * w + b)
    return err + HALF_STEP[dtype] * (y + err), (U32 * m + v)[:, 0], rel[:, 0]


# (H, offset, spread) of rows whose values share a large offset; float32 resolves the spread in 16 to 160 steps
OFFSETS = [(324, 1000.1, 0.01), (1020, -1e4, 0.02), (2052, 1000.1, 0.01), (4100, 3e5, 0.6), (8196, 1e4, 0.02),
           (16384, 1000.1, 0.01)]


# the same for bf16 within a binade, the spread 4, 9 and 1.5 of its steps
OFFSETS_BF16 = [(320, 768.0, 16.0), (2112, -24.0, 1.125), (16384, 3.0 * 2 ** 20, 24576.0)]


def offset_rows(T, H, offset, spread):
    """Values around the offset, at most a quarter of it away."""
    x = spread * np.random.default_rng(H).normal(size=(T, H))
    return (offset + np.clip(x, -abs(offset) / 4, abs(offset) / 4)).astype(np.float32)


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

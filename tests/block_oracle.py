"""Float64 references of the router, of dropout's mask and of 4-bit matrices, row by row in numpy (test infrastructure)."""
from __future__ import annotations

import math

import numpy as np

U32 = 2.0 ** -24  # half a float32 step, relative
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------------------ router
def scores(row: np.ndarray, score: str) -> np.ndarray:
    if score == "sigmoid":
        return np.array([1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 for v in row])
    m = row.max()
    if m == -np.inf:
        return np.zeros_like(row)
    e = np.exp(row - m)
    return e / e.sum()


def route_row(row, bias, score, G, limit, k):
    """The ids of one row, -1 where no expert is left."""
    E = len(row)
    key = row.copy()
    if bias is not None or 0 < limit < G:
        s = scores(row, score)
        key = np.array([s[e] + (0.0 if bias is None else bias[e])
                        if row[e] > -np.inf and (bias is None or np.isfinite(bias[e])) else -np.inf for e in range(E)])
    if 0 < limit < G:
        n = E // G
        total = [sum(sorted(key[g * n:(g + 1) * n])[-2:]) for g in range(G)]
        open_ = sorted(range(G), key=lambda g: (-total[g], g))[:limit]
        key = np.array([key[e] if e // n in open_ else -np.inf for e in range(E)])
    order = sorted(range(E), key=lambda e: (-key[e], e))
    ids = [e for e in order if key[e] > -np.inf][:k]
    return ids + [-1] * (k - len(ids))


def weights_row(row, ids, score, renorm, factor):
    """Weights of the ids, also where scores underflow (in extended precision)."""
    L = np.longdouble
    kept = [e for e in ids if e >= 0]
    if score == "sigmoid":
        s = {e: 1 / (1 + np.exp(-L(row[e]))) for e in kept}
    else:
        m = L(row.max())
        total = np.exp(row.astype(L) - m).sum() if kept else L(1)
        s = {e: np.exp(L(row[e]) - m) / total for e in kept}
    total = sum(s[e] for e in kept) if renorm else L(1)
    return [float(L(factor) * s[e] / total) if e >= 0 else 0.0 for e in ids]


def route_grad_row(row, ids, g, score, renorm, factor):
    """Gradient of the logits and the sum of magnitudes that its rounding is held to."""
    E = len(row)
    grad, size = np.zeros(E), np.zeros(E)
    kept = [j for j, e in enumerate(ids) if 0 <= e < E and row[e] > -np.inf]
    c = {j: factor * g[j] for j in kept}
    if not kept:
        return grad, size
    if renorm:
        w = weights_row(row, [ids[j] for j in kept], score, True, 1.0)
        q = dict(zip(kept, w))
        S, SA = sum(q[j] * c[j] for j in kept), sum(q[j] * abs(c[j]) for j in kept)
        for j in kept:
            tail = 1.0 / (1.0 + math.exp(min(row[ids[j]], 700.0))) if score == "sigmoid" else 1.0
            grad[ids[j]] += q[j] * (c[j] - S) * tail
            size[ids[j]] += q[j] * (abs(c[j]) + SA) * tail
        return grad, size
    p = scores(row, score)
    if score == "sigmoid":
        for j in kept:
            v = p[ids[j]] / (1.0 + math.exp(min(row[ids[j]], 700.0)))
            grad[ids[j]] += v * c[j]
            size[ids[j]] += v * abs(c[j])
        return grad, size
    S, SA = sum(p[ids[j]] * c[j] for j in kept), sum(p[ids[j]] * abs(c[j]) for j in kept)
    for j in kept:
        grad[ids[j]] += p[ids[j]] * c[j]
        size[ids[j]] += p[ids[j]] * abs(c[j])
    return grad - p * S, size + p * SA


# ------------------------------------------------------------------ dropout
def philox(c, k):
    """One block of Philox 4x32-10 on Python integers."""
    c, k, low = list(c), list(k), 0xFFFFFFFF
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & low, (a >> 32) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return c


def kept_mask(n: int, p: float, seed: int, offset: int, first: int = 0) -> np.ndarray:
    """Elements 8 * first .. 8 * first + n - 1."""
    least, low = min(65535, round(p * 65536)), 0xFFFFFFFF
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    halves = []
    for v in range(first, first + -(-n // 8)):
        w = philox((v & low, v >> 32, offset & low, offset >> 32), (seed & low, seed >> 32))
        halves += [h for x in w for h in (x & 0xFFFF, x >> 16)]
    return np.array(halves[:n]) >= least


# ------------------------------------------------------------------ 4-bit matrices
def quantize_row_major(x: np.ndarray):
    """Codes [rows][cols] and scale bytes [rows][cols/32] of float64 x."""
    rows, cols = x.shape
    g = x.reshape(rows, cols // 32, 32)
    codes, bytes_ = np.zeros(g.shape, np.uint8), np.zeros(g.shape[:2], np.uint8)
    for i in np.ndindex(*g.shape[:2]):
        v = g[i]
        if not np.isfinite(v).all():
            bytes_[i] = 255
            continue
        big = np.abs(v).max()
        s = -127
        if big > 0:
            s = max(-127, int(math.floor(math.log2(big))) - 3)
            while big > 6.0 * 2.0 ** s:
                s += 1
        bytes_[i] = s + 127
        a = np.minimum(np.abs(v) / 2.0 ** s, 3.0 if s == 126 else np.inf)
        d = np.abs(a[:, None] - E2M1[None, :])
        best = d.min(1, keepdims=True)
        # of two equally near codes the even one
        code = np.array([min((c for c in range(8) if d[j, c] == best[j, 0]), key=lambda c: c & 1) for j in range(32)])
        codes[i] = code + 8 * np.signbit(v)
    return codes.reshape(rows, cols), bytes_


def values(codes: np.ndarray, bytes_: np.ndarray) -> np.ndarray:
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    power = np.where(bytes_ == 255, np.nan, 2.0 ** (bytes_.astype(np.float64) - 127))
    return v * np.repeat(power, 32, axis=1)


def pack(codes: np.ndarray, bytes_: np.ndarray):
    """Packed values and scales, each byte placed by the layout's formula."""
    rows, cols = codes.shape
    nk, nq = cols // 64, -(-cols // 256)
    q, scale = np.zeros(rows * cols // 2, np.uint8), np.zeros(rows // 32 * nq * 256, np.uint8)
    r, c = np.meshgrid(np.arange(rows), np.arange(0, cols, 2), indexing="ij")
    at = ((r // 32) * nk + c // 64) * 1024 + ((c % 64 // 32) * 32 + r % 32) * 16 + c % 32 // 2
    q[at] = codes[:, 0::2] | codes[:, 1::2] << 4
    r, b = np.meshgrid(np.arange(rows), np.arange(cols // 32), indexing="ij")
    at = ((r // 32) * nq + b // 8) * 256 + ((b % 2) * 32 + r % 32) * 4 + b // 2 % 4
    scale[at] = bytes_
    return q, scale

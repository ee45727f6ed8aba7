"""FP64 oracle of the layer norm and of dropout (TEST INFRASTRUCTURE ONLY).

Plain numpy in float64, written from the closed forms; shares no code with the
CUDA library.  Besides the values it returns, element by element, how far an
FP32 evaluation of the same formulas may be from them (see `forward`), and
replays the order of the parameter gradients in float32.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24          # relative rounding error of one FP32 operation

# A row sum is a tree whose longest chain of additions is at most 64 (at most 32
# elements of a thread, 5 levels of a warp, at most 16 warps, and the rounding of
# 1/H and of the product), so a mean of terms t carries at most DEPTH * U * mean|t|.
DEPTH = 64


def keep_mask(seed: int, offset: int, rows, hidden: int, p: float) -> np.ndarray:
    """keep[i, h] of logical row rows[i]: 16 bits an element of Philox4x32-10 with
    key (seed) and counter (h // 8, row, offset)."""
    t = int(np.rint(p * 65536.0))
    rows = np.asarray(rows, dtype=np.uint64)
    u16 = np.empty((rows.size, hidden // 8, 8), dtype=np.int64)
    m = np.uint64(0xFFFFFFFF)
    s = np.uint64(32)
    a = np.broadcast_to(np.arange(hidden // 8, dtype=np.uint64), (rows.size, hidden // 8)).copy()
    b = np.broadcast_to(rows[:, None], a.shape).copy()
    c = np.full(a.shape, offset & 0xFFFFFFFF, dtype=np.uint64)
    d = np.full(a.shape, (offset >> 32) & 0xFFFFFFFF, dtype=np.uint64)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        p0, p1 = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)
        a, b, c, d = (p1 >> s) ^ b ^ np.uint64(k0), p1 & m, (p0 >> s) ^ d ^ np.uint64(k1), p0 & m
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    for i, w in enumerate((a, b, c, d)):
        u16[:, :, 2 * i] = (w & np.uint64(0xFFFF)).astype(np.int64)
        u16[:, :, 2 * i + 1] = (w >> np.uint64(16)).astype(np.int64)
    return u16.reshape(rows.size, hidden) >= t


def philox(ctr, key):
    """One evaluation on Python integers: four words of four counter words and two key words."""
    c, k = list(ctr), list(key)
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return tuple(c)


def drop_scale(p: float) -> float:
    t = int(np.rint(p * 65536.0))
    return 65536.0 / (65536 - t) if t < 65536 else 0.0


def forward(x, w, b, eps: float):
    """(y, mean, rstd, err) in float64 of x [n, H]; err bounds an FP32 evaluation
    before the rounding of y to its type.

    mean: off by DEPTH U A, A = mean|x|.  x - mean: that plus U|x - mean|.  The
    variance takes the error of the mean squared (the deviations sum to zero) and
    DEPTH U of itself, so rstd is off by less than (DEPTH / 2 + 8) U of itself and
    xhat by (DEPTH / 2 + 10) U |xhat| + (DEPTH + 2) U A rstd; y adds two roundings."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(1, keepdims=True)
    d = x - mean
    rstd = 1.0 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    xhat = d * rstd
    ex = xhat_error(x, xhat, rstd)
    y = xhat * w + b
    err = np.abs(w) * ex + 3 * U * (np.abs(xhat * w) + np.abs(b))
    return y, mean[:, 0], rstd[:, 0], err


def xhat_error(x, xhat, rstd):
    a = np.abs(x).mean(1, keepdims=True)
    return U * ((DEPTH / 2 + 10) * np.abs(xhat) + (DEPTH + 2) * a * rstd)


def backward(x, w, dy, eps: float):
    """(dx, dweight, dbias, err_dx, err_dw, err_db) in float64, dx unscaled and unrounded.

    With a = dy w: the two means carry (DEPTH + 3) U of the mean of their terms'
    sizes and, the second one, the mean of |a| times xhat's error; the three
    terms of dx and their sum are rounded a few times, and rstd's own error
    scales the whole.  The parameter gradients add their terms along chains of
    at most 8 + 8 + 31 additions."""
    x = np.asarray(x, dtype=np.float64)
    dy = np.asarray(dy, dtype=np.float64)
    mean = x.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    xhat = (x - mean) * rstd
    a = dy * w
    ma, mc = a.mean(1, keepdims=True), (a * xhat).mean(1, keepdims=True)
    dx = rstd * (a - ma - xhat * mc)
    ex = xhat_error(x, xhat, rstd)
    ama, amc = np.abs(a).mean(1, keepdims=True), np.abs(a * xhat).mean(1, keepdims=True)
    e_mc = (DEPTH + 3) * U * amc + (np.abs(a) * ex).mean(1, keepdims=True)
    size = np.abs(a) + ama + np.abs(xhat) * amc
    err = rstd * (ex * np.abs(mc) + np.abs(xhat) * e_mc + (DEPTH + 3) * U * ama + 6 * U * size
                  + (DEPTH / 2 + 8) * U * size)
    chain = 48
    err_dw = (np.abs(dy) * ex).sum(0) + chain * U * np.abs(dy * xhat).sum(0)
    err_db = chain * U * np.abs(dy).sum(0)
    return dx, (dy * xhat).sum(0), dy.sum(0), err, err_dw, err_db


def rounded(err, ref, dtype: str):
    """Bound of the error after one rounding to the type: half a step of the value, or
    half the smallest subnormal, on top of the FP32 error."""
    half, tiny = {"bfloat16": (2.0 ** -9, 2.0 ** -134), "float16": (2.0 ** -12, 2.0 ** -25),
                  "float32": (0.0, 0.0)}[dtype]
    # a value just above a power of two is at most 2^-p of itself off (p the type's
    # precision); relative to the reference that is the half step of eps / 2
    return err + 2 * half * (np.abs(ref) + err) + tiny


def grad_replay(dy: np.ndarray, xhat: np.ndarray = None) -> np.ndarray:
    """float32 replay of the parameter gradients' order for exact leaves dy * xhat
    (dy alone without xhat): groups of 8 rows from the first to the last, the groups
    of a 64-row block likewise, then adjacent pairs of blocks with odd carry."""
    leaf = dy.astype(np.float32) if xhat is None else dy.astype(np.float32) * xhat.astype(np.float32)
    n, H = leaf.shape
    blocks = []
    for b0 in range(0, n, 64):
        acc = None
        for g0 in range(b0, min(b0 + 64, n), 8):
            v = np.zeros(H, np.float32)
            for r in range(g0, min(g0 + 8, n)):
                v = v + leaf[r]
            acc = v if acc is None else acc + v
        blocks.append(acc)
    while len(blocks) > 1:
        blocks = [blocks[i] + blocks[i + 1] if i + 1 < len(blocks) else blocks[i] for i in range(0, len(blocks), 2)]
    return blocks[0] if blocks else np.zeros(H, np.float32)

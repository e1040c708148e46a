"""Plain 64-bit forms of the operators around and inside the expert sublayer
(norm, dropout, block-scaled e4m3 products and experts) and the bounds their
tests use.  numpy only; nothing here calls the CUDA library.

Roundings: u32 = 2^-24 is half a step of fp32, u16 = 2^-8 half a step of bf16.
A sum of n fp32 terms in any order is off by at most (n - 1) u32 times the sum of
their magnitudes; the tensor cores may cut instead of round, which doubles u32."""
from __future__ import annotations

import math

import numpy as np

U32, U16 = 2.0 ** -24, 2.0 ** -8
E4M3 = np.array([math.ldexp(m / 8.0, -6) if e == 0 else math.ldexp(1 + m / 8.0, e - 7)
                 for e in range(16) for m in range(8)])[:127]     # values of the codes 0 .. 126 (448)


def half_step(dtype: str) -> float:
    return U16 if dtype == "bf16" else U32


def blocks(n: int) -> int:
    return -(-n // 128)


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def norm(x, layer, gamma=None, beta=None, eps=1e-6):
    """(y, mean, rstd) of the rows of x."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1) if layer else np.zeros(x.shape[0])
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, np.float64)
    if beta is not None:
        y = y + np.asarray(beta, np.float64)
    return y, mean, rstd


def norm_bound(x, layer, gamma, y, mean, rstd, dtype):
    """|error| of y: the mean and the mean square are sums of d terms, by lanes of
    at most 32 and then trees of at most 10 levels, so 48 u32 covers each with the
    few operations around it; the mean's error moves c, rstd's scales it, and the
    mean's error enters the mean square squared."""
    x = np.abs(np.asarray(x, np.float64))
    g = np.ones(x.shape[1]) if gamma is None else np.abs(np.asarray(gamma, np.float64))
    c = np.abs(np.asarray(x) if not layer else x + np.abs(mean)[:, None])
    size = rstd[:, None] * g
    shift = 48 * U32 * x.mean(1, keepdims=True) * size if layer else 0.0
    square = 0.5 * (48 * U32 * x.mean(1) * rstd)[:, None] ** 2 if layer else 0.0
    return shift + 64 * U32 * c * size + (half_step(dtype) + 2 * U32 + square) * np.abs(y)


def norm_backward(dy, x, layer, gamma, mean, rstd, dres=None):
    """(dx, dgamma, dbeta) with the saved mean and rstd, and bounds of their errors."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    rstd = np.asarray(rstd, np.float64)[:, None]
    xhat = (x - np.asarray(mean, np.float64)[:, None] if layer else x) * rstd
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    m1 = g.mean(1, keepdims=True) if layer else 0.0
    m2 = (g * xhat).mean(1, keepdims=True)
    dx = rstd * (g - m1 - xhat * m2)
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    a1, a2 = np.abs(g).mean(1, keepdims=True), np.abs(g * xhat).mean(1, keepdims=True)
    return dx, (dy * xhat).sum(0), dy.sum(0), rstd * (np.abs(g) + a1 + np.abs(xhat) * a2)


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------
def philox(counter, key):
    """Philox4x32-10: [n, 4] words of 64-bit whole numbers, key two words."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.asarray(counter)[:, i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1)


def keep_mask(seed: int, draw: int, n: int, p: float, first: int = 0):
    """Which of the values first .. first + n - 1 are kept (first a multiple of 4)."""
    q = first // 4 + np.arange(-(-n // 4), dtype=np.uint64)
    m = 0xFFFFFFFF
    counter = np.stack([q & np.uint64(m), q >> np.uint64(32), np.full_like(q, draw & m),
                        np.full_like(q, draw >> 32)], 1)
    words = philox(counter, (seed & m, seed >> 32)).reshape(-1)[:n]
    return words.astype(np.float64) / 2.0 ** 32 >= p


# ---------------------------------------------------------------------------
# e4m3 in blocks of 128
# ---------------------------------------------------------------------------
def scale_of(top):
    """Smallest power of two >= 2^-126 that brings `top` to 448 or less; 1 for 0."""
    m, e = np.frexp(np.asarray(top, np.float64))
    s = np.exp2(np.maximum(e - 9 + (m > 0.875), -126).astype(np.float64))
    return np.where(np.asarray(top) == 0, 1.0, s)


def to_grid(v):
    """v (|v| <= 448) to the nearest e4m3 value, ties to the even code."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(E4M3, a, side="left"), 1, 126)
    lo = hi - 1
    below, above = a - E4M3[lo], E4M3[hi] - a
    pick = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(E4M3[pick], v)


def encode(v):
    """Codes of values that lie on the grid."""
    code = np.searchsorted(E4M3, np.abs(v)).astype(np.uint8)
    assert np.array_equal(E4M3[code], np.abs(v))
    return code | (np.signbit(v).astype(np.uint8) << 7)


def quantize_tiles(x):
    """(codes' values, scales) of 1 x 128 tiles."""
    x = np.asarray(x, np.float64)
    r, c = x.shape
    pad = np.zeros((r, blocks(c) * 128))
    pad[:, :c] = x
    t = pad.reshape(r, -1, 128)
    s = scale_of(np.abs(t).max(2))
    return to_grid(t / s[:, :, None]).reshape(r, -1)[:, :c], s


def quantize_blocks(w):
    """(codes' values, scales) of 128 x 128 blocks of [n, rows, cols]."""
    w = np.asarray(w, np.float64)
    n, r, c = w.shape
    pad = np.zeros((n, blocks(r) * 128, blocks(c) * 128))
    pad[:, :r, :c] = w
    t = pad.reshape(n, blocks(r), 128, blocks(c), 128)
    s = scale_of(np.abs(t).max((2, 4)))
    q = to_grid(t / s[:, :, None, :, None])
    return q.reshape(n, pad.shape[1], pad.shape[2])[:, :r, :c], s


def spread_tiles(s, cols):
    return np.repeat(s, 128, 1)[:, :cols]


def spread_blocks(s, rows, cols):
    return np.repeat(np.repeat(s, 128, -2)[..., :rows, :], 128, -1)[..., :cols]


def product(x, xs, w, ws):
    """(y, size) of the scaled product: size = sum over blocks of |scales| times the
    sum of the products' magnitudes, what a sum's error is measured against."""
    a, b = x * spread_tiles(xs, x.shape[1]), w * spread_blocks(ws, *w.shape)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def product_slack(k):
    """|error| / size of a product in fp32: sums of 128 and of the blocks, cutting."""
    return (160 + blocks(k)) * 2 * U32


def experts(x, xs, gate, sg, up, su, down, sd):
    """(y, bound) of one SwiGLU expert with its product in 1 x 128 tiles of e4m3.

    The bound follows the product A = SiLU(u) v through its quantization: where A
    lies within its own fp32 error of the border of two codes, the code may be the
    neighbour; where a tile's maximum lies that close to 448 scales, the tile's scale may be
    the double, and each of its values be off by both half steps."""
    k, f = x.shape[1], gate.shape[0]
    u, su_ = product(x, xs, gate, sg)
    v, sv_ = product(x, xs, up, su)
    silu = u / (1.0 + np.exp(-u))
    A = silu * v
    du, dv = product_slack(k) * su_, product_slack(k) * sv_
    # SiLU's slope is at most 1.1; exp's error in steps of fp32 grows with its argument
    dA = 1.1 * np.abs(v) * du + np.abs(silu) * dv + 1.1 * du * dv + (8 + 1.2 * np.abs(u)) * 2 * U32 * np.abs(A)
    q, s = quantize_tiles(A)
    S = spread_tiles(s, f)
    r = A / S
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(r), 2.0 ** -40))), -6) - 3)
    d = dA / S
    frac = np.abs(r) / step - np.floor(np.abs(r) / step)
    flip = np.abs(frac - 0.5) * step <= d
    err = np.where(flip, step, 0.0) * S
    pad = lambda m: np.pad(m, ((0, 0), (0, blocks(f) * 128 - f))).reshape(m.shape[0], -1, 128)  # noqa: E731
    top, dt = np.abs(pad(A)).max(2), pad(dA).max(2)
    lo, hi = scale_of(np.maximum(top - dt, 0.0)), scale_of(top + dt)
    moved = spread_tiles((lo != hi).astype(np.float64), f) > 0
    err = np.where(moved, np.maximum(err, 1.5 * 2 * step * S), err)
    y, size = product(q, s, down, sd)
    bound = err @ np.abs(down * spread_blocks(sd, *down.shape)).T + product_slack(f) * size * 1.07
    return y, bound

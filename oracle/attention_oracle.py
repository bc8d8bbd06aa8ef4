"""The layer's attention operators in 64 bits, from their formulas (numpy; test infrastructure, shares
nothing with the CUDA path).

Rows are [tokens, heads, D]. A cache is two lists of rows per slot, here dense arrays [slots, heads, D].
"""
from __future__ import annotations

import numpy as np


def rope_angles(positions, rope_dim: int, base: float = 10000.0) -> np.ndarray:
    """fp32 [positions, rope_dim]: cosines of p * base^(-2i/rope_dim), then sines."""
    inv = base ** (-np.arange(0, rope_dim, 2, dtype=np.float64) / rope_dim)
    a = np.arange(positions, dtype=np.float64)[:, None] * inv
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def norm_rope(x, weight, eps, table, positions, start=0, interleaved=False) -> np.ndarray:
    """x / sqrt(mean(x^2) + eps) * weight, then pairs of [start, start + R) as complex numbers times
    cos + i sin of their position."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    if table is not None:
        half = table.shape[1] // 2
        rows = np.asarray(table, dtype=np.float64)[np.clip(np.asarray(positions), 0, table.shape[0] - 1)]
        turn = (rows[:, :half] + 1j * rows[:, half:])[:, None, :]
        i = np.arange(half)
        ia, ib = (start + 2 * i, start + 2 * i + 1) if interleaved else (start + i, start + half + i)
        z = (y[..., ia] + 1j * y[..., ib]) * turn
        y[..., ia], y[..., ib] = z.real, z.imag
    return y


def _e4m3_values() -> np.ndarray:
    """The 127 finite values of codes 0 .. 126, ascending (OFP8 E4M3: bias 7, subnormals, no infinity)."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))


_VALUES = _e4m3_values()


def fp8_encode(x):
    """fp32 rows [..., D] -> (codes uint8 [..., D], scale bytes uint8 [..., D/32]): per block the smallest
    2^e >= 2^-126 with max|x| <= 448 * 2^e (2^127 with an infinity, 1 for zeros), codes by nearest value,
    ties to the even code."""
    b = np.asarray(x, dtype=np.float64)
    b = b.reshape(*b.shape[:-1], -1, 32)
    mag = np.abs(b)
    amax = np.max(np.where(np.isnan(mag), 0.0, mag), -1)
    e = np.full(amax.shape, -126, dtype=np.int64)
    for _ in range(127 + 126):
        e = np.where((amax > 448.0 * 2.0 ** e.astype(np.float64)) & (e < 127), e + 1, e)
    e = np.where(amax == 0, 0, e)
    u = mag / 2.0 ** e[..., None].astype(np.float64)
    u = np.where(np.isinf(mag), 448.0, np.minimum(u, 448.0))
    hi = np.searchsorted(_VALUES, np.where(np.isnan(u), 0.0, u))           # first value >= u
    hi = np.clip(hi, 0, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = u - _VALUES[lo], _VALUES[hi] - u
    code = np.where(dlo < dhi, lo, np.where(dhi < dlo, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isnan(b), 0x7F, code) | np.where(np.signbit(b), 0x80, 0)
    return code.reshape(np.shape(x)).astype(np.uint8), (127 + e).astype(np.uint8)


def fp8_decode(codes, scale_bytes) -> np.ndarray:
    """code value * the fp32 number whose exponent field is the byte (0 stands for zero, 255 for infinity)."""
    codes = np.asarray(codes)
    mag = codes & 0x7F
    v = np.where(mag == 0x7F, np.nan, _VALUES[np.minimum(mag, 126)]) * np.where(codes & 0x80, -1.0, 1.0)
    byte = np.asarray(scale_bytes).astype(np.float64)
    scale = np.where(byte == 0, 0.0, np.where(byte == 255, np.inf, 2.0 ** (np.minimum(byte, 254) - 127)))
    with np.errstate(invalid="ignore"):
        return v * np.repeat(scale, 32, -1)


def attention(q, keys, values, scale, q_rel: float = 0.0, p_rel: float = 0.0):
    """One sequence: q [Hq, D], keys and values [n, Hk, D] (only the attended ones). Returns (out [Hq, D],
    lse [Hq], a bound of out's error, a bound of lse's) where the bounds hold for products with fp32
    accumulation whose query operand is off by q_rel and whose weights are rounded by p_rel:
      score error ds <= ((D + 8) 2^-24 + q_rel) * scale * sum|q k| + 2^-22 |s|  (scaling, subtraction)
      weight error   <= 2 ds + 2^-21 (exp2) + p_rel + n 2^-24 (sums), times sum p|v|
    The output's own rounding is not in them."""
    q = np.asarray(q, dtype=np.float64)
    Hq, D = q.shape
    n, Hk, _ = keys.shape
    out, lse = np.zeros((Hq, D)), np.full(Hq, -np.inf)
    tol, tol_lse = np.zeros((Hq, D)), np.zeros(Hq)
    if n == 0:
        return out, lse, tol, tol_lse
    for h in range(Hq):
        k, v = keys[:, h * Hk // Hq].astype(np.float64), values[:, h * Hk // Hq].astype(np.float64)
        s = k @ q[h] * scale
        m = s.max()
        w = np.exp(s - m)
        lse[h] = m + np.log(w.sum())
        w /= w.sum()
        out[h] = w @ v
        ds = (((D + 8) * 2.0 ** -24 + q_rel) * abs(scale) * (np.abs(k) @ np.abs(q[h]))).max() + 2.0 ** -22 * np.abs(s).max()
        tol[h] = (2 * ds + 2.0 ** -21 + p_rel + n * 2.0 ** -24) * (w @ np.abs(v))
        tol_lse[h] = ds + 2.0 ** -21 + n * 2.0 ** -24 + 2.0 ** -22 * abs(lse[h])
    return out, lse, tol, tol_lse


def visible(n: int, length: int, causal: bool = True, window: int = 0, doc_starts=None, prefix_ends=None):
    """Positions and intervals [lo, hi) of the keys that n new tokens of a sequence of `length` see."""
    p = length - n + np.arange(n, dtype=np.int64)
    lo, hi = np.zeros(n, np.int64), np.full(n, length, np.int64)
    if causal:
        hi = p + 1
        if prefix_ends is not None:
            hi = np.maximum(hi, prefix_ends)
        hi = np.minimum(hi, length)
    if window:
        lo = np.maximum(lo, p + 1 - window)
    if doc_starts is not None:
        lo = np.maximum(lo, doc_starts)
    return p, lo, hi


def attention_rows(q, keys, values, seen, p, scale, cap: float = 0.0, slopes=None, q_rel: float = 0.0, p_rel: float = 0.0):
    """Rows q [T, Hq, D] at positions p over keys and values [n, Hk, D] at positions 0 .. n - 1; seen: bool [T, n]. Scores
    cap * tanh(x / cap) - slope |p - j|. Returns (out, lse, a bound of out's error, a bound of lse's) as `attention` does; beside
    its terms a capped score is off by 2^-19 of itself (tanh's slope is at most 1), a bias by 2^-22 of itself (its slope in
    other units, the product)."""
    q = np.asarray(q, dtype=np.float64)
    T, Hq, D = q.shape
    n, Hk, _ = keys.shape
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    tol, tol_lse = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    some = seen.any(1) if n else np.zeros(T, bool)
    if not some.any():
        return out, lse, tol, tol_lse
    far = np.abs(np.asarray(p)[:, None] - np.arange(n)[None, :]).astype(np.float64)
    for h in range(Hq):
        k, v = keys[:, h * Hk // Hq].astype(np.float64), values[:, h * Hk // Hq].astype(np.float64)
        x = q[:, h] @ k.T * scale
        ds = ((D + 8) * 2.0 ** -24 + q_rel) * abs(scale) * (np.abs(q[:, h]) @ np.abs(k).T) + 2.0 ** -22 * np.abs(x)
        s = cap * np.tanh(x / cap) if cap else x
        if cap:
            ds += 2.0 ** -19 * np.abs(s)
        if slopes is not None:
            s = s - slopes[h] * far
            ds += 2.0 ** -22 * (slopes[h] * far + np.abs(s))
        s = np.where(seen, s, -np.inf)
        m = np.where(some, s.max(1), 0.0)
        w = np.exp(s - m[:, None])
        total = np.where(some, w.sum(1), 1.0)
        lse[:, h] = np.where(some, m + np.log(total), -np.inf)
        w /= total[:, None]
        out[:, h] = w @ v
        # every weight by its own score's error, and all of them by their mean error in the sum
        mean = (w * ds).sum(1)
        tol[:, h] = (w * (ds + mean[:, None])) @ np.abs(v) * 1.01 + (2.0 ** -21 + p_rel + n * 2.0 ** -24) * (w @ np.abs(v))
        tol_lse[:, h] = 1.01 * mean + 2.0 ** -21 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(some, lse[:, h], 0.0))
    return out, lse, tol, tol_lse

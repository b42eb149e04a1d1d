"""Plain float64 definition of the 4-bit key/value cache and of the attention
over it (test infrastructure: only the test-suite uses it).

The SSD summary's AMD MI300X part rolls the key/value cache back by its valid
length alone; the cache's format, the visibility rule and the errors are those
include/spec_verify.h states.  numpy only; no code is shared with the library.
"""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32
NAN_SCALE = 255


def quantise(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """x [..., dim] -> (codes uint8 [..., dim], scale bytes uint8 [..., dim / 32]).

    The scale is the smallest power of two s with max|x| <= 7 s, its byte
    clamped to 3..252; a code is the nearest magnitude of |x| / s, ties to the
    even code, with the sign in bit 3.  A block that is not finite: codes 0,
    scale byte 255."""
    x = np.asarray(x, dtype=np.float64)
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    fine = np.isfinite(blocks).all(-1)
    blocks = np.where(fine[..., None], blocks, 0.0)
    a = np.abs(blocks).max(-1)
    m, e = np.frexp(a)                       # a = m 2^e, 1/2 <= m < 1 (0 for a = 0)
    e = np.where(a > 0, e - 3 + (m > 7 / 8), -1000)
    byte = np.clip(e + 127, 3, 252)
    y = np.abs(blocks) * 2.0 ** (127.0 - byte[..., None])
    d = np.abs(y[..., None] - MAGNITUDES)
    # the nearest; of two equally near ones, the even code
    best = np.argmin(np.where(d == d.min(-1, keepdims=True), np.arange(8) % 2, 9), -1)
    codes = np.where(np.signbit(blocks), 8, 0) + best
    codes = np.where(fine[..., None], codes, 0)
    return codes.reshape(x.shape).astype(np.uint8), np.where(fine, byte, NAN_SCALE).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """What codes [..., dim] under scale bytes [..., dim / 32] stand for."""
    mag = MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == NAN_SCALE, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return mag * np.repeat(s, BLOCK, -1)


def places(page: int, dim: int, r: int):
    """Of token r in a record: the byte of each number's key code and of its
    value code [dim], of its key scales and of its value scales [dim / 32]."""
    d, blk = np.arange(dim), np.arange(dim // BLOCK)
    share = dim // 16
    key = r * (dim // 2) + d // 2
    value = (page * dim // 2 + (r // 16) * 8 * dim + ((r % 16) // 4) * 2 * dim + (d // share) * (dim // 8)
             + (r % 4) * (dim // 32) + (d % share) // 2)
    key_scale = page * dim + r * (dim // BLOCK) + blk
    value_scale = page * dim + page * (dim // BLOCK) + (r // 16) * (dim // 2) + blk * 16 + r % 16
    return key, value, key_scale, value_scale


def write(data: np.ndarray, table_row, page: int, dim: int, t: int, k: np.ndarray, v: np.ndarray) -> None:
    """Quantise one token's k, v [heads, dim] into data [pages, heads, record] at position t."""
    rec = data[table_row[t // page]]
    at = places(page, dim, t % page)
    half = np.arange(dim) % 2
    for x, code_at, scale_at in ((k, at[0], at[2]), (v, at[1], at[3])):
        codes, scales = quantise(x)
        for h in range(rec.shape[0]):
            for side in (0, 1):
                pick = half == side
                old = rec[h, code_at[pick]]
                rec[h, code_at[pick]] = (old & (0xF0 if side == 0 else 0x0F)) | (codes[h, pick] << (4 * side))
            rec[h, scale_at] = scales[h]


def read(data: np.ndarray, table_row, page: int, dim: int, t: int) -> tuple[np.ndarray, np.ndarray]:
    """One token's keys and values [heads, dim] at position t."""
    rec = data[table_row[t // page]]
    at = places(page, dim, t % page)
    half = (np.arange(dim) % 2) * 4
    return tuple(values((rec[:, c] >> half) & 15, rec[:, s]) for c, s in ((at[0], at[2]), (at[1], at[3])))


def sees(pos: int, i: int, count: int, t: np.ndarray, window: int = 0, bits: int | None = None) -> np.ndarray:
    """Which of the positions t new token i sees, the first of count new tokens at pos."""
    if bits is None:
        ok = t <= pos + i
    else:
        new = np.clip(t - pos, 0, 63)
        set_ = np.array([(int(bits) >> int(j)) & 1 for j in new], dtype=bool)
        ok = (t < pos) | (set_ & (t < pos + count))
    if window:
        ok = ok & (t > pos + i - window)
    return ok


def attend(q: np.ndarray, K: np.ndarray, V: np.ndarray, scale: float):
    """One row: q [dim], the keys and values [T, dim] it sees.  Returns (out
    [dim], lse, the weighted mean of |V| [dim], the largest scaled sum of
    |q K|, the range of the scores): the last three are what error bounds need."""
    if len(K) == 0:
        z = np.zeros(q.shape)
        return z, -np.inf, z, 0.0, 0.0
    if np.isnan(K).any() or np.isnan(V).any():
        z = np.full(q.shape, np.nan)
        return z, np.nan, z, 0.0, 0.0
    s = scale * (K @ q)
    m = s.max()
    w = np.exp(s - m)
    l = w.sum()
    return w @ V / l, m + np.log(l), w @ np.abs(V) / l, abs(scale) * (np.abs(K) @ np.abs(q)).max(), m - s.min()


def read_span(data: np.ndarray, table_row, page: int, dim: int, t0: int, t1: int) -> tuple[np.ndarray, np.ndarray]:
    """The keys and values [t1 - t0, heads, dim] at positions t0 .. t1 - 1; NaN on pages outside the pool."""
    t = np.arange(t0, t1)
    pages = np.asarray(table_row, dtype=np.int64)[t // page]
    bad = (pages < 0) | (pages >= len(data))
    at = [np.stack(p)[t % page] for p in zip(*(places(page, dim, r) for r in range(page)))]
    half = (np.arange(dim) % 2) * 4
    heads = np.arange(data.shape[1])[None, :, None]
    pages = np.where(bad, 0, pages)[:, None, None]
    out = []
    for c, s in ((at[0], at[2]), (at[1], at[3])):
        v = values((data[pages, heads, c[:, None]] >> half) & 15, data[pages, heads, s[:, None]])
        out.append(np.where(bad[:, None, None], np.nan, v))
    return out[0], out[1]

"""NumPy oracle of the 8-bit paged KV cache, in float64, written from the
header's formulas: the two 8-bit forms, appending with rotation, and
attention with a window and sinks. Test infrastructure only; it shares no
code with the CUDA side."""

from __future__ import annotations

import numpy as np

BLOCK = 16
FLOOR = np.float32(2.0 ** -60)
TOP = {"int8": 127.0, "e4m3": 448.0}


def _e4m3_table() -> np.ndarray:
    """Value of each of the 256 bytes: sign, 4 exponent bits (bias 7), 3
    mantissa bits; exponent 0 is subnormal, 0x7f and 0xff are NaN."""
    out = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = np.nan if (b & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = -x if b & 128 else x
    return out


E4M3 = _e4m3_table()
_POS = E4M3[:127]                       # 0 .. 448, ascending with the byte
_MID = (_POS[1:] + _POS[:-1]) / 2


def decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    return codes.astype(np.float64) - 128 if fmt == "int8" else E4M3[codes]


def encode(t: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest code of each value (ties to even), clamped; e4m3 by way of fp32."""
    t = np.asarray(t, np.float64)
    if fmt == "e4m3":
        t = t.astype(np.float32).astype(np.float64)
    if fmt == "int8":
        return (np.clip(np.rint(t), -127, 127) + 128).astype(np.uint8)
    a = np.minimum(np.abs(t), 448.0)
    i = np.searchsorted(_MID, a, side="left")          # midpoints below a
    tie = (i < len(_MID)) & (_MID[np.minimum(i, len(_MID) - 1)] == a)
    i = np.where(tie & (i % 2 == 1), i + 1, i)          # the even one of the two neighbours
    return (i + np.where(np.signbit(t), 128, 0)).astype(np.uint8)


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [tokens, heads, dim] with the first 2 * cos.shape[1] channels turned."""
    x = np.array(x, np.float64)
    half = cos.shape[1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos.astype(np.float64)[:, None], sin.astype(np.float64)[:, None]
    xa, xb = x[..., a].copy(), x[..., b].copy()
    x[..., a] = xa * c - xb * s
    x[..., b] = xb * c + xa * s
    return x


class Cache:
    """codes [pages, heads, page, dim] and scales [pages, heads, page / 16] of
    keys (0) and values (1)."""

    def __init__(self, codes_k, codes_v, scales_k, scales_v, fmt):
        self.codes = [np.array(codes_k), np.array(codes_v)]
        self.scales = [np.array(scales_k, np.float32), np.array(scales_v, np.float32)]
        self.fmt = fmt
        self.page = self.codes[0].shape[2]

    def values(self, which, table, lo, hi):
        """[hi - lo, heads, dim] of a sequence whose pages are `table`."""
        pos = np.arange(lo, hi)
        pg, off = np.asarray(table)[pos // self.page], pos % self.page
        return decode(self.codes[which][pg, :, off], self.fmt) * \
            self.scales[which][pg, :, off // BLOCK].astype(np.float64)[..., None]

    def tops(self, which, table, lo, hi):
        """[hi - lo, heads]: the largest value a code can stand for."""
        pos = np.arange(lo, hi)
        pg, off = np.asarray(table)[pos // self.page], pos % self.page
        return self.scales[which][pg, :, off // BLOCK].astype(np.float64) * TOP[self.fmt]

    def append(self, which, table, past, x):
        """x [tokens, heads, dim] (float64) at positions past ..; returns for
        each token the quotients x / s that were rounded."""
        n = x.shape[0]
        quotients = np.zeros_like(x)
        for start in range(max(past, 0) // BLOCK * BLOCK, past + n, BLOCK):
            lo, hi = max(start, past, 0), min(start + BLOCK, past + n)
            if hi <= lo:
                continue
            pg, off = int(np.asarray(table)[start // self.page]), start % self.page
            new = x[lo - past:hi - past]
            old = self.scales[which][pg, :, off // BLOCK].copy() if lo > start else np.zeros(x.shape[1], np.float32)
            top = np.abs(new).max((0, 2))
            s = np.maximum(np.maximum((top / TOP[self.fmt]).astype(np.float32), old), FLOOR)
            codes = self.codes[which][pg, :, off:off + BLOCK]         # [heads, 16, dim], a view
            if lo > start:
                grown = s > old
                held = decode(codes[:, :lo - start], self.fmt) * old.astype(np.float64)[:, None, None]
                again = encode(held / s.astype(np.float64)[:, None, None], self.fmt)
                codes[:, :lo - start] = np.where(grown[:, None, None], again, codes[:, :lo - start])
            q = new / s.astype(np.float64)[None, :, None]
            codes[:, lo - start:hi - start] = encode(q, self.fmt).transpose(1, 0, 2)
            quotients[lo - past:hi - past] = q
            self.scales[which][pg, :, off // BLOCK] = s
        return quotients


def attention(q, k, v, past, scale, window=0, sinks=0, top=None, keep=None):
    """q [rows, heads, dim] at positions past .., k, v [len, kv_heads, dim]:
    (out, sum of weight * |v|, largest scale * sum |q| |k|, keys seen times the
    largest weight * top), the first two [rows, heads, dim], the others
    [rows, heads]. top [len, kv_heads]. keep [len]: keys that are there (None:
    all)."""
    rows, heads, dim = q.shape
    n, kv = k.shape[:2]
    group = heads // kv
    out, mass = np.zeros((rows, heads, dim)), np.zeros((rows, heads, dim))
    big, small = np.zeros((rows, heads)), np.zeros((rows, heads))
    j = np.arange(n)
    for i in range(rows):
        p = past + i
        see = j <= p
        if window:
            see &= (j > p - window) | (j < sinks)
        if keep is not None:
            see &= keep
        if not see.any():
            continue
        for h in range(heads):
            kh, vh = k[see, h // group], v[see, h // group]
            z = scale * (kh @ q[i, h])
            w = np.exp(z - z.max())
            w /= w.sum()
            out[i, h] = w @ vh
            mass[i, h] = w @ np.abs(vh)
            big[i, h] = abs(scale) * (np.abs(kh) @ np.abs(q[i, h])).max()
            small[i, h] = see.sum() * (w * top[see, h // group]).max()
    return out, mass, big, small

"""The 8-bit pools and the position rotation in numpy, from their definitions (include/pagedkv.h):
codes by search in the table of e4m3 values, writes token by token."""
from __future__ import annotations

import numpy as np


def _table():
    c = np.arange(128)
    e, m = c >> 3, (c & 7).astype(np.float64)
    v = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m * 2.0 ** -9)
    v[127] = np.nan
    return np.concatenate((v, -v))


VALUES = _table()            # of the 256 codes
_POS = VALUES[:127]
_MIDS = (_POS[1:] + _POS[:-1]) / 2


def encode(x):
    """Codes of values of at most 448 in magnitude (fp64), ties to even; NaN for what is no
    number."""
    x = np.asarray(x, np.float64)
    mag = np.abs(x)
    bad = ~np.isfinite(x)
    at = np.searchsorted(_MIDS, np.where(bad, 0, mag), side="left")
    tie = (at < 126) & (_MIDS[np.minimum(at, 125)] == mag) & (at % 2 == 1)
    code = np.minimum(at + tie, 126).astype(np.uint8)
    code = np.where(np.signbit(x), code | 0x80, code).astype(np.uint8)
    return np.where(bad, np.uint8(0x7F), code)


def canon(codes):
    """Codes with every NaN as 0x7f."""
    return np.where((codes & 0x7F) == 0x7F, np.uint8(0x7F), codes)


def values(codes, scale):
    """fp64 values of codes [..., B, d] with scales [...]."""
    return VALUES[codes] * np.asarray(scale, np.float64)[..., None, None]


def scale_for(a):
    """The least power of two n >= 2^-100 with a <= 448 n."""
    n = 2.0 ** -100
    while float(a) > 448.0 * n:
        n *= 2.0
    return n


def scale_up(s):
    """The least power of two >= s; NaN for what no page may have."""
    s = float(s)
    if not 0 <= s <= 2.0 ** 126:
        return float("nan")
    if s == 0:
        return 0.0
    n = 2.0 ** -126
    while n < s:
        n *= 2.0
    return n


def rotate(x, cos_sin, pos, mix):
    """fp32 rows x [N, H, d] at positions pos, every product and sum rounded to fp32."""
    x = np.asarray(x, np.float32).copy()
    rot = cos_sin.shape[1]
    h = rot // 2
    i = np.arange(h)
    a, b = (2 * i, 2 * i + 1) if mix else (i, i + h)
    c, s = cos_sin[pos][:, None, :h], cos_sin[pos][:, None, h:]
    xa, xb = x[..., a], x[..., b]
    ra = (xa * c).astype(np.float32) - (xb * s).astype(np.float32)
    rb = (xb * c).astype(np.float32) + (xa * s).astype(np.float32)
    x[..., a], x[..., b] = ra, rb
    return x


def cos_sin(positions, rot, theta=10000.0):
    ang = np.arange(positions)[:, None] * theta ** (-2.0 * np.arange(rot // 2) / rot)
    return np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)


def write(x, table, seq, pos, codes, scale, live):
    """Rows x [N, Hkv, d] (fp32, rotated) of the tokens with live[n] into codes
    [blocks, Hkv, B, d] and scale [blocks, Hkv] (fp32), in place."""
    block = codes.shape[2]
    n = 0
    while n < len(seq):
        s, pg = seq[n], pos[n] // block
        if s < 0:
            n += 1
            continue
        end = n
        while end < len(seq) and seq[end] == s and pos[end] // block == pg:
            end += 1
        rows = [t for t in range(n, end) if live[t]]
        page, front = table[s, pg], pos[n] % block
        if rows:
            for h in range(codes.shape[1]):
                v = x[rows, h].astype(np.float64)
                fin = np.abs(v[np.isfinite(v)])
                new = scale_for(fin.max(initial=0.0))
                if front:
                    old = float(scale[page, h])
                    up = scale_up(old)
                    new = up if up != up else max(new, up)
                    if new != old:
                        with np.errstate(invalid="ignore"):
                            codes[page, h, :front] = encode(
                                VALUES[codes[page, h, :front]] * (old / new))
                scale[page, h] = new
                for t, row in zip(rows, v):
                    with np.errstate(invalid="ignore"):
                        codes[page, h, pos[t] % block] = encode(row / new)
        n = end

"""Plain numpy model of the 4-bit row format and of the calls on 4-bit pools:
the stored bytes in fp32 steps (they are the format), everything computed from
them in 64 bits."""
from __future__ import annotations

import numpy as np


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """fp32 -> bf16 bits, ties to even; NaN -> 0x7fff as the hardware stores it."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FFF), r)


def bf16_value(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, np.uint32) << 16).view(np.float32)


def units(d: int):
    """(unit, nibble) of every dim of a row."""
    i = np.arange(d)
    return ((i % 32) // 4) * (d // 32) + i // 32, i % 4


def quantise(x: np.ndarray) -> np.ndarray:
    """fp32 [..., d] -> rows uint8 [..., 5 d / 8]."""
    x = np.ascontiguousarray(x, np.float32)
    d = x.shape[-1]
    ng = d // 32
    g = x.reshape(*x.shape[:-1], ng, 32)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)  # a NaN stays
        sb = bf16_bits((hi - lo) / np.float32(15))
        s = bf16_value(sb)
        tiny = s < np.float32(2.0 ** -126)
        sb, s = np.where(tiny, np.uint16(0), sb), np.where(tiny, np.float32(0), s)
        zb = bf16_bits((np.float32(0.5) * lo + np.float32(0.5) * hi) + np.float32(0.5) * s)
        z = bf16_value(zb)
        inv = np.where(s > 0, np.float32(1) / s, np.float32(0)).astype(np.float32)
        u = np.rint((g - z[..., None]) * inv[..., None]) + np.float32(8)
        u = np.where(np.isnan(u), 0, np.clip(u, 0, 15)).astype(np.uint8)
    u = u.reshape(*x.shape[:-1], d)
    rows = np.zeros((*x.shape[:-1], 5 * d // 8), np.uint8)
    unit, nib = units(d)
    for i in range(d):
        rows[..., 2 * unit[i] + nib[i] // 2] |= u[..., i] << np.uint8(4 * (nib[i] % 2))
    sz = np.stack((sb, zb), -1).astype("<u2").reshape(*x.shape[:-1], 2 * ng)
    rows[..., d // 2:] = np.ascontiguousarray(sz).view(np.uint8)
    return rows


def parts(rows: np.ndarray):
    """(u - 8, s, z) per dim, in 64 bits."""
    d = rows.shape[-1] * 8 // 5
    unit, nib = units(d)
    u = (rows[..., 2 * unit + nib // 2] >> (4 * (nib % 2))) & 15
    sz = np.ascontiguousarray(rows[..., d // 2:]).view("<u2").reshape(*rows.shape[:-1], d // 32, 2)
    v = bf16_value(sz).astype(np.float64)
    grp = np.arange(d) // 32
    return u.astype(np.float64) - 8, v[..., grp, 0], v[..., grp, 1]


def values(rows: np.ndarray) -> np.ndarray:
    u, s, z = parts(rows)
    return s * u + z


def rows_of(pool: np.ndarray, table_row, n: int) -> np.ndarray:
    """Rows [n, Hkv, R] of a sequence's first n positions."""
    b = pool.shape[2]
    pos = np.arange(n)
    return pool[np.asarray(table_row)[pos // b], :, pos % b]


def decode(q, kc, vc, table, lens, scale, skip=None):
    """(out, tolerance) in 64 bits.  skip[b]: positions not attended to (bad pages).

    Tolerance, per output value, with p the softmax weights:
      output rounding              r |out|            r = 2^-8 (bf16), 2^-24 (fp32)
      weights rounded to 8 bits or more  2^-8 sum p |s (u - 8)|   (the kernel keeps 11 with
      bf16 q; fp32 q: 2^-22)
      scores: fp32 sums of d products of q with whole numbers of at most 280 (the
      kernel's codes, two to a byte, and their offset stay below), each term rounded or
      cut (2^-23), 48 terms a group:
        e = 48 2^-23 280 sum_g s_g |q|_1,g + (2 d) 2^-23 sum |q| |k|,
      which moves every weight by a factor exp(2 scale e) at most
      exponential, sums and merges 2^-15 sum p |v| (fp32 q: 2^-19): thousands of
      fp32 additions with a random sign.
    """
    batch, hq, d = q.shape
    hkv = kc.shape[1]
    out = np.zeros((batch, hq, d))
    tol = np.zeros((batch, hq, d))
    bf = q.dtype == np.uint16
    q = bf16_value(q) if bf else q
    q = q.astype(np.float64)
    for b in range(batch):
        n = int(lens[b])
        pos = np.arange(n)
        if skip is not None and n:
            pos = pos[~np.isin(pos, skip[b])]
        if not len(pos):
            continue
        blk = np.asarray(table[b])
        bs = kc.shape[2]
        kr = kc[blk[pos // bs], :, pos % bs]
        vr = vc[blk[pos // bs], :, pos % bs]
        k, v = values(kr), values(vr)
        uk, sk, zk = parts(kr)
        uv, sv, zv = parts(vr)
        for h in range(hq):
            kh = h // (hq // hkv)
            s = scale * (k[:, kh] @ q[b, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            out[b, h] = p @ v[:, kh]
            e = 2 * d * 2.0 ** -23 * (np.abs(k[:, kh]) @ np.abs(q[b, h]))
            if bf:
                e = e + 48 * 2.0 ** -23 * 280 * (sk[:, kh] @ np.abs(q[b, h]))
            e = float(np.max(e)) * 2 * abs(scale)
            mag = p @ np.abs(v[:, kh])
            w = p @ np.abs(sv[:, kh] * uv[:, kh])
            tol[b, h] = ((2.0 ** -8 if bf else 2.0 ** -24) * np.abs(out[b, h]) +
                         (2.0 ** -8 if bf else 2.0 ** -22) * w +
                         (np.expm1(e) + (2.0 ** -15 if bf else 2.0 ** -19)) * (mag + w))
    return out, tol


def compact(pool, table, keep, cu, start, head_major):
    """The pool after compaction (a copy)."""
    new = pool.copy()
    b_size = pool.shape[2] if head_major else pool.shape[1]
    for b in range(len(cu) - 1):
        at = np.asarray(keep[cu[b]:cu[b + 1]], dtype=np.int64)
        to = (0 if start is None else int(start[b])) + np.arange(len(at))
        row = np.asarray(table[b])
        if head_major:
            new[row[to // b_size], :, to % b_size] = pool[row[at // b_size], :, at % b_size]
        else:
            new[row[to // b_size], to % b_size] = pool[row[at // b_size], at % b_size]
    return new

"""What the 4-bit decode may be off by, from the roundings it makes, tightly enough
that a lost tile, a coarser query or a coarser weight does not pass.

Rounding errors of different keys have no common sign, so they add in quadrature:
per output value, with p the softmax weights, v = s (u - 8) + z and o = sum p v,

  Var = sum_j (w_j |u_j - 8|)^2 + (p_j |v_j - o| e_j)^2,   E = 6 sqrt(Var) + D,
  tolerance = r (|o| + E) + E,   r = 2^-8 (bf16), 2^-24 (fp32): the output's half step.

w_j: standard deviation of a rounded p_j s_j.  A half step is 2^-11 of it (fp16), or
  2^-22 with fp32 queries (two parts); weights are held relative to at most the largest
  weight times twice the largest scale, with steps of 2^-24 there (and 2^-36 where fp32
  queries move them up by 2^12): half a step is 2^-24 (2^-36) of pmax smax.  A value
  that is uniform in a half step has 1 / sqrt(3) of it as its deviation.
e_j: deviation of a score, in nats (scale's factor included):
  bf16 queries: operands are exact; products of subnormal codes are cut 24 bits or more
  below the largest field exponent, which is Q = 2^-14 of the power of two at or below the
  largest |q|, per unit of code.  Products of a q whose last bit (2^-7 of its own power
  of two) is at or above Q are not cut.  Per group: s Q sqrt(cut products + 1) / sqrt(3).
  fp32 queries: two parts of q, 2^-22 of it; products are cut 24 bits below the largest,
  2^-24 of 8 max |q| each, 64 of them a group.
  Both: a handful of fp32 operations on the groups' parts, on the score and on its
  distance from the maximum, and the exponential: 2^-22 (parts + |score| + |maximum| + 1).
D: what has a common sign.  bf16 queries: a product with a weight below 2^-4 of the
  largest of its 16 keys (aligned to 16 in the sequence) is cut by up to 2^-14 of that
  weight times a unit of code; sums of 16 products of codes up to 16 with weights are
  cut 24 bits below: 16 2^-24 16 sum p s.  fp32 queries: sums of a warp's share,
  2^-18 sqrt(sum p^2 v^2) for up to 64 roundings in the same direction.  Both: the sums
  of weights, 2^-20 |o|.
"""
from __future__ import annotations

import numpy as np

import q4_oracle as Q


def _pow2(x):
    """The power of two at or below x (0 for 0)."""
    return np.where(x > 0, np.exp2(np.floor(np.log2(np.where(x > 0, x, 1)))), 0.0)


def decode(q, kc, vc, table, lens, scale):
    """(out, tolerance, root of the mean square that a value may be off by) in 64 bits."""
    batch, hq, d = q.shape
    hkv, bs, ng = kc.shape[1], kc.shape[2], q.shape[2] // 32
    out, tol, var = (np.zeros((batch, hq, d)) for _ in range(3))
    bf = q.dtype == np.uint16
    q = (Q.bf16_value(q) if bf else q).astype(np.float64)
    r = 2.0 ** -8 if bf else 2.0 ** -24
    for b in range(batch):
        n = int(lens[b])
        if not n:
            continue
        pos = np.arange(n)
        blk = np.asarray(table[b])
        kr, vr = (pool[blk[pos // bs], :, pos % bs] for pool in (kc, vc))
        for kh in range(hkv):
            uk, sk, zk = Q.parts(kr[:, kh])
            uv, sv, zv = Q.parts(vr[:, kh])
            k, v = sk * uk + zk, sv * uv + zv
            smax = np.abs(sv).max()
            for h in range(kh * (hq // hkv), (kh + 1) * (hq // hkv)):
                x = q[b, h]
                s = scale * (k @ x)
                p = np.exp(s - s.max())
                p /= p.sum()
                o = p @ v
                e = score_error(x, uk, sk, zk, s, scale, bf)
                w = np.maximum((2.0 ** -11 if bf else 2.0 ** -22) * p[:, None] * np.abs(sv),
                               (2.0 ** -24 if bf else 2.0 ** -36) * smax * p.max()) / np.sqrt(3)
                var_bh = (w ** 2 * uv ** 2).sum(0) + (p * e) ** 2 @ (v - o) ** 2
                cut = 2.0 ** -20 * np.abs(o)
                if bf:
                    ps = p[:, None] * np.abs(sv)
                    pad = -n % 16
                    sixteen = np.pad(ps, ((0, pad), (0, 0))).reshape(-1, 16, d)
                    top = sixteen.max(1)
                    few = ((sixteen < 2.0 ** -4 * top[:, None]) & (sixteen > 0)).sum(1)
                    cut += 2.0 ** -14 * (few * top).sum(0) + 2.0 ** -16 * ps.sum(0)
                else:
                    cut += 2.0 ** -18 * np.sqrt(p ** 2 @ v ** 2)
                err = 6 * np.sqrt(var_bh) + cut
                out[b, h] = o
                tol[b, h] = r * (np.abs(o) + err) + err
                var[b, h] = (r * np.abs(o)) ** 2 / 3 + var_bh + cut ** 2
    return out, tol, np.sqrt(var)


def score_error(x, uk, sk, zk, s, scale, bf):
    d = len(x)
    ng = d // 32
    g = x.reshape(ng, 32)
    sg, zg = np.abs(sk[:, ::32]), np.abs(zk[:, ::32])
    codes = np.abs(np.einsum("kgi,gi->kg", uk.reshape(-1, ng, 32), g))
    parts = (sg * codes + zg * np.abs(g.sum(1))).sum(1)
    if bf:
        quantum = 2.0 ** -14 * _pow2(np.abs(x).max())
        cut = ((np.abs(g) > 0) & (2.0 ** -7 * _pow2(np.abs(g)) < quantum)).sum(1)
        err2 = (sg ** 2 * np.where(cut > 0, cut + 1, 0)).sum(1) * quantum ** 2 / 3
    else:
        err2 = ((sk * uk * x) ** 2).sum(1) * 2.0 ** -44 / 3
        err2 = err2 + (sg * 8 * np.abs(g).max(1) * 2.0 ** -24 * 8) ** 2 @ np.ones(ng)
    return (abs(scale) * np.sqrt(err2) +
            2.0 ** -22 * (abs(scale) * parts + np.abs(s) + np.abs(s.max()) + 1))


def rejects(got, want, tol):
    """Whether the bound tells `got` from a right answer."""
    return not np.all(np.abs(got - want) <= tol)

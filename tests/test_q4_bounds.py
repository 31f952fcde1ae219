"""The decode's bounds told from mistakes: the oracle computes a wrong answer on
purpose (on the CPU) and the bound has to reject it."""
import numpy as np
import pytest

import q4_bounds as B
import q4_oracle as Q


def competing(hq, hkv, d, batch, n, seed, outliers=False):
    """Few keys with large scores: pairs that share the weight show a score's error."""
    rng = np.random.default_rng(seed)
    block = 16
    lens = [n] * batch
    table = np.arange(batch, dtype=np.int32)[:, None]
    k, v = (rng.standard_normal((batch, hkv, block, d)).astype(np.float32) for _ in range(2))
    if outliers:
        k[..., 3::29] *= 8
    q = Q.bf16_bits(rng.standard_normal((batch, hq, d)).astype(np.float32))
    return q, Q.quantise(k), Q.quantise(v), table, lens


def scores_of_differences(q, kc, vc, table, lens, scale, exact):
    """The output with the score product's operands in fp16: q0 - q1 / 16 beside the byte
    u0 + 16 u1 of two codes, or (exact) q0 and q1 / 16 beside u0 and 16 u1."""
    batch, hq, d = q.shape
    hkv = kc.shape[1]
    x = Q.bf16_value(q).astype(np.float64)
    up = 2.0 ** (11 - np.floor(np.log2(np.abs(x).max(-1, keepdims=True))))
    a = x * up
    a[..., 1::2] /= 16
    if not exact:
        a[..., 0::2] -= a[..., 1::2]
    a = a.astype(np.float16).astype(np.float64) / up
    out = np.zeros((batch, hq, d))
    for b, n in enumerate(lens):
        for h in range(hq):
            kh = h // (hq // hkv)
            u, s, z = Q.parts(kc[table[b, 0], kh, :n])
            c = u + 8
            c[:, 1::2] *= 16
            if not exact:
                c[:, 1::2] += u[:, 0::2] + 8
            e = scale * ((s * c) @ a[b, h] + (z - 8 * s) @ x[b, h])
            p = np.exp(e - e.max())
            out[b, h] = p / p.sum() @ Q.values(vc[table[b, 0], kh, :n])
    return out


@pytest.mark.parametrize("hq,hkv,d,outliers", [(4, 2, 128, False), (8, 2, 64, True)])
def test_differences_of_queries_in_fp16_are_rejected(hq, hkv, d, outliers):
    case = competing(hq, hkv, d, 48, 3, 5, outliers)
    want, tol, _ = B.decode(*case, 3.0)
    assert not B.rejects(scores_of_differences(*case, 3.0, True), want, tol)
    assert B.rejects(scores_of_differences(*case, 3.0, False), want, tol)

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


def long_case(dtype, n, d, seed):
    """One sequence of n keys as the decode tests make them."""
    rng = np.random.default_rng(seed)
    block = 256
    blocks = -(-n // block)
    k, v = (rng.standard_normal((blocks, 1, block, d)).astype(np.float32) for _ in range(2))
    for x in (k, v):
        x[..., 3::29] *= 4
    q = rng.standard_normal((1, 2, d)).astype(np.float32)
    table = np.arange(blocks, dtype=np.int32)[None]
    return Q.bf16_bits(q) if dtype == "bf16" else q, Q.quantise(k), Q.quantise(v), table, [n]


def without(case, dropped, scale):
    """The output with some positions left out."""
    return Q.decode(*case, scale, [dropped])[0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [12345, 20000])
def test_lost_keys_are_rejected_at_long_contexts(dtype, n):
    case = long_case(dtype, n, 128, n)
    scale = 128 ** -0.5
    want, tol, _ = B.decode(*case, scale)
    assert np.allclose(want, Q.decode(*case, scale)[0], rtol=1e-12, atol=1e-15)
    for got in (np.zeros_like(want),                                  # nothing
                without(case, range(n * 7 // 10, n), scale),          # the last pieces
                without(case, range(n // 2 // 32 * 32, n // 2 // 32 * 32 + 32), scale)):  # a tile
        assert np.mean(np.abs(got - want) > tol) > 0.5
    assert B.rejects(without(case, [n - 1], scale), want, tol)        # the last key


@pytest.mark.parametrize("n", [300, 9000])
def test_coarser_queries_and_weights_are_rejected(n):
    """fp32 queries held in fp16 or bf16, their weights in fp16, and bf16 queries'
    weights in bf16."""
    case = long_case("f32", n, 128, n)
    scale = 128 ** -0.5
    want, tol, _ = B.decode(*case, scale)
    q = case[0]
    for coarse in (q.astype(np.float16).astype(np.float32), Q.bf16_value(Q.bf16_bits(q))):
        assert B.rejects(Q.decode(coarse, *case[1:], scale)[0], want, tol)
    assert B.rejects(coarse_weights(case, scale, lambda w: w.astype(np.float16)), want, tol)
    case = long_case("bf16", n, 128, n)
    want, tol, _ = B.decode(*case, scale)
    half = coarse_weights(case, scale, lambda w: w.astype(np.float16))
    assert not B.rejects(half, want, tol)
    assert B.rejects(coarse_weights(case, scale, lambda w: Q.bf16_value(Q.bf16_bits(w))), want, tol)


def coarse_weights(case, scale, cast):
    """The output with the weights times V scales (relative to the largest) cast."""
    q, kc, vc, table, lens = case
    x = Q.bf16_value(q) if q.dtype == np.uint16 else q
    at = np.arange(lens[0])
    block = kc.shape[2]
    k = Q.values(kc[table[0, at // block], 0, at % block])
    u, s, z = Q.parts(vc[table[0, at // block], 0, at % block])
    out = np.zeros(q.shape)
    for h in range(q.shape[1]):
        e = scale * (k @ x[0, h].astype(np.float64))
        p = np.exp(e - e.max())
        w = np.asarray(cast((p[:, None] * s / s.max()).astype(np.float32)), np.float64) * s.max()
        out[0, h] = ((w * u).sum(0) + p @ z) / p.sum()
    return out

"""The 4-bit decode over values that its fp16 weights and their reference have to
follow: groups of equal values (scale 0) of any size, scales far apart, and of
either sign."""
import numpy as np
import pytest

import paged_kv_cache_70_gb300 as pkv
import q4_oracle as Q
from gpu_helpers import to_dev, widen

pytestmark = pytest.mark.gpu


def pool_of(rows, block=16):
    """One sequence's rows [n, Hkv, R] in pages 0, 1, .., and its table."""
    n, hkv, r = rows.shape
    blocks = -(-n // block)
    pool = np.zeros((blocks, hkv, block, r), np.uint8)
    pos = np.arange(n)
    pool[pos // block, :, pos % block] = rows
    return pool, np.arange(blocks, dtype=np.int32)[None]


def queries(hq, d, dtype, seed=0):
    q = np.random.default_rng(seed).standard_normal((1, hq, d)).astype(np.float32)
    return Q.bf16_bits(q) if dtype == "bf16" else q


def decode(q, k_rows, v_rows):
    """(the call's output, 64 bits, tolerance) of one sequence."""
    (kc, table), (vc, _) = pool_of(k_rows), pool_of(v_rows)
    n, d = len(k_rows), q.shape[-1]
    out = pkv.paged_decode_q4(to_dev(q), to_dev(kc), to_dev(vc), to_dev(table),
                              to_dev(np.asarray([n], np.int32)))
    want, tol = Q.decode(q, kc, vc, table, [n], d ** -0.5)
    assert pkv.paged_error_flags() == 0
    return widen(out), want, tol


def check(out, want, tol):
    assert np.all(np.abs(out - want) <= tol)  # (an infinity or a NaN is not)


HEADS = [(2, 1, 128), (4, 1, 128), (8, 1, 64), (2, 1, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("size", [1e-20, 1e12, 1e18, -1e30, 1e33, 3e38])
def test_groups_of_equal_values(dtype, hq, hkv, d, size):
    """Keys of equal score whose V is one value per group: the answer is that value."""
    n = 400
    k = np.zeros((n, hkv, d), np.float32)
    v = np.repeat(np.float32(size) / np.arange(1, d // 32 + 1, dtype=np.float32), 32)
    v = np.broadcast_to(v, (n, hkv, d))
    check(*decode(queries(hq, d, dtype), Q.quantise(k), Q.quantise(v)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_equal_values_beside_others(dtype, hq, hkv, d):
    """One group of equal, large values of either sign beside groups of ordinary ones,
    which keep their precision; the large ones grow along the keys."""
    rng = np.random.default_rng(d + hq)
    n = 700
    k = rng.standard_normal((n, hkv, d)).astype(np.float32)
    v = rng.standard_normal((n, hkv, d)).astype(np.float32)
    size = np.logspace(0, 33, n) * rng.choice([-1, 1], n)
    v[:, :, 32:64] = size[:, None, None]
    check(*decode(queries(hq, d, dtype), Q.quantise(k), Q.quantise(v)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("n", [400, 6000])
@pytest.mark.parametrize("small", [0.0, 1e-18, 1.0])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_scales_far_apart(dtype, hq, hkv, d, n, small, order):
    """Keys of equal score, half with V of 0 (or small), half with large V: both halves
    count in the sum of the weights, in one warp's keys and where pieces are merged."""
    large = 1e30 if small != 1.0 else 1e36
    ramp = np.tile(np.linspace(0.1, 1, 32), d // 32).astype(np.float32)
    at = np.arange(n)
    big = {"rising": at >= n // 2, "falling": at < n // 2, "mixed": at % 3 > 0}[order]
    v = np.where(big[:, None, None], np.float32(large), np.float32(small)) * ramp
    v = np.broadcast_to(v, (n, hkv, d)).astype(np.float32)
    k = np.zeros((n, hkv, d), np.float32)
    check(*decode(queries(hq, d, dtype), Q.quantise(k), Q.quantise(v)))

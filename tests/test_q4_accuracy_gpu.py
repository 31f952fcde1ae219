"""The 4-bit decode against bounds from the roundings it makes (q4_bounds)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_70_gb300 as pkv
import q4_bounds as B
import q4_oracle as Q
from gpu_helpers import to_dev, widen
from test_q4_bounds import competing, long_case
from test_q4_gpu import DECODE, decode_case

pytestmark = pytest.mark.gpu


def check(q, kc, vc, table, lens, scale):
    out = widen(pkv.paged_decode_q4(to_dev(q), to_dev(kc), to_dev(vc), to_dev(table),
                                    to_dev(np.asarray(lens, np.int32)), scale=scale))
    want, tol, rms = B.decode(q, kc, vc, table, lens, scale)
    err = np.abs(out - want)
    worst = np.max(err / np.maximum(tol, 1e-300))
    assert np.all(err <= tol), f"{worst:.3g} of the bound"
    mean = lambda x: np.sqrt(np.mean(x ** 2))
    assert mean(err) <= mean(rms), f"{mean(err) / mean(rms):.3g} of the mean bound"
    assert pkv.paged_error_flags() == 0


@pytest.mark.parametrize("i", range(len(DECODE)))
def test_lengths_and_heads(i):
    lens, hq, hkv, d, block, dtype = DECODE[i]
    q, kc, vc, table = decode_case(lens, hq, hkv, d, block, dtype, 100 + i)
    check(q, kc, vc, table, lens, d ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [300, 9000, 12345, 20000])
@pytest.mark.parametrize("d", [64, 128])
def test_long_contexts(dtype, n, d):
    check(*long_case(dtype, n, d, n), scale=d ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, 0.5, -0.3, 3.0])
def test_flat_and_peaked_weights(dtype, scale):
    q, kc, vc, table = decode_case([700, 45], 8, 4, 128, 16, dtype, 7)
    check(q, kc, vc, table, [700, 45], scale)


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (8, 2, 128), (16, 2, 128), (4, 2, 64), (8, 2, 64),
                                      (16, 2, 64)])
@pytest.mark.parametrize("outliers", [False, True])
def test_few_keys_with_large_scores(hq, hkv, d, outliers):
    case = competing(hq, hkv, d, 48, 3, 5, outliers)
    check(*case, scale=3.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (8, 2, 128), (16, 2, 64), (4, 2, 64)])
@pytest.mark.parametrize("share", [1.0, 0.5])
def test_scales_of_either_sign(dtype, hq, hkv, d, share):
    """Rows of another writer: the scales of some groups of K and V below 0."""
    rng = np.random.default_rng(d + hq)
    n, block = 300, 16
    lens = [n, 77]
    q = rng.standard_normal((2, hq, d)).astype(np.float32)
    q = Q.bf16_bits(q) if dtype == "bf16" else q
    table = np.arange(2 * 19, dtype=np.int32).reshape(2, 19)
    pools = []
    for _ in range(2):
        rows = Q.quantise(rng.standard_normal((38, hkv, block, d)).astype(np.float32))
        sz = rows[..., d // 2:].copy().view(np.uint16)
        sz[..., 0::2] |= np.where(rng.random(sz[..., 0::2].shape) < share, 0x8000, 0).astype(np.uint16)
        rows[..., d // 2:] = sz.view(np.uint8)
        pools.append(rows)
    check(q, *pools, table, lens, d ** -0.5)


def test_one_workspace_in_calls_with_other_tile_starts():
    """Calls back to back whose plans differ, in one workspace: each has its own bits."""
    rng = np.random.default_rng(3)
    hq, hkv, d, block = 16, 8, 128, 16
    pool = Q.quantise(rng.standard_normal((400, hkv, block, d)).astype(np.float32))
    kd = to_dev(pool)
    calls, ws = [], None
    for lens in ([3000, 20, 1], [7, 7, 7], [0, 2500, 900], [64, 0, 0]):
        table = rng.integers(0, 400, (3, 190)).astype(np.int32)
        q = torch.randn(3, hq, d, device="cuda", dtype=torch.bfloat16)
        args = q, kd, kd, to_dev(table), to_dev(np.asarray(lens, np.int32))
        if ws is None:
            ws = torch.empty(pkv.paged_decode_q4_workspace_size(3, hq, torch.bfloat16, kd),
                             dtype=torch.uint8, device="cuda")
        calls.append((args, pkv.paged_decode_q4(*args)))
    torch.cuda.synchronize()
    outs = [(want, pkv.paged_decode_q4(*args, workspace=ws))
            for _ in range(100) for args, want in calls]
    assert all(torch.equal(a, b) for a, b in outs)


@pytest.mark.parametrize("d", [64, 128])
def test_read_rounds_once(d):
    """Rows whose value lies beside the middle of two bf16 neighbours, nearer to it than
    fp32 can tell: scale 129/128 or 131/128, codes 3 or 5 off 8, offsets of 2^-30."""
    s, u, sign = np.meshgrid([0x3F81, 0x3F83], [11, 5, 13, 3], [1, -1], indexing="ij")
    s, u, sign = (x.reshape(-1) for x in (s, u, sign))
    rows = np.zeros((len(s), 1, 5 * d // 8), np.uint8)
    rows[..., :d // 2] = (u * 17)[:, None, None]
    sz = np.stack((s, Q.bf16_bits(sign * np.float32(2.0 ** -30))), -1).astype(np.uint16)
    rows[..., d // 2:] = np.tile(sz, (1, d // 32)).view(np.uint8)[:, None]
    pool = rows.reshape(1, 1, len(s), -1)
    k, v = pkv.paged_kv_read_q4(to_dev(pool), to_dev(pool),
                                to_dev(np.arange(len(s), dtype=np.int32)), torch.bfloat16)
    x = Q.values(rows)
    # the neighbours of 8 significant bits, and the nearer of the two
    step = np.exp2(np.floor(np.log2(np.abs(x))) - 7)
    lo = np.floor(x / step) * step
    want = np.where(x - lo < lo + step - x, lo, lo + step)
    middle = (Q.values(rows).astype(np.float32) - lo) / step == 0.5
    assert middle.sum() >= 4 * d  # (fp32 sees these in the middle)
    assert np.array_equal(widen(k), want) and np.array_equal(widen(v), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (8, 1, 64)])
@pytest.mark.parametrize("size", [1e-30, 1e-15, 1e15, 1e30])
def test_sizes_of_queries_and_keys(dtype, hq, hkv, d, size):
    """Queries of any size over keys of the inverse: scores of the usual size."""
    rng = np.random.default_rng(hq)
    lens, block = [90, 33], 16
    q = (rng.standard_normal((2, hq, d)) * size).astype(np.float32)
    k, v = (rng.standard_normal((12, hkv, block, d)).astype(np.float32) for _ in range(2))
    table = np.arange(12, dtype=np.int32).reshape(2, 6)
    check(Q.bf16_bits(q) if dtype == "bf16" else q, Q.quantise((k / size).astype(np.float32)),
          Q.quantise(v), table, lens, d ** -0.5)
    # every product at its largest, of one sign
    q[:], k[:] = size, 1 / size
    check(Q.bf16_bits(q) if dtype == "bf16" else q, Q.quantise(k), Q.quantise(v), table, lens, d ** -1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (8, 2, 128), (16, 2, 128), (4, 2, 64)])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_an_infinity_in_v_stays_in_its_group(dtype, hq, hkv, d, bad):
    """One value of V that is no number: its 32 dims are NaN, the others as without it."""
    rng = np.random.default_rng(d)
    n, block = 500, 16
    q = rng.standard_normal((1, hq, d)).astype(np.float32)
    q = Q.bf16_bits(q) if dtype == "bf16" else q
    k, v = (rng.standard_normal((32, hkv, block, d)).astype(np.float32) for _ in range(2))
    table = np.arange(32, dtype=np.int32)[None]
    kc, vc = Q.quantise(k), Q.quantise(v)
    v[7, 1, 5, 33] = bad
    broken = Q.quantise(v)
    out = widen(pkv.paged_decode_q4(to_dev(q), to_dev(kc), to_dev(broken), to_dev(table),
                                    to_dev(np.asarray([n], np.int32))))
    want, tol, _ = B.decode(q, kc, vc, table, [n], d ** -0.5)
    nan = np.zeros(out.shape, bool)
    nan[:, hq // hkv:, 32:64] = True
    assert np.array_equal(np.isnan(out), nan)
    assert np.all(np.abs(out - want)[~nan] <= tol[~nan])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (8, 2, 128), (16, 2, 128), (4, 2, 64)])
@pytest.mark.parametrize("size", [1e-18, 1.6e38])
def test_the_least_and_largest_values(dtype, hq, hkv, d, size):
    """V whose groups span nearly all that fp32 holds, and V far below 1."""
    rng = np.random.default_rng(hq + d)
    lens, block = [700, 33], 16
    q = rng.standard_normal((2, hq, d)).astype(np.float32)
    k = rng.standard_normal((88, hkv, block, d)).astype(np.float32)
    v = (rng.uniform(-1, 1, (88, hkv, block, d)) * size).astype(np.float32)
    table = np.arange(88, dtype=np.int32).reshape(2, 44)
    check(Q.bf16_bits(q) if dtype == "bf16" else q, Q.quantise(k), Q.quantise(v), table, lens,
          d ** -0.5)

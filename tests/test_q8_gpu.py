"""8-bit pools on the GPU: the write, the read and the decode against the numpy model of the
format (q8_oracle), and all of them together as a serving loop uses them."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_70_gb300 as pkv
import q4_oracle as Q4
import q8_oracle as Q
from gpu_helpers import to_dev, to_host, widen
from test_rope_write_gpu import new_tokens, rows

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def pool(codes):
    return to_dev(codes).view(F8)


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def random_pool(rng, total, hkv, block, d):
    """Any bytes (NaN codes among them) and scales from 2^-20 to 2^12, some no power of two,
    some 0."""
    codes = rng.integers(0, 256, (total, hkv, block, d), dtype=np.uint8)
    scale = np.exp2(rng.integers(-20, 13, (total, hkv))).astype(np.float32)
    scale[rng.random(scale.shape) < 0.1] *= 1.3
    scale[rng.random(scale.shape) < 0.05] = 0
    return codes, scale


# ---------------------------------------------------------------------------
# write and read
# ---------------------------------------------------------------------------
WRITES = [  # (cached, new), Hq, Hkv, d, rot (0: none), interleaved, B, type, padding, fused
    ([(0, 1)], 1, 1, 64, 0, False, 1, "f32", 0, 0),
    ([(5, 1), (0, 1), (77, 1), (15, 1), (16, 1)], 16, 8, 128, 128, False, 16, "bf16", 0, 0),
    ([(5, 1), (0, 1), (77, 1), (15, 1)], 16, 8, 128, 64, True, 16, "bf16", 3, 24),
    ([(3, 40), (0, 0), (100, 9)], 6, 3, 128, 0, False, 7, "bf16", 1, 0),
    ([(3, 40), (17, 300)], 4, 2, 64, 48, False, 24, "f32", 2, 2),
    ([(0, 33), (33, 33)], 22, 11, 64, 64, True, 33, "bf16", 2, 0),
    ([(1, 600), (255, 2), (250, 1)], 8, 2, 128, 128, False, 256, "bf16", 0, 2),
    ([(1, 600), (255, 2), (250, 1)], 8, 2, 128, 128, False, 256, "f32", 0, 0),
    ([(100, 1500)], 1, 1, 64, 32, False, 1000, "bf16", 0, 0),
    ([(100, 1500)], 1, 1, 128, 0, False, 700, "f32", 5, 0),
    ([(9, 5)] * 70, 17, 17, 128, 16, False, 32, "bf16", 40, 0),
    ([(i % 40, 1 + i % 3) for i in range(400)], 8, 8, 64, 64, False, 8, "bf16", 0, 0),
    ([(7, 3000), (0, 2000)], 2, 1, 64, 64, False, 16, "bf16", 0, 0),
    ([(0, 64)] * 3, 4, 4, 128, 128, False, 64, "bf16", 0, 0),
    ([(2, 130)], 4, 4, 128, 128, True, 128, "f32", 0, 0),
    # runs that go on for windows of 256 tokens, and end with one, behind one or before one
    ([(0, 768), (4090, 1), (1, 511), (40, 257)], 2, 1, 64, 64, False, 4096, "bf16", 0, 0),
    ([(3, 2500), (1900, 700)], 2, 2, 128, 0, False, 2048, "f32", 0, 0),
    ([(200, 1), (0, 255), (5, 513), (0, 1025)], 1, 1, 64, 32, True, 600, "bf16", 7, 0),
]


def special(x, rng):
    """Heads that a quantiser can go wrong at, among normal ones."""
    f = x.reshape(-1, x.shape[-1])
    n = len(f)
    d = x.shape[-1]
    rows_ = [np.zeros(d), np.full(d, -0.0), np.full(d, 1e-41), np.full(d, -3e38),
             np.r_[np.zeros(d - 1), 1e30], np.r_[np.inf, np.ones(d - 1)],
             np.r_[np.ones(d - 1), -np.inf], np.full(d, np.nan), np.r_[np.nan, np.ones(d - 1)],
             np.full(d, 448.0), np.full(d, 449.0), np.full(d, 464.0) * np.r_[np.ones(d - 1), 0],
             rng.standard_normal(d) * 2.0 ** -105, rng.standard_normal(d) * 1e4]
    for i, s in enumerate(rows_):
        if n > 8 * i + 3:
            f[(8 * i + 3) % n] = s.astype(np.float32)
    return x


@pytest.mark.parametrize("sizes,hq,hkv,d,rot,mix,block,dtype,pad,fused", WRITES)
@pytest.mark.parametrize("odd", [False, True])
def test_write_stores_the_formats_bytes_and_read_returns_their_values(sizes, hq, hkv, d, rot, mix,
                                                                      block, dtype, pad, fused,
                                                                      odd):
    rng = np.random.default_rng(d + rot + block)
    table, total, seq, pos = new_tokens(rng, sizes, block, pad)
    n = len(seq)
    x = []
    for _ in range(2):
        a, t = rows(rng, n, hkv, d, dtype, fused)
        if odd:
            a = special(a, rng)
            if dtype == "bf16":
                a = Q4.bf16_value(Q4.bf16_bits(a)).astype(np.float32)
            t.copy_(to_dev(a))
        x.append((a, t))
    (k, kt), (v, vt) = x
    before = [random_pool(rng, total, hkv, block, d) for _ in range(2)]
    if not odd:
        before = [(c & 0xBF, s) for c, s in before]  # (no NaN codes)
    (kb, ksb), (vb, vsb) = before
    kc, vc, ks, vs = pool(kb), pool(vb), to_dev(ksb), to_dev(vsb)
    kw, cs = {}, None
    if rot:
        cs = Q.cos_sin(max(pos.max(), 0) + 9, rot)
        q, qt = rows(rng, n, hq, d, dtype, fused)
        kw = dict(cos_sin=to_dev(cs), q=qt, interleaved=mix)
    out = pkv.paged_kv_write_q8(kt, vt, to_dev(table), to_dev(seq), to_dev(pos), kc, vc, ks, vs,
                                **kw)
    live = seq >= 0
    if rot:
        with np.errstate(invalid="ignore", over="ignore"):
            kr = k.copy()
            kr[live] = Q.rotate(k[live], cs, pos[live], mix)
            q[live] = Q.rotate(q[live], cs, pos[live], mix)
        assert np.array_equal(to_host(out), Q4.bf16_bits(q) if dtype == "bf16" else q)
        k = kr
    else:
        assert out is None
    for got, gots, c, s, val in ((kc, ks, kb, ksb, k), (vc, vs, vb, vsb, v)):
        c, s = c.copy(), s.copy()
        Q.write(val, table, seq, pos, c, s, live)
        assert np.array_equal(to_host(gots), s, equal_nan=True)
        assert np.array_equal(Q.canon(codes_of(got)), Q.canon(c))
    # every row of the sequences back, some twice, padding as zeros
    ask = np.array([table[b, p // block] * block + p % block for b, (o, m) in enumerate(sizes)
                    for p in range(o + m)] + [-1, -9], np.int32)
    ask = np.concatenate((ask, ask[:5]))
    for to in (torch.float32, torch.bfloat16):
        got = pkv.paged_kv_read_q8(kc, vc, ks, vs, to_dev(ask), to)
        for g, c, s in zip(got, (kc, vc), (ks, vs)):
            want = Q.values(codes_of(c), to_host(s))[np.maximum(ask, 0) // block, :,
                                                          np.maximum(ask, 0) % block]
            want = np.float32(np.where((ask < 0)[:, None, None], 0.0, want))
            if to == torch.bfloat16:
                assert np.array_equal(np.isnan(widen(g)), np.isnan(want))
                ok = ~np.isnan(want)
                assert np.array_equal(to_host(g)[ok], Q4.bf16_bits(want)[ok])
            else:
                assert np.array_equal(to_host(g), want, equal_nan=True)
    assert pkv.paged_error_flags() == 0


def test_one_token_at_a_time_or_all_at_once():
    """Without growth behind the first token the bytes are the same; with it, values differ by
    what a coarser scale cannot hold, 2^-10 of it per growth."""
    rng = np.random.default_rng(2)
    n, hkv, d, block = 40, 2, 64, 16
    for falling in (True, False):
        x = rng.uniform(0.5, 1, (n, hkv, d)) * rng.choice([-1, 1], (n, hkv, d))
        x = (x * np.exp2((-1 if falling else 1) * (np.arange(n) % block))[:, None, None]).astype(np.float32)
        table = to_dev(np.array([[2, 0, 1]], np.int32))
        res = []
        for parts in ([(0, n)], [(i, i + 1) for i in range(n)]):
            kc, vc = (torch.zeros(3, hkv, block, d, device="cuda").to(F8) for _ in range(2))
            ks, vs = (torch.zeros(3, hkv, device="cuda") for _ in range(2))
            for lo, hi in parts:
                t = to_dev(x[lo:hi])
                seq = torch.zeros(hi - lo, dtype=torch.int32, device="cuda")
                pos = torch.arange(lo, hi, dtype=torch.int32, device="cuda")
                pkv.paged_kv_write_q8(t, t, table, seq, pos, kc, vc, ks, vs)
            res.append((codes_of(kc), to_host(ks), codes_of(vc), to_host(vs)))
        (a, sa, va, ta), (b, sb, vb, tb) = res
        assert np.array_equal(sa, sb) and np.array_equal(a, va) and np.array_equal(sa, ta)
        assert np.array_equal(b, vb) and np.array_equal(sb, tb)
        if falling:
            assert np.array_equal(a, b)
        else:
            gap = np.abs(Q.values(a, sa) - Q.values(b, sb))
            assert np.all(gap <= 16 * 2.0 ** -10 * sa[..., None, None])


def test_tokens_that_are_not_written():
    d, hkv, block = 64, 2, 4
    table = torch.tensor([[2, 9], [0, -1]], dtype=torch.int32, device="cuda")
    seq = [0, 0, 1, 1, 2, 0, -7, 1]
    pos = [1, 4, 5, 8, 0, 2, 0, 3]
    at = [1, 4, 5, 8, 0, 50, 0, 3]
    flags = [0, pkv.PKV_FLAG_BAD_BLOCK, pkv.PKV_FLAG_BAD_BLOCK, pkv.PKV_FLAG_BAD_LENGTH,
             pkv.PKV_FLAG_BAD_SEQ, pkv.PKV_FLAG_BAD_LENGTH, 0, 0]
    x = np.random.default_rng(0).standard_normal((8, hkv, d)).astype(np.float32)
    cs = Q.cos_sin(50, d)
    dev = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")
    for some in [list(range(8)), [0, 5], [5, 0]] + [[i] for i in range(8)]:
        codes = np.full((3, hkv, block, d), 0x2A, np.uint8)
        scale = np.full((3, hkv), 0.125, np.float32)
        kc, vc, ks, vs = pool(codes), pool(codes), to_dev(scale), to_dev(scale)
        t = to_dev(x[some])
        pkv.paged_kv_write_q8(t, t, table, dev([seq[i] for i in some]), dev([pos[i] for i in some]),
                              kc, vc, ks, vs, cos_sin=to_dev(cs), rope_pos=dev([at[i] for i in some]))
        want = 0
        for i in some:
            want |= flags[i]
        assert pkv.paged_error_flags() == want
        for got, gots, turned in ((kc, ks, True), (vc, vs, False)):
            c, s = codes.copy(), scale.copy()
            for i in some:
                if i in (0, 7):
                    y = Q.rotate(x[i:i + 1], cs, np.array([at[i]]), False) if turned else x[i:i + 1]
                    Q.write(y, np.array([[2], [0]]), [seq[i]], [pos[i]], c, s, [True])
            assert np.array_equal(codes_of(got), c) and np.array_equal(to_host(gots), s)


def test_old_scales_that_no_page_may_have_read_as_nan():
    d, hkv, block = 128, 1, 8
    for bad in (-1.0, float("nan"), float("inf"), 2.0 ** 127):
        kc = pool(np.full((1, hkv, block, d), 0x38, np.uint8))
        ks = torch.full((1, hkv), bad, device="cuda")
        t = torch.ones(1, hkv, d, device="cuda")
        i = dict(dtype=torch.int32, device="cuda")
        pkv.paged_kv_write_q8(t, t, torch.zeros(1, 1, **i), torch.zeros(1, **i),
                              torch.full((1,), 3, **i), kc, kc.clone(), ks, ks.clone())
        assert bool(ks.isnan().all())
        k, _ = pkv.paged_kv_read_q8(kc, kc, ks, ks, torch.arange(4, **i), torch.float32)
        assert bool(k.isnan().all())


def test_read_slots_past_the_pool_are_flagged():
    rng = np.random.default_rng(4)
    codes, scale = random_pool(rng, 2, 3, 4, 64)
    kc, ks = pool(codes & 0xBF), to_dev(scale)
    ask = torch.tensor([8, 7, 2**31 - 1, -1], dtype=torch.int32, device="cuda")
    k, v = pkv.paged_kv_read_q8(kc, kc, ks, ks, ask, torch.float32)
    assert pkv.paged_error_flags() == pkv.PKV_FLAG_BAD_SLOT
    assert not k[[0, 2, 3]].any() and not v[[0, 2, 3]].any()
    assert np.array_equal(to_host(k)[1], Q.values(codes & 0xBF, scale)[1, :, 3].astype(np.float32))
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    k, v = pkv.paged_kv_read_q8(kc, kc, ks, ks, e)
    assert k.shape == (0, 3, 64) and v.dtype == torch.bfloat16


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
DECODE = [  # lens, Hq, Hkv, d, B, type
    ([30, 32, 70], 2, 1, 64, 32, "f32"),
    ([1], 1, 1, 128, 16, "bf16"),
    ([0], 4, 2, 64, 8, "bf16"),
    ([0, 1, 17, 0, 300, 16, 15], 16, 8, 128, 16, "bf16"),
    ([5, 1000, 64, 63, 65], 8, 8, 128, 8, "bf16"),
    ([77, 500], 16, 8, 64, 16, "bf16"),
    ([129, 33, 2000], 32, 8, 128, 256, "bf16"),
    ([400, 31], 32, 4, 64, 16, "bf16"),
    ([513, 100, 3], 64, 8, 128, 16, "bf16"),
    ([700, 90], 32, 2, 128, 64, "bf16"),
    ([260, 41], 32, 1, 128, 16, "bf16"),
    ([100, 257], 5, 1, 64, 48, "bf16"),
    ([64, 250, 7], 15, 3, 128, 24, "bf16"),
    ([90, 21], 12, 1, 128, 16, "bf16"),
    ([210, 5], 34, 17, 64, 32, "bf16"),
    ([99], 16, 16, 128, 16, "bf16"),
    ([150, 64], 48, 24, 128, 16, "bf16"),
    ([3000], 16, 8, 128, 16, "f32"),
    ([61, 0, 200], 32, 8, 64, 8, "f32"),
    ([128, 50], 24, 3, 128, 32, "f32"),
    ([45, 333], 16, 1, 64, 16, "f32"),
    ([20000, 9000, 1], 16, 8, 128, 256, "bf16"),
    ([12345], 2, 1, 128, 16, "bf16"),
    ([40] * 200 + [1500], 16, 8, 128, 16, "bf16"),
    ([500, 33], 10, 5, 128, 16, "bf16"),
    ([77, 410], 28, 7, 64, 32, "bf16"),
    ([96, 97, 95], 20, 10, 128, 16, "bf16"),
    ([385, 383], 24, 12, 128, 8, "f32"),
    ([1000, 20], 64, 1, 128, 16, "bf16"),
    ([700], 128, 2, 64, 16, "f32"),
    ([100, 3], 18, 6, 64, 64, "f32"),
    ([50] * 3, 32, 32, 128, 16, "bf16"),
    # sequences that a CTA takes whole, at the border to those that are split, empty ones
    ([192, 0, 1, 191], 16, 8, 128, 16, "bf16"),
    ([193, 5], 16, 8, 128, 1, "bf16"),
    ([0, 0, 0], 16, 8, 64, 8, "f32"),
    ([512, 0, 300], 2, 1, 64, 32, "f32"),
    ([0] + [47, 48, 49] * 21, 32, 8, 128, 16, "bf16"),
    ([630, 0, 7] * 25 + [600], 16, 8, 128, 16, "bf16"),
    ([9, 0, 160], 24, 1, 128, 20, "bf16"),
    ([100] * 152, 8, 4, 128, 16, "bf16"),
    ([100] * 153, 8, 4, 128, 16, "bf16"),
    # pages whose rows do not fill the swizzle's 8
    ([5, 100, 64], 8, 8, 128, 1, "bf16"),
    ([77, 200], 16, 8, 64, 2, "bf16"),
    ([90, 31], 6, 3, 128, 20, "f32"),
    ([90, 31], 6, 3, 128, 7, "bf16"),
    ([333, 1], 4, 4, 64, 6, "bf16"),
    ([640], 4, 2, 128, 300, "bf16"),
]


def decode_inputs(rng, lens, hq, hkv, d, block, dtype, spread=3):
    """Queries, pools whose rows outside the sequences are NaN (scales too), and the table."""
    need = [-(-n // block) for n in lens]
    total = sum(need) + 3
    ids = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(need + [1])), -1, np.int32)
    pools = []
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    for _ in range(2):
        codes = np.full((total, hkv, block, d), 0x7F, np.uint8)
        scale = np.full((total, hkv), np.nan, np.float32)
        for b, n in enumerate(lens):
            p = np.arange(n)
            scale[table[b, :need[b]]] = np.exp2(rng.integers(-spread, spread + 1, (need[b], hkv))) / 32
            codes[table[b, p // block], :, p % block] = Q.encode(
                np.clip(rng.standard_normal((n, hkv, d)) * 16, -448, 448))
        pools += [codes, scale]
    x, t = rows(rng, len(lens), hq, d, dtype)
    return x / 1.0, t, pools, table


def decode_want(q, kc, ks, vc, vs, table, lens, scale, block):
    """(output, sum p |v|, largest sum |q k| scale) in 64 bits."""
    n, hq, d = q.shape
    hkv = kc.shape[1]
    out, mass = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    reach = np.zeros((n, hq, 1))
    for b, m in enumerate(lens):
        if not m:
            continue
        pages = table[b, : -(-m // block)]
        k = Q.values(kc[pages], ks[pages]).transpose(0, 2, 1, 3).reshape(-1, hkv, d)[:m]
        v = Q.values(vc[pages], vs[pages]).transpose(0, 2, 1, 3).reshape(-1, hkv, d)[:m]
        for h in range(hq):
            g = h // (hq // hkv)
            s = k[:, g] @ q[b, h].astype(np.float64) * scale
            reach[b, h] = np.max(np.abs(k[:, g]) @ np.abs(q[b, h].astype(np.float64))) * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[b, h], mass[b, h] = p @ v[:, g], p @ np.abs(v[:, g])
    return out, mass, reach


def decode_bound(want, mass, reach, lens, dtype):
    """What roundings leave.  Scores: products of fp16 parts are exact, sums of 128 of them in
    fp32 lose 8 steps of 2^-23 (the tensor cores cut) of sum |q k|, the conversion to log2 units
    and the exponential 2^-22 of the score, fp32 queries' parts 2^-22 of sum |q k|: together
    2^-19 of it, twice (weight and sum).  Weights: 2^-11 (bf16) or 2^-22, and what lies below the
    least fp16, 2^-31 or 2^-37 of the largest.  Sums over the keys: one step of 2^-23 per 16 keys
    and 40 merges.  The output's own rounding."""
    keys = np.array(lens, np.float64)[:, None, None]
    score = 2 * 2.0 ** -19 * reach + 2.0 ** -21
    weight = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
    sums = (keys / 16 + 40) * 2.0 ** -23
    out = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    return out * np.abs(want) + 1.1 * mass * (score + weight + sums) + 1e-30


@pytest.mark.parametrize("lens,hq,hkv,d,block,dtype", DECODE)
def test_decode(lens, hq, hkv, d, block, dtype):
    rng = np.random.default_rng(len(lens) + hq * 3 + d + block)
    q, qt, (kc, ks, vc, vs), table = decode_inputs(rng, lens, hq, hkv, d, block, dtype)
    got = pkv.paged_decode_q8(qt, pool(kc), pool(vc), to_dev(ks), to_dev(vs), to_dev(table),
                              to_dev(np.array(lens, np.int32)))
    assert pkv.paged_error_flags() == 0
    want, mass, reach = decode_want(q, kc, ks, vc, vs, table, lens, 1 / math.sqrt(d), block)
    assert got.dtype == qt.dtype
    err = np.abs(widen(got) - want)
    bound = decode_bound(want, mass, reach, lens, dtype)
    assert np.all(np.isfinite(err)) and np.all(err <= bound), (err / bound).max()


@pytest.mark.parametrize("lens,hq,hkv,d,block,dtype", DECODE)
def test_decode_with_a_table_for_longer_contexts(lens, hq, hkv, d, block, dtype):
    """The same sequences where the table could hold 400,000 keys of each: what is a CTA's or a
    cluster's there is split here."""
    rng = np.random.default_rng(len(lens) + hq * 3 + d + block)
    q, qt, (kc, ks, vc, vs), table = decode_inputs(rng, lens, hq, hkv, d, block, dtype)
    wide = np.full((len(lens), 400000 // block), -1, np.int32)
    wide[:, :table.shape[1]] = table
    got = pkv.paged_decode_q8(qt, pool(kc), pool(vc), to_dev(ks), to_dev(vs), to_dev(wide),
                              to_dev(np.array(lens, np.int32)))
    assert pkv.paged_error_flags() == 0
    want, mass, reach = decode_want(q, kc, ks, vc, vs, table, lens, 1 / math.sqrt(d), block)
    err = np.abs(widen(got) - want)
    assert np.all(err <= decode_bound(want, mass, reach, lens, dtype))


CLUSTERS = [  # lens, Hq, Hkv, d, B, type, keys that the table holds
    ([0, 1, 191, 192, 193, 1536, 1537, 2000], 4, 1, 128, 16, "bf16", 2000),  # fewer tiles than CTAs
    ([0, 5, 3000], 32, 4, 64, 16, "bf16", 4096),
    ([0], 16, 8, 128, 16, "f32", 4096),
    ([1, 4096], 40, 2, 128, 32, "bf16", 4096),   # 20 queries per KV head: three warps' worth
    ([700, 0, 33, 1500] * 4, 16, 8, 128, 16, "f32", 1500),
    ([1000] * 30, 16, 8, 128, 64, "bf16", 1024),
    ([990, 77] * 30, 8, 4, 64, 2, "bf16", 1000),
    ([64, 900] * 9, 6, 6, 128, 1, "bf16", 900),
    ([800, 31], 64, 1, 64, 8, "f32", 800),
]


@pytest.mark.parametrize("lens,hq,hkv,d,block,dtype,keys", CLUSTERS)
def test_decode_of_sequences_that_clusters_share(lens, hq, hkv, d, block, dtype, keys):
    rng = np.random.default_rng(keys + hq)
    q, qt, (kc, ks, vc, vs), table = decode_inputs(rng, lens, hq, hkv, d, block, dtype)
    wide = np.full((len(lens), -(-keys // block)), -1, np.int32)
    wide[:, :table.shape[1]] = table
    args = (qt, pool(kc), pool(vc), to_dev(ks), to_dev(vs), to_dev(wide),
            to_dev(np.array(lens, np.int32)))
    got = pkv.paged_decode_q8(*args)
    assert pkv.paged_error_flags() == 0
    want, mass, reach = decode_want(q, kc, ks, vc, vs, table, lens, 1 / math.sqrt(d), block)
    err = np.abs(widen(got) - want)
    assert np.all(err <= decode_bound(want, mass, reach, lens, dtype))
    assert torch.equal(got, pkv.paged_decode_q8(*args))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("spread", [20, 60])
def test_decode_scales_far_apart(dtype, spread):
    """V scales from 2^-spread to 2^spread, next to one another and anywhere in the sequence:
    the weights' reference follows the products, so that the bound is relative to sum p |v| of
    each output whatever other pages hold."""
    rng = np.random.default_rng(spread)
    lens, hq, hkv, d, block = [700, 33, 2000], 8, 4, 128, 16
    q, qt, (kc, ks, vc, vs), table = decode_inputs(rng, lens, hq, hkv, d, block, dtype)
    vs *= np.exp2(rng.integers(-spread, spread + 1, vs.shape)).astype(np.float32)
    got = pkv.paged_decode_q8(qt, pool(kc), pool(vc), to_dev(ks), to_dev(vs), to_dev(table),
                              to_dev(np.array(lens, np.int32)))
    want, mass, reach = decode_want(q, kc, ks, vc, vs, table, lens, 1 / math.sqrt(d), block)
    err = np.abs(widen(got) - want)
    assert np.all(err <= decode_bound(want, mass, reach, lens, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_large_scales_before_keys_that_outweigh_them(dtype):
    """The first half of the keys has V scales of 2^60 and scores far below those of the second
    half, whose V are of ordinary size: nothing of the second half's bits is lost."""
    rng = np.random.default_rng(9)
    lens, hq, hkv, d, block = [1024], 4, 2, 128, 16
    q, qt, (kc, ks, vc, vs), table = decode_inputs(rng, lens, hq, hkv, d, block, dtype, spread=0)
    # the queries are one direction, the keys of the second half lie along it
    q[:] = 1.0
    qt.copy_(to_dev(q.astype(np.float32)))
    late = table[0, 32:]
    kc[late] = Q.encode(np.abs(Q.VALUES[kc[late] & 0x77]) + 32)
    kc[table[0, :32]] = Q.encode(-np.abs(Q.VALUES[kc[table[0, :32]] & 0x77]) - 32)
    vs[table[0, :32]] = 2.0 ** 60
    got = pkv.paged_decode_q8(qt, pool(kc), pool(vc), to_dev(ks), to_dev(vs), to_dev(table),
                              to_dev(np.array(lens, np.int32)), scale=1.0)
    want, mass, reach = decode_want(q, kc, ks, vc, vs, table, lens, 1.0, block)
    assert np.abs(want).max() < 1e3  # the large ones have no weight
    err = np.abs(widen(got) - want)
    assert np.all(err <= decode_bound(want, mass, reach, lens, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [64, 1024])
@pytest.mark.parametrize("first,then", [(0.0, 8.0), (0.0, 2.0 ** 100), (2.0 ** -100, 2.0 ** 40),
                                        (-(2.0 ** -100), -(2.0 ** 90)), (2.0 ** 40, 2.0 ** 90)])
def test_decode_larger_scales_behind_keys_that_outweigh_them(dtype, n, first, then):
    """The second half's keys have no weight (their scores are hundreds below the others'), whatever
    their V scales are: a weight of zero times a scale past the range of the reference is nothing,
    and no NaN.  (Also where a sequence begins with V scales of zero.)"""
    rng = np.random.default_rng(n)
    lens, hq, hkv, d, block = [n], 4, 2, 128, 16
    q, qt, (kc, ks, vc, vs), table = decode_inputs(rng, lens, hq, hkv, d, block, dtype, spread=0)
    q[:] = 1.0
    qt.copy_(to_dev(q.astype(np.float32)))
    early, late = table[0, : n // 32], table[0, n // 32:]
    kc[early] = Q.encode(np.abs(Q.VALUES[kc[early] & 0x77]) + 32)
    kc[late] = Q.encode(-np.abs(Q.VALUES[kc[late] & 0x77]) - 32)
    vs[early], vs[late] = first, then
    got = pkv.paged_decode_q8(qt, pool(kc), pool(vc), to_dev(ks), to_dev(vs), to_dev(table),
                              to_dev(np.array(lens, np.int32)), scale=2.0)
    # (in 64 bits the late keys would weigh 2^-700 and less)
    late_v = vs.copy()
    late_v[late] = 0.0
    want, mass, reach = decode_want(q, kc, ks, vc, late_v, table, lens, 2.0, block)
    err = np.abs(widen(got) - want)
    assert np.all(err <= decode_bound(want, mass, reach, lens, dtype))


def test_decode_nans_stay_with_their_own():
    rng = np.random.default_rng(3)
    lens, hq, hkv, d, block = [100, 64, 40], 8, 4, 128, 16
    for what in ("k", "v", "ks", "vs", "q", "k scale inf"):
        q, qt, (kc, ks, vc, vs), table = decode_inputs(rng, lens, hq, hkv, d, block, "bf16")
        bad = np.zeros((3, hq, d), bool)
        if what == "k":
            kc[table[0, 2], 1, 3, 7] = 0xFF
            bad[0, 2:4] = True
        elif what == "v":
            vc[table[0, 2], 1, 3, 7] = 0x7F
            bad[0, 2:4, 7] = True
        elif what == "ks":
            ks[table[1, 0], 3] = np.nan
            bad[1, 6:8] = True
        elif what == "vs":
            vs[table[1, 0], 3] = np.nan
            bad[1, 6:8] = True
        elif what == "k scale inf":
            ks[table[1, 0], 3] = np.inf
            bad[1, 6:8] = True
        else:
            qt[2, 5, 9] = float("nan")
            bad[2, 5] = True
        got = widen(pkv.paged_decode_q8(qt, pool(kc), pool(vc), to_dev(ks), to_dev(vs),
                                        to_dev(table), to_dev(np.array(lens, np.int32))))
        assert np.array_equal(np.isnan(got), bad), what


def test_decode_bad_pages_and_lengths():
    rng = np.random.default_rng(6)
    lens, hq, hkv, d, block = [100, 64, 40], 16, 8, 128, 16
    q, qt, (kc, ks, vc, vs), table = decode_inputs(rng, lens, hq, hkv, d, block, "bf16")
    tab = table.copy()
    tab[0, 2], tab[1, 0] = -1, 10**6
    got = pkv.paged_decode_q8(qt, pool(kc), pool(vc), to_dev(ks), to_dev(vs), to_dev(tab),
                              to_dev(np.array(lens, np.int32)))
    assert pkv.paged_error_flags() == pkv.PKV_FLAG_BAD_BLOCK
    # the same sequences without those pages
    short = table.copy()
    short[0, 2:-1] = table[0, 3:]
    short[1, :3] = table[1, 1:4]
    less = [84, 48, 40]
    want, mass, reach = decode_want(q, kc, ks, vc, vs, short, less, 1 / math.sqrt(d), block)
    err = np.abs(widen(got) - want)
    assert np.all(err <= decode_bound(want, mass, reach, less, "bf16"))
    # lengths past the table and below 0
    n = table.shape[1] * block
    tab = np.where(table < 0, table[2, 0], table)  # (every entry a page that holds numbers)
    kc2, vc2 = kc & 0xBF, vc & 0xBF
    ks2, vs2 = np.nan_to_num(ks, nan=0.5), np.nan_to_num(vs, nan=0.5)
    got = pkv.paged_decode_q8(qt, pool(kc2), pool(vc2), to_dev(ks2), to_dev(vs2), to_dev(tab),
                              to_dev(np.array([n + 1000, -3, 40], np.int32)))
    assert pkv.paged_error_flags() == pkv.PKV_FLAG_BAD_LENGTH
    want, mass, reach = decode_want(q, kc2, ks2, vc2, vs2, tab, [n, 0, 40], 1 / math.sqrt(d), block)
    err = np.abs(widen(got) - want)
    assert np.all(err <= decode_bound(want, mass, reach, [n, 0, 40], "bf16"))


def test_decode_no_valid_page_at_all():
    i = dict(dtype=torch.int32, device="cuda")
    kc = pool(np.full((2, 2, 16, 64), 0x7F, np.uint8))
    s = torch.full((2, 2), float("nan"), device="cuda")
    q = torch.randn(2, 4, 64, device="cuda")
    out = pkv.paged_decode_q8(q, kc, kc, s, s, torch.full((2, 3), -1, **i),
                              torch.tensor([40, 0], **i))
    assert pkv.paged_error_flags() == pkv.PKV_FLAG_BAD_BLOCK and not out.any()


def test_decode_does_not_depend_on_where_pages_are():
    rng = np.random.default_rng(11)
    lens, hq, hkv, d, block = [700, 33, 2000], 16, 8, 128, 16
    q, qt, (kc, ks, vc, vs), table = decode_inputs(rng, lens, hq, hkv, d, block, "bf16")
    n = to_dev(np.array(lens, np.int32))
    a = pkv.paged_decode_q8(qt, pool(kc), pool(vc), to_dev(ks), to_dev(vs), to_dev(table), n)
    perm = rng.permutation(len(kc))
    inv = np.argsort(perm).astype(np.int32)
    moved = np.where(table < 0, -1, inv[np.maximum(table, 0)]).astype(np.int32)
    b = pkv.paged_decode_q8(qt, pool(kc[perm]), pool(vc[perm]), to_dev(ks[perm]), to_dev(vs[perm]),
                            to_dev(moved), n)
    assert torch.equal(a, b)


def test_decode_workspace_and_refusals():
    lib = pkv.load_library()
    rng = np.random.default_rng(12)
    lens = [50, 60]
    q, qt, (kc, ks, vc, vs), table = decode_inputs(rng, lens, 16, 8, 128, 16, "bf16")
    kp, vp, kst, vst, t, n = pool(kc), pool(vc), to_dev(ks), to_dev(vs), to_dev(table), \
        to_dev(np.array(lens, np.int32))
    need = pkv.paged_decode_q8_workspace_size(2, 16, torch.bfloat16, kp)
    assert need > 0
    out = torch.empty_like(qt)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    a = pkv.paged_decode_q8(qt, kp, vp, kst, vst, t, n, out=out, workspace=ws)
    assert a is out
    assert torch.equal(out, pkv.paged_decode_q8(qt, kp, vp, kst, vst, t, n))
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.paged_decode_q8(qt, kp, vp, kst, vst, t, n, workspace=ws[:need - 1])
    assert e.value.status == -3
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.paged_decode_q8(qt, kp, vp, kst, vst, t, n,
                            workspace=torch.empty(need + 256, dtype=torch.uint8, device="cuda")[16:])
    assert e.value.status == -3
    g = pkv.Geom(16, 8, 64, 7, 10, pkv.PKV_Q8)  # odd pages of 64-byte rows
    assert lib.paged_decode_q8_workspace_size(2, 1, ctypes.byref(g)) == 0
    p = ctypes.c_void_p(256)
    assert lib.paged_decode_q8(p, 1, p, p, p, p, p, 4, p, 2, 1.0, p, p, 1 << 40, ctypes.byref(g),
                               None) == -2
    for bad in (dict(batch=5000), dict(hq=1600, hkv=1), dict(blocks=1 << 27, hkv=32, hq=32, block=8),
                dict(width=1 << 28)):
        f = dict(hq=16, hkv=8, block=16, blocks=100, batch=2, width=4)
        f.update(bad)
        g = pkv.Geom(f["hq"], f["hkv"], 128, f["block"], f["blocks"], pkv.PKV_Q8)
        assert lib.paged_decode_q8(p, 1, p, p, p, p, p, f["width"], p, f["batch"], 1.0, p, p,
                                   1 << 40, ctypes.byref(g), None) == -2, bad
    for bad, error in ((dict(k_scale=kst[:1]), ValueError), (dict(v_scale=vst.double()), TypeError),
                       (dict(v_cache=vp[:1]), ValueError), (dict(q=qt[..., :64]), ValueError),
                       (dict(cache_seqlens=n[:1]), ValueError), (dict(block_table=t[:1]), ValueError),
                       (dict(out=out[:1]), ValueError), (dict(out=out.float()), TypeError),
                       (dict(k_cache=kp.view(torch.uint8)), ValueError),
                       (dict(block_table=t.long()), TypeError)):
        ok = dict(q=qt, k_cache=kp, v_cache=vp, k_scale=kst, v_scale=vst, block_table=t,
                  cache_seqlens=n)
        with pytest.raises(error):
            pkv.paged_decode_q8(**{**ok, **bad})


def test_decode_of_the_largest_batch():
    """4096 sequences, the shortest empty; the table keeps them from being taken whole."""
    rng = np.random.default_rng(13)
    lens = [int(n) for n in rng.integers(0, 40, 4096)]
    q, qt, (kc, ks, vc, vs), table = decode_inputs(rng, lens, 4, 2, 64, 8, "bf16")
    got = pkv.paged_decode_q8(qt, pool(kc), pool(vc), to_dev(ks), to_dev(vs), to_dev(table),
                              to_dev(np.array(lens, np.int32)))
    want, mass, reach = decode_want(q, kc, ks, vc, vs, table, lens, 0.125, 8)
    assert np.all(np.abs(widen(got) - want) <= decode_bound(want, mass, reach, lens, "bf16"))
    assert pkv.paged_error_flags() == 0


@pytest.mark.parametrize("seed", range(30))
def test_decode_of_random_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    d = int(rng.choice([64, 128]))
    hkv = int(rng.integers(1, 13))
    hq = hkv * int(rng.integers(1, 18))
    block = int(rng.integers(1, 70)) * (2 if d == 64 else 1)
    batch = int(rng.integers(1, 9))
    top = int(np.exp(rng.uniform(0, np.log(3000))))
    lens = [int(n) for n in rng.integers(0, top + 1, batch)]
    dtype = ["bf16", "f32"][int(rng.integers(2))]
    wide = int(rng.integers(0, 2)) * 200  # a table that reaches further than any sequence
    q, qt, (kc, ks, vc, vs), table = decode_inputs(rng, lens, hq, hkv, d, block, dtype)
    table = np.concatenate((table, np.full((batch, wide), -1, np.int32)), 1)
    scale = float(rng.uniform(0.02, 0.2))
    got = pkv.paged_decode_q8(qt, pool(kc), pool(vc), to_dev(ks), to_dev(vs), to_dev(table),
                              to_dev(np.array(lens, np.int32)), scale=scale)
    want, mass, reach = decode_want(q, kc, ks, vc, vs, table, lens, scale, block)
    err = np.abs(widen(got) - want)
    bound = decode_bound(want, mass, reach, lens, dtype)
    assert np.all(err <= bound), (err / bound).max()
    assert pkv.paged_error_flags() == 0


def test_pages_past_four_gigabytes():
    """Pages at the end of pools whose byte offsets pass 32 bits: write, read, decode and copy;
    the write with the rotation into bf16 pools as well."""
    rng = np.random.default_rng(14)
    hq, hkv, d, block, lens = 16, 8, 128, 16, [300, 41]
    page = hkv * block * d
    total = (5 << 30) // page
    if torch.cuda.mem_get_info()[0] < 6 * total * page:
        pytest.skip("needs 30 GB of device memory")
    used = sum(-(-n // block) for n in lens)
    ids = rng.permutation(used)
    near = np.full((2, 19), -1, np.int32)
    near[0], near[1, :3] = ids[:19], ids[19:]
    far = np.where(near < 0, -1, total - 1 - near).astype(np.int32)
    kc, vc = (torch.empty(pkv.q8_cache_shape(total, block, hkv, d), dtype=F8, device="cuda")
              for _ in range(2))
    ks, vs = (torch.empty(total, hkv, device="cuda") for _ in range(2))
    seq = np.concatenate([np.full(n, i) for i, n in enumerate(lens)]).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    (k, kt), (v, vt) = (rows(rng, len(seq), hkv, d, "bf16") for _ in range(2))
    q, qt = rows(rng, 2, hq, d, "bf16")
    cs = Q.cos_sin(300, d)
    pkv.paged_kv_write_q8(kt, vt, to_dev(far), to_dev(seq), to_dev(pos), kc, vc, ks, vs,
                          cos_sin=to_dev(cs))
    model = []
    kr = Q.rotate(k, cs, pos, False)
    for x in (kr, v):
        c, s = np.zeros((used, hkv, block, d), np.uint8), np.zeros((used, hkv), np.float32)
        Q.write(x, near, seq, pos, c, s, np.ones(len(seq), bool))
        model += [c, s]
    slots = (far[seq, pos // block] * block + pos % block).astype(np.int32)
    got = pkv.paged_kv_read_q8(kc, vc, ks, vs, to_dev(slots), torch.float32)
    for g, c, s in zip(got, model[::2], model[1::2]):
        assert np.array_equal(to_host(g), Q.values(c, s)[near[seq, pos // block], :, pos % block]
                              .astype(np.float32))
    out = pkv.paged_decode_q8(qt, kc, vc, ks, vs, to_dev(far), to_dev(np.array(lens, np.int32)))
    kcm, ksm, vcm, vsm = model
    want, mass, reach = decode_want(q, kcm, ksm, vcm, vsm, near, lens, d ** -0.5, block)
    assert np.all(np.abs(widen(out) - want) <= decode_bound(want, mass, reach, lens, "bf16"))
    src, dst = to_dev(far[0, :1]), torch.tensor([3], dtype=torch.int32, device="cuda")
    pkv.paged_copy_blocks(kc, vc, src, dst, ks, vs)
    for t in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs):
        assert torch.equal(t[int(far[0, 0])], t[3])
    del kc, vc, got, out
    kb, vb = (torch.empty(total, block, hkv, d, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    pkv.paged_kv_write_rope(kt, vt, to_dev(cs), to_dev(far), to_dev(seq), to_dev(pos), kb, vb)
    at = torch.from_numpy(slots.astype(np.int64)).cuda()
    for p, x in ((kb, kr), (vb, v)):
        assert np.array_equal(to_host(p.view(-1, hkv, d)[at]), Q4.bf16_bits(x))
    assert pkv.paged_error_flags() == 0


def test_copy_blocks_of_8_bit_pools_needs_their_scales():
    kc = torch.zeros(4, 2, 8, 64, device="cuda").to(F8)
    s = torch.zeros(4, 2, device="cuda")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    for ks, vs in ((None, None), (s, None), (s[:2], s), (s, s[:, :1])):
        with pytest.raises(ValueError):
            pkv.paged_copy_blocks(kc, kc.clone(), i, i + 1, ks, vs)
    with pytest.raises(TypeError):
        pkv.paged_copy_blocks(kc, kc.clone(), i, i + 1, s.double(), s)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_a_serving_loop(dtype=torch.bfloat16):
    """Prompts rotated and written into 8-bit pools and attended to through the packed prefill,
    a fork with its copy-on-write, then decode steps, each against 64 bits over what the pools
    hold."""
    rng = np.random.default_rng(21)
    hq, hkv, d, block, blocks = 8, 4, 128, 16, 40
    bm = pkv.BlockManager(blocks, block)
    cs = to_dev(Q.cos_sin(400, d))
    kc, vc = (torch.zeros(pkv.q8_cache_shape(blocks, block, hkv, d), device="cuda").to(F8)
              for _ in range(2))
    ks, vs = (torch.zeros(blocks, hkv, device="cuda") for _ in range(2))
    prompts = [37, 90, 16]
    seqs = [bm.allocate(list(rng.integers(0, 10**6, n)))[0] for n in prompts]
    i32 = dict(dtype=torch.int32, device="cuda")

    def tables(which):
        t = [bm.table(s) for s in which]
        w = max(map(len, t))
        return torch.tensor([r + [-1] * (w - len(r)) for r in t], **i32)

    def oracle(qv, which, lens):
        want, mass, reach = decode_want(qv, codes_of(kc), to_host(ks), codes_of(vc), to_host(vs),
                                        tables(which).cpu().numpy(), lens, 1 / math.sqrt(d), block)
        return want, decode_bound(want, mass, reach, lens, "bf16")

    # prompts
    n = sum(prompts)
    q, k, v = (torch.randn(n, h, d, device="cuda").to(dtype) for h in (hq, hkv, hkv))
    seq = torch.tensor([b for b, m in enumerate(prompts) for _ in range(m)], **i32)
    pos = torch.tensor([p for m in prompts for p in range(m)], **i32)
    tab = tables(seqs)
    qr = pkv.paged_kv_write_q8(k, v, tab, seq, pos, kc, vc, ks, vs, cos_sin=cs, q=q)
    slots = pkv.paged_build_slot_mapping(tab, seq, pos, block)
    kp, vp = pkv.paged_kv_read_q8(kc, vc, ks, vs, slots)
    cu = torch.tensor(np.cumsum([0] + prompts), **i32)
    out = pkv.paged_varlen_prefill(qr, kp, vp, cu, cu, max(prompts), max(prompts), None)
    last = [int(c) - 1 for c in cu[1:]]
    want, _ = oracle(widen(qr)[last], seqs, prompts)
    err = np.abs(widen(out)[last] - want)
    assert err.max() <= 2e-2 and err.mean() <= 2e-3
    # a fork of the first: its partial last block is copied, with its scales, before its next token
    seqs.append(bm.fork(seqs[0]))
    lens = prompts + [prompts[0]]
    graph = None
    for step in range(20):
        pairs = [bm.append(s, int(rng.integers(0, 10**6))) for s in seqs]
        pairs = [p for p in pairs if p[0] >= 0]
        assert bool(pairs) == (step == 0)
        if pairs:
            src, dst = (torch.tensor(x, **i32) for x in zip(*pairs))
            pkv.paged_copy_blocks(kc, vc, src, dst, ks, vs)
            for t in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs):
                assert torch.equal(t[src.long()], t[dst.long()])
        tab = tables(seqs)
        q, k, v = (torch.randn(4, h, d, device="cuda").to(dtype) for h in (hq, hkv, hkv))
        at = torch.tensor(lens, **i32)
        qr = pkv.paged_kv_write_q8(k, v, tab, torch.arange(4, **i32), at, kc, vc, ks, vs,
                                   cos_sin=cs, q=q)
        lens = [m + 1 for m in lens]
        out = pkv.paged_decode_q8(qr, kc, vc, ks, vs, tab, torch.tensor(lens, **i32))
        want, bound = oracle(widen(qr), seqs, lens)
        assert np.all(np.abs(widen(out) - want) <= bound), step
    assert pkv.paged_error_flags() == 0


def test_a_captured_step_with_its_own_workspace():
    """Write and decode of a step in one graph, replayed with new rows, positions and lengths, on
    another stream; two graphs of two batches share nothing but the pools."""
    rng = np.random.default_rng(22)
    hq, hkv, d, block, blocks = 16, 8, 128, 16, 64
    kc, vc = (torch.zeros(pkv.q8_cache_shape(blocks, block, hkv, d), device="cuda").to(F8)
              for _ in range(2))
    ks, vs = (torch.zeros(blocks, hkv, device="cuda") for _ in range(2))
    cs = to_dev(Q.cos_sin(400, d))
    i32 = dict(dtype=torch.int32, device="cuda")
    steps = []
    for b in range(2):
        tab = torch.from_numpy(rng.permutation(32).astype(np.int32).reshape(4, 8) + 32 * b).cuda()
        st = dict(tab=tab, seq=torch.tensor([0, 1, 2, 3, -1], **i32), pos=torch.zeros(5, **i32),
                  lens=torch.zeros(4, **i32))
        for name, h in (("q", hq), ("k", hkv), ("v", hkv)):
            st[name] = torch.zeros(5, h, d, device="cuda", dtype=torch.bfloat16)
        st["qr"] = torch.zeros_like(st["q"])
        st["out"] = torch.zeros(4, hq, d, device="cuda", dtype=torch.bfloat16)
        st["ws"] = torch.empty(pkv.paged_decode_q8_workspace_size(4, hq, torch.bfloat16, kc),
                               dtype=torch.uint8, device="cuda")
        steps.append(st)

    def run(st):
        pkv.paged_kv_write_q8(st["k"], st["v"], st["tab"], st["seq"], st["pos"], kc, vc, ks, vs,
                              cos_sin=cs, q=st["q"], q_out=st["qr"])
        pkv.paged_decode_q8(st["qr"][:4], kc, vc, ks, vs, st["tab"], st["lens"], out=st["out"],
                            workspace=st["ws"])

    streams = [torch.cuda.Stream() for _ in steps]
    graphs = []
    for st, s in zip(steps, streams):
        run(st)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run(st)
        graphs.append(g)
    for t in range(100):
        for st in steps:
            for name in ("q", "k", "v"):
                st[name].normal_()
            st["pos"].fill_(t)
            st["lens"].fill_(t + 1)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        if t % 33 == 0 or t == 99:
            for st in steps:
                q = widen(st["qr"][:4])
                lens = [t + 1] * 4
                want, mass, reach = decode_want(q, codes_of(kc), to_host(ks), codes_of(vc),
                                                to_host(vs), st["tab"].cpu().numpy(), lens,
                                                1 / math.sqrt(d), block)
                err = np.abs(widen(st["out"]) - want)
                assert np.all(err <= decode_bound(want, mass, reach, lens, "bf16"))
    assert pkv.paged_error_flags() == 0

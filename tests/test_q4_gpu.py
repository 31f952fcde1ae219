"""4-bit pools on the GPU: the quantising write, the read and the decode against
the numpy model of the format (q4_oracle), and all of them together as a
serving loop uses them."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_70_gb300 as pkv
import q4_oracle as Q
from gpu_helpers import assert_close, to_dev, to_host, widen

pytestmark = pytest.mark.gpu


def bf16(x):
    return Q.bf16_bits(np.asarray(x, np.float32))


def pages(rng, lens, block, extra=3, width=None):
    """A table over a shuffled pool, padding -1, and the pool's page count."""
    need = [-(-int(n) // block) for n in lens]
    total = sum(need) + extra
    ids = rng.permutation(total).astype(np.int32)
    table = np.full((len(need), max(width or 0, max(need + [1]))), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    return table, total


def slots_of(table, seq, pos, block):
    return table[seq, pos // block] * block + pos % block


def row_values(rng, shape):
    """Rows with the groups a quantiser can go wrong at, among normal ones."""
    x = rng.standard_normal(shape).astype(np.float32)
    f = x.reshape(-1, 32)
    n = len(f)
    special = [np.zeros(32), np.full(32, 3.25), np.full(32, -1e-41), np.r_[np.zeros(31), 1e30],
               np.linspace(-1, 1, 32), np.r_[np.full(31, 100.0), 100.5], np.arange(32) - 16.0,
               np.r_[np.full(16, -2.0 ** -120), np.full(16, 2.0 ** -120)],
               np.r_[-3e38, np.zeros(30), 3e38], rng.standard_normal(32) * 1e-20 + 1e-18]
    for i, s in enumerate(special):
        if n > 8 * i + 3:
            f[(8 * i + 3) % n] = np.asarray(s, np.float32)
    return x


def make_pool(rng, total, hkv, block, d, table, lens):
    """Pool bytes 0xff (NaN scales) except the rows the sequences hold."""
    pool = np.full((total, hkv, block, 5 * d // 8), 0xFF, np.uint8)
    for b, n in enumerate(lens):
        pos = np.arange(int(n))
        x = rng.standard_normal((len(pos), hkv, d)).astype(np.float32)
        x[:, :, 3::29] *= 4
        pool[table[b, pos // block], :, pos % block] = Q.quantise(x)
    return pool


# ---------------------------------------------------------------------------
# write and read
# ---------------------------------------------------------------------------
CASES = [  # tokens, Hkv, d, B, dtype, padding
    (1, 1, 64, 1, "f32", 0.0), (1, 8, 128, 16, "bf16", 0.0), (3, 1, 128, 5, "bf16", 0.0),
    (37, 2, 64, 16, "bf16", 0.3), (64, 8, 128, 16, "bf16", 0.0), (129, 3, 64, 7, "f32", 0.1),
    (200, 5, 128, 24, "f32", 0.1), (333, 16, 128, 256, "bf16", 0.05), (50, 33, 64, 8, "bf16", 0.0),
    (1025, 8, 64, 32, "f32", 0.05), (40, 48, 128, 3, "bf16", 0.0),
]


@pytest.mark.parametrize("n,hkv,d,block,dtype,pad", CASES)
def test_write_stores_the_formats_bytes_and_read_returns_their_values(n, hkv, d, block, dtype, pad):
    rng = np.random.default_rng(n * 7 + d)
    total = -(-n // block) + 2
    slots = rng.permutation(total * block)[:n].astype(np.int32)
    slots[rng.random(n) < pad] = -1
    x = [row_values(rng, (n, hkv, d)) for _ in range(2)]
    if dtype == "bf16":
        rows = [bf16(a) for a in x]
        x = [Q.bf16_value(a) for a in rows]
    else:
        rows = x
    before = [rng.integers(0, 256, (total, hkv, block, 5 * d // 8), dtype=np.uint8) for _ in x]
    kc, vc = to_dev(before[0]), to_dev(before[1])
    pkv.paged_kv_write_q4(to_dev(rows[0]), to_dev(rows[1]), to_dev(slots), kc, vc)
    live = slots >= 0
    for got, was, val in zip((kc, vc), before, x):
        want = was.copy()
        want[slots[live] // block, :, slots[live] % block] = Q.quantise(val[live])
        assert np.array_equal(to_host(got), want)
    # every row back, some twice, padding as zeros
    ask = np.concatenate([slots, slots[: n // 2], [-1]]).astype(np.int32)
    for out in (torch.float32, torch.bfloat16):
        k, v = pkv.paged_kv_read_q4(kc, vc, to_dev(ask), out)
        for got, pool in ((k, kc), (v, vc)):
            p = to_host(pool)
            want = Q.values(p[ask // block, :, ask % block]).astype(np.float32)
            want[ask < 0] = 0
            if out == torch.bfloat16:
                assert np.array_equal(np.isnan(want), np.isnan(widen(got)))
                ok = ~np.isnan(want)
                assert np.array_equal(to_host(got)[ok], Q.bf16_bits(want)[ok])
            else:
                assert np.array_equal(to_host(got), want, equal_nan=True)
    assert pkv.paged_error_flags() == 0


def test_a_group_with_a_nan_or_an_infinity_reads_as_nan_and_no_other():
    x = np.ones((4, 2, 128), np.float32) * np.linspace(-1, 1, 128, dtype=np.float32)
    x[0, 0, 5] = np.nan
    x[1, 1, 40] = np.inf
    x[2, 0, 127] = -np.inf
    kc = torch.zeros(pkv.q4_cache_shape(1, 4, 2, 128), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    pkv.paged_kv_write_q4(to_dev(x), to_dev(x), slots, kc, vc)
    k, _ = pkv.paged_kv_read_q4(kc, vc, slots, torch.float32)
    nan = np.isnan(to_host(k)).reshape(4, 2, 4, 32)
    want = np.zeros((4, 2, 4, 32), bool)
    want[0, 0, 0] = want[1, 1, 1] = want[2, 0, 3] = True
    assert np.array_equal(nan, want)
    assert np.array_equal(to_host(kc)[0].transpose(1, 0, 2), Q.quantise(x))


def test_slots_past_the_pool_are_flagged_and_skipped():
    kc = torch.full(pkv.q4_cache_shape(2, 4, 2, 64), 7, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    x = torch.randn(3, 2, 64, device="cuda")
    slots = torch.tensor([8, 2, 2**31 - 1], dtype=torch.int32, device="cuda")
    pkv.paged_kv_write_q4(x, x, slots, kc, vc)
    assert pkv.paged_error_flags() == pkv.PKV_FLAG_BAD_SLOT
    want = np.full((2, 2, 4, 40), 7, np.uint8)
    want[0, :, 2] = Q.quantise(to_host(x)[1])
    assert np.array_equal(to_host(kc), want) and np.array_equal(to_host(vc), want)
    k, v = pkv.paged_kv_read_q4(kc, vc, slots, torch.float32)
    assert pkv.paged_error_flags() == pkv.PKV_FLAG_BAD_SLOT
    assert not k[0].any() and not k[2].any() and not v[0].any() and k[1].any()


def test_no_tokens():
    kc = torch.full(pkv.q4_cache_shape(2, 4, 2, 64), 7, dtype=torch.uint8, device="cuda")
    e = torch.empty(0, 2, 64, device="cuda")
    s = torch.empty(0, dtype=torch.int32, device="cuda")
    pkv.paged_kv_write_q4(e, e, s, kc, kc.clone())
    k, v = pkv.paged_kv_read_q4(kc, kc, s)
    assert k.shape == (0, 2, 64) and v.dtype == torch.bfloat16
    assert bool((kc == 7).all())


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
DECODE = [  # lens, Hq, Hkv, d, B, dtype
    ([30, 32, 70], 2, 1, 64, 32, "f32"),
    ([1], 1, 1, 128, 16, "bf16"),
    ([0], 4, 2, 64, 8, "bf16"),
    ([0, 1, 17, 0, 300, 16, 15], 16, 8, 128, 16, "bf16"),
    ([5, 1000, 64, 63, 65], 8, 8, 128, 1, "bf16"),
    ([77, 500], 16, 8, 64, 2, "bf16"),
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
]


def decode_case(lens, hq, hkv, d, block, dtype, seed):
    rng = np.random.default_rng(seed)
    table, total = pages(rng, lens, block)
    kc = make_pool(rng, total, hkv, block, d, table, lens)
    vc = make_pool(rng, total, hkv, block, d, table, lens)
    q = rng.standard_normal((len(lens), hq, d)).astype(np.float32)
    return (bf16(q) if dtype == "bf16" else q), kc, vc, table


def check(got, want, tol, what=""):
    err = np.abs(widen(got) - want)
    assert np.all(err <= tol), f"{what}: {np.max(err / np.maximum(tol, 1e-300)):.3g} of the bound"


@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode(i):
    lens, hq, hkv, d, block, dtype = DECODE[i]
    q, kc, vc, table = decode_case(lens, hq, hkv, d, block, dtype, 100 + i)
    scale = 1 / math.sqrt(d)
    out = pkv.paged_decode_q4(to_dev(q), to_dev(kc), to_dev(vc), to_dev(table),
                              to_dev(np.asarray(lens, np.int32)))
    want, tol = Q.decode(q, kc, vc, table, lens, scale)
    check(out, want, tol, str(DECODE[i]))
    assert not widen(out)[np.asarray(lens) == 0].any()
    assert pkv.paged_error_flags() == 0


@pytest.mark.parametrize("scale", [0.0, 0.5, -0.3, 3.0])
def test_decode_scales(scale):
    """Peaked and flat weights: a growing maximum, every key alike."""
    lens = [700, 45]
    q, kc, vc, table = decode_case(lens, 8, 4, 128, 16, "bf16", 7)
    out = pkv.paged_decode_q4(to_dev(q), to_dev(kc), to_dev(vc), to_dev(table),
                              to_dev(np.asarray(lens, np.int32)), scale=scale)
    want, tol = Q.decode(q, kc, vc, table, lens, scale)
    check(out, want, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 100, 299])
def test_decode_with_a_large_value_that_no_query_looks_at(dtype, at):
    """A V row 4096 times the others' with a weight near zero: the others keep the
    precision that the tolerance gives them (fp16 holds weights times scales above 2^-14
    of the largest scale in full, and the smaller ones to 2^-25 of it)."""
    rng = np.random.default_rng(at + 1)
    n, d, block = 300, 128, 16
    table, total = pages(rng, [n], block)
    q = bf16(rng.standard_normal((1, 2, d)))
    q[0, 1] = q[0, 0]
    qv = Q.bf16_value(q)[0, 0].astype(np.float32)
    x = [rng.standard_normal((n, 1, d)).astype(np.float32) for _ in range(2)]
    x[0][at, 0] = -5 * qv
    x[1][at, 0] *= 4096
    kc, vc = (np.full((total, 1, block, 80), 0xFF, np.uint8) for _ in range(2))
    pos = np.arange(n)
    for pool, rows in ((kc, x[0]), (vc, x[1])):
        pool[table[0, pos // block], :, pos % block] = Q.quantise(rows)
    if dtype == "f32":
        q = Q.bf16_value(q).astype(np.float32)
    out = pkv.paged_decode_q4(to_dev(q), to_dev(kc), to_dev(vc), to_dev(table),
                              to_dev(np.asarray([n], np.int32)))
    want, tol = Q.decode(q, kc, vc, table, [n], d ** -0.5)
    assert np.abs(want).max() < 1  # (the large row is not in it)
    check(out, want, tol)


def test_decode_bad_lengths_and_pages():
    lens = [100, 40, 64]
    block = 16
    q, kc, vc, table = decode_case(lens, 16, 8, 128, block, "bf16", 8)
    table = table[:, :7].copy()  # 112 keys at most
    t = table.copy()
    t[0, 2], t[2, 3] = 10**6, -5  # keys 32..47 of sequence 0, 48..63 of sequence 2
    out = pkv.paged_decode_q4(to_dev(q), to_dev(kc), to_dev(vc), to_dev(t),
                              to_dev(np.asarray(lens, np.int32)))
    assert pkv.paged_error_flags() == pkv.PKV_FLAG_BAD_BLOCK
    want, tol = Q.decode(q, kc, vc, table, lens, 128 ** -0.5,
                         [range(32, 48), [], range(48, 64)])
    check(out, want, tol)
    full = kc.copy()
    full[:] = kc[table[0, 0], :, :1]  # every page holds a row
    for bad, use in (([-3, 40, 64], [0, 40, 64]), ([113, 40, 2**31 - 1], [112, 40, 112])):
        tt = np.where(table < 0, 0, table)
        out = pkv.paged_decode_q4(to_dev(q), to_dev(full), to_dev(full), to_dev(tt),
                                  to_dev(np.asarray(bad, np.int32)))
        assert pkv.paged_error_flags() == pkv.PKV_FLAG_BAD_LENGTH
        want, tol = Q.decode(q, full, full, tt, use, 128 ** -0.5)
        check(out, want, tol)


def test_decode_keeps_a_nan_of_its_own_sequence_only():
    lens = [50, 50, 50]
    q, kc, vc, table = decode_case(lens, 4, 2, 64, 16, "bf16", 9)
    kc[table[1, 1], 0, 3, 32:34] = [0xFF, 0x7F]  # a NaN scale: key 19, head 0, of sequence 1
    out = widen(pkv.paged_decode_q4(to_dev(q), to_dev(kc), to_dev(vc), to_dev(table),
                                    to_dev(np.asarray(lens, np.int32))))
    assert np.isnan(out[1, :2]).all()
    assert np.isfinite(out[0]).all() and np.isfinite(out[2]).all() and np.isfinite(out[1, 2:]).all()
    q2 = q.copy()
    q2[0, 3] = 0x7FC0  # a NaN query
    out = widen(pkv.paged_decode_q4(to_dev(q2), to_dev(vc), to_dev(vc), to_dev(table),
                                    to_dev(np.asarray(lens, np.int32))))
    assert np.isnan(out[0, 3]).all() and np.isfinite(out[0, :3]).all()


def test_decode_does_not_depend_on_the_pages():
    """The same rows in other pages give the same bits."""
    lens = [900, 130, 17]
    rng = np.random.default_rng(4)
    q, kc, vc, table = decode_case(lens, 16, 8, 128, 16, "bf16", 10)
    args = to_dev(q), to_dev(np.asarray(lens, np.int32))
    a = pkv.paged_decode_q4(args[0], to_dev(kc), to_dev(vc), to_dev(table), args[1])
    perm = rng.permutation(len(kc)).astype(np.int32)
    k2, v2 = np.empty_like(kc), np.empty_like(vc)
    k2[perm], v2[perm] = kc, vc
    t2 = np.where(table < 0, -1, perm[table])
    b = pkv.paged_decode_q4(args[0], to_dev(k2), to_dev(v2), to_dev(t2), args[1])
    c = pkv.paged_decode_q4(args[0], to_dev(kc), to_dev(vc), to_dev(table), args[1])
    assert torch.equal(a, b) and torch.equal(a, c)


def test_decode_in_two_graphs_that_share_a_workspace_and_on_other_streams():
    cases = []
    ws = None
    for seed, lens in ((20, [300, 41, 9000]), (21, [64, 700, 5])):
        q, kc, vc, table = decode_case(lens, 16, 8, 128, 16, "bf16", seed)
        dev = [to_dev(x) for x in (q, kc, vc, table, np.asarray(lens, np.int32))]
        out = torch.empty_like(dev[0])
        want, tol = Q.decode(q, kc, vc, table, lens, 128 ** -0.5)
        cases.append((dev, out, want, tol))
        need = pkv.paged_decode_q4_workspace_size(3, 16, torch.bfloat16, dev[1])
        if ws is None:
            ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graphs = []
    for dev, out, _, _ in cases:
        pkv.paged_decode_q4(*dev, out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_decode_q4(*dev, out=out, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for dev, out, _, _ in cases:
            out.zero_()
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for _, out, want, tol in cases:
        check(out, want, tol)
    # eager calls at once on two streams, each with a workspace of its own
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for s, (dev, _, _, _) in zip(streams, cases):
            with torch.cuda.stream(s):
                outs.append(pkv.paged_decode_q4(*dev))
    torch.cuda.synchronize()
    for out, (_, _, want, tol) in zip(outs, cases):
        check(out, want, tol)


def test_the_largest_batch_and_one_more():
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 20, 4096).tolist()
    lens[77] = 3000
    q, kc, vc, table = decode_case(lens, 2, 1, 64, 16, "bf16", 8)
    dev = [to_dev(x) for x in (q, kc, vc, table, np.asarray(lens, np.int32))]
    want, tol = Q.decode(q, kc, vc, table, lens, 0.125)
    check(pkv.paged_decode_q4(*dev), want, tol)
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.paged_decode_q4(torch.cat([dev[0], dev[0][:1]]), dev[1], dev[2],
                            torch.cat([dev[3], dev[3][:1]]), torch.cat([dev[4], dev[4][:1]]))
    assert e.value.status == -2
    # more keys in all than the split can number: refused, whatever the lengths are
    wide = torch.zeros(4096, 5000, dtype=torch.int32, device="cuda")
    pool = torch.zeros(pkv.q4_cache_shape(2, 400000, 1, 64), dtype=torch.uint8, device="cuda")
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.paged_decode_q4(dev[0], pool, pool, wide, dev[4])
    assert e.value.status == -2
    assert pkv.paged_error_flags() == 0


def test_a_step_in_one_graph_replayed_as_the_lengths_move_on():
    """Slots, write, decode and lengths + 1, captured once and replayed; then the same
    rows evicted by a captured compaction."""
    rng = np.random.default_rng(6)
    hq, hkv, d, block, first, steps = 8, 4, 64, 16, [14, 0, 200], 5
    table, total = pages(rng, [n + steps for n in first], block, width=14)
    kc = make_pool(rng, total, hkv, block, d, table, first)
    vc = make_pool(rng, total, hkv, block, d, table, first)
    kd, vd, td = to_dev(kc), to_dev(vc), to_dev(table)
    lens = to_dev(np.asarray(first, np.int32))
    seq = to_dev(np.arange(3, dtype=np.int32))
    q, k, v = (torch.zeros(3, h, d, device="cuda", dtype=torch.bfloat16) for h in (hq, hkv, hkv))
    out = torch.empty_like(q)
    slots = torch.empty(3, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkv.paged_decode_q4_workspace_size(3, hq, torch.bfloat16, kd),
                     dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_build_slot_mapping(td, seq, lens, block, slots)
        pkv.paged_kv_write_q4(k, v, slots, kd, vd)
        lens += 1
        pkv.paged_decode_q4(q, kd, vd, td, lens, out=out, workspace=ws)
    assert lens.tolist() == first
    at = np.asarray(first)
    for step in range(steps):
        x = [bf16(rng.standard_normal((3, h, d))) for h in (hq, hkv, hkv)]
        for dst, src in zip((q, k, v), x):
            dst.copy_(to_dev(src))
        g.replay()
        for pool, rows in ((kc, x[1]), (vc, x[2])):
            pool[table[np.arange(3), at // block], :, at % block] = Q.quantise(Q.bf16_value(rows))
        at = at + 1
        assert np.array_equal(to_host(kd), kc) and np.array_equal(to_host(vd), vc)
        want, tol = Q.decode(x[0], kc, vc, table, at, d ** -0.5)
        check(out, want, tol, f"replay {step}")
    assert lens.tolist() == at.tolist() and pkv.paged_error_flags() == 0


def test_decode_workspace_and_shape_refusals():
    lens = [300, 41]
    q, kc, vc, table = decode_case(lens, 16, 8, 128, 16, "bf16", 30)
    dev = [to_dev(x) for x in (q, kc, vc, table, np.asarray(lens, np.int32))]
    need = pkv.paged_decode_q4_workspace_size(2, 16, torch.bfloat16, dev[1])
    if need:
        small = torch.empty(need - 1, dtype=torch.uint8, device="cuda")
        with pytest.raises(pkv.PagedKVError) as e:
            pkv.paged_decode_q4(*dev, workspace=small)
        assert e.value.status == -3
    with pytest.raises(ValueError):
        pkv.paged_decode_q4(dev[0][:, :, :64].contiguous(), *dev[1:])
    with pytest.raises(ValueError):
        pkv.paged_decode_q4(dev[0], dev[1], dev[2][:-1], *dev[3:])
    with pytest.raises(ValueError):
        pkv.paged_decode_q4(dev[0], dev[1], dev[2], dev[3][:1], dev[4])
    with pytest.raises(ValueError):
        pkv.paged_decode_q4(dev[0], dev[1].transpose(1, 2), *dev[2:])
    with pytest.raises(TypeError):
        pkv.paged_decode_q4(dev[0].half(), *dev[1:])
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_decode_q4(dev[0][:, :12].contiguous(), *dev[1:])  # 12 % 8
    for hq, hkv, d, block in ((65, 1, 128, 16), (130, 2, 64, 16), (4, 2, 64, 7)):
        q = torch.zeros(2, hq, d, device="cuda", dtype=torch.bfloat16)
        kc = torch.zeros(pkv.q4_cache_shape(4, block, hkv, d), dtype=torch.uint8, device="cuda")
        t = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
        with pytest.raises(pkv.PagedKVError) as e:
            pkv.paged_decode_q4(q, kc, kc, t, dev[4])
        assert e.value.status == -2


def test_pages_past_four_gigabytes():
    """Pages at the end of a pool whose byte offsets pass 32 bits: write, read,
    decode and copy."""
    hq, hkv, d, block, lens = 16, 8, 128, 16, [300, 41]
    page = hkv * block * 80
    total = (5 << 30) // page
    if torch.cuda.mem_get_info()[0] < 4 * total * page:
        pytest.skip("needs 20 GB of device memory")
    rng = np.random.default_rng(5)
    table, used = pages(rng, lens, block, extra=0)
    far = np.where(table < 0, -1, total - 1 - table).astype(np.int32)  # the last pages
    kd, vd = (torch.empty(pkv.q4_cache_shape(total, block, hkv, d), dtype=torch.uint8,
                          device="cuda") for _ in range(2))
    seq = np.concatenate([np.full(n, i) for i, n in enumerate(lens)]).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    slots = slots_of(far, seq, pos, block).astype(np.int32)
    x = [rng.standard_normal((len(seq), hkv, d)).astype(np.float32) for _ in range(2)]
    pkv.paged_kv_write_q4(to_dev(x[0]), to_dev(x[1]), to_dev(slots), kd, vd)
    k, v = pkv.paged_kv_read_q4(kd, vd, to_dev(slots), torch.float32)
    rows = [Q.quantise(a) for a in x]
    assert np.array_equal(to_host(k), Q.values(rows[0]).astype(np.float32))
    assert np.array_equal(to_host(v), Q.values(rows[1]).astype(np.float32))
    near = [np.zeros((used, hkv, block, 80), np.uint8) for _ in x]
    for pool, r in zip(near, rows):
        pool[table[seq, pos // block], :, pos % block] = r
    q = rng.standard_normal((2, hq, d)).astype(np.float32)
    out = pkv.paged_decode_q4(to_dev(q), kd, vd, to_dev(far), to_dev(np.asarray(lens, np.int32)))
    want, tol = Q.decode(q, near[0], near[1], table, lens, d ** -0.5)
    check(out, want, tol)
    src, dst = int(far[0, 0]), 3
    pkv.paged_copy_blocks(kd, vd, to_dev(np.asarray([src], np.int32)),
                          to_dev(np.asarray([dst], np.int32)))
    assert torch.equal(kd[src], kd[dst]) and torch.equal(vd[src], vd[dst])
    # the last page's tokens kept every other one, in place
    keep = np.arange(0, lens[0], 2, dtype=np.int32)[1:]
    keep = np.concatenate([[0], keep]).astype(np.int32)
    pkv.paged_kv_compact(kd, vd, to_dev(far[:1]), to_dev(keep),
                         to_dev(np.asarray([0, len(keep)], np.int32)))
    k, _ = pkv.paged_kv_read_q4(kd, vd, to_dev(slots[:len(keep)]), torch.float32)
    assert np.array_equal(to_host(k), Q.values(rows[0][keep]).astype(np.float32))
    assert pkv.paged_error_flags() == 0


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_prompts_then_tokens_then_eviction_over_a_4_bit_cache():
    """A serving loop: prompts written in 4 bits and attended to as packed
    values, tokens appended and decoded, a forked page copied, tokens evicted,
    decoded again; every attention against 64 bits over the stored rows."""
    rng = np.random.default_rng(77)
    hq, hkv, d, block = 16, 8, 128, 16
    scale = d ** -0.5
    prompts = [70, 33, 5]
    width = 8
    table, total = pages(rng, [width * block] * 3, block, extra=2)
    spare = np.setdiff1d(np.arange(total), table)[0]
    kc = np.full((total, hkv, block, 80), 0xFF, np.uint8)
    kd, vd, td = to_dev(kc), to_dev(kc), to_dev(table)
    seq = np.concatenate([np.full(n, i) for i, n in enumerate(prompts)]).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in prompts]).astype(np.int32)
    new = [bf16(rng.standard_normal((len(seq), hkv, d))) for _ in range(2)]
    q = bf16(rng.standard_normal((len(seq), hq, d)))
    slots = pkv.paged_build_slot_mapping(td, to_dev(seq), to_dev(pos), block)
    pkv.paged_kv_write_q4(to_dev(new[0]), to_dev(new[1]), slots, kd, vd)
    k, v = pkv.paged_kv_read_q4(kd, vd, slots)
    cu = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    out = pkv.paged_varlen_prefill(to_dev(q), k, v, to_dev(cu), to_dev(cu), max(prompts),
                                   max(prompts), None, scale=scale)
    want = oracle.prefill(q, to_host(k), to_host(v), cu, cu, scale, causal=True)
    assert_close(widen(out), want, "bf16", "prompts")
    lens = np.asarray(prompts, np.int32)
    for step in range(3):
        tok = [bf16(rng.standard_normal((3, hkv, d))) for _ in range(2)]
        qd = bf16(rng.standard_normal((3, hq, d)))
        s = pkv.paged_build_slot_mapping(td, to_dev(np.arange(3, dtype=np.int32)), to_dev(lens),
                                         block)
        pkv.paged_kv_write_q4(to_dev(tok[0]), to_dev(tok[1]), s, kd, vd)
        lens = lens + 1
        out = pkv.paged_decode_q4(to_dev(qd), kd, vd, td, to_dev(lens), scale)
        want, tol = Q.decode(qd, to_host(kd), to_host(vd), table, lens, scale)
        check(out, want, tol, f"step {step}")
    # sequence 1's second page moves to a spare one (a copy-on-write)
    old = table[1, 1]
    pkv.paged_copy_blocks(kd, vd, to_dev(np.asarray([old], np.int32)),
                          to_dev(np.asarray([spare], np.int32)))
    assert torch.equal(kd[int(old)], kd[int(spare)]) and torch.equal(vd[int(old)], vd[int(spare)])
    table[1, 1] = spare
    td = to_dev(table)
    # a third of the tokens behind the first four goes
    start = np.full(3, 4, np.int32)
    lists = [np.sort(rng.permutation(np.arange(4, n))[: (n - 4) * 2 // 3]) for n in lens]
    keep = np.concatenate(lists).astype(np.int32)
    cu_keep = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
    ks, vs = to_host(kd).copy(), to_host(vd).copy()
    ld = to_dev(lens)
    pkv.paged_kv_compact(kd, vd, td, to_dev(keep), to_dev(cu_keep), to_dev(start), ld)
    assert np.array_equal(to_host(kd), Q.compact(ks, table, keep, cu_keep, start, True))
    assert np.array_equal(to_host(vd), Q.compact(vs, table, keep, cu_keep, start, True))
    after = np.asarray([4 + len(x) for x in lists], np.int32)
    assert np.array_equal(to_host(ld), after)
    out = pkv.paged_decode_q4(to_dev(qd), kd, vd, td, ld, scale)
    want, tol = Q.decode(qd, to_host(kd), to_host(vd), table, after, scale)
    check(out, want, tol, "after eviction")
    assert pkv.paged_error_flags() == 0

"""paged_kv_compact: kept tokens moved together in place, against a copy made
with numpy, for every pool type and for lists, pages and rows of many sizes."""
import numpy as np
import pytest
import torch

import paged_kv_cache_70_gb300 as pkv
import q4_oracle as Q
from gpu_helpers import to_dev, to_host

pytestmark = pytest.mark.gpu


def make(rng, dtype, total, block, hkv, d):
    if dtype == "q4":
        return rng.integers(0, 256, (total, hkv, block, 5 * d // 8), dtype=np.uint8)
    x = rng.integers(0, 1 << 16, (total, block, hkv, d)).astype(np.uint16)  # any bits
    return x if dtype == "bf16" else rng.standard_normal((total, block, hkv, d)).astype(np.float32)


def tables(rng, lens, block, extra=2):
    need = [-(-n // block) for n in lens]
    total = sum(need) + extra
    ids = rng.permutation(total).astype(np.int32)
    t = np.full((len(lens), max(need + [1])), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = ids[at:at + n]
        at += n
    return t, total


def lists_of(rng, lens, starts, share):
    out = []
    for n, s in zip(lens, starts):
        rest = np.arange(s, n)
        out.append(np.sort(rng.permutation(rest)[: int(round(len(rest) * share))]))
    cu = np.concatenate([[0], np.cumsum([len(x) for x in out])]).astype(np.int32)
    return np.concatenate(out + [np.zeros(0, int)]).astype(np.int32), cu


def run(dtype, lens, starts, keep, cu, block, hkv, d, seed, use_start=True):
    rng = np.random.default_rng(seed)
    t, total = tables(rng, lens, block)
    k, v = (make(rng, dtype, total, block, hkv, d) for _ in range(2))
    kd, vd = to_dev(k), to_dev(v)
    new = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    st = np.asarray(starts, np.int32) if use_start else None
    pkv.paged_kv_compact(kd, vd, to_dev(t), to_dev(keep), to_dev(cu),
                         to_dev(st) if use_start else None, new)
    for got, was in ((kd, k), (vd, v)):
        assert np.array_equal(to_host(got).view(np.uint8),
                              Q.compact(was, t, keep, cu, st, dtype == "q4").view(np.uint8))
    assert np.array_equal(to_host(new), np.asarray(starts) + np.diff(cu))
    assert pkv.paged_error_flags() == 0


CASES = [  # dtype, lens, tail (0: from the start), share, B, Hkv, d
    ("bf16", [1], 0, 1.0, 16, 8, 128),
    ("bf16", [2, 1, 0, 5], 0, 0.5, 1, 1, 64),
    ("bf16", [300, 17, 1000], 0, 0.5, 16, 8, 128),
    ("bf16", [300, 17, 1000], 0, 0.02, 16, 8, 128),
    ("bf16", [300, 17, 1000], 0, 0.99, 16, 8, 128),
    ("bf16", [300, 17, 1000], 0, 0.0, 16, 8, 128),
    ("bf16", [300, 17, 1000], 0, 1.0, 16, 8, 128),
    ("f32", [257, 64], 0, 0.6, 24, 3, 64),
    ("f32", [40, 70], 16, 0.4, 7, 1, 128),
    ("bf16", [200, 513], 16, 0.3, 256, 2, 64),
    ("bf16", [90, 33], 0, 0.5, 8, 5, 3),     # rows of 30 bytes
    ("f32", [90, 33], 0, 0.5, 8, 1, 1),      # rows of 4 bytes
    ("bf16", [90, 33], 0, 0.5, 8, 3, 2),     # rows of 12 bytes
    ("bf16", [90, 33], 0, 0.5, 8, 1, 20),    # rows of 40 bytes
    ("q4", [300, 17, 1000], 0, 0.5, 16, 8, 128),
    ("q4", [300, 17, 1000], 0, 0.9, 8, 3, 64),
    ("q4", [64, 65, 1], 16, 0.3, 16, 1, 128),
    ("q4", [700], 64, 0.5, 5, 1, 64),
    ("bf16", [9000, 20, 4000], 0, 0.5, 256, 8, 128),
    ("q4", [9000, 20, 4000], 0, 0.7, 256, 4, 64),
    ("bf16", [7] * 300, 4, 0.5, 16, 2, 64),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_compact(i):
    dtype, lens, tail, share, block, hkv, d = CASES[i]
    starts = [max(0, n - tail) if tail else 0 for n in lens]
    keep, cu = lists_of(np.random.default_rng(50 + i), lens, starts, share)
    run(dtype, lens, starts, keep, cu, block, hkv, d, i, use_start=bool(tail))


@pytest.mark.parametrize("dtype", ["bf16", "q4"])
@pytest.mark.parametrize("gap", [1, 2, 63, 256, 4000])
def test_every_token_moves_a_fixed_way(dtype, gap):
    """The first `gap` tokens go: each destination is a later token's source,
    next to it, within a round, or rounds away."""
    n = 5000
    keep = np.arange(gap, n, dtype=np.int32)
    run(dtype, [n], [0], keep, np.asarray([0, n - gap], np.int32), 16, 4, 64, gap, use_start=False)


@pytest.mark.parametrize("dtype,hkv,d", [("bf16", 8, 128), ("q4", 8, 128), ("f32", 1, 128)])
@pytest.mark.parametrize("lens", [[3000], [700, 2500], [1500, 20, 900, 2100], [900, 600] * 4,
                                  [200] * 11, [100, 300] * 12, [70] * 150])
def test_any_number_of_sequences(dtype, hkv, d, lens):
    """From one sequence, cut into narrow slices, to so many that each has wide ones."""
    rng = np.random.default_rng(len(lens))
    keep, cu = lists_of(rng, lens, [0] * len(lens), 0.6)
    run(dtype, lens, [0] * len(lens), keep, cu, 16, hkv, d, 3, use_start=False)


def test_lists_need_not_ascend():
    """Any order whose i-th entry is at least start + i (here also one entry twice)."""
    keep = np.asarray([9, 3, 5, 12, 12, 8, 11, 7], np.int32)
    run("bf16", [16], [0], keep, np.asarray([0, 8], np.int32), 4, 2, 64, 1, use_start=False)


@pytest.mark.parametrize("dtype,block,hkv,d", [("bf16", 16, 8, 128), ("q4", 16, 2, 64), ("f32", 4, 40, 128)])
def test_the_starts_own_array_takes_the_new_lengths(dtype, block, hkv, d):
    """Lengths before a draft, moved on in place by its accepted tokens (every CTA of
    a sequence has to read the start before it changes)."""
    rng = np.random.default_rng(hkv)
    lens = [int(n) for n in rng.integers(0, 90, 300)] + [3000]
    starts = np.asarray([rng.integers(0, n + 1) for n in lens], np.int32)
    t, total = tables(rng, lens, block)
    k, v = (make(rng, dtype, total, block, hkv, d) for _ in range(2))
    keep, cu = lists_of(rng, lens, starts, 0.4)
    at = to_dev(starts)
    kd, vd = to_dev(k), to_dev(v)
    pkv.paged_kv_compact(kd, vd, to_dev(t), to_dev(keep), to_dev(cu), at, at)
    for got, was in ((kd, k), (vd, v)):
        assert np.array_equal(to_host(got).view(np.uint8),
                              Q.compact(was, t, keep, cu, starts, dtype == "q4").view(np.uint8))
    assert np.array_equal(to_host(at), starts + np.diff(cu))
    # starts out of range are flagged and brought into the table
    far = to_dev(np.asarray([-5, block * t.shape[1] + 9] + [0] * (len(lens) - 2), np.int32))
    pkv.paged_kv_compact(kd, vd, to_dev(t), to_dev(keep[:0]), to_dev(np.zeros_like(cu)), far, far)
    assert to_host(far).tolist() == [0, block * t.shape[1]] + [0] * (len(lens) - 2)
    assert pkv.paged_error_flags() == pkv.PKV_FLAG_BAD_LENGTH


def test_the_most_sequences():
    """65,535 of them, two tokens each, the second kept."""
    n = 65535
    k = torch.arange(2 * n, device="cuda", dtype=torch.float32).reshape(n, 2, 1, 1)
    kd, vd = k.clone(), -k
    i32 = dict(dtype=torch.int32, device="cuda")
    new = torch.full((n,), -1, **i32)
    pkv.paged_kv_compact(kd, vd, torch.arange(n, **i32)[:, None], torch.ones(n, **i32),
                         torch.arange(n + 1, **i32), None, new)
    want = k.clone()
    want[:, 0] = k[:, 1]
    assert torch.equal(kd, want) and torch.equal(vd, -want)
    assert bool((new == 1).all()) and pkv.paged_error_flags() == 0


@pytest.mark.parametrize("dtype", ["bf16", "q4"])
def test_with_the_block_managers_bookkeeping(dtype):
    """Forked sequences: the copies and the table that BlockManager.compact names, then
    the move; each sequence reads back its own rows."""
    rng = np.random.default_rng(9)
    block, hkv, d, total = 16, 2, 64, 40
    k, v = (make(rng, dtype, total, block, hkv, d) for _ in range(2))
    kd, vd = to_dev(k), to_dev(v)
    bm = pkv.BlockManager(total, block)
    a, _ = bm.allocate(range(100))
    b = bm.fork(a)
    c, _ = bm.allocate(range(1000, 1070))

    def rows(seq, x):
        t, n = np.asarray(bm.table(seq)), bm.seq_len(seq)
        pos = np.arange(n)
        x = to_host(x)
        return x[t[pos // block], :, pos % block] if dtype == "q4" else x[t[pos // block], pos % block]

    want = {s: [rows(s, x) for x in (kd, vd)] for s in (a, b, c)}
    for seq, start, keep in ((b, 20, [30, 31, 50, 77, 99]), (c, 0, list(range(3, 70, 2))),
                             (a, 90, [95]), (b, 25, [])):
        src, dst, table = bm.compact(seq, keep, start)
        if src:
            pkv.paged_copy_blocks(kd, vd, *(to_dev(np.asarray(x, np.int32)) for x in (src, dst)))
        one = lambda *x: to_dev(np.asarray(x, np.int32))  # noqa: E731
        at = one(start)
        pkv.paged_kv_compact(kd, vd, one(*table)[None], one(*keep), one(0, len(keep)), at, at)
        want[seq] = [np.concatenate([x[:start], x[keep]]) if keep else x[:start] for x in want[seq]]
        assert at.tolist() == [bm.seq_len(seq)]
        for s, w in want.items():
            for x, y in zip((kd, vd), w):
                assert np.array_equal(rows(s, x), y)
    assert pkv.paged_error_flags() == 0


def test_bad_entries_are_flagged_and_left_out():
    rng = np.random.default_rng(0)
    t, total = tables(rng, [32, 32, 32], 8)
    k, v = (make(rng, "bf16", total, 8, 2, 64) for _ in range(2))

    def call(tab, keep, cu, start, flag, moved):
        kd, vd = to_dev(k), to_dev(v)
        new = torch.full((3,), -9, dtype=torch.int32, device="cuda")
        pkv.paged_kv_compact(kd, vd, to_dev(tab), to_dev(np.asarray(keep, np.int32)),
                             to_dev(np.asarray(cu, np.int32)),
                             to_dev(np.asarray(start, np.int32)), new)
        assert pkv.paged_error_flags() == flag
        for got, was in ((kd, k), (vd, v)):
            want = was.copy()
            for b, src, dst in moved:
                want[t[b, dst // 8], dst % 8] = was[t[b, src // 8], src % 8]
            assert np.array_equal(to_host(got), want)
        return to_host(new).tolist()

    L, B = pkv.PKV_FLAG_BAD_LENGTH, pkv.PKV_FLAG_BAD_BLOCK
    # an entry below its place, one past the table, one negative
    assert call(t, [5, 0, 7, 32, 9, -1], [0, 3, 5, 6], [0, 0, 0], L,
                [(0, 5, 0), (0, 7, 2), (1, 9, 1)]) == [3, 2, 1]
    assert call(t, [5, -2 ** 31, 2 ** 31 - 1], [0, 1, 2, 3], [0, 0, 0], L, [(0, 5, 0)]) == [1, 1, 1]
    # a bad source page, a bad destination page
    bad = t.copy()
    bad[0, 1], bad[1, 0] = -1, total
    assert call(bad, [1, 9, 17, 9, 17], [0, 3, 5, 5], [0, 0, 0], B,
                [(0, 1, 0), (0, 17, 2)]) == [3, 2, 0]
    # a negative start, bounds that run backwards, a new length past the table
    assert call(t, [5, 6, 7], [0, 1, 2, 3], [-1, 0, 0], L, [(1, 6, 0), (2, 7, 0)]) == [0, 1, 1]
    assert call(t, [5, 6, 7], [0, 2, 1, 3], [0, 0, 0], L,
                [(0, 5, 0), (0, 6, 1), (2, 6, 0), (2, 7, 1)]) == [2, 0, 2]
    assert call(t, [5, 6, 7], [0, 1, 2, 9], [0, 0, 0], L, [(0, 5, 0), (1, 6, 0)]) == [1, 1, 0]
    assert call(t, [5, 31, 31], [0, 1, 3, 3], [0, 31, 0], L, [(0, 5, 0)]) == [1, 31, 0]


def test_no_lengths_out_no_tokens_other_stream_and_graph():
    rng = np.random.default_rng(1)
    lens = [400, 300]
    t, total = tables(rng, lens, 16)
    k, v = (make(rng, "bf16", total, 16, 8, 128) for _ in range(2))
    keep, cu = lists_of(rng, lens, [0, 0], 0.5)
    kd, vd = to_dev(k), to_dev(v)
    dev = [to_dev(x) for x in (t, keep, cu)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pkv.paged_kv_compact(kd, vd, *dev)
    torch.cuda.synchronize()
    assert np.array_equal(to_host(kd), k)  # captured, not run
    g.replay()
    torch.cuda.synchronize()
    once = Q.compact(k, t, keep, cu, None, False)
    assert np.array_equal(to_host(kd), once)
    with torch.cuda.stream(side):
        pkv.paged_kv_compact(kd, vd, *dev)
    torch.cuda.synchronize()
    assert np.array_equal(to_host(kd), Q.compact(once, t, keep, cu, None, False))
    kd = to_dev(k)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    pkv.paged_kv_compact(kd, vd, dev[0], none, torch.zeros(3, dtype=torch.int32, device="cuda"),
                         torch.tensor([7, 0], dtype=torch.int32, device="cuda"), new)
    assert new.tolist() == [7, 0] and np.array_equal(to_host(kd), k)
    pkv.paged_kv_compact(kd, vd, dev[0], none, none.new_zeros(1))  # no sequences
    assert pkv.paged_error_flags() == 0


def test_binding_refusals():
    k = torch.zeros(4, 8, 2, 64, device="cuda")
    both = torch.zeros(5, 8, 2, 64, device="cuda")
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    t = i(0, 1, 2, 3).reshape(2, 2)
    for v in (k, both[1:]):  # pools that share rows
        with pytest.raises(pkv.PagedKVError) as e:
            pkv.paged_kv_compact(k if v is k else both[:4], v, t, i(1), i(0, 1))
        assert e.value.status == -1
    with pytest.raises(ValueError):
        pkv.paged_kv_compact(k, k[:2], t, i(1), i(0, 1))
    with pytest.raises(ValueError):
        pkv.paged_kv_compact(k, k.clone(), t[:1], i(1), i(0, 1, 1))
    with pytest.raises(ValueError):
        pkv.paged_kv_compact(k, k.clone(), t, i(1), i(0, 1, 1), start=i(0))
    with pytest.raises(ValueError):
        pkv.paged_kv_compact(k, k.clone(), t, i(1), i(0, 1, 1), seqlens_out=i(0))
    with pytest.raises(TypeError):
        pkv.paged_kv_compact(k, k.clone(), t, i(1).long(), i(0, 1, 1))
    with pytest.raises(TypeError):
        pkv.paged_kv_compact(k.half(), k.half(), t, i(1), i(0, 1, 1))
    with pytest.raises(ValueError):
        pkv.paged_kv_compact(k.transpose(1, 2), k.transpose(1, 2), t, i(1), i(0, 1, 1))

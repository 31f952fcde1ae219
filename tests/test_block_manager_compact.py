"""paged_bm_compact against a plain Python model: tokens, tables, reference
counts, the free stack, copies of shared blocks, and what the prefix cache must
not hand out afterwards."""
import ctypes
import random

import numpy as np
import pytest

import paged_kv_cache_70_gb300 as pkv
from paged_kv_cache_70_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return pkv.load_library()


def move(rows, table, keep, start, block):
    """Contents of the blocks after paged_kv_compact through `table`."""
    new = rows.copy()
    for i, p in enumerate(keep):
        to = start + i
        new[table[to // block], to % block] = rows[table[p // block], p % block]
    return new


def held(rows, bm, seq, block):
    t = bm.table(seq)
    return [rows[t[i // block], i % block] for i in range(bm.seq_len(seq))]


def test_eviction_releases_the_blocks_behind_the_end():
    bm = pkv.BlockManager(10, 4)
    s, _ = bm.allocate(range(18))  # blocks 0 .. 4
    src, dst, table = bm.compact(s, [1, 2, 7, 8, 16], 0)
    assert (src, dst, table) == ([], [], [0, 1, 2, 3, 4])
    assert bm.table(s) == [0, 1] and bm.seq_len(s) == 5
    assert bm.free_stack()[-3:] == [4, 3, 2] and bm.num_free() == 8
    assert [bm.ref_count(b) for b in range(5)] == [1, 1, 0, 0, 0]


def test_shared_blocks_that_are_written_are_copied_first():
    bm = pkv.BlockManager(12, 4)
    a, _ = bm.allocate(range(14))
    b = bm.fork(a)
    src, dst, table = bm.compact(b, [5, 9, 10, 13], 4)
    # rows move into block 1 only (positions 4 .. 7)
    assert src == [1] and dst == [4] and table == [0, 4, 2, 3]
    assert bm.table(b) == [0, 4] and bm.table(a) == [0, 1, 2, 3]
    assert [bm.ref_count(x) for x in range(5)] == [2, 1, 1, 1, 1]
    assert bm.seq_len(a) == 14 and bm.seq_len(b) == 8


def test_moved_blocks_are_never_found_by_their_tokens():
    bm = pkv.BlockManager(30, 4)
    a, _ = bm.allocate([1, 2, 3, 4, 5, 6, 7, 8, 9])
    bm.compact(a, [1, 2, 3, 4], 0)  # now [2, 3, 4, 5], moved
    assert bm.allocate([1, 2, 3, 4])[1] == 0  # its old first block
    assert bm.allocate([2, 3, 4, 5])[1] == 0  # its new contents
    for t in (6, 7, 8, 9):
        bm.append(a, t)  # a block filled behind moved ones
    assert bm.allocate([2, 3, 4, 5, 6, 7, 8, 9])[1] == 4  # the plain sequence's own first block
    f = bm.fork(a)
    for t in (1, 1, 1, 1):
        bm.append(f, t)
    assert bm.allocate([2, 3, 4, 5, 6, 7, 8, 9, 1, 1, 1, 1])[1] == 8


def test_cutting_a_sequence_keeps_its_whole_blocks_cached():
    bm = pkv.BlockManager(20, 4)
    a, _ = bm.allocate(range(12))
    assert bm.compact(a, [], 10)[:2] == ([], [])
    assert bm.table(a) == [0, 1, 2] and bm.seq_len(a) == 10
    b, cached = bm.allocate(range(12))  # the third block is partial now
    assert cached == 8 and bm.table(b)[:2] == [0, 1] and bm.table(b)[2] != 2
    bm.append(a, 50)
    bm.append(a, 51)
    assert bm.allocate([*range(10), 50, 51])[1] == 12  # it did not move: cached when full again
    c = bm.fork(a)
    bm.compact(c, [], 9)  # a shared block cut: the other holder keeps it
    assert bm.append(c, 7) != (-1, -1)
    assert bm.allocate([*range(10), 50, 51])[1] == 12


def test_a_cut_block_whose_other_holder_left_is_not_found_after_a_write():
    bm = pkv.BlockManager(20, 4)
    a, _ = bm.allocate(range(12))
    c = bm.fork(a)
    bm.compact(c, [], 9)  # block 2 is shared and still whole for `a`
    bm.free(a)
    assert bm.append(c, 7) == (-1, -1)  # written in place: it is this sequence's alone
    b, cached = bm.allocate(range(12))
    assert cached == 8 and bm.table(b)[2] != bm.table(c)[2]


def test_refusals_change_nothing(lib):
    bm = pkv.BlockManager(4, 4)
    a, _ = bm.allocate(range(14))
    b = bm.fork(a)
    state = lambda: (bm.table(a), bm.table(b), bm.seq_len(b), bm.free_stack(),  # noqa: E731
                     [bm.ref_count(i) for i in range(4)])
    before = state()
    for keep, start in (([3, 3], 0), ([5, 4], 0), ([14], 0), ([-1], 0), ([2], 3), ([], 15), ([0], -1), ([1], 2**63 - 1)):
        with pytest.raises(pkv.PagedKVError) as e:
            bm.compact(b, keep, start)
        assert e.value.status == -1 and state() == before
    with pytest.raises(pkv.PagedKVError) as e:
        bm.compact(b, [1, 2], 0)  # block 0 is shared and no block is free
    assert e.value.status == -5 and state() == before
    with pytest.raises(pkv.PagedKVError):
        bm.compact(99, [], 0)
    with pytest.raises(ValueError, match="32-bit"):
        bm.compact(b, [2**32], 0)
    assert state() == before
    n, k = ctypes.c_int32(-7), (ctypes.c_int32 * 1)(3)
    t = (ctypes.c_int32 * 4)()
    f, vp = lib.paged_bm_compact, lambda x: ctypes.cast(x, ctypes.c_void_p)  # noqa: E731
    assert f(bm._h, b, 0, vp(k), 1, vp(t), 3, None, None, 0, ctypes.byref(n)) == -1  # table too small
    assert f(bm._h, b, 0, vp(k), 1, vp(t), 4, None, None, 0, ctypes.byref(n)) == -1
    assert n.value == 1 and state() == before
    assert f(None, b, 0, vp(k), 1, vp(t), 4, None, None, 0, ctypes.byref(n)) == -1
    assert f(bm._h, b, 0, None, 1, vp(t), 4, None, None, 0, ctypes.byref(n)) == -1
    assert f(bm._h, b, 0, vp(k), 1, vp(t), 4, None, None, 0, None) == -1


@pytest.mark.parametrize("seed", range(8))
def test_random_histories_keep_every_sequences_rows(seed):
    """Sequences allocated, forked, appended to, compacted and freed; each row
    carries the (token, when it was written) its sequence holds, blocks are copied
    as told, and every sequence must hold its own rows throughout."""
    rnd = random.Random(seed)
    block, total = rnd.choice([1, 3, 4, 8]), 80
    bm = pkv.BlockManager(total, block)
    rows = np.full((total, block), -1, np.int64)
    want, stamp = {}, 0
    for _ in range(300):
        op = rnd.random()
        try:
            if op < 0.2 or not want:
                toks = [rnd.randrange(3) for _ in range(rnd.randrange(0, 40))]
                s, cached = bm.allocate(toks)
                t = bm.table(s)
                for i in range(cached, len(toks)):
                    rows[t[i // block], i % block] = stamp * 10 + toks[i]
                    stamp += 1
                want[s] = [int(rows[t[i // block], i % block]) for i in range(len(toks))]
                assert [x % 10 for x in want[s]] == toks
            elif op < 0.3:
                p = rnd.choice(list(want))
                want[bm.fork(p)] = list(want[p])
            elif op < 0.6:
                s, tok = rnd.choice(list(want)), rnd.randrange(3)
                src, dst = bm.append(s, tok)
                if src >= 0:
                    rows[dst] = rows[src]
                n = bm.seq_len(s) - 1
                rows[bm.table(s)[n // block], n % block] = stamp * 10 + tok
                want[s].append(stamp * 10 + tok)
                stamp += 1
            elif op < 0.85:
                s = rnd.choice(list(want))
                n = len(want[s])
                start = rnd.randrange(n + 1)
                keep = [p for p in range(start, n) if rnd.random() < rnd.choice([0.2, 0.7, 1.0])]
                src, dst, table = bm.compact(s, keep, start)
                for x, y in zip(src, dst):
                    rows[y] = rows[x]
                rows = move(rows, table, keep, start, block)
                want[s] = want[s][:start] + [want[s][p] for p in keep]
            else:
                s = rnd.choice(list(want))
                bm.free(s)
                del want[s]
        except pkv.PagedKVError as e:
            assert e.status == pkv.PKV_ERR_NO_SPACE
        for s, w in want.items():
            assert held(rows, bm, s, block) == w
        counts = np.zeros(total, int)
        for s in want:
            for b in bm.table(s):
                counts[b] += 1
        assert [bm.ref_count(b) for b in range(total)] == counts.tolist()
        assert sorted(bm.free_stack()) == [b for b in range(total) if counts[b] == 0]

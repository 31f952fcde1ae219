"""Rows that are not written standing between the tokens of a page in a list for
paged_kv_write_q8: padding, sequences and positions past the table, positions past the angles.
The tokens in front of and behind them share the page's scale, which is set once for all of
them.  Bytes against the numpy model, which sees the list without the rows that have no place."""
import numpy as np
import pytest

import paged_kv_cache_70_gb300 as pkv
import q4_oracle as Q4
import q8_oracle as Q
from gpu_helpers import to_dev, to_host
from test_q8_gpu import codes_of, pool, random_pool
from test_rope_write_gpu import new_tokens, rows

pytestmark = pytest.mark.gpu

ANGLES = 5000  # positions that the table of angles has


def spread(rng, seq, pos, table, block, gaps, kinds):
    """The list with `gaps` (how many, rows at most) of rows without a place between its tokens:
    seq, pos, rope_pos, which have a place, which are written, and the flags that they set."""
    count, most = gaps
    n = len(seq)
    put = np.zeros(n + 1, int)
    np.add.at(put, rng.integers(0, n + 1, count), rng.integers(1, most + 1, count))
    out, flags = [], 0
    for i in range(n + 1):
        for _ in range(put[i]):
            s, p = (seq[i], pos[i]) if i < n else (0, 0)
            kind = kinds[int(rng.integers(len(kinds)))]
            if kind == "padding":  # (its position is nobody's, whatever it looks like)
                out.append((-1, int(rng.choice([p, p + 1, -1, 0])), 3, False, False))
            elif kind == "sequence":
                out.append((len(table) + int(rng.integers(0, 3)), p, 3, False, False))
                flags |= pkv.PKV_FLAG_BAD_SEQ
            else:
                past = table.shape[1] * block
                out.append((s, int(rng.choice([-1, -2**31, past, past + 7, 2**31 - 1])), 3, False,
                            False))
                flags |= pkv.PKV_FLAG_BAD_LENGTH
        if i < n:
            at, live = int(pos[i]), True
            if "angle" in kinds and rng.random() < 0.2:
                at, live = int(rng.choice([-1, ANGLES, 2**31 - 1, -2**31])), False
                flags |= pkv.PKV_FLAG_BAD_LENGTH
            out.append((seq[i], pos[i], at, True, live))
    s, p, a, placed, live = zip(*out)
    i32 = lambda x: np.array(x, np.int64).astype(np.int32)
    return i32(s), i32(p), i32(a), np.array(placed), np.array(live), flags


def check(rng, sizes, hq, hkv, d, rot, mix, block, dtype, gaps, kinds, fresh):
    table, total, seq, pos = new_tokens(rng, sizes, block, 0)
    if not rot:
        kinds = [k for k in kinds if k != "angle"]
    seq, pos, at, placed, live, flags = spread(rng, seq, pos, table, block, gaps, kinds)
    n = len(seq)
    (k, kt), (v, vt) = (rows(rng, n, hkv, d, dtype) for _ in range(2))
    # what lies in rows that are not written does not enter: infinities, NaN, large values
    for x, t in ((k, kt), (v, vt)):
        junk = np.array([np.inf, -np.inf, np.nan, 1e30], np.float32)[rng.integers(0, 4, n)]
        if dtype == "bf16":
            junk = Q4.bf16_value(Q4.bf16_bits(junk)).astype(np.float32)
        x[~live] = junk[~live, None, None]
        t.copy_(to_dev(x))
    before = [random_pool(rng, total, hkv, block, d) for _ in range(2)]
    before = [(np.zeros_like(c), np.zeros_like(s)) if fresh else (c & 0xBF, s) for c, s in before]
    kw, want_q = {}, None
    if rot:
        cs = Q.cos_sin(ANGLES, rot)
        q, qt = rows(rng, n, hq, d, dtype)
        kw = dict(cos_sin=to_dev(cs), q=qt, interleaved=mix, rope_pos=to_dev(at))
        turned = (seq >= 0) & (at >= 0) & (at < ANGLES)
        want_q = q.copy()
        want_q[turned] = Q.rotate(q[turned], cs, at[turned], mix)
        k = k.copy()
        k[live] = Q.rotate(k[live], cs, at[live], mix)
    want = []
    for x, (c, s) in ((k, before[0]), (v, before[1])):
        c, s = c.copy(), s.copy()
        Q.write(x[placed], table, seq[placed], pos[placed], c, s, live[placed])
        want.append((c, s))
    for _ in range(3):
        (kc, ks), (vc, vs) = ((pool(c), to_dev(s)) for c, s in before)
        out = pkv.paged_kv_write_q8(kt, vt, to_dev(table), to_dev(seq), to_dev(pos), kc, vc, ks, vs,
                                    **kw)
        assert pkv.paged_error_flags() == flags
        if rot:
            assert np.array_equal(to_host(out),
                                  Q4.bf16_bits(want_q) if dtype == "bf16" else want_q)
        for (c, s), codes, scale in zip(want, (kc, vc), (ks, vs)):
            assert np.array_equal(to_host(scale), s)
            assert np.array_equal(Q.canon(codes_of(codes)), Q.canon(c))


ALL = ["padding", "sequence", "position", "angle"]
CASES = [  # (cached, new), Hq, Hkv, d, rot (0: none), interleaved, B, type, gaps (count, most), rows
    ([(0, 2)], 1, 1, 64, 0, False, 16, "f32", (3, 1), ["padding"]),
    ([(3, 6), (14, 5)], 4, 2, 128, 128, False, 16, "bf16", (8, 2), ["padding"]),
    ([(3, 6), (14, 5)], 4, 2, 128, 128, False, 16, "bf16", (8, 2), ALL),
    ([(0, 16)] * 8, 8, 8, 128, 64, True, 16, "f32", (60, 3), ALL),
    ([(5, 60), (0, 0), (100, 9), (0, 200)], 6, 3, 64, 48, False, 7, "bf16", (90, 4), ALL),
    ([(0, 64), (30, 64)], 4, 4, 128, 128, False, 64, "bf16", (50, 2), ALL),
    ([(0, 128), (2, 130)], 4, 4, 128, 0, False, 128, "f32", (50, 2), ALL),
    ([(1, 600), (255, 2), (250, 1)], 8, 2, 128, 128, False, 256, "bf16", (200, 3), ALL),
    ([(1, 600), (255, 2), (250, 1)], 8, 2, 64, 64, True, 256, "f32", (200, 3), ALL),
    ([(0, 768), (4090, 1), (1, 511), (40, 257)], 2, 1, 64, 64, False, 4096, "bf16", (400, 2), ALL),
    ([(200, 1), (0, 255), (5, 513), (0, 1025)], 1, 1, 64, 32, True, 600, "bf16", (300, 2), ALL),
    ([(i % 40, 1 + i % 3) for i in range(300)], 8, 8, 64, 64, False, 8, "bf16", (300, 3), ALL),
    # windows of 256 tokens, and many of them, without a token that has a place
    ([(2, 3)], 2, 2, 64, 64, False, 16, "bf16", (4, 300), ["padding"]),
    ([(2, 5), (0, 9)], 2, 2, 64, 0, False, 16, "f32", (7, 1400), ["padding"]),
    ([(2, 5), (0, 9)], 2, 2, 128, 128, False, 16, "bf16", (12, 700), ALL),
    ([(7, 1000)], 2, 1, 64, 64, False, 2048, "bf16", (9, 1500), ALL),
    ([(60, 4), (0, 4)], 2, 1, 128, 128, False, 64, "bf16", (2, 5000), ["padding"]),
]


@pytest.mark.parametrize("sizes,hq,hkv,d,rot,mix,block,dtype,gaps,kinds", CASES)
@pytest.mark.parametrize("fresh", [True, False])
def test_rows_that_are_not_written_do_not_part_a_page(sizes, hq, hkv, d, rot, mix, block, dtype,
                                                      gaps, kinds, fresh):
    rng = np.random.default_rng(d + rot + block + len(kinds) + fresh)
    check(rng, sizes, hq, hkv, d, rot, mix, block, dtype, gaps, kinds, fresh)


@pytest.mark.parametrize("before", [0, 1, 254, 255, 256, 257, 511])
@pytest.mark.parametrize("between", [1, 2, 254, 255, 256, 257, 511, 512, 767, 768, 1279, 1280, 1281,
                                     2304, 2305])
def test_padding_of_every_length_around_a_windows_border(before, between):
    """`before` padding rows, a token that begins a page, `between` padding rows, the page's next
    token, and one of another sequence behind it."""
    rng = np.random.default_rng(before * 10000 + between)
    hkv, d, block = 1, 64, 8
    table = np.array([[2, 0], [1, -1]], np.int32)
    seq = np.r_[[-1] * before, 0, [-1] * between, 0, 1].astype(np.int32)
    pos = np.r_[[1] * before, 0, [1] * between, 1, 3].astype(np.int32)
    x, t = rows(rng, len(seq), hkv, d, "f32")
    x[np.flatnonzero(seq >= 0)[0]] *= 100  # (a scale by itself would be another)
    t.copy_(to_dev(x))
    codes, scale = random_pool(rng, 3, hkv, block, d)
    codes &= 0xBF
    kc, vc, ks, vs = pool(codes), pool(codes), to_dev(scale), to_dev(scale)
    pkv.paged_kv_write_q8(t, t, to_dev(table), to_dev(seq), to_dev(pos), kc, vc, ks, vs)
    live = seq >= 0
    Q.write(x[live], table, seq[live], pos[live], codes, scale, live[live])
    for c, s in ((kc, ks), (vc, vs)):
        assert np.array_equal(to_host(s), scale) and np.array_equal(codes_of(c), codes)
    assert pkv.paged_error_flags() == 0


@pytest.mark.parametrize("seed", range(20))
def test_random_lists(seed):
    rng = np.random.default_rng(7000 + seed)
    d = int(rng.choice([64, 128]))
    block = int(rng.choice([1, 4, 16, 33, 64, 100, 256, 300]))
    sizes = [(int(rng.integers(0, 2 * block)), int(rng.integers(0, 1 + min(3 * block, 400))))
             for _ in range(int(rng.integers(1, 9)))] + [(0, 1)]
    hkv = int(rng.integers(1, 5))
    kinds = list(rng.permutation(ALL)[: int(rng.integers(1, 5))])
    if kinds == ["angle"]:
        kinds = ALL
    check(rng, sizes, hkv, hkv, d, int(rng.choice([0, 16, d])), bool(rng.integers(2)), block,
          ["bf16", "f32"][int(rng.integers(2))], (int(rng.integers(1, 200)), int(rng.integers(1, 9))),
          kinds, bool(rng.integers(2)))

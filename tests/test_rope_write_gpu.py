"""The cache write with the position rotation (paged_kv_write_rope): bytes of the pools and of
the rotated queries against numpy, where every product and sum is rounded to fp32."""
import numpy as np
import pytest
import torch

import paged_kv_cache_70_gb300 as pkv
import q4_oracle as Q4
import q8_oracle as Q
from gpu_helpers import to_dev, to_host, widen

pytestmark = pytest.mark.gpu


def new_tokens(rng, sizes, block, pad, extra=3):
    """(table, pages, seq, pos) of sequences with (cached, new) tokens, padding at the end."""
    need = [-(-(o + n) // block) for o, n in sizes]
    total = sum(need) + extra
    ids = rng.permutation(total).astype(np.int32)
    table = np.full((len(sizes), max(need + [1])), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    seq = np.array([i for i, (_, n) in enumerate(sizes) for _ in range(n)] + [-1] * pad, np.int32)
    pos = np.array([o + j for o, n in sizes for j in range(n)] + [-5] * pad, np.int32)
    return table, total, seq, pos


def rows(rng, n, heads, d, dtype, fused=0):
    """fp32 values [N, H, d] of `dtype`, and a tensor of them (columns of a wider one)."""
    x = (rng.standard_normal((n, heads, d)) * 2).astype(np.float32)
    if dtype == "bf16":
        x = Q4.bf16_value(Q4.bf16_bits(x)).astype(np.float32)
    t = to_dev(x)
    t = t.to(torch.bfloat16) if dtype == "bf16" else t
    if fused:
        wide = torch.full((n, heads + fused, d), 77.0, dtype=t.dtype, device="cuda")
        wide[:, 1:1 + heads] = t
        t = wide[:, 1:1 + heads]
    return x, t


def as_pool(x, dtype):
    return Q4.bf16_bits(x) if dtype == "bf16" else np.asarray(x, np.float32)


CASES = [  # (cached, new), Hq, Hkv, d, rot, interleaved, B, rows' type, pools' type, padding, fused
    ([(0, 1)], 1, 1, 64, 64, False, 1, "f32", "f32", 0, 0),
    ([(5, 1), (0, 1), (77, 1)], 16, 8, 128, 128, False, 16, "bf16", "bf16", 0, 0),
    ([(5, 1), (0, 1), (77, 1)], 16, 8, 128, 128, True, 16, "bf16", "bf16", 4, 24),
    ([(3, 40), (0, 0), (100, 9)], 5, 5, 128, 64, False, 7, "bf16", "f32", 1, 3),
    ([(3, 40), (17, 300)], 6, 2, 64, 16, False, 24, "f32", "bf16", 3, 2),
    ([(3, 40), (17, 300)], 6, 2, 64, 16, True, 24, "f32", "bf16", 0, 0),
    ([(0, 33)], 33, 11, 64, 48, False, 16, "bf16", "bf16", 2, 0),
    ([(0, 33)], 33, 11, 128, 112, True, 16, "bf16", "bf16", 0, 1),
    ([(1, 600)], 64, 1, 128, 128, False, 256, "bf16", "bf16", 0, 2),
    ([(9, 5)] * 70, 32, 32, 128, 32, False, 32, "f32", "f32", 11, 0),
    ([(0, 3)], 0, 3, 128, 128, False, 8, "bf16", "bf16", 0, 0),
]


@pytest.mark.parametrize("sizes,hq,hkv,d,rot,mix,block,src,dst,pad,fused", CASES)
def test_bytes(sizes, hq, hkv, d, rot, mix, block, src, dst, pad, fused):
    rng = np.random.default_rng(d + rot + len(sizes))
    table, total, seq, pos = new_tokens(rng, sizes, block, pad)
    n = len(seq)
    k, kt = rows(rng, n, hkv, d, src, fused)
    v, vt = rows(rng, n, hkv, d, src, fused)
    cs = Q.cos_sin(2000, rot)
    before = [as_pool(rng.standard_normal((total, block, hkv, d)), dst) for _ in range(2)]
    kc, vc = to_dev(before[0]), to_dev(before[1])
    rope_pos = np.where(seq >= 0, pos + 3 * seq + 11, -1).astype(np.int32)
    slots = torch.full((n,), 99, dtype=torch.int32, device="cuda")
    kw = {}
    if hq:
        q, qt = rows(rng, n, hq, d, src, fused)
        kw["q"] = qt
    out = pkv.paged_kv_write_rope(kt, vt, to_dev(cs), to_dev(table), to_dev(seq), to_dev(pos), kc,
                                  vc, rope_pos=to_dev(rope_pos), interleaved=mix,
                                  slot_mapping_out=slots, **kw)
    live = seq >= 0
    s, p = seq[live], pos[live]
    want = np.full(n, -1, np.int32)
    want[live] = table[s, p // block] * block + p % block
    assert np.array_equal(to_host(slots), want)
    for got, was, x, turned in ((kc, before[0], k, True), (vc, before[1], v, False)):
        x = Q.rotate(x[live], cs, rope_pos[live], mix) if turned else x[live]
        was = was.copy()
        was[table[s, p // block], p % block] = as_pool(x, dst)
        assert np.array_equal(to_host(got), was)
    if hq:
        turned = q.copy()
        turned[live] = Q.rotate(q[live], cs, rope_pos[live], mix)
        assert np.array_equal(to_host(out), as_pool(turned, src))
        # in place, the other columns left alone
        rest = qt.clone() if not fused else None
        res = pkv.paged_kv_write_rope(kt, vt, to_dev(cs), to_dev(table), to_dev(seq), to_dev(pos),
                                      kc, vc, q=qt, q_out=qt, rope_pos=to_dev(rope_pos),
                                      interleaved=mix)
        assert res is qt and torch.equal(qt, out) and (rest is None or rest.shape == qt.shape)
        if fused:
            base = qt._base
            assert bool((base[:, 0] == 77).all()) and bool((base[:, 1 + hq:] == 77).all())
    else:
        assert out is None
    assert pkv.paged_error_flags() == 0


def test_a_rotation_of_64_bits_is_met_to_the_roundings():
    """Queries at far positions against angles and rotation in 64 bits: the table's values are
    within 2^-25 of the cosines, two products and a sum add 2^-24 each, relative to |x_a| + |x_b|."""
    rng = np.random.default_rng(5)
    pos = np.array([0, 1, 40959, 131071, 1000000], np.int32)
    q, qt = rows(rng, 5, 4, 128, "f32")
    ang = pos[:, None] * 1e6 ** (-np.arange(64) / 64.0)
    cs = np.zeros((1000001, 128), np.float32)
    cs[pos] = np.concatenate((np.cos(ang), np.sin(ang)), 1)
    pool = torch.zeros(5, 1, 1, 128, device="cuda")
    table = torch.arange(5, dtype=torch.int32, device="cuda")[:, None].contiguous()
    out = pkv.paged_kv_write_rope(torch.zeros(5, 1, 128, device="cuda"),
                                  torch.zeros(5, 1, 128, device="cuda"), to_dev(cs), table,
                                  torch.arange(5, dtype=torch.int32, device="cuda"),
                                  torch.zeros(5, dtype=torch.int32, device="cuda"), pool,
                                  pool.clone(), q=qt, rope_pos=to_dev(pos))
    a, b = q[..., :64].astype(np.float64), q[..., 64:].astype(np.float64)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    want = np.concatenate((a * c - b * s, b * c + a * s), -1)
    bound = (2.0 ** -25 + 2 * 2.0 ** -24) * np.tile(np.abs(a) + np.abs(b), 2)
    assert np.all(np.abs(widen(out) - want) <= bound)


def test_tokens_that_are_not_written_are_flagged_and_nothing_else_is_touched():
    d, hkv, block = 64, 2, 4
    table = torch.tensor([[2, 9], [0, -1]], dtype=torch.int32, device="cuda")  # 9: no page
    #      ok  page 9  page -1  past the table  past the sequences  angle  padding  ok
    seq = [0, 0, 1, 1, 2, 0, -7, 1]
    pos = [1, 4, 5, 8, 0, 2, 0, 3]
    at = [1, 4, 5, 8, 0, 50, 0, 3]
    flags = [0, pkv.PKV_FLAG_BAD_BLOCK, pkv.PKV_FLAG_BAD_BLOCK, pkv.PKV_FLAG_BAD_LENGTH,
             pkv.PKV_FLAG_BAD_SEQ, pkv.PKV_FLAG_BAD_LENGTH, 0, 0]
    k = torch.randn(8, hkv, d, device="cuda")
    cs = to_dev(Q.cos_sin(50, d))
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for bad in [list(range(8))] + [[i] for i in range(8)]:
        kc = torch.full((3, block, hkv, d), 7.0, device="cuda")
        vc = kc.clone()
        slots = dev([99] * len(bad))
        q = torch.randn(len(bad), 4, d, device="cuda")
        out = pkv.paged_kv_write_rope(
            k[bad].contiguous(), k[bad].contiguous(), cs, table, dev([seq[i] for i in bad]),
            dev([pos[i] for i in bad]), kc, vc, q=q, rope_pos=dev([at[i] for i in bad]),
            slot_mapping_out=slots)
        want = 0
        for i in bad:
            want |= flags[i]
        assert pkv.paged_error_flags() == want
        live = {0: 2 * block + 1, 7: 3}
        assert slots.tolist() == [live.get(i, -1) for i in bad]
        rows_ = [live[i] for i in bad if i in live]
        rest = torch.ones(3 * block, dtype=torch.bool)
        rest[rows_] = False
        assert bool((kc.view(-1, hkv, d)[rest.cuda()] == 7).all())
        assert bool((vc.view(-1, hkv, d)[rest.cuda()] == 7).all())
        for j, i in enumerate(bad):  # passed on: padding and the angle outside the table
            if i in (5, 6):
                assert torch.equal(out[j], q[j])


def test_no_tokens_and_broadcast_rows():
    d, hkv = 128, 2
    kc = torch.zeros(2, 4, hkv, d, device="cuda")
    vc = torch.zeros_like(kc)
    i32 = dict(dtype=torch.int32, device="cuda")
    cs = to_dev(Q.cos_sin(16, d))
    table = torch.tensor([[1, 0]], **i32)
    e = torch.empty(0, hkv, d, device="cuda")
    none = torch.empty(0, **i32)
    out = pkv.paged_kv_write_rope(e, e, cs, table, none, none, kc, vc, q=e)
    assert out.shape == (0, hkv, d) and not kc.any()
    one = torch.randn(1, hkv, d, device="cuda")
    k = one.expand(6, hkv, d)  # a token stride of 0
    pos = torch.arange(6, **i32)
    pkv.paged_kv_write_rope(k, k, cs, table, torch.zeros(6, **i32), pos, kc, vc)
    want = Q.rotate(np.repeat(to_host(one), 6, 0), to_host(cs), np.arange(6), False)
    slot = [4, 5, 6, 7, 0, 1]
    assert np.array_equal(to_host(kc).reshape(8, hkv, d)[slot], want)
    assert torch.equal(vc.view(8, hkv, d)[slot], k)


def test_binding_refuses_shapes():
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.zeros(3, 2, 64, device="cuda")
    kc = torch.zeros(2, 4, 2, 64, device="cuda")
    cs = torch.zeros(9, 64, device="cuda")
    table, idx = torch.zeros(1, 2, **i32), torch.zeros(3, **i32)
    ok = dict(k=k, v=k, cos_sin=cs, block_table=table, token_seq=idx, token_pos=idx, k_cache=kc,
              v_cache=kc.clone())
    pkv.paged_kv_write_rope(**ok)
    for bad, error in ((dict(v=k[:2]), ValueError), (dict(k=k[..., :32], v=k[..., :32]), ValueError),
                       (dict(token_seq=idx[:2]), ValueError), (dict(token_pos=idx.long()), TypeError),
                       (dict(rope_pos=idx[:1]), ValueError), (dict(cos_sin=cs.double()), TypeError),
                       (dict(cos_sin=cs[0]), ValueError), (dict(q=k[:2]), ValueError),
                       (dict(q=k.double()), TypeError), (dict(q_out=k), ValueError),
                       (dict(q=k, q_out=k[:, :1]), ValueError), (dict(v=k.bfloat16()), TypeError),
                       (dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                       (dict(v_cache=kc[:1]), ValueError), (dict(v_cache=kc.bfloat16()), TypeError),
                       (dict(slot_mapping_out=idx[:2]), ValueError),
                       (dict(cos_sin=cs[:, :24].contiguous()), pkv.PagedKVError),
                       (dict(k_cache=kc.half(), v_cache=kc.half()), TypeError),
                       (dict(block_table=table.cpu()), ValueError)):
        with pytest.raises(error):
            pkv.paged_kv_write_rope(**{**ok, **bad})
    assert pkv.paged_error_flags() == 0


def test_captured_and_replayed_on_another_stream():
    rng = np.random.default_rng(8)
    table, total, seq, pos = new_tokens(rng, [(3, 1), (40, 1), (0, 1)], 16, 1)
    k, kt = rows(rng, 4, 8, 128, "bf16")
    q, qt = rows(rng, 4, 16, 128, "bf16")
    cs = Q.cos_sin(100, 128)
    kc = torch.zeros(total, 16, 8, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    out = torch.empty_like(qt)
    args = (to_dev(cs), to_dev(table), to_dev(seq), to_dev(pos), kc, vc)
    pkv.paged_kv_write_rope(kt, kt, *args, q=qt, q_out=out)
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=st):
        pkv.paged_kv_write_rope(kt, kt, *args, q=qt, q_out=out)
    k2, kt2 = rows(rng, 4, 8, 128, "bf16")
    kt.copy_(kt2)
    kc.zero_()
    out.zero_()
    with torch.cuda.stream(st):
        st.wait_stream(torch.cuda.default_stream())
        g.replay()
    st.synchronize()
    s, p = seq[:3], pos[:3]
    got = to_host(kc)[table[s, p // 16], p % 16]
    assert np.array_equal(got, Q4.bf16_bits(Q.rotate(k2[:3], cs, p, False)))
    assert np.array_equal(to_host(out)[:3], Q4.bf16_bits(Q.rotate(q[:3], cs, p, False)))

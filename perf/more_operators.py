"""Cases of the cache write with the position rotation and of the 8-bit KV-cache calls.

``paged_kv_write_rope``   new K/V rows into fp32 or bf16 pools, K (and q) rotated on the way
``paged_kv_write_q8``     the same into 8-bit pools, with or without the rotation
``paged_kv_read_q8``      rows of 8-bit pools as values
``paged_decode_q8``       one query per sequence over an 8-bit cache

Rotation.  cos_sin [positions, rot] (fp32) holds rot / 2 cosines, then rot / 2 sines, of every
position.  The dims (i, i + rot / 2), or (2 i, 2 i + 1) interleaved, i < rot / 2, of a row x
at position p become
    x_a c - x_b s,    x_b c + x_a s        c = cos_sin[p, i], s = cos_sin[p, rot / 2 + i]
where every product and sum is rounded to fp32; dims from rot on stay.

An 8-bit pool is float8_e4m3fn [num_blocks, Hkv, B, d] with a scale for each block and head,
fp32 [num_blocks, Hkv]: a value is its code times its block's scale.  The rows that one call
puts into a block, with the largest finite magnitude a, need the least power of two
    n = 2^e >= 2^-100    with    a <= 448 n.
If they begin the block its scale becomes s = n.  Else it becomes s = max(n, the least power
of two >= the old scale), and the codes of the rows in front of them e4m3(code * (old / s)).
The new codes are e4m3(x / s), rounded to nearest even.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELT = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one decode step of a 64-sequence batch: 64 new tokens rotated and written (latency)
        dict(name="rope step 64", op="rope", seqs=64, new_lo=1, new_hi=1, old_lo=128, old_hi=4096,
             hq=16, hkv=8, d=128, rot=128, mix=False, block=16, dtype="bf16", cache="bf16",
             fused=False, shift=0, pad=0),
        # the new rows of a chunked prefill: 16 requests of up to 2048 new tokens, large pages
        dict(name="rope prefill rows", op="rope", seqs=16, new_lo=1, new_hi=2048, old_lo=0,
             old_hi=2048, hq=16, hkv=8, d=128, rot=128, mix=False, block=256, dtype="bf16",
             cache="bf16", fused=True, shift=0, pad=0),
        # a continuous-batching step in fp32 into bf16 pools, padded at its end, small heads of
        # which one half is rotated in neighbouring pairs, q, k, v the parts of one projection
        dict(name="rope mixed f32 d64 half", op="rope", seqs=40, new_lo=1, new_hi=120, old_lo=0,
             old_hi=2048, hq=16, hkv=8, d=64, rot=32, mix=True, block=16, dtype="f32",
             cache="bf16", fused=True, shift=0, pad=121),
        # the decode step over 8-bit pools: 64 tokens into begun pages, read back with their pages
        dict(name="q8 write step 64", op="write", seqs=64, new_lo=1, new_hi=1, old_lo=128,
             old_hi=4096, hq=16, hkv=8, d=128, rot=128, mix=False, block=16, dtype="bf16",
             fused=True, shift=0, pad=0),
        # the chunked prefill's rows into 8-bit pools with large pages
        dict(name="q8 write prefill rows", op="write", seqs=16, new_lo=1, new_hi=2048, old_lo=0,
             old_hi=2048, hq=16, hkv=8, d=128, rot=128, mix=False, block=256, dtype="bf16",
             fused=False, shift=0, pad=0),
        # the keys of a chunked prefill's requests (new and cached) as packed K/V for the
        # varlen prefill
        dict(name="q8 read prefill keys", op="read", tokens=34567, hkv=8, d=128, block=256,
             dtype="bf16", pad=0.0),
        # one short request's keys, in fp32
        dict(name="q8 read short f32", op="read", tokens=513, hkv=8, d=128, block=16, dtype="f32",
             pad=0.0),
        # the three-sequence example of the decode tests: the smallest call
        dict(name="q8 decode tiny f32", op="decode", batch=3, lo=30, hi=70, hq=2, hkv=1, d=64,
             block=32, dtype="f32"),
        # a served batch of ordinary contexts, small pages
        dict(name="q8 decode batch 64", op="decode", batch=64, lo=128, hi=4096, hq=16, hkv=8,
             d=128, block=16, dtype="bf16"),
        # few sequences with long contexts, large pages
        dict(name="q8 decode long", op="decode", batch=8, lo=16384, hi=40960, hq=16, hkv=8, d=128,
             block=256, dtype="bf16"),
        # the same contexts with 8 query heads per KV head
        dict(name="q8 decode long gqa 8", op="decode", batch=8, lo=16384, hi=40960, hq=64, hkv=8,
             d=128, block=256, dtype="bf16"),
        # one user, one middling context, small heads, 8 query heads per KV head
        dict(name="q8 decode one d64 gqa 8", op="decode", batch=1, lo=7777, hi=7777, hq=32, hkv=4,
             d=64, block=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "write", "write", "read", "decode", "decode", "decode"])
    d = rng.choice([64, 128, 128])
    block = rng.choice([8, 16, 16, 24, 32, 48, 64, 128, 256])
    if op == "read":
        hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 34567 * 8 * 128 * 2 // (hkv * d * ELT[dtype])
        return dict(op=op, tokens=_log(rng, 1, min(most, 34567)), hkv=hkv, d=d, block=block,
                    dtype=dtype, pad=rng.choice([0.0, 0.0, 0.05]))
    if op == "decode":
        hkv = rng.choice([1, 2, 3, 4, 8, 8])
        group = rng.choice([1, 2, 2, 4, 5, 8])
        batch = _log(rng, 1, 192)
        hi = _log(rng, 16, max(64, min(40960, 200000 // batch)))
        return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, hq=hkv * group, hkv=hkv,
                    d=d, block=block, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    hkv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 4])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if rng.random() < 0.4:  # a decode step
        seqs, new_hi = _log(rng, 1, 256), 1
    else:
        seqs = _log(rng, 1, 32)
        new_hi = _log(rng, 2, 2048)
    while seqs * new_hi * hkv * group * d * ELT[dtype] > 16 * 2048 * 16 * 128 * 2:
        new_hi = max(1, new_hi // 2)
    case = dict(op=op, seqs=seqs, new_lo=rng.randint(1, new_hi), new_hi=new_hi, old_lo=0,
                old_hi=_log(rng, 1, 4096), hq=hkv * group, hkv=hkv, d=d,
                rot=rng.choice([d, d, d // 2, 16, 48]), mix=rng.random() < 0.4, block=block,
                dtype=dtype, fused=rng.random() < 0.5, shift=rng.choice([0, 0, 0, 30000]),
                pad=rng.choice([0, 0, 7]))
    if op == "rope":
        case["cache"] = rng.choice(["bf16", "bf16", dtype])
    return case


# ---------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------
def _spread(n, lo, hi, step=0.6180339887498949):
    """n lengths spread over lo..hi, the same for every seed."""
    return [lo + int((hi - lo) * ((0.5 + i * step) % 1.0) + 0.5) for i in range(n)]


def _lens(case):
    return _spread(case["batch"], case["lo"], case["hi"])


def _old_new(case):
    """(tokens cached before, new tokens) of each sequence."""
    return list(zip(_spread(case["seqs"], case["old_lo"], case["old_hi"], 0.7548776662466927),
                    _spread(case["seqs"], case["new_lo"], case["new_hi"])))


def _touched(case):
    """(first, end) positions of the pages that each sequence's new tokens lie in."""
    b = case["block"]
    return [(old // b * b, old + new) for old, new in _old_new(case)]


def work(case):
    op, kv = case["op"], case["hkv"] * case["d"]
    if op == "decode":
        keys = sum(_lens(case))
        io = 2 * case["batch"] * case["hq"] * case["d"] * ELT[case["dtype"]]
        pages = keys // case["block"]
        return {"bytes": 2 * keys * kv + io + pages * (4 + 8 * case["hkv"]),
                "flops": 4.0 * keys * case["hq"] * case["d"]}
    elt = ELT[case["dtype"]]
    if op == "read":
        n = case["tokens"]
        return {"bytes": n * (2 * kv * (elt + 1) + 4), "flops": 2.0 * n * kv}
    n = sum(new for _, new in _old_new(case))
    rows = n + case["pad"]
    q = 2 * rows * case["hq"] * case["d"] * elt
    index = 8 * rows + 4 * n * case["rot"]
    flops = 3.0 * n * (case["hq"] + case["hkv"]) * case["rot"]
    if op == "rope":
        return {"bytes": q + index + 2 * n * kv * (elt + ELT[case["cache"]]), "flops": flops}
    # the new rows in and out, then the values of every row of their pages
    seen = sum(end - first for first, end in _touched(case))
    return {"bytes": q + index + 2 * n * kv * (elt + 1) + seen * (2 * kv * (elt + 1) + 4),
            "flops": flops + 4.0 * n * kv + 2.0 * seen * kv}


# ---------------------------------------------------------------------------
# plain form: rotation, codes, rows, slots
# ---------------------------------------------------------------------------
def _rotate(x, cos_sin, pos, mix):
    """fp32 rows x [N, H, d] at positions pos [N], rotated."""
    rot = cos_sin.shape[1]
    t = cos_sin[pos][:, None, :]
    c, s = t[..., : rot // 2], t[..., rot // 2:]
    x = x.float()
    if mix:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
    ra, rb = a * c - b * s, b * c + a * s
    if mix:
        head = torch.stack((ra, rb), -1).flatten(-2)
    else:
        head = torch.cat((ra, rb), -1)
    return torch.cat((head, x[..., rot:]), -1)


def _pow2(e):
    """2^e in fp32 of whole numbers e in -126 .. 127, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _needed(a):
    """The least power of two n >= 2^-100 with a <= 448 n, of fp32 magnitudes a."""
    m, e = torch.frexp(a)  # a = m 2^e, 1/2 <= m < 1; 448 = 7/8 2^9
    e = torch.where(m > 0.875, e + 1, e) - 9
    e = torch.where(a > 0, e, torch.full_like(e, -100)).clamp(min=-100)
    return _pow2(e)


def _codes(x):
    """e4m3 codes (uint8) of fp32 values of at most 448 in magnitude, or non-finite ones."""
    bad = ~torch.isfinite(x)
    return torch.where(bad, torch.full_like(x, float("nan")), x).to(torch.float8_e4m3fn).view(
        torch.uint8)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _slots(table, seq, pos, block):
    return table[seq, pos // block].long() * block + pos % block


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _table(cos_len, rot):
    """cos and sin of every position, of angles in 64 bits."""
    inv = 1e6 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") * 2 / rot)
    a = torch.arange(cos_len, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float()


def _q8_pool(case, num_blocks, gen):
    """An 8-bit pool of N(0, 1) rows with a few large channels, as K has them, and heads of
    different size; its scales."""
    hkv, d, b = case["hkv"], case["d"], case["block"]
    gain = torch.exp2(torch.rand(hkv, 1, d, device="cuda", generator=gen) * 2 - 1)
    gain[:, :, 5::37] *= 4.0
    codes = torch.empty(num_blocks, hkv, b, d, dtype=torch.uint8, device="cuda")
    scale = torch.empty(num_blocks, hkv, device="cuda")
    step = max(1, (1 << 26) // (hkv * b * d))
    for i in range(0, num_blocks, step):
        n = min(step, num_blocks - i)
        x = torch.randn(n, hkv, b, d, device="cuda", generator=gen) * gain
        s = _needed(x.abs().amax((2, 3)))
        scale[i:i + n] = s
        codes[i:i + n] = _codes(x / s[:, :, None, None])
    return codes.view(torch.float8_e4m3fn), scale


def _pages(lens, block, rnd):
    """Block tables over a shuffled pool with a tenth of it free; padding is -1."""
    need = [-(-n // block) for n in lens]
    num_blocks = sum(need) + max(1, sum(need) // 10)
    ids = torch.randperm(num_blocks, generator=rnd, dtype=torch.int64).tolist()
    rows, at = [], 0
    for n in need:
        rows.append(ids[at:at + n] + [-1] * (max(max(need), 1) - n))
        at += n
    return torch.tensor(rows, dtype=torch.int32, device="cuda"), num_blocks


def _prepare_new(case, st, rnd, gen):
    """The new tokens of a write: rows, sequences, positions, rotation."""
    sizes = _old_new(case)
    block, d, hq, hkv = case["block"], case["d"], case["hq"], case["hkv"]
    st["table"], num_blocks = _pages([old + new for old, new in sizes], block, rnd)
    seq = [b for b, (_, new) in enumerate(sizes) for _ in range(new)] + [-1] * case["pad"]
    pos = [old + i for old, new in sizes for i in range(new)] + [0] * case["pad"]
    st["seq"], st["pos"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (seq, pos))
    n = len(seq)
    st["n_live"] = n - case["pad"]
    if case["fused"]:  # the projection's output, of which q, k and v are columns
        x = torch.randn(n, hq + 2 * hkv, d, device="cuda", generator=gen).to(
            DTYPES[case["dtype"]])
        st["q"], st["k"], st["v"] = x.split([hq, hkv, hkv], 1)
    else:
        st["q"], st["k"], st["v"] = (
            torch.randn(n, h, d, device="cuda", generator=gen).to(DTYPES[case["dtype"]])
            for h in (hq, hkv, hkv))
    st["rope_pos"] = None
    if case["shift"]:  # keys were evicted before: the rotation goes on counting them
        by = torch.randint(0, case["shift"], (case["seqs"],), generator=rnd).cuda()
        st["rope_pos"] = (st["pos"] + by[st["seq"].long().clamp(min=0)]).to(torch.int32)
    st["cos_sin"] = _table(max(pos) + case["shift"] + 1, case["rot"])
    return num_blocks


def prepare(case, seed):
    rnd = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, d, block, hkv = case["op"], case["d"], case["block"], case["hkv"]
    st = {"case": case}
    if op == "decode":
        lens = _lens(case)
        st["table"], num_blocks = _pages(lens, block, rnd)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["q"] = torch.randn(case["batch"], case["hq"], d, device="cuda", generator=gen).to(
            DTYPES[case["dtype"]])
    elif op == "read":
        n = case["tokens"]
        num_blocks = -(-n // block) + 8
        page = torch.randperm(num_blocks, generator=rnd)
        at = torch.arange(n)
        slots = page[at // block] * block + at % block  # the tokens fill shuffled pages
        if case["pad"]:
            slots[torch.rand(n, generator=rnd) < case["pad"]] = -1
        st["slots"] = slots.to(torch.int32).cuda()
    else:
        num_blocks = _prepare_new(case, st, rnd, gen)
    if op == "rope":
        st["kc"], st["vc"] = (torch.randn(num_blocks, block, hkv, d, device="cuda", generator=gen)
                              .to(DTYPES[case["cache"]]) for _ in range(2))
        return st
    st["kc"], st["ks"] = _q8_pool(case, num_blocks, gen)
    st["vc"], st["vs"] = _q8_pool(case, num_blocks, gen)
    if op == "write":  # every row of the pages that the new tokens lie in
        seen = _touched(case)
        seq = torch.tensor([b for b, (lo, hi) in enumerate(seen) for _ in range(lo, hi)],
                           device="cuda")
        pos = torch.tensor([p for lo, hi in seen for p in range(lo, hi)], device="cuda")
        st["slots"] = _slots(st["table"], seq, pos, block).to(torch.int32)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _run_own(st):
    import paged_kv_cache_70_gb300 as pkv
    case = st["case"]
    op = case["op"]
    if op == "decode":
        return pkv.paged_decode_q8(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["table"],
                                   st["lens"])
    if op == "rope":
        q = pkv.paged_kv_write_rope(st["k"], st["v"], st["cos_sin"], st["table"], st["seq"],
                                    st["pos"], st["kc"], st["vc"], q=st["q"],
                                    rope_pos=st["rope_pos"], interleaved=case["mix"])
        return q, st["kc"], st["vc"]
    if op == "write":
        q = pkv.paged_kv_write_q8(st["k"], st["v"], st["table"], st["seq"], st["pos"], st["kc"],
                                  st["vc"], st["ks"], st["vs"], cos_sin=st["cos_sin"], q=st["q"],
                                  rope_pos=st["rope_pos"], interleaved=case["mix"])
    k, v = pkv.paged_kv_read_q8(st["kc"], st["vc"], st["ks"], st["vs"], st["slots"],
                                DTYPES[case["dtype"]])
    return (q, k, v, st["ks"], st["vs"]) if op == "write" else (k, v)


def _read(codes, scale, slots, dtype):
    b = codes.shape[2]
    at = slots.clamp(min=0).long()
    v = _values(codes.view(torch.uint8)[at // b, :, at % b]) * scale[at // b][:, :, None]
    return torch.where((slots >= 0)[:, None, None], v, torch.zeros_like(v)).to(dtype)


def _write_q8(x, table, seq, pos, codes, scale, first):
    """fp32 rows x [N, Hkv, d] into a pool; first [N]: the lowest new position of a row's page."""
    codes = codes.view(torch.uint8)
    b = codes.shape[2]
    page = table[seq, pos // b].long()
    amax = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)  # [N, Hkv]
    most = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand_as(amax), amax, "amax")
    need = _needed(most)
    offset = torch.zeros(len(scale), dtype=torch.int64, device=x.device)
    offset[page] = first % b
    hit = torch.zeros(len(scale), dtype=torch.bool, device=x.device)
    hit[page] = True
    pages = hit.nonzero()[:, 0]
    old, at = scale[pages], offset[pages][:, None]
    m, e = torch.frexp(old)  # the least power of two >= old
    up = torch.where(old > 0, _pow2(torch.where(m > 0.5, e, e - 1)), torch.zeros_like(old))
    new = torch.where(at == 0, need[pages], torch.maximum(need[pages], up))
    front = (torch.arange(b, device=x.device) < at)[:, None, :, None]
    was = codes[pages]
    ratio = torch.where(at == 0, torch.ones_like(old), old / new)[:, :, None, None]
    codes[pages] = torch.where(front, _codes(_values(was) * ratio), was)
    scale[pages] = new
    codes[page, :, pos % b] = _codes(x / scale[page][:, :, None])


def _run_new(st):
    case, n = st["case"], st["n_live"]
    seq, pos = st["seq"].long(), st["pos"].long()
    at = pos if st["rope_pos"] is None else st["rope_pos"].long()
    table, b, cs = st["table"], case["block"], st["cos_sin"]
    q = torch.cat((_rotate(st["q"][:n], cs, at[:n], case["mix"]), st["q"][n:].float()))
    q = q.to(st["q"].dtype)
    k, v = _rotate(st["k"][:n], cs, at[:n], case["mix"]), st["v"][:n].float()
    seq, pos = seq[:n], pos[:n]
    if case["op"] == "rope":
        page = table[seq, pos // b].long()
        st["kc"][page, pos % b] = k.to(st["kc"].dtype)
        st["vc"][page, pos % b] = v.to(st["vc"].dtype)
        return q, st["kc"], st["vc"]
    lowest = torch.full((len(table),), 2**31, device=pos.device).scatter_reduce(
        0, seq, pos, "amin")  # of a sequence
    first = torch.maximum(lowest[seq], pos // b * b)
    _write_q8(k, table, seq, pos, st["kc"], st["ks"], first)
    _write_q8(v, table, seq, pos, st["vc"], st["vs"], first)
    dtype = DTYPES[case["dtype"]]
    return (q, _read(st["kc"], st["ks"], st["slots"], dtype),
            _read(st["vc"], st["vs"], st["slots"], dtype), st["ks"], st["vs"])


def _keys(codes, scale, table):
    """fp32 [batch, Hkv, keys, d] of the tables' pages."""
    page = table.clamp(min=0).long()
    x = _values(codes.view(torch.uint8)[page]) * scale[page][..., None, None]
    b, p, h, s, d = x.shape
    return x.transpose(1, 2).reshape(b, h, p * s, d)


def _run_decode(st):
    q, table, lens = st["q"], st["table"], st["lens"]
    b, hq, d = q.shape
    k, v = _keys(st["kc"], st["ks"], table), _keys(st["vc"], st["vs"], table)
    hkv, n = k.shape[1], k.shape[2]
    if n == 0:
        return torch.zeros_like(q)
    qg = q.float().reshape(b, hkv, hq // hkv, d)
    s = torch.matmul(qg, k.transpose(2, 3)) / math.sqrt(d)  # [batch, Hkv, G, keys]
    dead = torch.arange(n, device=q.device)[None, :] >= lens[:, None]
    s = s.masked_fill(dead[:, None, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m > float("-inf"), m, torch.zeros_like(m)))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.reshape(b, hq, d).to(q.dtype)


def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    if op == "decode":
        return _run_decode(st)
    if op == "read":
        dtype = DTYPES[st["case"]["dtype"]]
        return (_read(st["kc"], st["ks"], st["slots"], dtype),
                _read(st["vc"], st["vs"], st["slots"], dtype))
    return _run_new(st)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exp2(i):
    """2^i in fp64 of whole numbers i."""
    return ((i.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3_value(codes):
    """fp64 values of e4m3 codes (uint8), from their fields."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * _exp2(e - 7), m * 2.0 ** -9)
    mag = torch.where((c & 127) == 127, torch.full_like(mag, float("nan")), mag)
    return torch.where(c >> 7 > 0, -mag, mag)


def _e4m3_round(x):
    """The e4m3 value nearest to x (fp64, |x| <= 448), ties to even."""
    _, e = torch.frexp(x)
    step = _exp2(torch.clamp(e - 4, min=-9))  # 4 significant bits, 2^-9 at least
    return torch.round(x / step) * step


def _pow2_at_least(x):
    """Smallest 2^i >= x for fp64 x > 0."""
    i = torch.ceil(torch.log2(x)).to(torch.int64)
    i = torch.where(_exp2(i - 1) >= x, i - 1, i)  # (log2 may be off beside a power)
    return _exp2(torch.where(_exp2(i) < x, i + 1, i))


def _rotated64(x, cos_sin, pos, mix, cut):
    """Rows rotated in 64 bits; with `cut`, products and sums rounded to fp32 as the format says."""
    def fl(y):
        return y.float().double() if cut else y

    rot = cos_sin.shape[1]
    h = rot // 2
    i = torch.arange(h, device=x.device)
    a, b = (2 * i, 2 * i + 1) if mix else (i, i + h)
    t = cos_sin.double()[pos]
    c, s = t[:, None, :h], t[:, None, h:]
    out = x.double().clone()
    xa, xb = out[..., a], out[..., b]
    out[..., a] = fl(fl(xa * c) - fl(xb * s))
    out[..., b] = fl(fl(xb * c) + fl(xa * s))
    return out


def _stored64(case, table, x, codes, scale):
    """The values of the touched pages' rows after x [N, Hkv, d] went in, row by row as
    `slots` lists them, and the scales."""
    b = case["block"]
    val, scale = _e4m3_value(codes.view(torch.uint8)), scale.double().clone()
    out, at = [], 0
    for s, (old, new) in enumerate(_old_new(case)):
        rows, at = x[at:at + new], at + new
        lo = old
        while lo < old + new:
            hi = min((lo // b + 1) * b, old + new)
            page, off = int(table[s, lo // b]), lo % b
            part = rows[lo - old:hi - old]
            need = torch.clamp(part.abs().amax((0, 2)) / 448.0, min=2.0 ** -100)
            need = _pow2_at_least(need)
            if off:
                was = scale[page].clone()
                grown = torch.maximum(need, _pow2_at_least(was))
                kept = _e4m3_round(val[page, :, :off] * (was / grown)[:, None, None])
                scale[page] = grown
                out.append((kept * grown[:, None, None]).transpose(0, 1))
            else:
                scale[page] = need
            sc = scale[page][None, :, None]
            out.append(_e4m3_round(part / sc) * sc)
            lo = hi
    return torch.cat(out), scale


def exact(case, seed):
    st = prepare(case, seed)
    op, block = case["op"], case["block"]
    if op == "read":
        out = []
        for codes, scale in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
            s = st["slots"].long().clamp(min=0)
            v = _e4m3_value(codes.view(torch.uint8)[s // block, :, s % block])
            v = v * scale.double()[s // block][:, :, None]
            out.append(v.masked_fill((st["slots"] < 0)[:, None, None], 0.0))
        return tuple(out)
    if op == "decode":
        tables, group = st["table"].cpu(), case["hq"] // case["hkv"]
        out = torch.zeros(case["batch"], case["hq"], case["d"], dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lens(case)):
            if not n:
                continue
            pages = tables[b, : -(-n // block)].long().cuda()
            for h in range(case["hkv"]):
                k, v = ((_e4m3_value(codes.view(torch.uint8)[pages, h])
                         * scale.double()[pages, h][:, None, None]).reshape(-1, case["d"])[:n]
                        for codes, scale in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
                q = st["q"][b, h * group:(h + 1) * group].double()
                p = torch.softmax(q @ k.T / math.sqrt(case["d"]), -1)
                out[b, h * group:(h + 1) * group] = p @ v
        return out
    n = st["n_live"]
    at = (st["pos"] if st["rope_pos"] is None else st["rope_pos"]).long()[:n]
    q = torch.cat((_rotated64(st["q"][:n], st["cos_sin"], at, case["mix"], False),
                   st["q"][n:].double()))
    k = _rotated64(st["k"][:n], st["cos_sin"], at, case["mix"], op == "write")
    table = st["table"].cpu()
    if op == "write":
        kv, ks = _stored64(case, table, k, st["kc"], st["ks"])
        vv, vs = _stored64(case, table, st["v"][:n].double(), st["vc"], st["vs"])
        return q, kv, vv, ks, vs
    kc, vc = st["kc"].double(), st["vc"].double()
    seq, pos = st["seq"].cpu().long()[:n], st["pos"].cpu().long()[:n]
    page = table[seq, pos // block].long().cuda()
    kc[page, (pos % block).cuda()] = k
    vc[page, (pos % block).cuda()] = st["v"][:n].double()
    return q, kc, vc


if __name__ == "__main__":
    r = random.Random(0)
    for c in listed() + [draw(r) for _ in range(6)]:
        w = work(c)
        print("%-90s %10.1f MB %10.3f GFLOP" % (c, w["bytes"] / 1e6, w["flops"] / 1e9))

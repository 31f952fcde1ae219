"""The bounds of the 8-bit decode's tests see what they are for: mistakes planted in the
64-bit oracle break them (no GPU needed)."""
import numpy as np
import pytest

import q4_oracle as Q4
import q8_oracle as Q
from test_q8_gpu import decode_bound, decode_want


def inputs(dtype, n=700, hq=4, hkv=2, d=64, block=16):
    rng = np.random.default_rng(3)
    pages = -(-n // block)
    kc, vc = (Q.encode(np.clip(rng.standard_normal((pages, hkv, block, d)) * 16, -448, 448))
              for _ in range(2))
    ks, vs = (np.exp2(rng.integers(-2, 3, (pages, hkv))).astype(np.float32) / 32 for _ in range(2))
    q = rng.standard_normal((1, hq, d)).astype(np.float32)
    if dtype == "bf16":
        q = Q4.bf16_value(Q4.bf16_bits(q))
    return q, kc, ks, vc, vs, np.arange(pages, dtype=np.int32)[None], [n], 0.125, block


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["nothing", "lost key", "key behind the end", "lost tile",
                                  "neighbour's V scale", "K scale halved", "coarse queries",
                                  "coarse weights", "one V code off", "scale off"])
def test_bounds(dtype, what):
    q, kc, ks, vc, vs, table, lens, scale, block = inputs(dtype)
    want, mass, reach = decode_want(q, kc, ks, vc, vs, table, lens, scale, block)
    bound = decode_bound(want, mass, reach, lens, dtype)
    kc = kc.copy()
    if what in ("lost key", "one V code off", "neighbour's V scale"):
        kc[3, :, 5] = Q.encode(np.clip(q[0, ::2] * 60, -448, 448))
        ks = ks.copy()
        ks[3] = 1 / 8
        want, mass, reach = decode_want(q, kc, ks, vc, vs, table, lens, scale, block)
        bound = decode_bound(want, mass, reach, lens, dtype)
    if what == "lost key":
        kc[3, :, 5] = Q.encode(-np.clip(q[0, ::2] * 60, -448, 448))
    elif what == "key behind the end":
        lens = [704]
    elif what == "lost tile":
        lens = [lens[0] - 48]
    elif what == "neighbour's V scale":
        vs = vs.copy()
        vs[3] = vs[3] * 2
    elif what == "K scale halved":
        ks = ks.copy()
        ks[7] /= 2
    elif what == "coarse queries":
        q = Q.VALUES[Q.encode(q * 64)] / 64
    elif what == "one V code off":
        vc = vc.copy()
        vc[3, :, 5] ^= 1
    elif what == "scale off":
        scale *= 1 + 2.0 ** -6
    if what == "coarse weights":  # 4 bits, as e4m3 weights would have
        got = np.zeros_like(want)
        k = Q.values(kc, ks).transpose(0, 2, 1, 3).reshape(-1, 2, 64)[:lens[0]]
        v = Q.values(vc, vs).transpose(0, 2, 1, 3).reshape(-1, 2, 64)[:lens[0]]
        for h in range(4):
            s = k[:, h // 2] @ q[0, h] * scale
            p = np.exp(s - s.max())
            got[0, h] = (Q.VALUES[Q.encode(p * 448)] / 448) @ v[:, h // 2] / p.sum()
    else:
        got = decode_want(q, kc, ks, vc, vs, table, lens, scale, block)[0]
    out = Q4.bf16_value(Q4.bf16_bits(got.astype(np.float32))) if dtype == "bf16" else got
    inside = np.all(np.abs(out - want) <= bound)
    assert inside == (what == "nothing")

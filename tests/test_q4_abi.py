"""Host-side checks of the calls on 4-bit pools and of cache compaction: what
they refuse before any CUDA call (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_70_gb300 as pkv
from paged_kv_cache_70_gb300 import build

import q4_oracle as Q


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pkv.load_library()


def geom(hq=16, hkv=8, d=128, block=16, blocks=100, dtype=pkv.PKV_Q4):
    return ctypes.byref(pkv.Geom(hq, hkv, d, block, blocks, dtype))


P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(264)  # not 16-byte aligned


def test_write_and_read_refusals(lib):
    w, r = lib.paged_kv_write_q4, lib.paged_kv_read_q4
    assert w(P, P, 1, P, 1, P, P, None, None) == -1
    assert w(P, P, 1, P, 1, P, P, geom(dtype=pkv.PKV_BF16), None) == -1  # not a 4-bit pool
    assert w(P, P, 2, P, 1, P, P, geom(), None) == -1  # rows are fp32 or bf16
    assert w(P, P, 1, P, -1, P, P, geom(), None) == -1
    assert w(P, P, 1, P, 1 << 40, P, P, geom(), None) == -1
    assert w(None, P, 1, P, 1, P, P, geom(), None) == -1
    assert w(P, P, 1, None, 1, P, P, geom(), None) == -1
    assert w(ODD, P, 1, P, 1, P, P, geom(), None) == -1
    assert w(P, P, 1, P, 1, P, ODD, geom(), None) == -1
    assert w(P, P, 1, P, 1, P, P, geom(d=96), None) == -2
    assert w(P, P, 1, P, 1, P, P, geom(block=256, blocks=1 << 24), None) == -2  # slots > int32
    assert w(None, None, 1, None, 0, None, None, geom(), None) == 0
    assert r(P, P, P, 1, P, P, 1, None, None) == -1
    assert r(P, P, P, 1, P, None, 1, geom(), None) == -1
    assert r(P, P, P, 1, P, P, 2, geom(), None) == -1
    assert r(P, P, P, 1, ODD, P, 1, geom(), None) == -1
    assert r(P, P, P, 1, P, P, 1, geom(d=32), None) == -2
    assert r(None, None, None, 0, None, None, 1, geom(), None) == 0


def test_decode_refusals(lib):
    f = lib.paged_decode_q4
    assert f(P, 1, P, P, P, 4, P, 2, 1.0, P, P, 1 << 40, None, None) == -1
    assert f(P, 1, P, P, P, 4, P, 2, 1.0, P, P, 1 << 40, geom(dtype=pkv.PKV_F32), None) == -1
    assert f(P, 2, P, P, P, 4, P, 2, 1.0, P, P, 1 << 40, geom(), None) == -1
    assert f(P, 1, P, P, P, 4, P, -1, 1.0, P, P, 1 << 40, geom(), None) == -1
    assert f(P, 1, P, P, P, -4, P, 2, 1.0, P, P, 1 << 40, geom(), None) == -1
    assert f(P, 1, P, P, P, 4, None, 2, 1.0, P, P, 1 << 40, geom(), None) == -1
    assert f(ODD, 1, P, P, P, 4, P, 2, 1.0, P, P, 1 << 40, geom(), None) == -1
    assert f(P, 1, P, P, P, 4, P, 2, 1.0, P, P, 1 << 40, geom(hq=12, hkv=8), None) == -1
    assert f(P, 1, P, P, P, 4, P, 2, 1.0, P, P, 1 << 40, geom(d=256), None) == -2
    assert f(None, 1, None, None, None, 4, None, 0, 1.0, None, None, 0, geom(), None) == 0
    assert lib.paged_decode_q4_workspace_size(2, 1, None) == 0
    assert lib.paged_decode_q4_workspace_size(-1, 1, geom()) == 0
    assert lib.paged_decode_q4_workspace_size(2, 2, geom()) == 0


def test_compact_refusals(lib):
    f = lib.paged_kv_compact
    for dtype in (pkv.PKV_F32, pkv.PKV_BF16, pkv.PKV_Q4):
        g = geom(dtype=dtype)
        assert f(P, P, P, 4, P, P, 3, P, -1, P, g, None) == -1
        assert f(P, P, P, 4, P, P, -3, P, 2, P, g, None) == -1
        assert f(P, P, P, -4, P, P, 3, P, 2, P, g, None) == -1
        assert f(P, P, P, 4, P, None, 3, P, 2, P, g, None) == -1
        assert f(P, P, P, 4, P, P, 3, None, 2, P, g, None) == -1
        assert f(P, P, None, 4, P, P, 3, P, 2, P, g, None) == -1
        assert f(P, None, P, 4, P, P, 3, P, 2, P, g, None) == -1
        assert f(P, P, P, 4, P, P, 3, P, 70000, P, g, None) == -2
        assert f(P, P, P, 1 << 28, P, P, 3, P, 2, P, g, None) == -2  # positions > int32
        assert f(None, None, None, 4, None, None, 0, None, 0, None, g, None) == 0
        # the new lengths share a part of the starts (the whole of them is a call)
        for by in (4, -4, 36):
            at, new = ctypes.c_void_p(1024), ctypes.c_void_p(1024 + by)
            assert f(P, P, P, 4, at, P, 3, P, 10, new, g, None) == -1
        # pools that share their rows, or some
        assert f(P, P, P, 4, P, P, 3, P, 2, P, g, None) == -1
        assert f(P, ctypes.c_void_p(4096), P, 4, P, P, 3, P, 2, P, g, None) == -1
    assert f(P, P, P, 4, P, P, 3, P, 2, P, None, None) == -1
    assert f(P, P, P, 4, P, P, 3, P, 2, P, geom(dtype=7), None) == -1
    assert f(ODD, P, P, 4, P, P, 3, P, 2, P, geom(), None) == -1
    assert f(P, P, P, 4, P, P, 3, P, 2, P, geom(d=96), None) == -2


def test_other_calls_refuse_4_bit_pools(lib):
    assert lib.paged_kv_write(P, P, 1, P, 1, P, P, geom(), None) == -1
    assert lib.paged_decode(P, P, P, P, 4, P, 2, 1.0, P, P, 1 << 40, geom(), None) == -1
    assert lib.paged_copy_blocks(P, P, P, P, 1, geom(), None) == -1


def test_binding_shapes():
    assert pkv.q4_cache_shape(7, 16, 8, 128) == (7, 8, 16, 80)
    assert pkv.q4_cache_shape(7, 16, 2, 64) == (7, 2, 16, 40)
    with pytest.raises(ValueError):
        pkv.q4_cache_shape(7, 16, 8, 96)
    g = pkv.q4_geom_of(torch.zeros(7, 8, 16, 80, dtype=torch.uint8), 32)
    assert (g.num_heads, g.num_kv_heads, g.head_dim, g.block_size, g.num_blocks, g.dtype) == \
        (32, 8, 128, 16, 7, pkv.PKV_Q4)
    with pytest.raises(ValueError):
        pkv.q4_geom_of(torch.zeros(7, 8, 16, 64, dtype=torch.uint8), 32)
    with pytest.raises(ValueError):
        pkv.q4_geom_of(torch.zeros(7, 8, 16, 80, dtype=torch.int8), 32)
    with pytest.raises(ValueError):  # not on a GPU
        pkv.paged_kv_compact(torch.zeros(2, 4, 1, 64), torch.zeros(2, 4, 1, 64),
                             torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                             torch.zeros(2, dtype=torch.int32))


def test_oracle_rows_hold_their_values():
    """The numpy format: a value is within half a step of what its row holds, or
    what the two bf16 constants leave at the ends of the range."""
    rng = np.random.default_rng(3)
    for d in (64, 128):
        x = rng.standard_normal((50, 3, d)).astype(np.float32)
        x[0] = 0
        x[1] = 1.7
        x[2] += 40
        got = Q.values(Q.quantise(x))
        u, s, z = Q.parts(Q.quantise(x))
        g = x.reshape(50, 3, d // 32, 32)
        ends = np.repeat(np.abs(g.min(-1)) + np.abs(g.max(-1)), 32, -1)
        assert np.all(np.abs(got - x) <= 0.5 * s * (1 + 2.0 ** -20) + 2.0 ** -8 * ends)
        assert np.all(Q.values(Q.quantise(np.float32(got)))[0] == 0)

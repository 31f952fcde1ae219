"""Sizes at which the calls on 4-bit pools and the compaction count past their integers:
refused before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

import paged_kv_cache_70_gb300 as pkv
from paged_kv_cache_70_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pkv.load_library()


P = ctypes.c_void_p(256)


@pytest.mark.parametrize("hkv,d", [((1 << 23) + 1, 128), (1 << 27, 128), ((1 << 24) + 1, 64),
                                   ((1 << 31) - 1, 64)])
def test_rows_that_32_bits_do_not_count(lib, hkv, d):
    g = ctypes.byref(pkv.Geom(hkv, hkv, d, 1, 1, pkv.PKV_Q4))
    assert lib.paged_kv_write_q4(P, P, 1, P, 1, P, P, g, None) == -2
    assert lib.paged_kv_read_q4(P, P, P, 1, P, P, 1, g, None) == -2


def meta(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_the_binding_cuts_no_size_off():
    """Sizes of 2^32 and some: ctypes passes an int32 their low bits."""
    q4 = meta(4, 2, 16, 80, dtype=torch.uint8)
    with pytest.raises(ValueError, match="2\\^31"):
        pkv.paged_kv_compact(q4, q4, meta(1, 4), meta(2**32 + 5), meta(2))
    with pytest.raises(ValueError, match="2\\^31"):
        pkv.paged_kv_compact(q4, q4, meta(2**32 + 1, 4), meta(5), meta(2**32 + 2))
    with pytest.raises(ValueError, match="2\\^31"):
        pkv.paged_kv_compact(q4, q4, meta(1, 2**32 + 4), meta(3), meta(2))
    with pytest.raises(ValueError, match="2\\^31"):
        pkv.paged_decode_q4(meta(1, 2, 128, dtype=torch.bfloat16), q4, q4, meta(1, 2**32 + 4),
                            meta(1))
    for shape in ((1, 1, 2**32 + 16, 80), (1, 2**32 + 2, 1, 80)):
        wide = meta(*shape, dtype=torch.uint8)
        with pytest.raises(ValueError, match="32-bit"):
            pkv.paged_kv_compact(wide, wide, meta(1, 4), meta(3), meta(2))
        with pytest.raises(ValueError, match="32-bit"):
            pkv.q4_geom_of(wide, shape[1])
    wide = meta(1, 2**32 + 16, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="32-bit"):
        pkv.paged_kv_compact(wide, wide, meta(1, 4), meta(3), meta(2))

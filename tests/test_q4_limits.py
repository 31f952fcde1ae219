"""Sizes at which the calls on 4-bit pools and the compaction count past their integers:
refused before any CUDA call (no GPU needed)."""
import ctypes

import pytest

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

"""paged_decode_q8 over a block table of no columns (what a batch of sequences without keys has):
rows of zeros, as for lengths of 0.  torch gives such a table no address."""
import ctypes

import pytest
import torch

import paged_kv_cache_70_gb300 as pkv
from paged_kv_cache_70_gb300 import build


def test_a_table_of_no_columns_needs_no_address():
    build.build()
    lib = pkv.load_library()
    p = ctypes.c_void_p(256)
    g = ctypes.byref(pkv.Geom(16, 8, 128, 16, 100, pkv.PKV_Q8))
    # (without a workspace: refused, but for that, or where there is no device)
    for width, table, invalid in ((0, None, False), (0, p, False), (4, None, True)):
        st = lib.paged_decode_q8(p, 1, p, p, p, p, table, width, p, 2, 1.0, p, None, 0, g, None)
        assert st != 0 and (st == -1) == invalid, (width, table, st)


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 5, 150, 500])
@pytest.mark.parametrize("hq,hkv,d,dtype", [(16, 8, 128, torch.bfloat16), (4, 1, 64, torch.float32),
                                            (64, 2, 128, torch.bfloat16)])
def test_sequences_without_a_page_give_zeros(batch, hq, hkv, d, dtype):
    i32 = dict(dtype=torch.int32, device="cuda")
    kc = torch.full((3, hkv, 16, d), float("nan"), device="cuda").to(torch.float8_e4m3fn)
    s = torch.full((3, hkv), float("nan"), device="cuda")
    q = torch.randn(batch, hq, d, device="cuda").to(dtype)
    for lens, flags in ((torch.zeros(batch, **i32), 0),
                        (torch.full((batch,), 7, **i32), pkv.PKV_FLAG_BAD_LENGTH)):
        out = torch.full_like(q, float("nan"))
        pkv.paged_decode_q8(q, kc, kc, s, s, torch.empty(batch, 0, **i32), lens, out=out)
        assert not out.any()
        assert pkv.paged_error_flags() == flags

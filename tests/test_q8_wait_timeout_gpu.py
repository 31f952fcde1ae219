"""An 8-bit decode whose pipeline wait runs out, on a test-only build of its split
kernel: the producers issue no copy and every wait gives up after 1 ms.  The call must
return, the kernels must finish, and that build's device error word must carry
PKV_FLAG_TIMEOUT, whether the sequences are split or taken whole.  The default library
is not changed."""
import ctypes

import pytest
import torch

import paged_kv_cache_70_gb300 as pkv
from paged_kv_cache_70_gb300 import build as B

pytestmark = pytest.mark.gpu

DEFINES = ("-DPKV_WAIT_LIMIT_NS=1000000ull", "-DPKV_TEST_SPLIT_PRODUCER_IDLE")


@pytest.fixture(scope="module")
def timeout_lib():
    return pkv.load_library(B.build_variant("test_q8_wait_timeout", DEFINES, ("q8_decode.cu",)))


def _flags(lib):
    v = ctypes.c_uint32(0)
    assert lib.paged_error_flags(ctypes.byref(v), 1) == 0
    return v.value


@pytest.mark.parametrize("width", [25000, 125, 7])
@pytest.mark.parametrize("hq,hkv,dtype", [(16, 8, torch.bfloat16), (4, 2, torch.bfloat16),
                                          (8, 1, torch.bfloat16), (4, 2, torch.float32)])
def test_decode_wait_timeout_sets_flag_and_returns(timeout_lib, hq, hkv, dtype, width):
    lib = timeout_lib
    lens = torch.tensor([100, 37, min(500, width * 16), width * 16], dtype=torch.int32, device="cuda")
    kc = torch.zeros(pkv.q8_cache_shape(200, 16, hkv, 128), device="cuda").to(torch.float8_e4m3fn)
    sc = torch.ones(200, hkv, device="cuda")
    table = (torch.arange(4 * width, dtype=torch.int32, device="cuda") % 200).reshape(4, width)
    q = torch.randn(4, hq, 128, device="cuda").to(dtype)
    out = torch.empty_like(q)
    g = ctypes.byref(pkv.q8_geom_of(kc, hq))
    code = pkv.PKV_BF16 if dtype == torch.bfloat16 else pkv.PKV_F32
    need = lib.paged_decode_q8_workspace_size(4, code, g)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    _flags(lib)
    pkv.paged_error_flags()
    st = lib.paged_decode_q8(q.data_ptr(), code, kc.data_ptr(), kc.data_ptr(), sc.data_ptr(),
                             sc.data_ptr(), table.data_ptr(), width, lens.data_ptr(), 4, 0.1,
                             out.data_ptr(), ws.data_ptr(), need, g,
                             torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()  # every wait gave up after 1 ms
    assert _flags(lib) & pkv.PKV_FLAG_TIMEOUT
    assert pkv.paged_error_flags() == 0  # the default library saw nothing
    got = pkv.paged_decode_q8(q, kc, kc, sc, sc, table, lens)  # and still works: rows of zeros
    assert not got.any()

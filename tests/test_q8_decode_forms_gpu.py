"""Which form of the 8-bit decode a call takes: a CTA or a cluster of CTAs for each sequence, in
one kernel, or shares of all tiles and a second kernel that merges them.  Every form is right for
every call, so that no output shows a plan that fell back to the third."""
import json

import pytest
import torch

import paged_kv_cache_70_gb300 as pkv

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def inputs(batch, keys, hq, hkv, d, block, dtype):
    width = -(-keys // block)
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = torch.randn(width, hkv, block, d, device="cuda").to(torch.float8_e4m3fn)
    scale = torch.ones(width, hkv, device="cuda")
    table = torch.arange(width, **i32).repeat(batch, 1)
    return (torch.randn(batch, hq, d, device="cuda").to(dtype), pool, pool, scale, scale, table,
            torch.full((batch,), keys, **i32))


# near sizes that the rule's comment gives figures for, of the form chosen there
FORMS = [  # (sequences, keys, Hq, Hkv, d, B, type), CTAs of a sequence and its heads (0: split)
    ((1, 20, 16, 8, 128, 16, BF16), 1),
    ((60, 190, 16, 8, 128, 16, BF16), 1),
    ((3, 70, 2, 1, 64, 32, F32), 1),
    ((1, 1000, 16, 8, 128, 16, BF16), 8),
    ((4, 2000, 16, 8, 128, 16, BF16), 4),
    ((16, 1000, 16, 8, 128, 16, BF16), 2),
    ((1, 7777, 32, 4, 64, 16, BF16), 16),
    ((16, 1000, 32, 4, 64, 16, BF16), 2),
    ((30, 1024, 16, 8, 128, 64, BF16), 2),
    ((2, 800, 64, 1, 64, 8, F32), 8),
    ((1, 8000, 16, 8, 128, 16, BF16), 0),
    ((1, 16000, 32, 4, 64, 16, BF16), 0),
    ((64, 4096, 16, 8, 128, 16, BF16), 0),
    ((300, 100, 16, 8, 128, 16, BF16), 0),
]


@pytest.mark.parametrize("sizes,ctas", FORMS)
def test_only_a_split_needs_the_workspace(sizes, ctas):
    args = inputs(*sizes)
    need = pkv.paged_decode_q8_workspace_size(sizes[0], sizes[2], sizes[6], args[1])
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    pkv.paged_decode_q8(*args, workspace=ws)
    assert bool((ws == 0xA5).all()) == (ctas > 0)


def test_kernels_and_grids(tmp_path):
    """The kernels of each call as the profiler names them, and their CTAs per sequence."""
    calls = [(sizes, ctas, inputs(*sizes)) for sizes, ctas in FORMS]
    for _ in range(2):  # (the profiler's first session may see nothing)
        torch.cuda.synchronize()
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
            for _, _, args in calls:
                pkv.paged_decode_q8(*args)
            torch.cuda.synchronize()
    path = str(tmp_path / "trace.json")
    prof.export_chrome_trace(path)
    with open(path) as f:
        kernels = sorted((e for e in json.load(f)["traceEvents"] if e.get("cat") == "kernel"),
                         key=lambda e: e["ts"])
    if not kernels:
        pytest.skip("the profiler sees no kernels here")
    for sizes, ctas, _ in calls:
        k = kernels.pop(0)
        mode = 2 if ctas > 1 else ctas
        assert "q8_split_kernel" in k["name"] and f"Mode){mode}" in k["name"], (sizes, k["name"])
        if ctas:
            assert k["args"]["grid"][0] == sizes[0] * ctas, (sizes, k["args"]["grid"])
        else:
            assert "split_combine_kernel" in kernels.pop(0)["name"], sizes
    assert not kernels

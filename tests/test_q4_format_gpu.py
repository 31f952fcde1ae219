"""The stored bytes of 4-bit rows over every quotient by 15 and every reciprocal that
the format can meet: the kernel forms both from an approximation and one step with the
exact remainder, the format says one rounding of the exact value."""
import numpy as np
import pytest
import torch

import paged_kv_cache_70_gb300 as pkv
import q4_oracle as Q
from gpu_helpers import to_dev, to_host

pytestmark = pytest.mark.gpu

HKV, D, BLOCK = 8, 128, 64
NG = D // 32


def written(x):
    """The rows [tokens, Hkv, 5 D / 8] that fp32 CUDA values [tokens, Hkv, D] are stored as."""
    n = x.shape[0]
    kc, vc = (torch.zeros(pkv.q4_cache_shape(-(-n // BLOCK), BLOCK, HKV, D), dtype=torch.uint8,
                          device="cuda") for _ in range(2))
    pkv.paged_kv_write_q4(x, x, torch.arange(n, dtype=torch.int32, device="cuda"), kc, vc)
    assert torch.equal(kc, vc) and pkv.paged_error_flags() == 0
    return kc.transpose(1, 2).reshape(-1, HKV, 5 * D // 8)[:n]


@pytest.mark.parametrize("exponent", [0, -124, -123, -122, 127])
def test_every_quotient_by_15(exponent):
    """Groups of 0 and one value x, for every x of a binade: 1 .. 2 stands for all others
    but those beside 15 * 2^-126, below which a scale is stored as 0, and the last."""
    bits = np.arange(1 << 23, dtype=np.uint32) | np.uint32((exponent + 127) << 23)
    hi = bits.view(np.float32)
    with np.errstate(all="ignore"):
        sb = Q.bf16_bits(hi / np.float32(15))
        sb = np.where(Q.bf16_value(sb) < np.float32(2.0 ** -126), np.uint16(0), sb)
        s = Q.bf16_value(sb)
        zb = Q.bf16_bits((np.float32(0) + np.float32(0.5) * hi) + np.float32(0.5) * s)
    want = np.stack((sb, zb), -1)
    tokens = len(hi) // (HKV * NG)
    x = torch.zeros(tokens, HKV, NG, 32, device="cuda")
    x[..., 17] = to_dev(hi.reshape(tokens, HKV, NG))
    got = to_host(written(x.reshape(tokens, HKV, D))[..., D // 2:])
    got = np.ascontiguousarray(got).view(np.uint16).reshape(-1, 2)
    assert np.array_equal(got, want)


def test_every_reciprocal():
    """For every scale s, a group -8 s .. 7 s (offset 0) of the values at and beside the
    middles between two codes, where the last bit of 1 / s decides."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    s = Q.bf16_value(bits)
    with np.errstate(all="ignore"):
        s = s[(s >= np.float32(2.0 ** -126)) & np.isfinite(s * np.float32(15))]
    assert len(s) > 30000
    x = np.zeros((len(s), 2, 32), np.float32)
    x[:, :, 0], x[:, :, 1] = -8 * s[:, None], 7 * s[:, None]
    for i in range(15):
        mid = s * np.float32(i - 7.5)
        at = 2 + 3 * (i // 2)
        x[:, i % 2, at] = mid
        x[:, i % 2, at + 1] = np.nextafter(mid, np.float32(np.inf))
        x[:, i % 2, at + 2] = np.nextafter(mid, np.float32(-np.inf))
    rows = x.reshape(-1, 32)
    pad = -len(rows) % (HKV * NG)
    rows = np.concatenate([rows, np.zeros((pad, 32), np.float32)]).reshape(-1, HKV, D)
    want = Q.quantise(rows)
    sz = np.ascontiguousarray(want[..., D // 2:]).view(np.uint16).reshape(-1, 2)
    assert np.array_equal(Q.bf16_value(sz[:len(s) * 2:2, 0]), s) and not sz[:, 1].any()
    assert np.array_equal(to_host(written(to_dev(rows))), want)

"""The 4-bit decode against bounds from the roundings it makes (q4_bounds)."""
import numpy as np
import pytest

import paged_kv_cache_70_gb300 as pkv
import q4_bounds as B
from gpu_helpers import to_dev, widen
from test_q4_bounds import competing

pytestmark = pytest.mark.gpu


def check(q, kc, vc, table, lens, scale):
    out = widen(pkv.paged_decode_q4(to_dev(q), to_dev(kc), to_dev(vc), to_dev(table),
                                    to_dev(np.asarray(lens, np.int32)), scale=scale))
    want, tol, rms = B.decode(q, kc, vc, table, lens, scale)
    err = np.abs(out - want)
    worst = np.max(err / np.maximum(tol, 1e-300))
    assert np.all(err <= tol), f"{worst:.3g} of the bound"
    mean = lambda x: np.sqrt(np.mean(x ** 2))
    assert mean(err) <= mean(rms), f"{mean(err) / mean(rms):.3g} of the mean bound"
    assert pkv.paged_error_flags() == 0


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (8, 2, 128), (16, 2, 128), (4, 2, 64), (8, 2, 64),
                                      (16, 2, 64)])
@pytest.mark.parametrize("outliers", [False, True])
def test_few_keys_with_large_scores(hq, hkv, d, outliers):
    case = competing(hq, hkv, d, 48, 3, 5, outliers)
    check(*case, scale=3.0)

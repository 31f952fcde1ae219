"""Host-side checks of the cache write with the position rotation and of the calls on 8-bit
pools: what they refuse before any CUDA call (no GPU needed); the numpy model of the format."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_70_gb300 as pkv
from paged_kv_cache_70_gb300 import build

import q8_oracle as Q


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pkv.load_library()


def geom(hq=16, hkv=8, d=128, block=16, blocks=100, dtype=pkv.PKV_Q8):
    return ctypes.byref(pkv.Geom(hq, hkv, d, block, blocks, dtype))


P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(264)  # not 16-byte aligned


def rope(**kw):
    f = dict(cos_sin=P, num_positions=100, rotary_dim=128, interleaved=0, positions=None, q=None,
             q_stride=0, q_out=None, q_out_stride=0)
    f.update(kw)
    return ctypes.byref(pkv.Rope(**f))


def write(lib, func, k=P, ks=1024, v=P, vs=1024, dtype=1, r=None, table=P, width=4, rows=2,
          seq=P, pos=P, n=3, kc=P, vc=P, k_scale=P, v_scale=P, g=None):
    if func == "paged_kv_write_rope":
        g = geom(dtype=pkv.PKV_BF16) if g is None else g
        return lib.paged_kv_write_rope(k, ks, v, vs, dtype, r, table, width, rows, seq, pos, n,
                                       None, kc, vc, g, None)
    g = geom() if g is None else g
    return lib.paged_kv_write_q8(k, ks, v, vs, dtype, r, table, width, rows, seq, pos, n, kc, vc,
                                 k_scale, v_scale, g, None)


@pytest.mark.parametrize("func", ["paged_kv_write_rope", "paged_kv_write_q8"])
def test_write_refusals(lib, func):
    def f(**kw):
        kw.setdefault("r", rope())
        return write(lib, func, **kw)

    own = pkv.PKV_BF16 if func == "paged_kv_write_rope" else pkv.PKV_Q8
    for bad in (dict(k=None), dict(v=None), dict(seq=None), dict(pos=None), dict(kc=None),
                dict(vc=None), dict(table=None), dict(k=ODD), dict(v=ODD), dict(kc=ODD),
                dict(vc=ODD), dict(dtype=2), dict(dtype=3), dict(n=-1), dict(width=-1),
                dict(rows=-1), dict(ks=1020), dict(vs=-1024), dict(ks=1026, dtype=0),
                dict(g=geom(dtype=7)), dict(g=geom(hq=12, dtype=own)),
                dict(g=geom(dtype=pkv.PKV_Q4))):
        assert f(**bad) == -1, bad
    for bad in (dict(cos_sin=None), dict(cos_sin=ODD), dict(rotary_dim=0), dict(rotary_dim=24),
                dict(rotary_dim=144), dict(rotary_dim=-16), dict(num_positions=-1),
                dict(q=ODD, q_out=P, q_stride=2048, q_out_stride=2048),
                dict(q=P, q_out=None, q_stride=2048, q_out_stride=2048),
                dict(q=P, q_out=P, q_stride=2049, q_out_stride=2048),
                dict(q=P, q_out=P, q_stride=2048, q_out_stride=1024),
                dict(q=P, q_out=P, q_stride=-2048, q_out_stride=2048)):
        assert f(r=rope(**bad)) == -1, bad
    for bad in (dict(g=geom(d=96, dtype=own)), dict(g=geom(block=256, blocks=1 << 24, dtype=own)),
                dict(g=geom(hq=1 << 24, hkv=1 << 24, dtype=own)), dict(n=1 << 40)):
        assert f(**bad) == -2, bad
    assert f(n=0, k=None, v=None, seq=None, pos=None, kc=None, vc=None, table=None) == 0
    # a rotary_dim past the heads is refused for no tokens as well
    assert f(n=0, r=rope(rotary_dim=256)) == -1


@pytest.mark.parametrize("func", ["paged_kv_write_rope", "paged_kv_write_q8"])
def test_queries_in_place_keep_their_stride(lib, func):
    for q_stride, out_stride in ((4096, 2048), (2048, 4096), (0, 2048)):
        r = rope(q=P, q_out=P, q_stride=q_stride, q_out_stride=out_stride)
        assert write(lib, func, r=r, n=3) == -1


def test_write_rope_needs_a_rotation_and_write_q8_its_scales(lib):
    assert write(lib, "paged_kv_write_rope", r=None) == -1
    assert write(lib, "paged_kv_write_q8", k_scale=None) == -1
    assert write(lib, "paged_kv_write_q8", v_scale=None) == -1
    assert lib.paged_kv_write_q8(P, 1024, P, 1024, 1, None, P, 4, 2, P, P, 3, P, P, P, P, None,
                                 None) == -1
    assert lib.paged_kv_write_rope(P, 1024, P, 1024, 1, rope(), P, 4, 2, P, P, 3, None, P, P, None,
                                   None) == -1
    assert write(lib, "paged_kv_write_q8", g=geom(dtype=pkv.PKV_BF16)) == -1
    assert write(lib, "paged_kv_write_rope", r=rope(), g=geom(dtype=pkv.PKV_Q8)) == -1


def test_read_refusals(lib):
    f = lib.paged_kv_read_q8
    assert f(P, P, P, P, P, 1, P, P, 1, None, None) == -1
    assert f(P, P, P, P, P, 1, P, P, 1, geom(dtype=pkv.PKV_BF16), None) == -1
    assert f(P, P, P, P, P, 1, P, P, 3, geom(), None) == -1
    assert f(P, P, P, P, P, -1, P, P, 1, geom(), None) == -1
    for i in range(8):
        a = [P, P, P, P, P, 1, P, P, 1]
        if i == 5:
            continue
        a[i] = None
        assert f(*a, geom(), None) == -1, i
    for i in (0, 1, 6, 7):
        a = [P, P, P, P, P, 1, P, P, 1]
        a[i] = ODD
        assert f(*a, geom(), None) == -1, i
    assert f(P, P, P, P, P, 1, P, P, 1, geom(d=32), None) == -2
    assert f(P, P, P, P, P, 1 << 40, P, P, 1, geom(), None) == -2
    assert f(None, None, None, None, None, 0, None, None, 1, geom(), None) == 0


def test_decode_refusals(lib):
    f = lib.paged_decode_q8

    def call(g=None, **kw):
        a = dict(q=P, qd=1, k=P, v=P, ks=P, vs=P, t=P, w=4, l=P, b=2, s=1.0, o=P, ws=P, n=1 << 40)
        a.update(kw)
        return f(*a.values(), geom() if g is None else g, None)

    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(ks=None), dict(vs=None),
                dict(t=None), dict(l=None), dict(o=None), dict(q=ODD), dict(k=ODD), dict(v=ODD),
                dict(o=ODD), dict(qd=2), dict(qd=3), dict(b=-1), dict(w=-1),
                dict(g=geom(dtype=pkv.PKV_Q4)), dict(g=geom(hq=12))):
        assert call(**bad) == -1, bad
    assert f(P, 1, P, P, P, P, P, 4, P, 2, 1.0, P, P, 1 << 40, None, None) == -1
    assert call(g=geom(d=256)) == -2
    assert call(q=None, k=None, v=None, ks=None, vs=None, t=None, l=None, o=None, ws=None, n=0,
                b=0) == 0
    assert lib.paged_decode_q8_workspace_size(2, 1, None) == 0
    assert lib.paged_decode_q8_workspace_size(-1, 1, geom()) == 0
    assert lib.paged_decode_q8_workspace_size(2, 2, geom()) == 0


def test_other_calls_refuse_8_bit_pools(lib):
    assert lib.paged_kv_write(P, P, 1, P, 1, P, P, geom(), None) == -1
    assert lib.paged_decode(P, P, P, P, 4, P, 2, 1.0, P, P, 1 << 40, geom(), None) == -1
    assert lib.paged_decode_q4(P, 1, P, P, P, 4, P, 2, 1.0, P, P, 1 << 40, geom(), None) == -1
    assert lib.paged_copy_blocks(P, P, P, P, 1, geom(), None) == -1
    assert lib.paged_kv_compact(P, ctypes.c_void_p(1 << 30), P, 4, None, P, 1, P, 1, None, geom(),
                                None) == -1


def test_binding_shapes():
    assert pkv.q8_cache_shape(7, 16, 8, 128) == (7, 8, 16, 128)
    with pytest.raises(ValueError):
        pkv.q8_cache_shape(7, 16, 8, 96)
    pool = torch.zeros(7, 8, 16, 128).to(torch.float8_e4m3fn)
    g = pkv.q8_geom_of(pool, 32)
    assert (g.num_heads, g.num_kv_heads, g.head_dim, g.block_size, g.num_blocks, g.dtype) == \
        (32, 8, 128, 16, 7, pkv.PKV_Q8)
    for bad in (torch.zeros(7, 8, 16, 128), torch.zeros(7, 8, 16, 96).to(torch.float8_e4m3fn),
                torch.zeros(7, 8, 128).to(torch.float8_e4m3fn)):
        with pytest.raises(ValueError):
            pkv.q8_geom_of(bad, 32)
    idx = torch.zeros(1, dtype=torch.int32)
    k, s = torch.zeros(1, 8, 128), torch.zeros(7, 8)
    with pytest.raises(ValueError):  # not on a GPU
        pkv.paged_kv_write_q8(k, k, idx[None], idx, idx, pool, pool.clone(), s, s.clone())
    with pytest.raises(ValueError):
        pkv.paged_kv_write_rope(k, k, None, idx[None], idx, idx, torch.zeros(7, 16, 8, 128),
                                torch.zeros(7, 16, 8, 128))
    with pytest.raises(TypeError):  # tokens do not move between pages
        pkv.paged_kv_compact(pool, pool.clone(), idx[None], idx, torch.zeros(2, dtype=torch.int32))


def test_oracle_codes_are_torchs():
    """The numpy table and rounding against torch's conversion, ties and subnormals among them."""
    x = np.concatenate((Q.VALUES[:127], Q._MIDS, -Q._MIDS, Q._MIDS * (1 + 2.0 ** -20),
                        np.random.default_rng(0).standard_normal(5000) * 50, [0.0, -0.0, np.nan]))
    x = x[~(np.abs(x) > 448)].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(Q.canon(Q.encode(x)), Q.canon(want))
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, Q.VALUES, equal_nan=True)


def test_oracle_write_keeps_what_the_header_promises():
    """Values within 2^-4 of themselves or 2^-10 of the scale, 2^-10 of it more per growth."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((23, 2, 64)) * np.exp2(rng.integers(-6, 7, (23, 1, 1)))).astype(np.float32)
    codes = rng.integers(0, 256, (2, 2, 16, 64), dtype=np.uint8)
    scale = np.full((2, 2), np.nan, np.float32)
    table = np.array([[1, 0]])
    grew = np.zeros((2, 2))
    for n in range(23):  # one token at a time
        was = scale.copy()
        Q.write(x[n:n + 1], table, [0], [n], codes, scale, [True])
        grew += (scale != was) & (n % 16 > 0) & (np.arange(2) == table[0, n // 16])[:, None]
    got = Q.values(codes, scale)
    for n in range(23):
        page = table[0, n // 16]
        s = scale[page].astype(np.float64)[:, None]
        err = np.abs(got[page, :, n % 16] - x[n])
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x[n]), 2.0 ** -10 * s)
                      + 2.0 ** -10 * s * grew[page][:, None])


def test_compiled_binding_fails_loudly_without_its_module(lib, monkeypatch, tmp_path):
    from paged_kv_cache_70_gb300 import _binding
    monkeypatch.setattr(_binding, "_native_module", None)
    monkeypatch.setattr(build, "binding_path", lambda: str(tmp_path / "missing.so"))
    with pytest.raises(RuntimeError, match="not found"):
        pkv.paged_decode_q8(*[torch.zeros(1)] * 7)


def test_compiled_binding_checks_its_arguments(lib):
    from paged_kv_cache_70_gb300 import _binding
    m = _binding._native()
    for f in (m.write, m.read_q8, m.decode_q8, m.bind):
        with pytest.raises(TypeError):
            f()
    t = torch.zeros(1)
    with pytest.raises(TypeError):  # no tensor
        m.decode_q8(None, *[t] * 9)
    with pytest.raises(ValueError):  # not on a GPU
        m.decode_q8(*[t] * 7, None, None, None)
    with pytest.raises(ValueError):
        m.read_q8(*[t] * 5, torch.float32, None, None)
    with pytest.raises(ValueError):
        m.bind(print, 0, 0, 0, 0, 0)

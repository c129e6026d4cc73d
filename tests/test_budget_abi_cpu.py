"""Refusals of the bounded-cache operators that need no GPU: every one is a
status before any CUDA call, and the rotary frequencies' host arithmetic."""
import ctypes as C
import math

import numpy as np
import pytest

F = C.c_float


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_236_gb300 import build
    build.build()
    import paged_kv_cache_236_gb300 as pkv
    return pkv.lib()


def rope(lib, T=3, NB=4, bs=16, Hq=8, Hkv=4, D=128, rot=128, amp=1.0, qs=0, ks=0, vs=0, dt=1, fp8=None):
    a = [None] * 9 + [T, NB, bs, Hq, Hkv, D, rot, 0, F(amp), qs, ks, vs, dt]
    if fp8 is None:
        return lib.paged_kv_write_rope(*a, None)
    return lib.paged_kv_write_rope_fp8(*a, F(fp8[0]), F(fp8[1]), None)


def test_rope_refusals(lib):
    assert rope(lib, T=0) == 0                                    # nothing to do
    assert rope(lib) == 1 and b"null" in lib.pkv_last_error()
    assert rope(lib, dt=2) == 2 and rope(lib, dt=7) == 2
    for bad in (dict(T=-1), dict(NB=0), dict(bs=0), dict(Hq=0), dict(Hkv=0), dict(D=0)):
        assert rope(lib, **bad) == 1, bad
    for rot in (0, 3, 130, -2):
        assert rope(lib, rot=rot) == 1 and b"rotary_dim" in lib.pkv_last_error()
    for amp in (0.0, -1.0, math.inf, math.nan):
        assert rope(lib, amp=amp) == 1 and b"amplitude" in lib.pkv_last_error()
    assert rope(lib, qs=8 * 128 - 1) == 1 and rope(lib, ks=100) == 1 and rope(lib, vs=100) == 1
    assert rope(lib, D=2048, rot=2) == 2
    assert rope(lib, T=0, fp8=(0.0, 1.0)) == 1 and rope(lib, T=0, fp8=(1.0, math.inf)) == 1
    assert rope(lib, T=0, fp8=(1.0, 1.0)) == 0


def scores(lib, B=1, T=1, Hq=8, Hkv=4, D=128, NB=4, bs=16, mb=2, rows=1, maxlen=32, scale=0.1, decay=1.0, dt=1,
           k_scale=None):
    a = [None] * 8 + [B, T, Hq, Hkv, D, NB, bs, mb, rows, maxlen, 0, F(scale), 1, F(decay)]
    if k_scale is None:
        return lib.paged_attention_scores(*a, None, 0, dt, None)
    return lib.paged_attention_scores_fp8kv(*a, F(k_scale), None, 0, None)


def test_scores_refusals(lib):
    assert scores(lib, B=0, T=0) == 0 and scores(lib, T=0) == 0
    assert scores(lib) == 1 and b"null" in lib.pkv_last_error()
    assert scores(lib, Hq=6) == 1 and b"num_kv_heads" in lib.pkv_last_error()
    assert scores(lib, D=96) == 2 and scores(lib, bs=24) == 2 and scores(lib, dt=2) == 2
    assert scores(lib, Hq=129, Hkv=1) == 2 and scores(lib, B=32769) == 2
    for bad in (dict(B=-1), dict(T=-1), dict(NB=0), dict(mb=0), dict(rows=0), dict(maxlen=0), dict(scale=0.0),
                dict(scale=math.nan), dict(decay=-0.5), dict(decay=math.inf), dict(decay=math.nan)):
        assert scores(lib, **bad) == 1, bad
    # row tiles of one sequence: 2 tokens each with 64 heads to a kv head
    wide = dict(Hq=64, Hkv=1, D=64, NB=1 << 20, mb=1 << 14, maxlen=1 << 20)
    assert scores(lib, T=(1 << 17) + 1, **wide) == 2 and b"query rows" in lib.pkv_last_error()
    assert scores(lib, T=1 << 17, **wide) == 1                          # allowed: stops at the null pointers
    assert scores(lib, T=(1 << 17) + 1, **{**wide, "maxlen": 4096}) == 1  # no sequence has so many
    assert scores(lib, T=(1 << 17) + 1, dt=0, **wide) == 1              # fp32 has no such limit
    assert scores(lib, k_scale=0.0) == 1 and scores(lib, D=64, k_scale=1.0) == 2


def test_scores_workspace_is_host_arithmetic(lib):
    size, least = lib.paged_attention_scores_workspace_size, lib.paged_attention_scores_workspace_min
    assert 0 < least(64, 64, 32, 8, 4096) <= size(64, 64, 32, 8, 4096)
    assert size(64, 64, 32, 0, 4096) == 0 and size(-1, 64, 32, 8, 4096) == 0 and size(1, 1, 1, 1, -1) == 0
    assert size(0, 0, 32, 8, 0) >= 0


def select(lib, B=1, Hkv=2, rows=1, maxlen=8, budget=4, sink=0, recent=0):
    return lib.paged_kv_select(None, None, None, None, B, Hkv, rows, maxlen, budget, sink, recent, None)


def test_select_refusals(lib):
    assert select(lib, B=0) == 0
    assert select(lib) == 1 and b"null" in lib.pkv_last_error()
    for bad in (dict(B=-1), dict(Hkv=0), dict(rows=0), dict(maxlen=0), dict(budget=0), dict(sink=-1),
                dict(recent=-1), dict(sink=3, recent=2), dict(sink=2**31 - 1, recent=2**31 - 1)):
        assert select(lib, **bad) == 1, bad
    assert select(lib, B=32769) == 2


def compact(lib, B=1, Hkv=2, D=64, NB=4, bs=16, mb=2, budget=4, rows=0, maxlen=0, dt=1, scores=None):
    return lib.paged_kv_compact(None, None, None, None, None, None, scores, B, Hkv, D, NB, bs, mb, budget, rows,
                                maxlen, dt, None)


def test_compact_refusals(lib):
    assert compact(lib, B=0) == 0
    assert compact(lib) == 1 and b"null" in lib.pkv_last_error()
    assert compact(lib, dt=3) == 2 and compact(lib, D=8, dt=2) == 2 and compact(lib, D=4, dt=1) == 2
    for bad in (dict(B=-1), dict(Hkv=0), dict(D=0), dict(NB=0), dict(bs=0), dict(mb=0), dict(budget=0),
                dict(scores=16, rows=0, maxlen=4), dict(scores=16, rows=4, maxlen=0)):
        assert compact(lib, **bad) == 1, bad


def test_rope_frequencies():
    import paged_kv_cache_236_gb300 as pkv
    f = lambda *a, **k: pkv.rope_frequencies(*a, device="cpu", **k).numpy()  # noqa: E731
    plain = f(64)
    assert plain.dtype == np.float64 and np.allclose(plain, 10000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-15)
    assert np.allclose(f(64, scaling="linear", factor=4.0), plain / 4)
    ntk = f(64, scaling="ntk", factor=8.0)
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(plain[-1] / 8, rel=1e-12)
    for kind, kw in (("bands", dict(low_freq_factor=1.0, high_freq_factor=4.0)), ("yarn", {})):
        g = f(128, 500000.0, scaling=kind, factor=8.0, original_max_position=8192, **kw)
        p = f(128, 500000.0)
        assert g[0] == p[0] and g[-1] == pytest.approx(p[-1] / 8, rel=1e-12)
        assert np.all(np.diff(g) < 0) and np.all(g <= p * (1 + 1e-15)) and np.all(g >= p / 8 * (1 - 1e-15))
    turns = 8192 * p / (2 * math.pi)
    g = f(128, 500000.0, scaling="bands", factor=8.0, original_max_position=8192)
    assert np.array_equal(g[turns > 4], p[turns > 4]) and np.allclose(g[turns < 1], p[turns < 1] / 8)
    assert pkv.rope_amplitude(1.0) == 1.0 and pkv.rope_amplitude(math.e ** 10) == pytest.approx(2.0)
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, factor=0.0),
                dict(rotary_dim=8, scaling="yarn"), dict(rotary_dim=8, scaling="other"),
                dict(rotary_dim=8, scaling="bands", original_max_position=10, low_freq_factor=4.0),
                dict(rotary_dim=2, scaling="ntk")):
        with pytest.raises(ValueError):
            pkv.rope_frequencies(device="cpu", **bad)

"""Refusals of the windowed attention, the normed writes and the pools with
block scales that need no GPU: every one is a status before any CUDA call.
And the host arithmetic of their workspaces."""
import ctypes as C
import math

import numpy as np
import pytest

F = C.c_float
WORKSPACE = 4  # PKV_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_236_gb300 import build
    build.build()
    import paged_kv_cache_236_gb300 as pkv
    return pkv.lib()


def window(lib, B=1, T=1, Hq=8, Hkv=4, D=128, NB=4, bs=16, mb=2, mql=0, scale=0.1, window=8, sink=0, dt=1, ptr=None,
           ws=None):
    return lib.paged_attention_window_forward(*[ptr] * 7, B, T, Hq, Hkv, D, NB, bs, mb, mql, F(scale), window, sink,
                                              ws, 0, dt, None)


def test_window_refusals(lib):
    assert window(lib, B=0, T=0) == 0 and window(lib, T=0) == 0
    assert window(lib) == 1 and b"null" in lib.pkv_last_error()
    for bad in (dict(window=0), dict(window=-1), dict(sink=-1)):
        assert window(lib, **bad) == 1 and b"window" in lib.pkv_last_error()
    assert window(lib, window=(1 << 30) + 1) == 2 and window(lib, sink=(1 << 30) + 1) == 2
    assert window(lib, T=0, window=1 << 30, sink=1 << 30) == 0
    assert window(lib, Hq=6) == 1 and b"num_kv_heads" in lib.pkv_last_error()
    assert window(lib, D=96) == 2 and window(lib, bs=24) == 2 and window(lib, dt=2) == 2
    assert window(lib, Hq=129, Hkv=1) == 2
    for bad in (dict(B=-1), dict(T=-1), dict(NB=0), dict(mb=0), dict(scale=0.0), dict(scale=math.nan)):
        assert window(lib, **bad) == 1, bad
    # aligned pointers that are never read: the workspace comes last
    assert window(lib, ptr=4096) == WORKSPACE and window(lib, ptr=4096, ws=4096) == WORKSPACE
    assert window(lib, ptr=4096 + 8) == 1 and b"16-byte" in lib.pkv_last_error()


def norm(lib, T=3, NB=4, bs=16, Hq=8, Hkv=4, D=128, rot=128, eps=1e-6, amp=1.0, qs=0, ks=0, vs=0, dt=1, wdt=1,
         fp8=None, ptrs=()):
    p = dict.fromkeys("q k v qw kw pos freq slots q_out k_out kc vc".split())
    p.update(ptrs)
    a = [*p.values(), T, NB, bs, Hq, Hkv, D, rot, 0, F(eps), F(amp), qs, ks, vs, dt, wdt]
    if fp8 is None:
        return lib.paged_kv_write_norm_rope(*a, None)
    return lib.paged_kv_write_norm_rope_fp8(*a, F(fp8[0]), F(fp8[1]), None)


def test_norm_rope_refusals(lib):
    some = dict(q=4096, k=4096, v=4096, pos=4096, freq=4096, slots=4096, q_out=4096, kc=4096, vc=4096)
    assert norm(lib, T=0) == 0 and norm(lib, T=0, NB=0, bs=0) == 0
    assert norm(lib) == 1 and b"null" in lib.pkv_last_error()
    for name in some:  # each of them is needed
        assert norm(lib, ptrs={**some, name: None}) == 1 and b"null" in lib.pkv_last_error(), name
    dense = dict(q=4096, k=4096, pos=4096, freq=4096, q_out=4096)
    assert norm(lib, ptrs=dense) == 1 and b"neither pools nor k_out" in lib.pkv_last_error()
    for name, off in (("q", 1), ("k_out", 1), ("qw", 1), ("pos", 4), ("freq", 4), ("kc", 8), ("vc", 8)):
        assert norm(lib, ptrs={**some, name: 4096 + off}) == 1 and b"aligned" in lib.pkv_last_error(), name
    assert norm(lib, dt=2) == 2 and norm(lib, dt=7) == 2 and norm(lib, wdt=2) == 2
    assert norm(lib, dt=0, wdt=1) == 2 and norm(lib, T=0, dt=1, wdt=0) == 0 and norm(lib, T=0, dt=0, wdt=0) == 0
    for bad in (dict(T=-1), dict(NB=-1), dict(bs=-1), dict(Hq=0), dict(Hkv=0), dict(D=0)):
        assert norm(lib, **bad) == 1, bad
    assert norm(lib, NB=0, ptrs=some) == 1 and norm(lib, bs=0, ptrs=some) == 1  # pools of no blocks
    for rot in (0, 3, 130, -2):
        assert norm(lib, rot=rot) == 1 and b"rotary_dim" in lib.pkv_last_error()
    for eps in (0.0, -1e-6, math.inf, math.nan):
        assert norm(lib, eps=eps) == 1 and b"eps" in lib.pkv_last_error()
    for amp in (0.0, -1.0, math.inf, math.nan):
        assert norm(lib, amp=amp) == 1 and b"amplitude" in lib.pkv_last_error()
    assert norm(lib, qs=8 * 128 - 1) == 1 and norm(lib, ks=100) == 1 and norm(lib, vs=100) == 1
    assert norm(lib, D=2048, rot=2) == 2 and norm(lib, Hq=1 << 18, D=128) == 2
    assert norm(lib, T=(1 << 30) + 1) == 2
    for scales in ((0.0, 1.0), (1.0, math.inf), (math.nan, 1.0), (1.0, -1.0)):
        assert norm(lib, T=0, fp8=scales) == 1 and b"scale" in lib.pkv_last_error()
    assert norm(lib, T=0, fp8=(1.0, 1.0)) == 0 and norm(lib, T=0, NB=0, fp8=(1.0, 1.0)) == 1


def block_write(lib, T=3, NB=8, bs=16, Hkv=4, D=128, ks=0, vs=0, ws=None, wsb=0, dt=1, ptrs=()):
    p = dict.fromkeys("k v slots kc vc ks vs".split())
    p.update(ptrs)
    return lib.paged_kv_write_fp8block(*p.values(), T, NB, bs, Hkv, D, ks, vs, ws, wsb, dt, None)


def test_block_write_refusals(lib):
    some = dict.fromkeys("k v slots kc vc ks vs".split(), 4096)
    assert block_write(lib, T=0) == 0
    assert block_write(lib) == 1 and b"null" in lib.pkv_last_error()
    for name in some:
        assert block_write(lib, ptrs={**some, name: None}) == 1 and b"null" in lib.pkv_last_error(), name
    for name, off in (("k", 1), ("v", 1), ("slots", 4), ("kc", 8), ("vc", 8), ("ks", 2), ("vs", 2)):
        assert block_write(lib, ptrs={**some, name: 4096 + off}) == 1 and b"aligned" in lib.pkv_last_error(), name
    assert block_write(lib, dt=2) == 2
    for bs in (1, 4, 24, 128):
        assert block_write(lib, bs=bs) == 2 and b"block_size" in lib.pkv_last_error()
    for D in (8, 100, 1040):
        assert block_write(lib, D=D) == 2 and b"head_dim" in lib.pkv_last_error()
    for bad in (dict(T=-1), dict(NB=0), dict(Hkv=0), dict(D=0), dict(ks=511), dict(vs=511)):
        assert block_write(lib, **bad) == 1, bad
    assert block_write(lib, Hkv=1 << 18, D=128) == 2 and block_write(lib, NB=1 << 31) == 2
    assert block_write(lib, T=(1 << 30) + 1) == 2


def test_block_write_workspace(lib):
    """Few tokens look their blocks up among themselves; more want a table
    with one int for each slot, without which the call is refused."""
    size = lib.paged_kv_write_fp8block_workspace
    some = dict.fromkeys("k v slots kc vc ks vs".split(), 4096)
    assert size(1, 1000, 16) == 0
    many = next(t for t in (1 << i for i in range(20)) if size(t, 1000, 16) > 0)
    want = size(many, 1000, 16)
    assert want >= 4 * 1000 * 16 and size(2 * many, 1000, 16) == want and size(many, 2000, 16) >= 4 * 2000 * 16
    big = dict(T=many, NB=1000, bs=16, ptrs=some)
    assert block_write(lib, **big) == WORKSPACE and b"workspace" in lib.pkv_last_error()
    assert block_write(lib, ws=4096, wsb=want - 1, **big) == WORKSPACE
    assert block_write(lib, ws=4096 + 8, wsb=want, **big) == WORKSPACE
    assert size(0, 1000, 16) == 0 and size(-1, 1000, 16) == 0 and size(many, 0, 16) == 0
    huge = size(1 << 20, (1 << 31) - 1, 64)  # past 32 bits
    assert huge >= 4 * ((1 << 31) - 1) * 64


def copy_scales(lib, pairs=None, n=None, layers=1, stride=0, NB=8, Hkv=4, ptr=4096):
    a = np.ascontiguousarray(pairs if pairs is not None else [[0, 1]], np.int32)
    return lib.paged_kv_copy_block_scales(ptr, ptr, a.ctypes.data, len(a) if n is None else n, layers, stride, NB, Hkv,
                                          None)


def test_copy_scales_refusals(lib):
    assert copy_scales(lib, n=0) == 0
    assert copy_scales(lib, ptr=None) == 1 and b"null" in lib.pkv_last_error()
    assert copy_scales(lib, ptr=4098) == 1 and b"aligned" in lib.pkv_last_error()
    for bad in (dict(n=-1), dict(layers=0), dict(NB=0), dict(Hkv=0), dict(stride=31)):
        assert copy_scales(lib, **bad) == 1, bad
    assert copy_scales(lib, NB=1 << 31) == 2 and copy_scales(lib, layers=1 << 30) == 2
    for pairs in ([[0, 8]], [[8, 0]], [[-1, 0]], [[0, 1], [2, 1]], [[0, 1], [1, 2]], [[3, 3]]):
        assert copy_scales(lib, pairs=pairs) == 1, pairs


def block_attend(lib, B=1, T=1, Hq=8, Hkv=4, D=128, NB=4, bs=16, mb=2, mql=0, scale=0.1, causal=1, window=0, sink=0,
                 ptr=None, scales=None, ws=None):
    return lib.paged_attention_forward_fp8block(ptr, ptr, ptr, scales, scales, ptr, ptr, ptr, ptr, B, T, Hq, Hkv, D,
                                                NB, bs, mb, mql, F(scale), causal, window, sink, ws, 0, None)


def test_block_attention_refusals(lib):
    assert block_attend(lib, B=0, T=0) == 0 and block_attend(lib, T=0) == 0
    assert block_attend(lib) == 1 and b"null" in lib.pkv_last_error()
    assert block_attend(lib, ptr=4096) == 1 and b"null" in lib.pkv_last_error()  # no scales
    assert block_attend(lib, ptr=4096, scales=4098) == 1 and b"aligned" in lib.pkv_last_error()
    assert block_attend(lib, ptr=4096, scales=4096) == WORKSPACE
    assert block_attend(lib, D=64) == 2 and b"head_dim" in lib.pkv_last_error()
    assert block_attend(lib, causal=0, window=8) == 1 and b"causal" in lib.pkv_last_error()
    assert block_attend(lib, T=0, causal=0) == 0 and block_attend(lib, T=0, sink=3) == 0
    assert block_attend(lib, window=-1) == 1 and block_attend(lib, sink=-1) == 1
    assert block_attend(lib, window=(1 << 30) + 1) == 2 and block_attend(lib, window=1, sink=(1 << 30) + 1) == 2
    assert block_attend(lib, Hq=6) == 1 and block_attend(lib, bs=24) == 2 and block_attend(lib, Hq=129, Hkv=1) == 2
    for bad in (dict(B=-1), dict(T=-1), dict(NB=0), dict(mb=0), dict(scale=0.0), dict(scale=math.inf)):
        assert block_attend(lib, **bad) == 1, bad


def test_copy_blocks_takes_codes(lib):
    """A block of codes whose bytes are no multiple of 16 is refused, as for
    the other types."""
    a = np.array([[0, 1]], np.int32)
    args = (4096, 4096, a.ctypes.data)
    assert lib.paged_kv_copy_blocks(*args, 0, 1, 0, 8, 16, 4, 128, 2, None) == 0  # no pairs
    assert lib.paged_kv_copy_blocks(*args, 1, 1, 0, 8, 1, 1, 8, 2, None) != 0
    assert lib.paged_kv_copy_blocks(*args, 1, 1, 0, 8, 16, 4, 128, 3, None) == 2

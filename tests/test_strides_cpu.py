"""Tensors that the C calls would take for others, and that the binding refuses:
those that repeat one row or layer (a stride of 0: dense), and pools without a
block (a null pointer: none).  The library is stubbed, so that what a call would be
given is seen without a GPU."""
import contextlib

import pytest
import torch

import paged_kv_cache_236_gb300 as pkv


@pytest.fixture
def calls(monkeypatch):
    """The C calls made, as (name, arguments): each is accepted and does nothing."""
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: made.append((name, a)) or 0

    monkeypatch.setattr(pkv, "lib", Lib)
    monkeypatch.setattr(pkv, "_need_cuda", lambda *t: torch.device("cpu"))
    monkeypatch.setattr(pkv, "_stream", lambda dev: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    return made


def pools(layers):
    return torch.zeros(layers, 4, 16, 2, 32, dtype=torch.uint8), torch.zeros(layers, 4, 16, 2, 32, dtype=torch.uint8)


def test_scales_of_one_layer_for_all(calls):
    k, v = pools(3)
    one = torch.ones(1, 4, 2)
    with pytest.raises(ValueError, match="layer stride"):
        pkv.copy_blocks(k, v, [[0, 1]], one.expand(3, 4, 2), one.expand(3, 4, 2))
    assert not calls  # nothing of the call has run
    # one layer has no stride, and layers may lie apart
    pkv.copy_blocks(k[:1], v[:1], [[0, 1]], one.expand(1, 4, 2), one.expand(1, 4, 2))
    pkv.copy_blocks(k[0], v[0], [[0, 1]], one[0], one[0])
    apart = torch.ones(3, 5, 4, 2)[:, 0]
    pkv.copy_blocks(k, v, [[0, 1]], apart, apart)
    scales = [a for name, a in calls if name == "paged_kv_copy_block_scales"]
    assert [(a[4], a[5]) for a in scales] == [(1, 0), (1, 0), (3, 40)]


def test_a_pool_of_one_layer_for_all(calls):
    k, v = (t[:1] for t in pools(1))
    with pytest.raises(ValueError, match="layer stride"):
        pkv.copy_blocks(k.expand(3, -1, -1, -1, -1), v.expand(3, -1, -1, -1, -1), [[0, 1]])
    assert not calls
    pkv.copy_blocks(k, v, [[0, 1]])
    k, v = torch.zeros(3, 2, 4, 16, 2, 32).unbind(1)
    pkv.copy_blocks(k, v, [[0, 1]])
    layer = 4 * 16 * 2 * 32
    assert [(a[4], a[5]) for _, a in calls] == [(1, layer), (3, 2 * layer)]


WRITES = ["paged_kv_write", "paged_kv_write_fp8", "paged_kv_write_attention_forward",
          "paged_kv_write_attention_forward_fp8kv"]


@pytest.mark.parametrize("name", WRITES)
def test_a_row_of_one_token_for_all(calls, monkeypatch, name):
    """The strides that a write is given, and that it is not given a 0 for several tokens."""
    monkeypatch.setattr(pkv, "_forward_args", lambda *a: ((), None, None))
    monkeypatch.setattr(pkv, "_fp8_forward_args", lambda *a: ((), None, None))
    fp8 = "fp8" in name
    cache = torch.zeros(4, 16, 2, 32, dtype=torch.uint8 if fp8 else torch.float32)
    at = torch.arange(5)
    scales = (1.0, 1.0) if fp8 else ()

    def write(k, v):
        slots = at[:k.shape[0]]
        if "attention" in name:
            getattr(pkv, name)(k, v, slots, None, cache, cache, None, None, None, 0.1, *scales)
        else:
            getattr(pkv, name)(k, v, slots, cache, cache, *scales)

    dense, one = torch.zeros(5, 2, 32), torch.zeros(1, 2, 32)
    for k, v in ((one.expand(5, 2, 32), dense), (dense, one.expand(5, 2, 32))):
        with pytest.raises(ValueError, match="token stride"):
            write(k, v)
    assert not calls
    fused = torch.zeros(5, 4, 32)
    write(dense, fused[:, :2])
    write(one, one)
    write(dense[:0], dense[:0])
    assert [n for n, _ in calls] == [name] * 3
    wide = [tuple(x for x in a if x in (64, 128)) for _, a in calls]
    assert wide[0] == (64, 128) and wide[1] == (64, 64) and wide[2] == ()


@pytest.mark.parametrize("shape", [(0, 16), (4, 0)])
def test_pools_without_a_block(calls, monkeypatch, shape):
    """Slots of a pool without a block are past it, and not left out unreported."""
    monkeypatch.setattr(pkv, "_device_of", lambda *t: -1)
    monkeypatch.setattr(pkv, "_call", lambda fn, dev, *a: fn(*a))
    q = k = v = torch.zeros(3, 2, 32)
    at, inv = torch.arange(3), torch.ones(16, dtype=torch.float64)

    def write(kc, vc):
        return pkv.paged_kv_write_norm_rope(q, k, v, None, None, at, inv, at, kc, vc, k_out=torch.zeros(3, 2, 32))

    none = torch.zeros(*shape, 2, 32)
    with pytest.raises(ValueError, match="blocks"):
        write(none, none.clone())
    assert not calls
    write(torch.zeros(4, 16, 2, 32), torch.zeros(4, 16, 2, 32))
    assert [n for n, _ in calls] == ["paged_kv_write_norm_rope"]

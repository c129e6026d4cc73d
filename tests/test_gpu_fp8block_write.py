"""paged_kv_write_fp8block against its definition, code by code.

Scales are powers of two, so that codes and scales are those of the definition
exactly: nothing to tolerate.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from oracle import serving

pytestmark = pytest.mark.gpu


class Pools:
    """Pools and scales on the device, and the same kept by the definition."""

    def __init__(self, NB, bs, Hkv, D, seed=0):
        g = np.random.default_rng(seed)
        self.host = []
        for _ in range(2):
            codes = g.integers(0, 256, (NB, bs, Hkv, D), dtype=np.uint8)
            self.host.append((codes, np.zeros((NB, Hkv), np.float32)))
        self.k, self.ks, self.v, self.vs = (torch.from_numpy(a.copy()).cuda() for pair in self.host for a in pair)

    def write(self, k, v, slots, **kw):
        pkv.paged_kv_write_fp8block(k, v, slots, self.k, self.v, self.ks, self.vs, **kw)
        for rows, (codes, scales) in zip((k, v), self.host):
            serving.write_blocks(rows.float().cpu().numpy(), slots.cpu().numpy(), codes, scales)
        self.check()

    def check(self):
        for (codes, scales), (c, s) in zip(self.host, ((self.k, self.ks), (self.v, self.vs))):
            assert np.array_equal(s.cpu().numpy(), scales)
            got, nan = c.cpu().numpy(), lambda a: (a & 0x7F) == 0x7F  # noqa: E731
            assert np.array_equal(nan(got), nan(codes)) and np.array_equal(got[~nan(got)], codes[~nan(codes)])


def rows(g, T, Hkv, D, dtype, fused=False, spread=1.5):
    gain = torch.exp(spread * torch.randn(T, 1, 1, generator=g))
    x = (gain * torch.randn(T, 2 * Hkv, D, generator=g)).to(dtype).cuda()
    k, v = x[:, :Hkv], x[:, Hkv:]
    return (k, v) if fused else (k.contiguous(), v.contiguous())


SHAPES = [(8, 1, 16), (16, 2, 128), (16, 8, 128), (32, 3, 64), (64, 2, 256), (64, 9, 48)]  # bs, Hkv, D


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bs,Hkv,D", SHAPES)
def test_a_sequence_grows(bs, Hkv, D, dtype):
    """A prompt in pieces, then single tokens: blocks begin, go on and outgrow their scale."""
    g = torch.Generator().manual_seed(bs + D)
    p = Pools(9, bs, Hkv, D)
    order = torch.randperm(9, generator=g)[:6]
    at = 0
    for n in (bs // 2 + 1, 1, 2 * bs, 3, 1, 1, bs - 1, 1, 1):
        place = torch.arange(at, at + n)
        slots = order[place // bs] * bs + place % bs
        p.write(*rows(g, n, Hkv, D, dtype, fused=n % 2 == 1), slots.cuda())
        at += n
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("T", [500, 513, 900])
@pytest.mark.parametrize("bs,Hkv,D", [(16, 2, 64), (64, 1, 128), (8, 4, 32)])
def test_many_rows_in_any_order(bs, Hkv, D, T):
    """Both ways of finding a block's rows; skipped slots, slots past the pool."""
    g = torch.Generator().manual_seed(T)
    NB = 2 * T // bs + 1
    p = Pools(NB, bs, Hkv, D)
    p.write(*rows(g, T, Hkv, D, torch.bfloat16), torch.randperm(NB * bs, generator=g)[:T].cuda())
    slots = torch.randperm(NB * bs, generator=g)[:T]
    slots[::5] = -1
    p.write(*rows(g, T, Hkv, D, torch.bfloat16, fused=True), slots.cuda())
    assert pkv.device_errors() == 0
    slots[7], slots[11] = NB * bs, (1 << 40) + 3
    k, v = rows(g, T, Hkv, D, torch.bfloat16)
    pkv.paged_kv_write_fp8block(k, v, slots.cuda(), p.k, p.v, p.ks, p.vs)
    assert pkv.device_errors() == pkv.DEVERR["slot_out_of_range"]
    slots[7] = slots[11] = -1
    for x, (codes, scales) in zip((k, v), p.host):
        serving.write_blocks(x.float().cpu().numpy(), slots.numpy(), codes, scales)
    p.check()


def test_values_at_the_edges():
    """Zeros, the scale's two ends, infinities, NaN, the last value a scale covers."""
    p = Pools(8, 16, 1, 16)
    one = torch.ones(1, 1, 16)
    for i, x in enumerate((0.0, 1e-30, 448.0, 448.0 * (1 + 2.0 ** -20), 2.0 ** 69, 3e38, float("inf"), float("nan"))):
        k = (one * x).cuda()
        k[0, 0, 3] = -k[0, 0, 3]
        p.write(k, k.clone(), torch.tensor([i * 16], device="cuda"))
    # a block without a first row: its scale counts as 0, and its codes end as zeros
    q = Pools(1, 16, 1, 16)
    q.write(one.cuda(), one.cuda(), torch.tensor([5], device="cuda"))
    # from the smallest scale to the largest in one block
    r = Pools(1, 8, 1, 16)
    for i, x in enumerate((1e-25, 1e-10, 1.0, 1e10, 1e25, 1e-10)):
        r.write((one * x).cuda(), (one * -x).cuda(), torch.tensor([i], device="cuda"))


def test_the_same_slot_twice():
    """One of the two lands, whole, under a scale that covers it."""
    for T in (2, 600):
        k = torch.ones(T, 1, 16, device="cuda")
        k[0] = 100.0
        slots = torch.arange(T, device="cuda") + 16
        slots[1] = slots[0]
        c = torch.zeros(64, 16, 1, 16, dtype=torch.uint8, device="cuda")
        s = torch.zeros(64, 1, device="cuda")
        c2, s2 = c.clone(), s.clone()
        pkv.paged_kv_write_fp8block(k, k, slots, c, c2, s, s2)
        got = serving.block_values(c.cpu().numpy(), s.cpu().numpy())[1, 0, 0]
        assert np.all(got == got[0]) and got[0] in (1.0, 96.0, 100.0, 104.0)
        assert torch.equal(c, c2) and torch.equal(s, s2)


def test_copies_take_their_scales():
    g = torch.Generator().manual_seed(3)
    for layers in (1, 3):
        shape = (layers, 12, 16, 3, 32)
        k = torch.randint(0, 256, shape, generator=g, dtype=torch.int32).to(torch.uint8).cuda()
        v = torch.randint(0, 256, shape, generator=g, dtype=torch.int32).to(torch.uint8).cuda()
        ks, vs = torch.rand(layers, 12, 3, generator=g).cuda(), torch.rand(layers, 12, 3, generator=g).cuda()
        want = [t.clone() for t in (k, v, ks, vs)]
        for t in want:
            t[:, 5], t[:, 7] = t[:, 2].clone(), t[:, 11].clone()
        if layers == 1:
            pkv.copy_blocks(k[0], v[0], [[2, 5], [11, 7]], ks[0], vs[0])
        else:
            pkv.copy_blocks(k, v, [[2, 5], [11, 7]], ks, vs)
        for t, w in zip((k, v, ks, vs), want):
            assert torch.equal(t, w)
    with pytest.raises(ValueError):
        pkv.copy_blocks(k, v, [[2, 5]], ks)
    with pytest.raises(ValueError):
        pkv.copy_blocks(k, v, [[2, 5]], ks[:2], vs[:2])
    with pytest.raises(ValueError):
        pkv.copy_blocks(k, v, [[2, 5]], ks.double(), vs.double())


def test_captured_and_replayed():
    g = torch.Generator().manual_seed(4)
    p = Pools(80, 16, 2, 64)
    T = 700
    k, v = rows(g, T, 2, 64, torch.bfloat16)
    slots = torch.arange(T, device="cuda")
    p.write(k, v, slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_kv_write_fp8block(k, v, slots, p.k, p.v, p.ks, p.vs)
    k2, v2 = rows(g, T, 2, 64, torch.bfloat16)
    k.copy_(k2), v.copy_(v2), slots.add_(37)
    graph.replay()
    torch.cuda.synchronize()
    for x, (codes, scales) in zip((k, v), p.host):
        serving.write_blocks(x.float().cpu().numpy(), slots.cpu().numpy(), codes, scales)
    p.check()


def test_refusals():
    g = torch.Generator().manual_seed(5)
    k, v = rows(g, 4, 2, 64, torch.bfloat16)
    slots = torch.arange(4, device="cuda")
    p = Pools(80, 16, 2, 64)
    f = pkv.paged_kv_write_fp8block
    for bad in (lambda: f(k, v, slots, p.k, p.v, p.ks[:4], p.vs), lambda: f(k, v, slots, p.k, p.v, p.ks.double(), p.vs),
                lambda: f(k, v.float(), slots, p.k, p.v, p.ks, p.vs), lambda: f(k.half(), v.half(), slots, p.k, p.v, p.ks, p.vs),
                lambda: f(k, v, slots.int(), p.k, p.v, p.ks, p.vs), lambda: f(k, v, slots, p.k.float(), p.v.float(), p.ks, p.vs),
                lambda: f(k[:1].expand(4, -1, -1), v, slots, p.k, p.v, p.ks, p.vs),
                lambda: f(k.cpu(), v, slots, p.k, p.v, p.ks, p.vs)):
        with pytest.raises(ValueError):
            bad()
    kk, vv = rows(g, 700, 2, 64, torch.bfloat16)
    with pytest.raises(ValueError):
        f(kk, vv, torch.arange(700, device="cuda"), p.k, p.v, p.ks, p.vs,
          workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    odd = torch.zeros(4, 24, 2, 64, dtype=torch.uint8, device="cuda")
    with pytest.raises(pkv.LibraryError):
        f(k, v, slots, odd, odd.clone(), torch.zeros(4, 2, device="cuda"), torch.zeros(4, 2, device="cuda"))
    f(k[:0], v[:0], slots[:0], p.k, p.v, p.ks, p.vs)
    p.check()

"""paged_attention_forward_fp8block against the fp64 definition over the pools'
values.

Tolerance, as a share of the largest |v| a row could mix: the weights keep at
least 9 bits (2^-9 of each), q's split is off by 2^-18 of a row's largest |q| in
each of 128 products (below 2^-8 of a unit of logit here: |q| <= 9, values of K
below 16, scale 2^-3.5, and of random sign), the output rounds to bf16 (half a
step, 2^-9 below a power of two): 2 * 2^-9 + 2^-8 of 4.5, below 4e-2; the mean
error, of random signs, a tenth of it.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from gpu_util import to_f64
from oracle import serving

pytestmark = pytest.mark.gpu

TMAX, TMEAN = 4e-2, 4e-3
NAN = 0x7F


def scale_of(top):
    return 2.0 ** np.ceil(np.log2(np.maximum(top, 1e-30) / 448))


class Batch:
    """Pools of rows with magnitudes by block and head (V's undone by its mixing
    size: values stay below 4.5), NaN codes and scales wherever no token is."""

    def __init__(self, seed, lens, n, Hq, Hkv, bs, spread=0.7, small_v=False):
        g = torch.Generator().manual_seed(seed)
        need = [-(-L // bs) for L in lens]
        NB = sum(need) + 3
        order = torch.randperm(NB, generator=g).numpy()
        self.tables = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
        kv = np.full((2, NB, bs, Hkv, 128), np.nan)
        at = 0
        for s, L in enumerate(lens):
            self.tables[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
            for j in range(need[s]):
                m = min(bs, L - j * bs)
                size = torch.exp(spread * torch.randn(1, Hkv, 1, generator=g)).clamp(max=4)
                kv[0, self.tables[s, j], :m] = (size * torch.randn(m, Hkv, 128, generator=g)).numpy()
                size = torch.exp(-3 * torch.rand(1, Hkv, 1, generator=g)) if small_v else 1.0
                kv[1, self.tables[s, j], :m] = (size * torch.randn(m, Hkv, 128, generator=g).clamp(-4.5, 4.5)).numpy()
        self.codes, self.scales = [], []
        for x in kv:
            top = np.where(np.isnan(x), 0, np.abs(x)).max((1, 3))
            scale = np.where(top > 0, scale_of(top), np.nan).astype(np.float32)
            c = torch.from_numpy((x / scale[:, None, :, None]).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
            c[torch.from_numpy(np.isnan(x))] = NAN
            self.codes.append(c.numpy())
            self.scales.append(scale)
        self.lens, self.n = list(lens), list(n)
        self.qsl = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.q = torch.randn(int(self.qsl[-1]), Hq, 128, generator=g).to(torch.bfloat16)
        self.scale = 128 ** -0.5
        self.up()

    def up(self):
        t = lambda a: torch.from_numpy(np.array(a)).cuda()  # noqa: E731
        self.args = (self.q.cuda(), t(self.codes[0]), t(self.codes[1]), t(self.scales[0]), t(self.scales[1]),
                     t(self.tables), t(np.array(self.lens, np.int32)), t(self.qsl), self.scale)

    def rows(self, i, s):
        L, bs = self.lens[s], self.codes[i].shape[1]
        blocks = self.tables[s, :-(-L // bs)]
        # scales outside [2^-60, 2^60] count as the nearest end
        x = serving.block_values(self.codes[i][blocks], np.clip(self.scales[i][blocks], 2.0 ** -60, 2.0 ** 60))
        return x.reshape((-1,) + x.shape[2:])[:L]

    def check(self, out, window=0, sink=0, causal=True, tol=(TMAX, TMEAN)):
        got, q = to_f64(out), to_f64(self.q)
        worst = total = count = 0
        for s in range(len(self.lens)):
            a, b = int(self.qsl[s]), int(self.qsl[s + 1])
            if a == b:
                continue
            want = serving.window_attend(q[a:b], self.rows(0, s), self.rows(1, s), self.scale, window, sink, causal)
            err = np.abs(got[a:b] - want)
            assert np.all(np.isfinite(err)), f"sequence {s}"
            worst, total, count = max(worst, err.max()), total + err.sum(), count + err.size
        assert worst <= tol[0] and total <= tol[1] * count, (worst, total / count)


LENS = [700, 1, 333, 129, 64, 512, 40, 257]
GROUPS = [(8, 2, 16), (4, 1, 8), (8, 8, 32), (16, 2, 64), (16, 1, 16), (6, 2, 16), (7, 1, 32), (12, 1, 16), (20, 1, 16)]
IDS = lambda s: "-".join(map(str, s))  # noqa: E731


@pytest.mark.parametrize("group", GROUPS, ids=IDS)
def test_single_tokens(group):
    Hq, Hkv, bs = group
    b = Batch(Hq + bs, LENS, [1] * len(LENS), Hq, Hkv, bs)
    for hint in (1, 0):
        b.check(pkv.paged_attention_forward_fp8block(*b.args, max_query_len=hint))
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("group", GROUPS, ids=IDS)
def test_several_queries(group):
    """Prompt chunks, verify windows, single tokens and sequences without a query, side by side."""
    Hq, Hkv, bs = group
    n = [150, 1, 5, 129, 0, 3, 40, 2]
    b = Batch(Hq + 2 * bs, LENS, n, Hq, Hkv, bs)
    for hint in (0, 150):
        b.check(pkv.paged_attention_forward_fp8block(*b.args, max_query_len=hint))
    b.check(pkv.paged_attention_forward_fp8block(*b.args, False), causal=False)
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("n", [[1, 1, 1], [1, 3, 2], [60, 1, 130]])
@pytest.mark.parametrize("window,sink", [(1, 0), (7, 2), (130, 4), (256, 140), (600, 1)])
def test_windows(window, sink, n):
    """Blocks out of sight have no valid entry, rows out of sight hold NaN codes."""
    lens = [700, 333, 512]
    b = Batch(window, lens, n, 8, 2, 16)
    kept = b.tables.copy()
    for s, L in enumerate(lens):
        first = L - n[s] + 1 - window
        for j in range(sink, first):
            b.codes[0][b.tables[s, j // 16], j % 16] = b.codes[1][b.tables[s, j // 16], j % 16] = NAN
        for blk in range(-(-sink // 16), max(first, 0) // 16):
            b.tables[s, blk] = -1 if blk % 2 else 1 << 30
    b.up()
    out = pkv.paged_attention_forward_fp8block(*b.args, window=window, num_sink=sink)
    assert pkv.device_errors() == 0
    b.tables = kept
    b.check(out, window, sink)


@pytest.mark.parametrize("n", [[1, 1], [3, 4], [200, 5]])
def test_scales_far_apart(n):
    """V's blocks differ by many powers of two, and K's: the output follows the large ones, and the small alone."""
    for shift in (0, -50, 40):
        b = Batch(9, [600, 300], n, 8, 2, 16, spread=0.3, small_v=True)
        for i in range(2):
            b.scales[i] = b.scales[i] * np.float32(2.0 ** (shift if i else 0))
        b.up()
        out = pkv.paged_attention_forward_fp8block(*b.args)
        unit = 2.0 ** shift
        b.check(out, tol=(TMAX * unit, TMEAN * unit))
    # one large block among small ones
    b = Batch(10, [600, 300], n, 8, 2, 16, small_v=True)
    b.scales[1][b.tables[0, 3]] *= np.float32(2.0 ** 30)
    b.scales[1][b.tables[1, 7]] *= np.float32(2.0 ** 30)
    b.up()
    b.check(pkv.paged_attention_forward_fp8block(*b.args), tol=(TMAX * 2.0 ** 30, TMEAN * 2.0 ** 30))
    # scales that are no powers of two, and zero for a block of zeros
    b = Batch(11, [600, 300], n, 8, 2, 16)
    for i in range(2):
        b.scales[i] = (b.scales[i] * 0.7).astype(np.float32)
    blk = b.tables[0, 5]
    b.codes[0][blk] = b.codes[1][blk] = 0
    b.scales[0][blk] = b.scales[1][blk] = 0
    b.up()
    b.check(pkv.paged_attention_forward_fp8block(*b.args))


@pytest.mark.parametrize("n", [[1], [20]])
def test_many_small_weights_beside_a_large_one(n):
    """The first key takes half of the weight, thousands share the rest: each far below the largest."""
    b = Batch(12, [20000], n, 4, 1, 16, spread=0.0)
    q = to_f64(b.q)
    b.scales[0][b.tables[0, 0]] = 0.25
    b.codes[0][b.tables[0, 0]] = 0
    b.codes[0][b.tables[0, 0], 0, 0, 0] = 0x58  # 16
    b.q[..., 0] = 28.0  # 4 * 28 / sqrt(128) = 9.9 = log(20000)
    b.codes[0][b.tables[0, 1:1250], :, :, 0] = 0
    b.codes[1][b.tables[0, :1250]] = torch.full((1,), 1.0).to(torch.float8_e4m3fn).view(torch.uint8).item()
    b.codes[1][b.tables[0, 0]] = 0
    b.scales[1][:] = 1.0
    del q
    b.up()
    out = pkv.paged_attention_forward_fp8block(*b.args)
    b.check(out)


def test_long_contexts_split():
    b = Batch(13, [20000, 9000], [1, 2], 8, 2, 16)
    least = pkv.workspace_min(2, 3, 8, 2, 128)
    for ws in (None, torch.empty(least, dtype=torch.uint8, device="cuda")):
        b.check(pkv.paged_attention_forward_fp8block(*b.args, workspace=ws, max_query_len=2))
    b.check(pkv.paged_attention_forward_fp8block(*b.args, window=6001, num_sink=4), 6001, 4)


def test_rising_logits():
    """Rows of one tile whose maximum rises at different key tiles."""
    for n in (1, 4, 64):
        b = Batch(14, [640], [n], 8, 2, 16, spread=0.0)
        tile = np.arange(40 * 16).reshape(40, 16) // 128
        b.scales[0][b.tables[0, :40]] = 2.0 ** -3
        codes = torch.from_numpy(2.0 * tile / 2.0 ** -3).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        b.codes[0][b.tables[0, :40], :, :, 0] = codes[:, :, None]
        b.q[..., 0] = 5.0 * 128 ** 0.5 * torch.tensor([1.0, -1.0]).repeat(4)
        b.up()
        b.check(pkv.paged_attention_forward_fp8block(*b.args), tol=(2 * TMAX, 2 * TMEAN))


def test_bad_batches():
    b = Batch(15, [100, 50, 300], [1, 1, 40], 8, 2, 16)
    bad = torch.tensor([100, 0, 300], dtype=torch.int32, device="cuda")  # a query of an empty sequence
    out = pkv.paged_attention_forward_fp8block(*b.args[:6], bad, *b.args[7:])
    assert pkv.device_errors() == pkv.DEVERR["bad_sequence"]
    assert torch.all(out[1] == 0) and torch.all(torch.isfinite(out.float()))
    # an invalid block is a block of zeros
    b.tables[0, 2], keep = 1 << 30, b.tables[0, 2]
    b.up()
    out = pkv.paged_attention_forward_fp8block(*b.args)
    assert pkv.device_errors() == pkv.DEVERR["block_out_of_range"]
    b.tables[0, 2] = keep
    for i in range(2):
        b.codes[i][keep], b.scales[i][keep] = 0, 1.0
    b.check(out)


def test_refusals():
    b = Batch(16, [100], [1], 8, 2, 16)
    f = pkv.paged_attention_forward_fp8block
    q, kc, vc, ks, vs, *rest = b.args
    for bad in (lambda: f(q.float(), kc, vc, ks, vs, *rest), lambda: f(q, kc, vc, ks[:2], vs, *rest),
                lambda: f(q, kc, vc, ks, vs.double(), *rest), lambda: f(q, kc.float(), vc.float(), ks, vs, *rest),
                lambda: f(q, kc, vc, ks.T, vs, *rest), lambda: f(q, kc, vc, ks, vs.cpu(), *rest),
                lambda: f(*b.args, window=-1), lambda: f(*b.args, window=4, num_sink=-1),
                lambda: f(*b.args, window=1 << 31)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(pkv.LibraryError):
        f(*b.args, False, window=5)
    half = torch.zeros(4, 16, 2, 64, dtype=torch.uint8, device="cuda")
    s = torch.ones(4, 2, device="cuda")
    with pytest.raises(pkv.LibraryError):
        f(q[..., :64].contiguous(), half, half, s, s, *rest)


def test_captured_and_replayed():
    b = Batch(17, [700, 333], [1, 1], 8, 2, 16)
    out = torch.empty_like(b.args[0])
    pkv.paged_attention_forward_fp8block(*b.args, out=out, max_query_len=1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_attention_forward_fp8block(*b.args, out=out, max_query_len=1)
    b.lens = [650, 200]
    b.args[6].copy_(torch.tensor(b.lens, dtype=torch.int32))
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    b.check(out)

"""paged_attention_scores and its FP8 form against the fp64 definition.

Tolerance.  A logit (in log2 units) is a dot product of D terms, summed in
fp32 in any order, times a constant: it is off by at most
  e = scale * log2(e) * (D + 2) * 2^-24 * sum |q k|.
A weight is exp2 of a logit less the row's log-sum-exp, itself as far off, so
its relative error is at most 2 ln2 e plus the exponentials' (2^-22 each, two of
them) and the sums' (each running sum of up to 512 terms, rescaled with
exponentials: 512 * 2^-22 < 1.3e-4).  Weights below 2^-126 flush to zero.
"""
import math
import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
import workloads as wl
from gpu_util import to_f64
from oracle import budget as ob
from oracle import fp8

pytestmark = pytest.mark.gpu


class Batch:
    """A ragged batch over a shuffled pool whose other slots are NaN."""

    def __init__(self, seed, lens, qlens, Hq, Hkv, D, bs, dtype=torch.bfloat16, f8=False, gain=1.5, rows=None,
                 max_len=None, extra_blocks=3):
        rng = np.random.default_rng(seed)
        need = [-(-L // bs) for L in lens]
        NB = sum(need) + extra_blocks
        order = rng.permutation(NB)
        self.tables = np.full((len(lens), max(max(need, default=1), 1)), -1, np.int32)
        at = 0
        for s, c in enumerate(need):
            self.tables[s, :c] = order[at:at + c]
            at += c
        pool = rng.standard_normal((NB, bs, Hkv, D)).astype(np.float32)
        live = np.zeros((NB, bs), bool)
        for s, L in enumerate(lens):
            for j in range(L):
                live[self.tables[s, j // bs], j % bs] = True
        self.k_scale = 0.011 if f8 else 1.0
        if f8:
            codes = fp8.quantize(pool, self.k_scale)
            codes[~live] = 0x7F
            self.kc = torch.from_numpy(codes).cuda()
            self.K = fp8.dequantize(codes, self.k_scale)
        else:
            pool[~live] = np.nan
            self.kc = torch.from_numpy(pool).to(dtype).cuda()
            self.K = to_f64(self.kc)
        T = int(sum(qlens))
        self.q = torch.from_numpy((gain * rng.standard_normal((T, Hq, D))).astype(np.float32)).to(dtype).cuda()
        self.lens, self.qlens, self.bs, self.Hq, self.Hkv, self.D, self.f8 = lens, qlens, bs, Hq, Hkv, D, f8
        self.qsl = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        self.scale = 1 / math.sqrt(D)
        self.rows = list(range(len(lens))) if rows is None else rows
        self.old = torch.from_numpy(rng.random((max(self.rows, default=0) + 2, Hkv,
                                                max_len or max(lens, default=1) + 5)).astype(np.float32) * 3).cuda()
        dev = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
        self.args = dict(block_tables=dev(self.tables), context_lens=dev(lens), query_start_loc=dev(self.qsl))
        self.row_arg = None if rows is None else dev(rows)

    def run(self, causal=True, decay=1.0, out=None, q=None, **kw):
        args = {**self.args, **kw}
        q = self.q if q is None else q
        scores = args.pop("scores", self.old)
        if self.f8:
            return pkv.paged_attention_scores_fp8kv(q, self.kc, args.pop("block_tables"), args.pop("context_lens"),
                                                    args.pop("query_start_loc"), scores, self.scale, self.k_scale,
                                                    causal, decay=decay, score_rows=self.row_arg, out=out, **args)
        return pkv.paged_attention_scores(q, self.kc, args.pop("block_tables"), args.pop("context_lens"),
                                          args.pop("query_start_loc"), scores, self.scale, causal, decay=decay,
                                          score_rows=self.row_arg, out=out, **args)

    def keys(self, s):
        L = self.lens[s]
        return self.K[self.tables[s, :-(-L // self.bs)]].reshape(-1, self.Hkv, self.D)[:L]

    def check(self, got, before, old=None, causal=True, decay=1.0, seqs=None):
        got, before = got.cpu().numpy(), before.cpu().numpy()
        old = before if old is None else old.cpu().numpy()
        want_all = before.astype(np.float64)
        tol_all = np.zeros_like(want_all)
        qf = to_f64(self.q)
        for s, L in enumerate(self.lens):
            r, n = self.rows[s], self.qlens[s]
            if r < 0 or n == 0 or (seqs is not None and s not in seqs):
                continue
            q, K = qf[self.qsl[s]:self.qsl[s + 1]], self.keys(s)
            w = ob.scores_update(q, K, old[r, :, :L], self.scale, causal, decay)
            dots = np.abs(q).reshape(-1, self.D).max(0) @ np.abs(K).reshape(-1, self.D).max(0)
            rel = 2 * self.scale * (self.D + 2) * 2.0 ** -24 * dots + 2 * 2.0 ** -22 + 1.3e-4
            paid = ob.scores_update(q, K, old[r, :, :L], self.scale, causal, 0.0)
            want_all[r, :, :L] = w
            tol_all[r, :, :L] = rel * paid + 2.0 ** -22 * w + n * self.Hq * 2.0 ** -120
            total = got[r, :, :L].astype(np.float64).sum() - (decay * old[r, :, :L - n].astype(np.float64)).sum()
            assert total == pytest.approx(n * self.Hq, rel=2e-4, abs=1e-3 * max(1.0, L * self.Hkv * 2e-4))
        err = np.abs(got - want_all)
        assert np.all(np.isfinite(got)) and np.all(err <= tol_all), float((err - tol_all).max())


SHAPES = [  # Hq, Hkv, D, bs
    (8, 2, 128, 16), (4, 4, 64, 8), (16, 2, 128, 32), (14, 2, 64, 64), (6, 2, 128, 64), (32, 1, 128, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_ragged_batches(shape, dtype):
    Hq, Hkv, D, bs = shape
    if dtype == "fp8" and D != 128:
        pytest.skip("FP8 pools: head_dim 128")
    b = Batch(Hq * D + bs, [1, 2, 300, 129, 64, 517, 40, 0, 33], [1, 2, 1, 5, 1, 40, 40, 0, 3], Hq, Hkv, D, bs,
              torch.float32 if dtype == "f32" else torch.bfloat16, dtype == "fp8")
    for causal, decay in ((True, 1.0), (True, 0.0), (False, 0.5)):
        before = b.old.clone()
        got = b.run(causal, decay, out=b.old.clone())
        assert torch.equal(b.old, before)
        b.check(got, before, causal=causal, decay=decay)
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("hint", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 8, 16])
def test_decode(group, dtype, hint):
    """Single tokens, one length on each side of the tiles' edges."""
    lens = [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000]
    b = Batch(group, lens, [1] * len(lens), 2 * group, 2, 128, 16,
              torch.float32 if dtype == "f32" else torch.bfloat16, dtype == "fp8")
    before = b.old.clone()
    b.check(b.run(max_query_len=hint), before)
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_long_context_and_large_logits(dtype):
    """A 20 000-key context, logits up to about +-40: most weights underflow."""
    b = Batch(5, [20000, 7000], [1, 4], 8, 2, 128, 16, f8=dtype == "fp8", gain=12.0)
    before = b.old.clone()
    b.check(b.run(decay=0.5), before, decay=0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("n,L", [(33, 700), (64, 64), (128, 2000), (200, 1111), (513, 600)])
def test_many_queries(n, L, dtype):
    if dtype != "bf16" and n > 200:
        pytest.skip("covered by bf16")
    b = Batch(n, [L, 50], [n, 1], 8, 2, 128, 16, torch.float32 if dtype == "f32" else torch.bfloat16, dtype == "fp8")
    before = b.old.clone()
    b.check(b.run(), before)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("Hq,Hkv,bs", [(8, 2, 16), (32, 2, 32), (8, 8, 64)])
def test_prompts_from_the_first_token(Hq, Hkv, bs, dtype):
    """No context before the queries: row tiles that see one, two, ... K tiles
    of a range, in odd and even numbers, and short sequences of one K tile in a
    row; over and over, since only the timing of the roles could go wrong."""
    lens = [700, 128, 90, 33, 127, 385, 64, 1100, 100, 100, 1]
    b = Batch(Hq + bs, lens, lens, Hq, Hkv, 128, bs, torch.float32 if dtype == "f32" else torch.bfloat16, dtype == "fp8")
    before = b.old.clone()
    first = b.run(out=b.old.clone())
    b.check(first, before)
    for _ in range(50):
        assert torch.equal(b.run(out=b.old.clone()), first)
    assert pkv.device_errors() == 0


def test_chunk_equals_steps():
    """Scores of a prompt's tokens: all queries at once, or one step after
    another with decay 1, add up to the same."""
    b = Batch(21, [40], [40], 4, 2, 64, 8, torch.float32)
    whole = b.run(decay=0.0, out=torch.zeros_like(b.old))
    step = torch.full_like(b.old, 7.0)  # stale scores of other tokens
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for i in range(40):
        b.run(q=b.q[i:i + 1].contiguous(), scores=step, context_lens=torch.tensor([i + 1], dtype=torch.int32, device="cuda"),
              query_start_loc=one)
    # fp32 sums of up to 40 weights below 1 each, and each weight within 1.3e-4 + 2^-21
    assert torch.allclose(step[0, :, :40], whole[0, :, :40], rtol=3e-4, atol=1e-6)
    assert torch.all(step[0, :, 40:] == 7.0)


def test_rows_left_out_and_shared_blocks():
    """score_rows: permuted, -1 (left out), out of range (flagged); blocks
    that two sequences share are scored in each one's own row."""
    b = Batch(31, [100, 60, 200, 30], [1, 3, 1, 2], 8, 2, 128, 16, rows=[3, -1, 0, 1])
    b.tables[2, :3] = b.tables[0, :3]
    b.args["block_tables"] = torch.from_numpy(b.tables).cuda()
    before = b.old.clone()
    b.check(b.run(), before)
    assert pkv.device_errors() == 0
    b.row_arg = torch.tensor([3, -1, 0, b.old.shape[0]], dtype=torch.int32, device="cuda")
    b.rows = [3, -1, 0, -1]
    before = b.old.clone()
    b.check(b.run(), before)
    assert pkv.device_errors() == pkv.DEVERR["bad_sequence"]


def test_invalid_metadata():
    """Bad sequences leave their rows as they were; an out-of-pool block
    reads as zeros; nothing faults."""
    b = Batch(41, [100, 60, 80, 50], [1, 2, 1, 1], 8, 2, 128, 16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for kw, good in ((dict(context_lens=i32([100, 1, 80, 50])), [0, 2, 3]),          # more queries than tokens
                     (dict(context_lens=i32([100, 60, 81 * 16, 50])), [0, 1, 3]),    # past its table
                     (dict(context_lens=i32([100, 60, -4, 50])), [0, 1, 3]),
                     (dict(query_start_loc=i32([0, 1, 3, 4, 9])), [0, 1, 2]),        # past q
                     (dict(query_start_loc=i32([0, 4, 0, 4, 5])), [3]),              # overlapping queries
                     (dict(query_start_loc=i32([0, 4, 0, 4, 5]), max_query_len=4), [3])):
        before = b.old.clone()
        if kw.get("query_start_loc") is not None and len(good) == 1:
            got = b.run(out=b.old.clone(), **kw)
            assert torch.equal(got[1:3], before[1:3])
            pkv.device_errors()
            continue
        got = b.run(out=b.old.clone(), **kw)
        b.check(got, before, seqs=good)
        assert pkv.device_errors() == pkv.DEVERR["bad_sequence"], kw
    short = b.old[:, :, :70].contiguous()
    before = short.clone()
    got = b.run(scores=short)
    b.check(got, before, seqs=[1, 3])
    assert pkv.device_errors() == pkv.DEVERR["bad_sequence"]
    # a block of zeros in place of an id outside the pool
    for bad in (-1, b.kc.shape[0], 2 ** 31 - 1):
        t = b.tables.copy()
        t[0, 2] = bad
        keep = b.K.copy()
        b.K = np.concatenate([b.K, np.zeros((1,) + b.K.shape[1:])])
        held, b.tables = b.tables, t.copy()
        b.tables[0, 2] = len(keep)
        before = b.old.clone()
        b.check(b.run(out=b.old.clone(), block_tables=torch.from_numpy(t).cuda()), before)
        assert pkv.device_errors() == pkv.DEVERR["block_out_of_range"]
        b.K, b.tables = keep, held


def test_broken_query_length_promise():
    """A sequence with more queries than max_query_len is flagged and left
    out; the others get their scores."""
    b = Batch(45, [300, 200, 90], [1, 30, 2], 8, 2, 128, 16)
    for most, good in ((1, [0]), (2, [0, 2]), (29, [0, 2]), (30, [0, 1, 2]), (0, [0, 1, 2])):
        before = b.old.clone()
        b.check(b.run(out=b.old.clone(), max_query_len=most), before, seqs=good)
        assert pkv.device_errors() == (0 if len(good) == 3 else pkv.DEVERR["bad_sequence"])


@pytest.mark.parametrize("count", [31, 33, 64, 255, 256, 257, 700])
def test_many_sequences(count):
    """Plans of one, two and more sequences a thread, and past what shared
    memory holds; every seventh sequence has no queries, one is invalid."""
    rng = np.random.default_rng(count)
    lens = rng.integers(1, 60, count).tolist()
    q = [0 if s % 7 == 3 else 1 for s in range(count)]
    b = Batch(count, lens, q, 4, 2, 64, 8)
    bad = count // 2
    ctx = b.args["context_lens"].clone()
    ctx[bad] = 61 * 8
    for hint in (0, 1):
        before = b.old.clone()
        good = [s for s in range(count) if s != bad or q[s] == 0]
        b.check(b.run(out=b.old.clone(), max_query_len=hint, context_lens=ctx), before, seqs=good)
        assert pkv.device_errors() == pkv.DEVERR["bad_sequence"]


def test_nan_in_masked_places():
    """NaN old scores count only where they are read: at the step's own
    tokens, and everywhere with decay 0, they are overwritten."""
    b = Batch(51, [90, 90], [2, 1], 4, 1, 128, 16)
    b.old[:, :, 88:] = float("nan")
    got = b.run(out=torch.zeros_like(b.old))
    assert torch.isfinite(got[0, :, :90]).all() and torch.isnan(got[1, :, 88]).all()
    b.old.fill_(float("nan"))
    got = b.run(decay=0.0)
    assert torch.isfinite(got[:2, :, :90]).all() and torch.isnan(got[:2, :, 90:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 3, 4, 40])
def test_logits_of_minus_infinity(n, dtype):
    """Infinite keys whose logits are -inf weigh nothing: the first key, a run
    that fills whole tiles, every seventh after it."""
    L = 700
    b = Batch(55 + n, [L], [n], 8, 2, 128, 16, torch.float32 if dtype == "f32" else torch.bfloat16)
    off = sorted({0, *range(128, 400), *range(400, L - n, 7)})
    b.q[..., 0] = -1.0
    for j in off:
        b.kc[b.tables[0, j // 16], j % 16, :, 0] = math.inf
        b.K[b.tables[0, j // 16], j % 16, :, 0] = math.inf
    before = b.old.clone()
    got = b.run(decay=0.0, out=b.old.clone()).cpu().numpy()
    q, K = to_f64(b.q), b.keys(0)
    paid = ob.scores_update(q, K, before[0, :, :L].cpu().numpy(), b.scale, True, 0.0)
    seen = np.setdiff1d(np.arange(L), off)
    # the bounds of Batch.check, over the finite keys
    dots = np.abs(q).reshape(-1, 128).max(0) @ np.abs(K[seen]).reshape(-1, 128).max(0)
    rel = 2 * b.scale * 130 * 2.0 ** -24 * dots + 2 * 2.0 ** -22 + 1.3e-4
    assert np.all(np.abs(got[0, :, :L] - paid) <= rel * paid + n * b.Hq * 2.0 ** -120)
    assert np.all(got[0][:, off] == 0.0)


def test_same_bits_each_time_and_workspaces():
    """Equal calls give equal bits, with the least workspace too the same
    numbers; back-to-back calls share the cached workspace."""
    b = Batch(61, [3000, 500, 40, 1500], [1, 1, 40, 4], 8, 2, 128, 16)
    T = b.q.shape[0]
    first = b.run(out=torch.zeros_like(b.old)).clone()
    for _ in range(3):
        assert torch.equal(b.run(out=torch.zeros_like(b.old)), first)
    context = min(b.old.shape[2], b.tables.shape[1] * 16)
    need = pkv.scores_workspace_min(4, T, 8, 2, context)
    small = b.run(out=torch.zeros_like(b.old), workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert torch.allclose(small, first, rtol=5e-4, atol=1e-7)
    with pytest.raises(ValueError):
        b.run(workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    other = Batch(62, [700, 900], [3, 1], 8, 2, 128, 16)
    want = other.run(out=torch.zeros_like(other.old)).clone()
    for _ in range(10):
        x = b.run(out=torch.zeros_like(b.old))
        y = other.run(out=torch.zeros_like(other.old))
    assert torch.equal(x, first) and torch.equal(y, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("group,D", [(1, 128), (7, 64), (16, 128)])
def test_least_workspace(group, D, dtype):
    """Few rows whose logits there is no room for are computed twice."""
    if dtype == "fp8" and D != 128:
        pytest.skip("FP8 pools: head_dim 128")
    lens, qlens = [900, 64, 1, 130, 257], [1, 2, 1, 0, 1]
    b = Batch(group + D, lens, qlens, 2 * group, 2, D, 16, torch.float32 if dtype == "f32" else torch.bfloat16,
              dtype == "fp8")
    need = pkv.scores_workspace_min(len(lens), b.q.shape[0], 2 * group, 2, min(b.old.shape[2], b.tables.shape[1] * 16))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for causal, decay in ((True, 1.0), (False, 0.5)):
        before = b.old.clone()
        b.check(b.run(causal, decay, out=b.old.clone(), workspace=ws), before, causal=causal, decay=decay)
    assert pkv.device_errors() == 0


def test_graph_replay_follows_its_inputs():
    """A captured step replayed with longer sequences and other queries."""
    b = Batch(71, [300, 900], [1, 1], 8, 2, 128, 16)
    ctx = torch.tensor([100, 200], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(b.old)
    ws = torch.empty(pkv.scores_workspace_size(2, 2, 8, 2, 1 << 10), dtype=torch.uint8, device="cuda")
    b.run(out=out, context_lens=ctx, workspace=ws, max_query_len=1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(out=out, context_lens=ctx, workspace=ws, max_query_len=1)
    for lens in ([300, 900], [1, 17], [257, 128]):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        out.copy_(b.old)
        g.replay()
        torch.cuda.synchronize()
        held, b.lens = b.lens, lens
        b.check(out, b.old)
        b.lens = held


def test_graphs_keep_their_own_workspace():
    """Two steps captured on one stream without a workspace, and later eager
    calls there that need a larger one: each replay is right, also both at
    once on two streams."""
    pair = [Batch(75 + i, [900 + 50 * i, 300], [1, 1 + 39 * i], 8, 2, 128, 16) for i in range(2)]
    large = Batch(79, [6000, 5000], [40, 1], 8, 2, 128, 16)
    want = [b.run(out=b.old.clone()) for b in pair]
    want_large = large.run(out=large.old.clone())
    outs = [b.old.clone() for b in pair]
    graphs = [torch.cuda.CUDAGraph() for _ in pair]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for b in pair:
            b.run(out=b.old.clone())  # eager on the stream of the captures
        for b, g, out in zip(pair, graphs, outs):
            with torch.cuda.graph(g, stream=st):
                b.run(out=out)
        got = large.run(out=large.old.clone())
    torch.cuda.synchronize()
    assert torch.equal(got, want_large)
    fill = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(32)]
    streams = [torch.cuda.Stream() for _ in pair]
    for _ in range(20):
        for b, out in zip(pair, outs):
            out.copy_(b.old)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert all(bool((x == 7).all()) for x in fill)
    assert pkv.device_errors() == 0


def test_other_stream():
    b = Batch(81, [5000, 300], [1, 1], 8, 2, 128, 16)
    want = b.run(out=torch.zeros_like(b.old)).clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = b.run(out=torch.zeros_like(b.old))
    st.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    b = Batch(91, [30], [1], 4, 2, 64, 16)
    for bad in (dict(scores=b.old.double()), dict(scores=b.old[:, :1]), dict(scores=b.old[0]), dict(q=b.q.float()),
                dict(context_lens=b.args["context_lens"].long()), dict(block_tables=b.args["block_tables"].long()),
                dict(query_start_loc=b.args["query_start_loc"][:1]), dict(scores=b.old.transpose(1, 2)),
                dict(out=b.old[:1]), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                dict(q=b.q.cpu()), dict(score_rows=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        if "score_rows" in bad:
            b.row_arg, bad = bad["score_rows"], {}
        with pytest.raises(ValueError):
            b.run(**bad)
        b.row_arg = None
    with pytest.raises(pkv.LibraryError):
        b.run(decay=-1.0)
    assert torch.equal(b.run(q=b.q[:0], out=torch.zeros_like(b.old),
                             query_start_loc=torch.zeros(2, dtype=torch.int32, device="cuda")), torch.zeros_like(b.old))


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("Hkv,group", [(1, 1), (1, 2), (3, 1), (3, 2), (1, 3)])
def test_wider_sequences_after_narrow_ones(Hkv, group, dtype):
    """One or two rows over an odd number of keys (of all kv heads) end their
    kept logits between 16-byte boundaries; the sequences after them have four
    rows and more, whose logits are read 16 bytes at a time.  With the plan made
    by the kernel (a promised query length) and by a launch of its own."""
    lens = [3, 8, 1, 41, 129, 77, 255, 300, 5, 513]
    for qlens, most in (([1, 3, 1, 2, 1, 5, 2, 5, 1, 5], 5), ([1, 3, 1, 2, 1, 5, 2, 9, 1, 20], 0)):
        b = Batch(Hkv * 8 + group, lens, qlens, Hkv * group, Hkv, 128, 16,
                  torch.float32 if dtype == "f32" else torch.bfloat16, dtype == "fp8")
        before = b.old.clone()
        b.check(b.run(out=b.old.clone(), max_query_len=most), before)
        assert pkv.device_errors() == 0


@pytest.mark.parametrize("n,L", [(512, 1 << 20), (4096, 5000)])
def test_many_row_tiles_over_many_ranges(n, L):
    """The lse of a head's rows are combined row tile by row tile: 4096 rows
    over 1024 ranges of keys are 8 million partials, which one warp would read
    in tens of milliseconds while the column items wait.  No wait may last
    longer than 10 ms here.

    Tolerance: that of Batch.check, and the partials' running sum: each of the
    ranges rescales it by an exponential (2^-22) and rounds twice (2^-24)."""
    g = torch.Generator("cuda").manual_seed(n)
    D, G, bs = 64, 8, 64
    NB = -(-L // bs)
    kc = torch.randn(NB, bs, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(n, G, D, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(NB, generator=g, device="cuda", dtype=torch.int32).view(1, NB)
    old = torch.rand(1, 1, L, generator=g, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    call = lambda: pkv.paged_attention_scores(q, kc, table, i32([L]), i32([0, n]), old, 0.125, out=torch.empty_like(old))  # noqa: E731
    call()  # sets up the kernel
    pkv.debug_fault(0, 10_000_000)
    got = call()
    assert pkv.device_errors() == 0
    Q, K = q.double().reshape(n * G, D), kc[table[0].long()].reshape(-1, D)[:L]
    last = torch.arange(n, device="cuda").repeat_interleave(G).view(-1, 1) + (L - n)  # the key each row sees last
    step = 8192
    logits = lambda j: (Q @ K[j:j + step].double().T * 0.125).masked_fill_(  # noqa: E731
        torch.arange(j, min(L, j + step), device="cuda") > last, -math.inf)
    lse = torch.full((n * G, 1), -math.inf, dtype=torch.float64, device="cuda")
    for j in range(0, L, step):
        lse = torch.logaddexp(lse, logits(j).logsumexp(1, keepdim=True))
    paid = torch.cat([(logits(j) - lse).exp_().sum(0) for j in range(0, L, step)])
    want = paid + torch.where(torch.arange(L, device="cuda") < L - n, old[0, 0].double(), 0.0)
    dots = float(Q.abs().amax(0) @ K.abs().amax(0).double())
    rel = 2 * 0.125 * (D + 2) * 2.0 ** -24 * dots + 2 * 2.0 ** -22 + 1.3e-4 + -(-L // 1024) * (2.0 ** -22 + 2 * 2.0 ** -24)
    assert torch.all((got[0, 0] - want).abs() <= rel * paid + 2.0 ** -22 * want + n * G * 2.0 ** -120)


def test_two_threads_on_one_stream():
    """Calls of different shapes from two threads, whose launches fall between
    one another's on the stream they share: each has a workspace of its own, and
    a third thread's larger calls leave theirs alone."""
    many = [Batch(111, [900, 300, 2000], [1, 40, 3], 8, 2, 128, 16), Batch(112, [64] * 40, [1] * 40, 16, 4, 128, 16),
            Batch(113, [6000, 5000], [70, 1], 8, 2, 128, 16)]
    want = [b.run(out=b.old.clone()) for b in many]
    outs = [[b.old.clone() for _ in range(60)] for b in many]
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(many)), []

    def calls(b, mine):
        try:
            start.wait()
            for out in mine:
                b.run(out=out)
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=calls, args=a) for a in zip(many, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and pkv.device_errors() == 0
    for w, mine in zip(want, outs):
        assert all(torch.equal(x, w) for x in mine)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("n", [1, 3, 4, 40])
@pytest.mark.parametrize("first", [0, 1024])
def test_keys_of_nan_among_others(first, n, dtype):
    """A row that sees a NaN logit has no weights, also where the NaN keys fill
    whole chunks of the sequence (1024 keys of 128, 256 and 1024 each), whose
    maximum is none: all its keys get NaN.  The other kv head is as it was."""
    L = 5000
    b = Batch(135 + n, [L, 700], [n, n], 8, 2, 128, 16, torch.float32 if dtype == "f32" else torch.bfloat16,
              dtype == "fp8")
    want = b.run(out=b.old.clone())
    for j in range(first, first + 1024):
        b.kc[b.tables[0, j // 16], j % 16, 1] = 0x7F if dtype == "fp8" else math.nan
    for workspace in (None, pkv.scores_workspace_min(2, 2 * n, 8, 2, b.old.shape[2])):
        ws = None if workspace is None else torch.empty(workspace, dtype=torch.uint8, device="cuda")
        got = b.run(out=b.old.clone(), workspace=ws)
        assert torch.isnan(got[0, 1, :L]).all()
        assert torch.isfinite(got[0, 0]).all() and torch.isfinite(got[1:]).all()
        assert ws is not None or torch.equal(got[0, 0], want[0, 0]) and torch.equal(got[1:], want[1:])
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("Hq,n", [(2, 4), (8, 3), (8, 4), (8, 40), (6, 150)])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_of_nan_keep_to_what_they_see(causal, Hq, n, dtype):
    """A NaN query makes the weights of the keys it sees NaN, and leaves those
    of the step's later tokens, which it does not see, to the other rows."""
    lens = [700, 1500, 300]
    b = Batch(141 + Hq + n, lens, [n] * 3, Hq, 2, 128, 16, torch.float32 if dtype == "f32" else torch.bfloat16,
              dtype == "fp8")
    group, at = Hq // 2, n // 2 - 1
    plain = b.run(causal, decay=0.0, out=b.old.clone())
    b.check(plain, b.old, causal=causal, decay=0.0)
    b.q[n + at, group:] = math.nan  # of the second sequence, the second kv head's
    for workspace in (None, pkv.scores_workspace_min(3, 3 * n, Hq, 2, min(b.old.shape[2], b.tables.shape[1] * 16))):
        ws = None if workspace is None else torch.empty(workspace, dtype=torch.uint8, device="cuda")
        got = b.run(causal, decay=0.0, out=b.old.clone(), workspace=ws)
        seen = 1500 - n + at + 1 if causal else 1500
        assert torch.isnan(got[1, 1, :seen]).all()
        if ws is None:
            assert torch.equal(got[0], plain[0]) and torch.equal(got[2:], plain[2:]) and torch.equal(got[1, 0], plain[1, 0])
        # the other rows' weights, one after another in another order: at most n * group additions of 2^-24 of the sum
        assert torch.allclose(got[1, 1, seen:1500], plain[1, 1, seen:1500], rtol=5e-4 + n * group * 2.0 ** -23, atol=0)
        assert torch.equal(got[1, 1, 1500:], plain[1, 1, 1500:])
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("most", [0, 4])
@pytest.mark.parametrize("qsl,good", [([0, 4, 0, 4, 5], [0, 3]), ([0, 2, 2, 1, 5], [0]), ([1, 0, 1, 3, 5], [2, 3]),
                                      ([0, 3, 1, 4, 5], [0, 3]), ([0, 1, 5, 4, 5], [0, 1])])
def test_overlapping_queries_are_reported(qsl, good, most, dtype):
    """A query_start_loc entry below an earlier one makes its sequences invalid
    (reported, their rows as they were); the others get the scores of the
    queries that are theirs."""
    b = Batch(151, [100, 60, 80, 50], [1, 2, 1, 1], 8, 2, 128, 16, torch.float32 if dtype == "f32" else torch.bfloat16,
              dtype == "fp8")
    b.qsl, b.qlens = np.array(qsl), np.diff(qsl).tolist()
    before = b.old.clone()
    got = b.run(out=b.old.clone(), query_start_loc=torch.tensor(qsl, dtype=torch.int32, device="cuda"), max_query_len=most)
    assert pkv.device_errors() == pkv.DEVERR["bad_sequence"]
    b.check(got, before, seqs=good)

"""A serving loop that keeps every sequence within a budget, end to end on the
GPU: rotary write, attention, running scores, and, when a sequence has grown
past its limit, selection, compaction and the block manager's compaction,
with a shared cached prefix, a fork and sequences that come and go.  At every
step each sequence's cache read through its table is bit for bit the rows that
a host simulation of the kept tokens says it holds, the attention is the fp64
oracle's over them, and the scores follow the fp64 definition."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from gpu_util import TOL, to_f64
from oracle import budget as ob
from oracle import paged_oracle as po

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS = 8, 2, 128, 16


class Seq:
    def __init__(self, row):
        self.row = row         # of the running scores
        self.pos = 0           # next position (runs ahead of the cache after an eviction)
        self.k = [[] for _ in range(HKV)]   # rows the cache of each head holds (fp64 of what was written)
        self.v = [[] for _ in range(HKV)]
        self.s = [np.zeros(0) for _ in range(HKV)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bounded_cache_serving_loop(dtype):
    rng = np.random.default_rng(11)
    tname = "bf16" if dtype == torch.bfloat16 else "f32"
    NB, MB, ROWS, LEN = 160, 24, 6, 24 * BS
    limit, budget, sink, recent = 150, 90, 4, 24
    mgr = pkv.BlockManager(NB, BS, MB)
    kc = torch.full((NB, BS, HKV, D), float("nan"), dtype=dtype, device="cuda")
    vc = kc.clone()
    scores = torch.full((ROWS, HKV, LEN), 1e9, device="cuda")   # stale
    inv = pkv.rope_frequencies(D, 10000.0, scaling="bands", factor=4.0, original_max_position=512)
    f = inv.cpu().numpy()
    scale = 1 / math.sqrt(D)
    dev = lambda a, t=np.int32: torch.from_numpy(np.ascontiguousarray(a, dtype=t)).cuda()  # noqa: E731
    seqs = {}

    def step(ids, n_new):
        T = sum(n_new)
        meta = mgr.step(ids, n_new)
        pkv.copy_blocks(kc, vc, meta["copies"])
        rows = torch.from_numpy(rng.standard_normal((T, HQ + 2 * HKV, D)).astype(np.float32)).to(dtype).cuda()
        q, k, v = rows[:, :HQ], rows[:, HQ:HQ + HKV], rows[:, HQ + HKV:]
        pos = np.concatenate([seqs[s].pos + np.arange(n) for s, n in zip(ids, n_new)] or [np.zeros(0)])
        bt, ctx, qsl = dev(meta["block_tables"]), dev(meta["context_lens"]), dev(meta["query_start_loc"])
        qr = pkv.paged_kv_write_rope(q, k, v, dev(pos, np.int64), inv, dev(meta["slot_mapping"], np.int64), kc, vc)
        out = pkv.paged_attention_forward(qr, kc, vc, bt, ctx, qsl, scale, True)
        pkv.paged_attention_scores(qr, kc, bt, ctx, qsl, scores, scale, True, decay=0.9,
                                   score_rows=dev([seqs[s].row for s in ids]))
        torch.cuda.synchronize()
        # the rotation itself is checked elsewhere: the pool's rows must be one rounding off the fp64 ones
        got_k = to_f64(kc).reshape(-1, HKV, D)[meta["slot_mapping"]]
        want_k = ob.rope(to_f64(k.contiguous()), pos.astype(np.int64), f)
        assert np.all(np.abs(got_k - want_k) <= 2.0 ** -8 * np.abs(want_k) + 1e-5)
        got_q, got_v, got_o, got_s = to_f64(qr), to_f64(v.contiguous()), to_f64(out), scores.cpu().numpy()
        at = 0
        for i, (s, n) in enumerate(zip(ids, n_new)):
            sq = seqs[s]
            sq.pos += n
            for h in range(HKV):
                sq.k[h] += list(got_k[at:at + n, h])
                sq.v[h] += list(got_v[at:at + n, h])
            L = len(sq.k[0])
            assert L == meta["context_lens"][i]
            table = meta["block_tables"][i][:-(-L // BS)]
            K = to_f64(kc)[table].reshape(-1, HKV, D)[:L]
            V = to_f64(vc)[table].reshape(-1, HKV, D)[:L]
            for h in range(HKV):
                assert np.array_equal(K[:, h], np.array(sq.k[h])) and np.array_equal(V[:, h], np.array(sq.v[h])), (s, h)
            if n == 0:
                continue
            want_o = po.attend(got_q[at:at + n], K, V, scale, True)
            err = np.abs(got_o[at:at + n] - want_o)
            assert err.max() <= TOL[tname][0] and err.mean() <= TOL[tname][1]
            old = np.zeros((HKV, L))
            for h in range(HKV):
                old[h, :len(sq.s[h])] = sq.s[h]
            want_s = ob.scores_update(got_q[at:at + n], K, old, scale, True, 0.9)
            # each weight within 3e-4 of itself (the scores' own tests derive it); the old scores are the device's own
            assert np.all(np.abs(got_s[sq.row, :, :L] - want_s) <= 3e-4 * want_s + 1e-6)
            sq.s = [got_s[sq.row, h, :L].astype(np.float64) for h in range(HKV)]   # follow the device's ties
            at += n

    def evict(ids):
        lens = [len(seqs[s].k[0]) for s in ids]
        rows = dev([seqs[s].row for s in ids])
        kept = pkv.paged_kv_select(scores, dev(lens), budget, num_sink=sink, num_recent=recent, score_rows=rows)
        moved = mgr.compact(ids, budget)
        pkv.paged_kv_compact(kc, vc, dev(moved["block_tables"]), kept, dst_block_tables=dev(moved["dst_block_tables"]),
                             scores=scores, score_rows=rows)
        kept = kept.cpu().numpy()
        for i, s in enumerate(ids):
            sq = seqs[s]
            assert moved["context_lens"][i] == min(lens[i], budget) == mgr.num_tokens(s)
            for h in range(HKV):
                want = ob.select(sq.s[h].astype(np.float32), lens[i], budget, sink, recent)
                assert kept[i, h, :len(want)].tolist() == want
                sq.k[h] = [sq.k[h][j] for j in want]
                sq.v[h] = [sq.v[h][j] for j in want]
                sq.s[h] = sq.s[h][want]

    # a prompt whose full blocks go to the prefix cache, two more on them, and a fork
    tokens = list(range(100))
    seqs[0] = Seq(0)
    step([0], [100])
    mgr.add_prefix(0, tokens)
    for s in (1, 2):
        seqs[s] = Seq(s)
        got = mgr.try_get_prefix_blocks(s, tokens + [500 + s] * 60)
        assert got == 96
        seqs[s].pos = got
        for h in range(HKV):
            seqs[s].k[h] = list(seqs[0].k[h][:got])
            seqs[s].v[h] = list(seqs[0].v[h][:got])
            seqs[s].s[h] = np.zeros(got)
    scores[1:3, :, :96] = 0.0   # a reader of cached tokens starts their scores itself
    step([1, 2], [64, 64])
    mgr.fork(1, 3)
    seqs[3] = Seq(3)
    seqs[3].pos = seqs[1].pos
    for h in range(HKV):
        seqs[3].k[h], seqs[3].v[h], seqs[3].s[h] = list(seqs[1].k[h]), list(seqs[1].v[h]), seqs[1].s[h].copy()
    scores[3] = scores[1]
    used = mgr.stats()["in_use"]
    evict([0, 1, 2, 3])                       # 0 is short enough; 1, 2, 3 share blocks
    assert len(seqs[0].k[0]) == 90 and mgr.stats()["in_use"] <= used + 12
    step([0, 1, 2, 3], [1, 1, 5, 0])
    for it in range(24):
        ids = [s for s in seqs if rng.random() < 0.9]
        step(ids, [int(rng.choice([1, 1, 1, 5, 17])) for _ in ids])
        over = [s for s in seqs if len(seqs[s].k[0]) > limit]
        if over:
            evict(over)
        if it == 10:
            mgr.free(2)
            del seqs[2]
            seqs[7] = Seq(5)
            step([7], [33])
    # the cached prefix is still what it was
    n = mgr.try_get_prefix_blocks(50, tokens + [1])
    assert n == 96
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("steps", [3])
def test_captured_step_replays(steps):
    """Rotary write, attention, scores, selection and compaction of one step
    captured in one graph and replayed give what the eager calls give."""
    g = torch.Generator().manual_seed(1)
    NB, MB, B, L = 96, 24, 3, 300
    bt = torch.arange(B * MB, dtype=torch.int32).view(B, MB).cuda()
    pools = [torch.randn(NB, BS, HKV, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    rows = torch.randn(B, HQ + 2 * HKV, D, generator=g).to(torch.bfloat16).cuda()
    sc0 = torch.rand(B, HKV, MB * BS, generator=g).cuda()
    ctx = torch.tensor([L, L - 7, 250], dtype=torch.int32, device="cuda")
    qsl = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([int(bt[s, (int(ctx[s]) - 1) // BS]) * BS + (int(ctx[s]) - 1) % BS for s in range(B)],
                         device="cuda")
    pos = torch.tensor([5000, 6000, 7000], device="cuda")
    inv = pkv.rope_frequencies(D)
    q_out, out = torch.empty(B, HQ, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, HQ, D, dtype=torch.bfloat16,
                                                                                         device="cuda")
    kept = torch.empty(B, HKV, 128, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(pkv.workspace_size(B, B, HQ, HKV, D), pkv.scores_workspace_size(B, B, HQ, HKV, MB * BS)),
                     dtype=torch.uint8, device="cuda")

    def one(kc, vc, sc):
        pkv.paged_kv_write_rope(rows[:, :HQ], rows[:, HQ:HQ + HKV], rows[:, HQ + HKV:], pos, inv, slots, kc, vc,
                                q_out=q_out)
        pkv.paged_attention_forward(q_out, kc, vc, bt, ctx, qsl, 0.09, out=out, workspace=ws, max_query_len=1)
        pkv.paged_attention_scores(q_out, kc, bt, ctx, qsl, sc, 0.09, workspace=ws, max_query_len=1)
        pkv.paged_kv_select(sc, ctx, 128, num_sink=2, num_recent=16, out=kept)
        pkv.paged_kv_compact(kc, vc, bt, kept, scores=sc)

    state = [pools[0].clone(), pools[1].clone(), sc0.clone()]
    for _ in range(steps):
        one(*state)
    want = [x.clone() for x in state] + [out.clone(), kept.clone()]
    torch.cuda.synchronize()
    live = [pools[0].clone(), pools[1].clone(), sc0.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(*live)
    for a, b in zip(live, [pools[0], pools[1], sc0]):
        a.copy_(b)
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(live + [out, kept], want):
        assert torch.equal(a, b)
    assert pkv.device_errors() == 0

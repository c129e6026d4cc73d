"""paged_kv_select and paged_kv_compact: exact against the definitions."""
import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from oracle import budget as ob

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def check_select(scores, lens, budget, sink=0, recent=0, rows=None, **kw):
    got = pkv.paged_kv_select(scores, i32(lens), budget, num_sink=sink, num_recent=recent,
                              score_rows=None if rows is None else i32(rows), **kw).cpu().numpy()
    s = scores.cpu().numpy()
    for b, L in enumerate(lens):
        r = b if rows is None else rows[b]
        for h in range(scores.shape[1]):
            want = ob.select(s[r, h], L, budget, sink, recent) if r >= 0 else []
            assert got[b, h, :len(want)].tolist() == want, (b, h, L)
            assert np.all(got[b, h, len(want):] == -1)
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (7, 2, 3), (64, 4, 60), (64, 0, 0),
                                                (300, 4, 32), (1024, 0, 1024), (2000, 16, 128)])
def test_select(budget, sink, recent):
    rng = np.random.default_rng(budget + sink)
    lens = [0, 1, 2, budget - 1, budget, budget + 1, budget + 2, 1023, 1024, 1025, 2049, 3001]
    s = rng.random((len(lens), 3, 3001)).astype(np.float32) ** 4
    s[:, 1] = np.floor(s[:, 1] * 8)      # many ties
    s[:, 2] = rng.standard_normal(s[:, 2].shape) * 1e-3
    check_select(torch.from_numpy(s).cuda(), lens, budget, sink, recent)


def test_select_odd_values():
    """Ties throughout, infinities, NaN, signed zeros, subnormals, and values
    that differ in their last bits only."""
    rng = np.random.default_rng(7)
    pool = np.array([np.inf, -np.inf, np.nan, 0.0, -0.0, 1e-42, -1e-42, 1.0, np.nextafter(np.float32(1), np.float32(2)),
                     3.4e38, -3.4e38], np.float32)
    s = np.stack([np.zeros((2, 500), np.float32), rng.choice(pool, (2, 500)),
                  np.full((2, 500), np.nan, np.float32),
                  (1 + rng.integers(0, 40, (2, 500)) * 2.0 ** -23).astype(np.float32)])
    for budget in (1, 13, 250, 499):
        check_select(torch.from_numpy(s).cuda(), [500, 500, 500, 500], budget, min(1, budget // 2), budget // 3)


def test_select_long_rows():
    rng = np.random.default_rng(8)
    L = 131072 + 37
    s = rng.random((2, 2, L + 1)).astype(np.float32)
    s[1, 0] = np.floor(s[1, 0] * 100)
    check_select(torch.from_numpy(s).cuda(), [L, 70001], 16384, 4, 1000)


def test_select_rows_and_errors():
    rng = np.random.default_rng(9)
    s = torch.from_numpy(rng.random((5, 2, 300)).astype(np.float32)).cuda()
    check_select(s, [300, 250, 10], 40, 2, 8, rows=[4, -1, 0])
    out = torch.full((2, 2, 40), 5, dtype=torch.int32, device="cuda")
    pkv.paged_kv_select(s, i32([301, 100]), 40, out=out)          # longer than its scores
    assert (out[0] == -1).all() and (out[1] >= 0).all()
    assert pkv.device_errors() == pkv.DEVERR["bad_sequence"]
    pkv.paged_kv_select(s, i32([100, 100]), 40, out=out, score_rows=i32([5, 1]))
    assert (out[0] == -1).all() and pkv.device_errors() == pkv.DEVERR["bad_sequence"]
    pkv.paged_kv_select(s, i32([-3, 100]), 40, out=out)
    assert (out[0] == -1).all() and pkv.device_errors() == pkv.DEVERR["bad_sequence"]
    for bad in (dict(budget=40, num_sink=30, num_recent=11), dict(budget=0), dict(budget=4, num_sink=-1)):
        with pytest.raises(pkv.LibraryError):
            pkv.paged_kv_select(s, i32([10, 10]), **bad)
    for bad in (dict(scores=s.double()), dict(scores=s[:, :, ::2]), dict(out=out[:, :, :39]), dict(scores=s[:1]),
                dict(context_lens=torch.tensor([1, 2], device="cuda"))):
        with pytest.raises(ValueError):
            pkv.paged_kv_select(**{**dict(scores=s, context_lens=i32([10, 10]), budget=40), **bad})
    assert pkv.paged_kv_select(s, i32([]), 40).shape == (0, 2, 40)


DT = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.uint8}


def make_pool(rng, NB, bs, Hkv, D, dtype):
    if dtype == "fp8":
        a = torch.from_numpy(rng.integers(0, 256, (NB, bs, Hkv, D)).astype(np.uint8)).cuda()
    else:
        a = torch.from_numpy(rng.standard_normal((NB, bs, Hkv, D)).astype(np.float32)).to(DT[dtype]).cuda()
    return a


def bits(t):
    return (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy()


def kept_of(rng, lens, Hkv, budget, how):
    kept = np.full((len(lens), Hkv, budget), -1, np.int32)
    for s, L in enumerate(lens):
        for h in range(Hkv):
            n = min(L, budget)
            if how == "random":
                p = np.sort(rng.choice(L, n, replace=False)) if L else []
            elif how == "last":
                p = np.arange(L - n, L)
            elif how == "first":
                p = np.arange(n)
            else:  # sinks, then the last ones
                p = np.concatenate([np.arange(min(3, n)), np.arange(L - n + min(3, n), L)])
            kept[s, h, :n] = p
    return kept


@pytest.mark.parametrize("how", ["random", "last", "first", "sinks"])
@pytest.mark.parametrize("dtype,Hkv,D,bs", [("bf16", 2, 128, 16), ("bf16", 3, 64, 8), ("f32", 1, 64, 64),
                                            ("f32", 2, 128, 32), ("fp8", 4, 128, 16), ("fp8", 1, 16, 16),
                                            ("bf16", 2, 40, 24)])
def test_compact_in_place(dtype, Hkv, D, bs, how):
    rng = np.random.default_rng(D + bs + len(how))
    lens, budget = [0, 1, 5, 70, 300, 299, 1500], 200
    need = [-(-L // bs) for L in lens]
    NB = sum(need) + 2
    order, at = rng.permutation(NB), 0
    tables = np.full((len(lens), max(need)), -1, np.int32)
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += n
    kept = kept_of(rng, lens, Hkv, budget, how)
    kc, vc = make_pool(rng, NB, bs, Hkv, D, dtype), make_pool(rng, NB, bs, Hkv, D, dtype)
    rows = [6, 2, 0, 1, 5, 3, 4]
    sc = torch.from_numpy(rng.random((8, Hkv, 1500)).astype(np.float32)).cuda()
    want_k, want_v, want_s = bits(kc).copy(), bits(vc).copy(), sc.cpu().numpy()
    was_k, was_v, was_s = want_k.copy(), want_v.copy(), want_s.copy()
    for s in range(len(lens)):
        for h in range(Hkv):
            p = [int(x) for x in kept[s, h] if x >= 0]
            ob.compact_head(want_k, tables[s], tables[s], p, h, was_k)
            ob.compact_head(want_v, tables[s], tables[s], p, h, was_v)
            want_s[rows[s], h, :len(p)] = was_s[rows[s], h, p]
    pkv.paged_kv_compact(kc, vc, i32(tables), i32(kept), scores=sc, score_rows=i32(rows))
    assert np.array_equal(bits(kc), want_k, equal_nan=dtype == "f32")
    assert np.array_equal(bits(vc), want_v, equal_nan=dtype == "f32")
    assert np.array_equal(sc.cpu().numpy(), want_s)
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_compact_to_other_blocks(dtype):
    """A shared first block goes to a fresh one, the others stay in place;
    the shared block keeps its rows; no scores."""
    rng = np.random.default_rng(3)
    bs, Hkv, D, NB = 16, 2, 128, 40
    lens, budget = [200, 150], 60
    tables = np.full((2, 13), -1, np.int32)
    tables[0, :13] = rng.permutation(20)[:13]
    tables[1, :10] = 20 + rng.permutation(12)[:10]
    tables[1, 0] = tables[0, 0]
    dst = np.full_like(tables, -1)
    dst[0, :4], dst[1, :4] = tables[0, :4], tables[1, :4]
    dst[0, 0], dst[1, 0] = 38, 39
    kept = kept_of(rng, lens, Hkv, budget, "random")
    kc, vc = make_pool(rng, NB, bs, Hkv, D, dtype), make_pool(rng, NB, bs, Hkv, D, dtype)
    want_k, want_v = bits(kc).copy(), bits(vc).copy()
    was_k, was_v = want_k.copy(), want_v.copy()
    for s in range(2):
        for h in range(Hkv):
            ob.compact_head(want_k, tables[s], dst[s], kept[s, h].tolist(), h, was_k)
            ob.compact_head(want_v, tables[s], dst[s], kept[s, h].tolist(), h, was_v)
    pkv.paged_kv_compact(kc, vc, i32(tables), i32(kept), dst_block_tables=i32(dst))
    assert np.array_equal(bits(kc), want_k) and np.array_equal(bits(vc), want_v)
    assert np.array_equal(want_k[tables[0, 0]], was_k[tables[0, 0]])
    assert pkv.device_errors() == 0


def test_compact_long_in_place():
    """Many rounds of one (sequence, head): 30 000 kept of 40 000."""
    rng = np.random.default_rng(5)
    bs, NB = 16, 2500
    tables = rng.permutation(NB).astype(np.int32)[None]
    kept = np.sort(rng.choice(40000, 30000, replace=False)).astype(np.int32)[None, None]
    kc, vc = make_pool(rng, NB, bs, 1, 64, "bf16"), make_pool(rng, NB, bs, 1, 64, "bf16")
    sc = torch.from_numpy(rng.random((1, 1, 40000)).astype(np.float32)).cuda()
    want_k, want_v, want_s = bits(kc).copy(), bits(vc).copy(), sc.cpu().numpy().copy()
    want_s[0, 0, :30000] = want_s[0, 0, kept[0, 0]]
    ob.compact_head(want_k, tables[0], tables[0], kept[0, 0].tolist(), 0)
    ob.compact_head(want_v, tables[0], tables[0], kept[0, 0].tolist(), 0)
    pkv.paged_kv_compact(kc, vc, i32(tables), i32(kept), scores=sc)
    assert np.array_equal(bits(kc), want_k) and np.array_equal(bits(vc), want_v)
    assert np.array_equal(sc.cpu().numpy(), want_s)


def test_compact_bad_inputs():
    rng = np.random.default_rng(6)
    bs, Hkv, D, NB = 16, 1, 64, 8
    tables = np.array([[3, 5, 1, 7]], np.int32)
    kc, vc = make_pool(rng, NB, bs, Hkv, D, "bf16"), make_pool(rng, NB, bs, Hkv, D, "bf16")
    was = bits(kc).copy()
    # a source past the table, and one in a block outside the pool: zeros
    t = tables.copy()
    t[0, 2] = 99
    k1 = kc.clone()
    pkv.paged_kv_compact(k1, vc.clone(), i32(t), i32([[[2, 40, 64, -1]]]))
    assert pkv.device_errors() == pkv.DEVERR["block_out_of_range"]
    assert np.array_equal(bits(k1)[3, 0], was[3, 2]) and not bits(k1)[3, 1:3].any()
    # a destination outside the pool is skipped
    k1 = kc.clone()
    pkv.paged_kv_compact(k1, vc.clone(), i32(tables), i32([[[2, 40, -1, 9]]]), dst_block_tables=i32([[-1, 0, 0, 0]]))
    assert pkv.device_errors() == pkv.DEVERR["block_out_of_range"] and np.array_equal(bits(k1), was)
    # not ascending: flagged, nothing outside the sequence's first rows is written
    k1 = kc.clone()
    pkv.paged_kv_compact(k1, vc.clone(), i32(tables), i32([[[9, 4, 4]]]))
    assert pkv.device_errors() == pkv.DEVERR["bad_sequence"]
    now = bits(k1)
    now[3, :3] = was[3, :3]
    assert np.array_equal(now, was)
    sc = torch.zeros(1, 1, 20, device="cuda")
    pkv.paged_kv_compact(k1, vc, i32(tables), i32([[[9, 24]]]), scores=sc, score_rows=i32([1]))
    assert pkv.device_errors() == pkv.DEVERR["bad_sequence"]
    pkv.paged_kv_compact(k1, vc, i32(tables), i32([[[9, 24]]]), scores=sc)
    assert pkv.device_errors() == pkv.DEVERR["block_out_of_range"]
    for bad in (dict(kept=i32([[[1]], [[2]]])), dict(kept=i32([[[1], [2]]])), dict(v_cache=vc.float()),
                dict(dst_block_tables=i32([[1]])), dict(scores=sc.double()), dict(block_tables=i32(tables).long()),
                dict(k_cache=kc[:, :, :, :32])):
        with pytest.raises(ValueError):
            pkv.paged_kv_compact(**{**dict(k_cache=kc, v_cache=vc, block_tables=i32(tables), kept=i32([[[1]]])), **bad})


@pytest.mark.parametrize("kept,scores", [([0, 1, 2, 3, 4, 5], [0, 1, 2, 3]),    # stay where they are
                                         ([0, 1, 3, 5, 6, 7], [0, 1, 3, None]),  # go past the scores too
                                         ([0, 1, 2, 3, 9, -1], [0, 1, 2, 3])])
def test_compact_positions_past_the_scores(kept, scores):
    """A kept position that the running scores have no place for is reported,
    whether its row moves or not, and whether it has a place after the move."""
    rng = np.random.default_rng(9)
    kc, vc = make_pool(rng, 4, 16, 1, 64, "bf16"), make_pool(rng, 4, 16, 1, 64, "bf16")
    sc = torch.tensor([[[10.0, 11.0, 12.0, 13.0]]], device="cuda")
    want = [0.0 if j is None else 10.0 + j for j in scores]
    was = bits(kc).copy()
    pkv.paged_kv_compact(kc, vc, i32([[2]]), i32([[kept]]), scores=sc)
    assert pkv.device_errors() == pkv.DEVERR["block_out_of_range"]
    assert sc.cpu().tolist() == [[want]]
    live = [j for j in kept if j >= 0]
    assert np.array_equal(bits(kc)[2, :len(live)], was[2, live])

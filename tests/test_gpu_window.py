"""paged_attention_window_forward against the fp64 definition.

Tolerances.  bf16: the softmax weights are rounded to bf16 (2^-9 of each, half
a step below its power of two) and the output once more (2^-9 of it), and the
logits, weights and sums are fp32 over at most 700 keys (below 2^-13 together
for |logit| <= 16): with |v| <= 4.5 at most (2^-9 + 2^-13) * 4.5 + 2^-9 * 4.5 <
2e-2.  fp32: exponentials good to 2^-21 (two units and a logit's rounding at
|logit| <= 16), at most 700 sums' rounding: 1e-4 with |v| <= 4.5.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from gpu_util import TOL, to_f64
from oracle import serving

pytestmark = pytest.mark.gpu


def batch(seed, lens, n, Hq, Hkv, D, bs, dtype):
    """Pools whose unused rows are NaN, and a batch's tensors on the device."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-L // bs) for L in lens]
    NB = sum(need) + 3
    order = torch.randperm(NB, generator=g)
    tables = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
    kc = torch.full((NB, bs, Hkv, D), float("nan"))
    vc = kc.clone()
    at = 0
    for s, L in enumerate(lens):
        tables[s, :need[s]] = order[at:at + need[s]].to(torch.int32)
        at += need[s]
        for j in range(need[s]):
            m = min(bs, L - j * bs)
            kc[tables[s, j], :m] = torch.randn(m, Hkv, D, generator=g)
            vc[tables[s, j], :m] = torch.randn(m, Hkv, D, generator=g).clamp(-4.5, 4.5)
    qsl = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = torch.randn(int(qsl[-1]), Hq, D, generator=g).to(dtype)
    return dict(q=q.cuda(), kc=kc.to(dtype).cuda(), vc=vc.to(dtype).cuda(), tables=tables.cuda(),
                lens=torch.tensor(lens, dtype=torch.int32).cuda(), qsl=torch.from_numpy(qsl).cuda())


def rows(pool, table, L):
    bs = pool.shape[1]
    return pool[table[:-(-L // bs)].long().cpu().numpy()].reshape((-1,) + pool.shape[2:])[:L]


def check(b, out, scale, window, sink, dtype):
    kc, vc, q, got = (to_f64(b[x]) if x != "out" else to_f64(out) for x in ("kc", "vc", "q", "out"))
    qsl, lens = b["qsl"].tolist(), b["lens"].tolist()
    tmax, tmean = TOL["bf16" if dtype == torch.bfloat16 else "f32"]
    worst, total, count = 0.0, 0.0, 0
    for s, L in enumerate(lens):
        if qsl[s + 1] == qsl[s]:
            continue
        table = b["tables"][s]
        want = serving.window_attend(q[qsl[s]:qsl[s + 1]], rows(kc, table, L), rows(vc, table, L), scale, window, sink)
        err = np.abs(got[qsl[s]:qsl[s + 1]] - want)
        assert np.all(np.isfinite(err)), f"sequence {s}"
        worst, total, count = max(worst, err.max()), total + err.sum(), count + err.size
    assert worst <= tmax and total <= tmean * count, (worst, total / count)


LENS = [700, 1, 333, 129, 64, 512, 40, 257]
SHAPES = [  # Hq, Hkv, D, bs, dtype
    (8, 2, 128, 16, torch.bfloat16),
    (16, 1, 128, 64, torch.bfloat16),
    (4, 4, 128, 8, torch.bfloat16),
    (7, 1, 128, 32, torch.bfloat16),   # a group that no tensor-core item of 16 rows holds: the CUDA-core kernel
    (6, 2, 64, 16, torch.bfloat16),
    (4, 1, 64, 32, torch.float32),
    (6, 2, 128, 16, torch.float32),
]


@pytest.mark.parametrize("window,sink", [(1, 0), (5, 1), (64, 0), (100, 4), (128, 200), (300, 129), (600, 3)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:4])) + ("-bf16" if s[4] == torch.bfloat16 else "-f32"))
def test_decode(shape, window, sink):
    Hq, Hkv, D, bs, dtype = shape
    b = batch(window + D, LENS, [1] * len(LENS), Hq, Hkv, D, bs, dtype)
    for hint in (0, 1):
        out = pkv.paged_attention_window_forward(b["q"], b["kc"], b["vc"], b["tables"], b["lens"], b["qsl"], D ** -0.5,
                                                 window, sink, max_query_len=hint)
        check(b, out, D ** -0.5, window, sink, dtype)
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("window,sink", [(1, 0), (7, 2), (130, 4), (256, 140), (500, 1)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:4])) + ("-bf16" if s[4] == torch.bfloat16 else "-f32"))
def test_several_queries(shape, window, sink):
    """Prompt chunks, verify windows, single tokens and sequences without a query, side by side."""
    Hq, Hkv, D, bs, dtype = shape
    n = [150, 1, 5, 129, 0, 3, 40, 2] if dtype == torch.bfloat16 else [9, 1, 5, 3, 0, 3, 6, 2]
    b = batch(3 * window + D, LENS, n, Hq, Hkv, D, bs, dtype)
    for hint in (0, max(n)):
        out = pkv.paged_attention_window_forward(b["q"], b["kc"], b["vc"], b["tables"], b["lens"], b["qsl"], D ** -0.5,
                                                 window, sink, max_query_len=hint)
        check(b, out, D ** -0.5, window, sink, dtype)
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:4])) + ("-bf16" if s[4] == torch.bfloat16 else "-f32"))
def test_hidden_blocks_and_rows(shape):
    """Blocks that no query sees have no valid table entry, and rows before
    every window hold NaN and infinities."""
    Hq, Hkv, D, bs, dtype = shape
    lens, n, window, sink = [700, 333, 512], [1, 2, 1], 90, 5
    b = batch(17, lens, n, Hq, Hkv, D, bs, dtype)
    for s, L in enumerate(lens):
        first = L - n[s] + 1 - window  # the first key of the first query's window
        for j in range(sink, first):
            blk = int(b["tables"][s, j // bs])
            b["kc"][blk, j % bs] = float("nan") if j % 2 else float("inf")
            b["vc"][blk, j % bs] = float("nan") if j % 3 else float("-inf")
    kept = b["tables"].clone()
    for s, L in enumerate(lens):
        first = L - n[s] + 1 - window
        for blk in range(-(-sink // bs), first // bs):
            b["tables"][s, blk] = -1 if blk % 2 else 1 << 30
    out = pkv.paged_attention_window_forward(b["q"], b["kc"], b["vc"], b["tables"], b["lens"], b["qsl"], D ** -0.5,
                                             window, sink)
    assert pkv.device_errors() == 0
    b["tables"] = kept
    check(b, out, D ** -0.5, window, sink, dtype)
    # an invalid block inside the window is reported and read as zeros
    b["tables"][0, (lens[0] - 20) // bs] = -1
    pkv.paged_attention_window_forward(b["q"], b["kc"], b["vc"], b["tables"], b["lens"], b["qsl"], D ** -0.5, window,
                                       sink)
    assert pkv.device_errors() == pkv.DEVERR["block_out_of_range"]


def test_long_context_splits():
    """A window of thousands of keys over a long context, split and unsplit."""
    lens, n = [20000, 9000], [1, 3]
    b = batch(5, lens, n, 8, 2, 128, 16, torch.bfloat16)
    least = pkv.workspace_min(2, 4, 8, 2, 128)
    for ws in (None, torch.empty(least, dtype=torch.uint8, device="cuda")):
        out = pkv.paged_attention_window_forward(b["q"], b["kc"], b["vc"], b["tables"], b["lens"], b["qsl"], 128 ** -0.5,
                                                 6001, 4, workspace=ws)
        check(b, out, 128 ** -0.5, 6001, 4, torch.bfloat16)


def test_a_window_past_every_context_is_none():
    b = batch(6, LENS, [1] * len(LENS), 8, 2, 128, 16, torch.bfloat16)
    args = b["q"], b["kc"], b["vc"], b["tables"], b["lens"], b["qsl"], 128 ** -0.5
    whole = pkv.paged_attention_forward(*args)
    for window in (700, 5000, 1 << 30):
        assert torch.equal(pkv.paged_attention_window_forward(*args, window, 3), whole)


def test_invalid_sequences_and_refusals():
    b = batch(7, [100, 50, 30], [1, 1, 1], 8, 2, 128, 16, torch.bfloat16)
    args = b["q"], b["kc"], b["vc"], b["tables"]
    bad = torch.tensor([100, 0, 30], dtype=torch.int32, device="cuda")  # a query of an empty sequence
    out = pkv.paged_attention_window_forward(*args, bad, b["qsl"], 0.1, 20, 2)
    assert pkv.device_errors() == pkv.DEVERR["bad_sequence"]
    assert torch.all(out[1] == 0) and torch.all(torch.isfinite(out.float()))
    for window, sink in ((0, 0), (-1, 0), (5, -1), ((1 << 30) + 1, 0), (5, 1 << 31), (1 << 32, 0)):
        with pytest.raises(ValueError):
            pkv.paged_attention_window_forward(*args, b["lens"], b["qsl"], 0.1, window, sink)
    empty = pkv.paged_attention_window_forward(b["q"][:0], b["kc"], b["vc"], b["tables"], b["lens"],
                                               torch.zeros(4, dtype=torch.int32, device="cuda"), 0.1, 20)
    assert empty.shape[0] == 0


def test_captured_and_replayed():
    b = batch(8, [700, 333], [1, 1], 8, 2, 128, 16, torch.bfloat16)
    out = torch.empty_like(b["q"])
    call = lambda: pkv.paged_attention_window_forward(b["q"], b["kc"], b["vc"], b["tables"], b["lens"], b["qsl"],  # noqa: E731
                                                      128 ** -0.5, 50, 4, out=out, max_query_len=1)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    b["lens"].copy_(torch.tensor([650, 200], dtype=torch.int32))
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check(b, out, 128 ** -0.5, 50, 4, torch.bfloat16)

"""A serving loop over two layers' caches, end to end on the GPU: the block
manager's step, its copies (codes with their scales), q and k heads normed and
rotated, the rows' write, and the attention over them.  One layer keeps codes
with block scales and sees every key, one keeps bf16 rows and sees a window
and sinks.  Prompts in chunks, single tokens, forks, freed and reused blocks.
At every step the pools hold what a host copy of them holds, code by code, and
each attention is the fp64 definition's over it.

Tolerances are those of the operators' own tests.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from gpu_util import TOL, to_f64
from oracle import serving
from test_gpu_fp8block_attention import TMAX, TMEAN
from test_gpu_norm_rope import CASES, HALF_STEP, expect, near
from test_gpu_norm_rope import test_fp8_pools as fp8_pools
from test_gpu_norm_rope import test_pools_and_rows as pools_and_rows

pytestmark = pytest.mark.gpu

HQ, HKV, D, ROT = 8, 2, 128, 64


def close(got, want, tol):
    err = np.abs(got - want)
    assert np.all(np.isfinite(err))
    assert err.max() <= tol[0] and err.mean() <= tol[1], (err.max(), err.mean())


@pytest.mark.parametrize("bs", [16, 8])
def test_serving_loop(bs):
    g = torch.Generator().manual_seed(bs)
    NB, MB = 640 // bs, 320 // bs
    window, sink = 40, 3
    mgr = pkv.BlockManager(NB, bs, MB)
    codes = [torch.full((NB, bs, HKV, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(NB, HKV, device="cuda") for _ in range(2)]
    plain = [torch.full((NB, bs, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    host = [(c.cpu().numpy().copy(), s.cpu().numpy().copy()) for c, s in zip(codes, scales)]
    inv = pkv.rope_frequencies(ROT)
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    dev = lambda a, t=np.int32: torch.from_numpy(np.ascontiguousarray(a, dtype=t)).cuda()  # noqa: E731
    scale = D ** -0.5
    work = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")  # one for all the calls

    def step(ids, n_new):
        T = sum(n_new)
        meta = mgr.step(ids, n_new)
        pkv.copy_blocks(*codes, meta["copies"], *scales)
        pkv.copy_blocks(*plain, meta["copies"])
        for c, s in host:
            for src, dst in meta["copies"]:
                c[dst], s[dst] = c[src], s[src]
        rows = torch.randn(T, HQ + 2 * HKV, D, generator=g).clamp(-4.5, 4.5)
        rows = (rows * torch.exp(torch.randn(T, 1, 1, generator=g)).clamp(max=1.0)).to(torch.bfloat16).cuda()
        q, k, v = rows[:, :HQ], rows[:, HQ:HQ + HKV], rows[:, HQ + HKV:]
        ctx = meta["context_lens"]
        pos = dev(np.concatenate([L - n + np.arange(n) for L, n in zip(ctx, n_new)]), np.int64)
        slots, bt = dev(meta["slot_mapping"], np.int64), dev(meta["block_tables"])
        lens, qsl = dev(ctx), dev(meta["query_start_loc"])
        hint = 1 if max(n_new) == 1 else 0
        # the layer with block scales
        k1 = torch.empty(T, HKV, D, dtype=torch.bfloat16, device="cuda")
        q1 = pkv.paged_kv_write_norm_rope(q, k, None, qw, kw, pos, inv, k_out=k1)
        pkv.paged_kv_write_fp8block(k1, v, slots, *codes, *scales)
        out1 = pkv.paged_attention_forward_fp8block(q1, *codes, *scales, bt, lens, qsl, scale, max_query_len=hint,
                                                    workspace=work)
        # the layer with a window
        q2 = pkv.paged_kv_write_norm_rope(q, k, v, qw, kw, pos, inv, slots, *plain)
        out2 = pkv.paged_attention_window_forward(q2, *plain, bt, lens, qsl, scale, window, sink, max_query_len=hint,
                                                  workspace=work)
        torch.cuda.synchronize()
        near(q1, *expect(q, qw, 1e-6, pos, inv, False, 1.0), HALF_STEP[torch.bfloat16])
        near(k1, *expect(k, kw, 1e-6, pos, inv, False, 1.0), HALF_STEP[torch.bfloat16])
        assert torch.equal(q1, q2)
        for x, (c, s), got_c, got_s in zip((k1, v), host, codes, scales):
            serving.write_blocks(x.float().cpu().numpy(), meta["slot_mapping"], c, s)
            assert np.array_equal(got_s.cpu().numpy(), s) and np.array_equal(got_c.cpu().numpy(), c)
        flat = [p.view(-1, HKV, D) for p in plain]
        assert torch.equal(flat[0][slots], k1) and torch.equal(flat[1][slots], v)
        K1, V1 = (serving.block_values(c, s) for c, s in host)
        K2, V2 = (to_f64(p) for p in plain)
        qf, o1, o2 = to_f64(q1), to_f64(out1), to_f64(out2)
        at = 0
        for i, n in enumerate(n_new):
            if n == 0:
                continue
            table = meta["block_tables"][i][:-(-ctx[i] // bs)]
            take = lambda p: p[table].reshape(-1, HKV, D)[:ctx[i]]  # noqa: E731
            mine = slice(at, at + n)
            close(o1[mine], serving.window_attend(qf[mine], take(K1), take(V1), scale), (TMAX, TMEAN))
            close(o2[mine], serving.window_attend(qf[mine], take(K2), take(V2), scale, window, sink), TOL["bf16"])
            at += n

    step([0, 1], [70, 33])
    step([0, 1], [1, 1])
    mgr.fork(0, 2)                      # shares a block that is not full
    step([0, 1, 2], [1, 1, 1])          # 0 or 2 copies it first
    step([0, 1, 2], [3, 0, 130])        # a verify window, a chunk
    mgr.free(1)
    step([3, 0], [45, 1])               # blocks of another sequence, with its codes and scales
    mgr.fork(3, 4)
    mgr.fork(3, 5)
    for _ in range(12):
        step([0, 2, 3, 4, 5], [1] * 5)
    step([4, 5], [8, 1])
    assert pkv.device_errors() == 0


BULK = [  # as the cases there, in steps of many tokens: rows come by bulk copies
    (7000, 16, 4, 128, 128, False, 16, True, True),   # several tokens to a warp
    (5000, 16, 4, 128, 64, True, 16, False, False),
    (1500, 6, 3, 80, 48, True, 16, True, False),
    (1501, 5, 2, 80, 48, False, 32, False, True),
    (1300, 8, 2, 256, 64, False, 16, True, True),
    (1250, 3, 1, 64, 32, True, 8, True, False),
    (1217, 40, 8, 256, 256, False, 16, False, True),  # too long for them
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", BULK, ids=lambda c: "-".join(map(str, c)))
def test_norm_of_many_tokens(case, dtype):
    assert case not in CASES
    pools_and_rows(case, dtype)
    if case[0] < 3000:
        fp8_pools(case, dtype)


def test_norm_of_many_tokens_past_the_pool():
    T = 2000
    q = torch.randn(T, 2, 64, device="cuda").to(torch.bfloat16)
    k = torch.randn(T, 1, 64, device="cuda").to(torch.bfloat16)
    kc = torch.full((8, 16, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    slots = torch.full((T,), -1, device="cuda")
    slots[1] = 3
    slots[1990] = 128
    pos = torch.arange(T, device="cuda")
    pkv.paged_kv_write_norm_rope(q, k, k, None, None, pos, pkv.rope_frequencies(64), slots, kc, vc)
    assert pkv.device_errors() == pkv.DEVERR["slot_out_of_range"]
    assert torch.equal(vc[0, 3], k[1])
    kc[0, 3], vc[0, 3] = 5.0, 5.0
    assert torch.all(kc == 5.0) and torch.all(vc == 5.0)


def test_norm_captured_and_replayed():
    """A captured step takes the rows, positions and slots that its tensors hold at the replay."""
    for T in (3, 1300):
        q, k = (torch.randn(T, h, 128, device="cuda").to(torch.bfloat16) for h in (4, 2))
        v = torch.randn(T, 2, 128, device="cuda").to(torch.bfloat16)
        kc = torch.zeros(100, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
        vc, inv = kc.clone(), pkv.rope_frequencies(128)
        pos, slots = torch.arange(T, device="cuda"), torch.arange(T, device="cuda")
        out = torch.empty_like(q)
        call = lambda: pkv.paged_kv_write_norm_rope(q, k, v, None, None, pos, inv, slots, kc, vc, q_out=out)  # noqa: E731
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda").to(torch.bfloat16))
        pos += 77
        slots.copy_(torch.randperm(1600, device="cuda")[:T])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got, got_k, got_v = out.clone(), kc.view(-1, 2, 128)[slots], vc.view(-1, 2, 128)[slots]
        near(got, *expect(q, None, 1e-6, pos, inv, False, 1.0), HALF_STEP[torch.bfloat16])
        near(got_k, *expect(k, None, 1e-6, pos, inv, False, 1.0), HALF_STEP[torch.bfloat16])
        assert torch.equal(got_v, v)

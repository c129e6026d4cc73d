"""Edges of the layer operators: pools whose elements pass 2^31, rows behind the
last sequence, the least workspace with many rows, windows over groups of any
size, and a batch in which nothing is valid.

Tolerances are those of the operators' own tests.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from gpu_util import TOL, to_f64
from oracle import serving
from test_gpu_fp8block_attention import TMAX, TMEAN, Batch
from test_gpu_norm_rope import HALF_STEP, expect, near
from test_gpu_window import batch, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 40])
def test_blocks_past_two_to_the_31_elements(n):
    """The last blocks of pools of 2.7e9 elements: written, copied and read."""
    NB, bs, Hq, Hkv, D, L = 41000, 64, 8, 8, 128, 200
    assert NB * bs * Hkv * D > 2 ** 31
    g = torch.Generator().manual_seed(n)
    blocks = [NB - 1, 5, NB - 2, NB - 7]
    slots = torch.cat([torch.arange(b * bs, b * bs + bs) for b in blocks])[:L].cuda()
    q = torch.randn(n, Hq, D, generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn(L, Hkv, D, generator=g).clamp(-4.5, 4.5).to(torch.bfloat16).cuda() for _ in range(2))
    table = torch.tensor([blocks], dtype=torch.int32).cuda()
    lens, qsl = torch.tensor([L], dtype=torch.int32).cuda(), torch.tensor([0, n], dtype=torch.int32).cuda()
    scale = D ** -0.5

    codes = [torch.full((NB, bs, Hkv, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(NB, Hkv, device="cuda") for _ in range(2)]
    pkv.paged_kv_write_fp8block(k, v, slots, *codes, *scales)
    pkv.copy_blocks(*codes, [[NB - 1, NB - 3]], *scales)
    for c, s in zip(codes, scales):
        assert torch.equal(c[NB - 3], c[NB - 1]) and torch.equal(s[NB - 3], s[NB - 1])
        assert torch.all(c[NB - 4:NB - 3] == 0x7F) and torch.all(c[6:9] == 0x7F)
    out = pkv.paged_attention_forward_fp8block(q, *codes, *scales, table, lens, qsl, scale, max_query_len=n)
    K, V = (serving.block_values(c[blocks].cpu().numpy(), s[blocks].cpu().numpy()).reshape(-1, Hkv, D)[:L]
            for c, s in zip(codes, scales))
    err = np.abs(to_f64(out) - serving.window_attend(to_f64(q), K, V, scale))
    assert err.max() <= TMAX and err.mean() <= TMEAN
    del codes, out

    pools = [torch.full((NB, bs, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pos, inv = torch.arange(L).cuda(), pkv.rope_frequencies(D)
    pkv.paged_kv_write_norm_rope(k, k, v, None, None, pos, inv, slots, *pools)
    flat = pools[0].view(-1, Hkv, D)[slots]
    near(flat, *expect(k, None, 1e-6, pos, inv, False, 1.0), HALF_STEP[torch.bfloat16])
    assert torch.equal(pools[1].view(-1, Hkv, D)[slots], v)
    out = pkv.paged_attention_window_forward(q, *pools, table, lens, qsl, scale, 70, 3, max_query_len=n)
    err = np.abs(to_f64(out) - serving.window_attend(to_f64(q), to_f64(flat), to_f64(v), scale, 70, 3))
    assert err.max() <= TOL["bf16"][0] and err.mean() <= TOL["bf16"][1]
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("group", [(8, 2), (7, 1), (20, 1)], ids=lambda g: "-".join(map(str, g)))
@pytest.mark.parametrize("n", [[1, 1, 1], [3, 1, 2], [130, 1, 60]])
def test_rows_behind_the_last_sequence(n, group):
    """A padded batch: query rows that no sequence owns are neither read for others nor written."""
    b = Batch(20, [300, 40, 129], n, *group, 16)
    T = sum(n)
    q = torch.cat([b.args[0], torch.full((11, group[0], 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    for hint in (0, max(n)):
        out = torch.full_like(q, 7.0)
        pkv.paged_attention_forward_fp8block(q, *b.args[1:], out=out, max_query_len=hint)
        b.check(out[:T])
        assert torch.all(out[T:] == 7.0)
    w = batch(21, [300, 40, 129], n, *group, 128, 16, torch.bfloat16)
    out = torch.full_like(q, 7.0)
    q[:T] = w["q"]
    pkv.paged_attention_window_forward(q, w["kc"], w["vc"], w["tables"], w["lens"], w["qsl"], 0.1, 50, 2, out=out)
    check(w, out[:T], 0.1, 50, 2, torch.bfloat16)
    assert torch.all(out[T:] == 7.0)
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("n", [[64], [300, 1], [17, 40, 2]])
def test_least_workspace(n):
    """Splits give way where the workspace has no room for their rows."""
    lens = [9000, 5000, 300][:len(n)]
    b = Batch(22, lens, n, 8, 2, 32)
    least = torch.empty(pkv.workspace_min(len(n), sum(n), 8, 2, 128), dtype=torch.uint8, device="cuda")
    for ws in (least, None):
        b.check(pkv.paged_attention_forward_fp8block(*b.args, workspace=ws))
        b.check(pkv.paged_attention_forward_fp8block(*b.args, workspace=ws, window=2000, num_sink=5), 2000, 5)
    assert pkv.device_errors() == 0


@pytest.mark.parametrize("group", [(7, 1, 32), (12, 1, 16), (20, 1, 8), (6, 2, 64), (8, 8, 16)], ids=lambda g: "-".join(map(str, g)))
@pytest.mark.parametrize("n", [[1, 1], [4, 70]])
def test_windows_over_any_group(n, group):
    Hq, Hkv, bs = group
    b = Batch(23, [400, 211], n, Hq, Hkv, bs)
    for window, sink in ((100, 4), (1, 0), (33, 200)):
        b.check(pkv.paged_attention_forward_fp8block(*b.args, window=window, num_sink=sink), window, sink)
    assert pkv.device_errors() == 0


def test_nothing_valid():
    """Every sequence of the batch is invalid, or has no query: zeros, flagged, and a clean call after."""
    b = Batch(24, [100, 50], [2, 3], 8, 2, 16)
    bad = torch.tensor([1, 0], dtype=torch.int32, device="cuda")  # fewer tokens than queries
    for kw in (dict(), dict(window=5, num_sink=1)):
        out = pkv.paged_attention_forward_fp8block(*b.args[:6], bad, *b.args[7:], **kw)
        assert pkv.device_errors() == pkv.DEVERR["bad_sequence"]
        assert torch.all(out == 0)
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.full_like(b.args[0], 3.0)
    pkv.paged_attention_forward_fp8block(*b.args[:7], none, b.args[8], out=out)
    assert torch.all(out == 3.0) and pkv.device_errors() == 0
    b.check(pkv.paged_attention_forward_fp8block(*b.args))


def test_two_streams_at_once():
    """Calls on two streams, each with the default workspaces of its own."""
    few = Batch(31, [700, 33, 5000], [1, 1, 1], 8, 2, 16)
    many = Batch(32, [700, 333, 60], [100, 1, 60], 8, 2, 16)
    win = batch(33, [700, 333, 60], [100, 1, 60], 8, 2, 128, 16, torch.bfloat16)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        with torch.cuda.stream(streams[0]):
            outs[0].append(pkv.paged_attention_forward_fp8block(*few.args, max_query_len=1))
            outs[0].append(pkv.paged_attention_forward_fp8block(*many.args))
        with torch.cuda.stream(streams[1]):
            outs[1].append(pkv.paged_attention_forward_fp8block(*many.args))
            outs[1].append(pkv.paged_attention_window_forward(win["q"], win["kc"], win["vc"], win["tables"], win["lens"],
                                                              win["qsl"], 0.1, 100, 2))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(o[i], o[i % 2]) for i in range(len(o)))
    few.check(outs[0][0])
    many.check(outs[0][1])
    assert torch.equal(outs[1][0], outs[0][1])
    check(win, outs[1][1], 0.1, 100, 2, torch.bfloat16)
    assert pkv.device_errors() == 0

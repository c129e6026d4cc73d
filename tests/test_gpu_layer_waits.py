"""The bounded waits of the attention over block scales and of the windowed
kernels, made to run out through the testing hook ``pkv_debug_fault`` (one CTA's
producer leaves out one key tile's load; no bad address, no trap): the call
comes back with PKV_DEVERR_TIMEOUT after about the short limit, and the next
ordinary call gives what the one before gave.  Then calls that share a
workspace, or run on another stream."""
import functools
import time

import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from test_gpu_fp8block_attention import Batch
from test_gpu_window import batch, check

pytestmark = pytest.mark.gpu

LIMIT_NS = 50_000_000  # 50 ms

DECODE = [2600 - 13 * i for i in range(64)], [1] * 64, 8, 2
PROMPT = [1900 + 40 * i for i in range(8)], [384] * 8, 8, 2
MIXED = [1900 + 40 * i for i in range(8)] + [3000] * 24, [384] * 8 + [1] * 24, 8, 2


def runs_out(call, fault_tile):
    before = call().clone()
    assert pkv.device_errors(clear=True) == 0
    pkv.debug_fault(fault_tile, LIMIT_NS)
    t0 = time.perf_counter()
    call()
    flags = pkv.device_errors(clear=True)  # synchronises
    secs = time.perf_counter() - t0
    assert flags == pkv.DEVERR["timeout"], f"flags {flags:#x}"
    assert secs < 1.5, f"the call took {secs:.2f} s: the short limit was not used"
    assert torch.equal(call(), before)
    assert pkv.device_errors() == 0


@functools.lru_cache(maxsize=1)
def block_batch(shape):
    return Batch(70, *dict(decode=DECODE, prompt=PROMPT, mixed=MIXED)[shape], 16)


@pytest.mark.parametrize("fault_tile", [1, 2, 5, 9])
@pytest.mark.parametrize("shape", ["decode", "prompt", "mixed"])
def test_block_scales(shape, fault_tile):
    b = block_batch(shape)
    runs_out(lambda: pkv.paged_attention_forward_fp8block(*b.args, max_query_len=int(shape == "decode")), fault_tile)


@pytest.mark.parametrize("fault_tile", [1, 3])
@pytest.mark.parametrize("shape,D,dtype", [("decode", 128, torch.bfloat16), ("decode", 64, torch.bfloat16),
                                           ("decode", 128, torch.float32), ("prompt", 128, torch.bfloat16),
                                           ("prompt", 64, torch.bfloat16)])
def test_windows(shape, D, dtype, fault_tile):
    lens, n, Hq, Hkv = dict(decode=DECODE, prompt=PROMPT)[shape]
    b = batch(80, lens, n, Hq, Hkv, D, 16, dtype)
    runs_out(lambda: pkv.paged_attention_window_forward(
        b["q"], b["kc"], b["vc"], b["tables"], b["lens"], b["qsl"], D ** -0.5, 1500, 4,
        max_query_len=int(shape == "decode")), fault_tile)


def test_one_workspace_call_after_call():
    """Calls of different shapes and operators follow one another on a stream
    of their own and in one workspace, without a synchronisation between them."""
    few = Batch(90, [700, 33, 5000], [1, 1, 1], 8, 2, 16)
    many = Batch(91, [700, 333, 60], [100, 1, 60], 8, 2, 16)
    win = batch(92, [700, 333, 60], [100, 1, 60], 8, 2, 128, 16, torch.bfloat16)
    work = torch.empty(pkv.workspace_size(3, 200, 8, 2, 128), dtype=torch.uint8, device="cuda")
    attend = pkv.paged_attention_forward_fp8block
    windowed = lambda w, s: pkv.paged_attention_window_forward(  # noqa: E731
        win["q"], win["kc"], win["vc"], win["tables"], win["lens"], win["qsl"], 0.1, w, s, workspace=work)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    outs = []
    with torch.cuda.stream(stream):
        for _ in range(4):
            outs.append((attend(*few.args, workspace=work, max_query_len=1), windowed(100, 2),
                         attend(*many.args, workspace=work), attend(*few.args, workspace=work, window=65, num_sink=3),
                         windowed(30, 0), attend(*many.args, False, workspace=work)))
    stream.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(o, outs[0]))
    a, w1, m, f, w2, full = outs[0]
    few.check(a)
    many.check(m)
    few.check(f, 65, 3)
    many.check(full, causal=False)
    check(win, w1, 0.1, 100, 2, torch.bfloat16)
    check(win, w2, 0.1, 30, 0, torch.bfloat16)
    assert pkv.device_errors() == 0


def test_two_graphs_share_a_workspace():
    few = Batch(93, [700, 33, 5000], [1, 1, 1], 8, 2, 16)
    many = Batch(94, [700, 333, 60], [100, 1, 60], 8, 2, 16)
    work = torch.empty(pkv.workspace_size(3, 200, 8, 2, 128), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(few.args[0]), torch.zeros_like(many.args[0])]
    graphs = []
    for b, out in zip((few, many), outs):
        pkv.paged_attention_forward_fp8block(*b.args, out=out, workspace=work)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            pkv.paged_attention_forward_fp8block(*b.args, out=out, workspace=work)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for out in outs:
            out.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        few.check(outs[0])
        many.check(outs[1])


@pytest.mark.parametrize("n", [[3, 1, 5, 2], [1, 17, 1, 130]])
def test_a_hint_below_the_query_counts(n):
    """The hint chooses kernels: a batch of more queries than it says gets its rows all the same."""
    b = Batch(95, [700, 333, 60, 257], n, 8, 2, 16)
    out = pkv.paged_attention_forward_fp8block(*b.args, max_query_len=1)
    assert pkv.device_errors() == 0
    b.check(out)
    w = batch(96, [700, 333, 60, 257], n, 8, 2, 128, 16, torch.bfloat16)
    out = pkv.paged_attention_window_forward(w["q"], w["kc"], w["vc"], w["tables"], w["lens"], w["qsl"], 0.1, 90, 3,
                                             max_query_len=1)
    assert pkv.device_errors() == 0
    check(w, out, 0.1, 90, 3, torch.bfloat16)

"""Workspaces of calls captured into graphs that torch does not manage."""
import ctypes
import time

import pytest
import torch

import paged_kv_cache_236_gb300 as pkv
from test_gpu_scores import Batch

pytestmark = pytest.mark.gpu


class Runtime:
    """The CUDA runtime's capture calls."""

    def __init__(self):
        self.lib = ctypes.CDLL("libcudart.so.13")
        self.lib.cudaStreamBeginCapture.argtypes = [ctypes.c_void_p, ctypes.c_int]
        self.lib.cudaStreamEndCapture.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]
        self.lib.cudaGraphInstantiate.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_void_p, ctypes.c_ulonglong]
        self.lib.cudaGraphLaunch.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
        self.lib.cudaGraphDestroy.argtypes = self.lib.cudaGraphExecDestroy.argtypes = [ctypes.c_void_p]

    def __getattr__(self, name):
        def call(*args):
            status = getattr(self.lib, name)(*args)
            assert status == 0, (name, status)
        return call

    def capture(self, stream, fn):
        """(graph, executable graph) of fn's calls on a torch stream."""
        graph, run = ctypes.c_void_p(), ctypes.c_void_p()
        self.cudaStreamBeginCapture(stream.cuda_stream, 2)  # relaxed
        with torch.cuda.stream(stream):
            fn()
        self.cudaStreamEndCapture(stream.cuda_stream, ctypes.byref(graph))
        self.cudaGraphInstantiate(ctypes.byref(run), graph, 0)
        return graph, run


def _gone():
    for _ in range(100):
        with pkv._graphs_lock:
            pkv._drop_graphs_gone()
        if not pkv._graphs_hold:
            return True
        time.sleep(0.05)
    return False


def test_graphs_of_other_captures_keep_their_workspace():
    """Two graphs captured outside torch, each of a small and a larger call:
    later eager calls and tensors of the capture's stream take none of their
    workspaces, both replay at once, and the memory is given up with them."""
    rt = Runtime()
    assert _gone()
    pairs = [[Batch(121 + 2 * i + j, [900 + 50 * i, 300 + 3000 * j], [1, 1 + 39 * j], 8, 2, 128, 16) for j in range(2)]
             for i in range(2)]
    large = Batch(129, [6000, 5000], [40, 1], 8, 2, 128, 16)
    want = [[b.run(out=b.old.clone()) for b in p] for p in pairs]
    want_large = large.run(out=large.old.clone())
    outs = [[b.old.clone() for b in p] for p in pairs]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        pairs[0][0].run(out=outs[0][0])  # a warm buffer of the stream, which the graphs leave alone
    torch.cuda.synchronize()
    graphs = [rt.capture(st, lambda: [b.run(out=o) for b, o in zip(p, out)]) for p, out in zip(pairs, outs)]
    assert len(pkv._graphs_hold) == 2
    with torch.cuda.stream(st):
        fill = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    streams = [torch.cuda.Stream() for _ in pairs]
    for _ in range(20):
        for p, out in zip(pairs, outs):
            for b, o in zip(p, out):
                o.copy_(b.old)
        torch.cuda.synchronize()
        for (_, run), s in zip(graphs, streams):
            rt.cudaGraphLaunch(run, s.cuda_stream)
        with torch.cuda.stream(st):
            got = large.run(out=large.old.clone())
        torch.cuda.synchronize()
        assert torch.equal(got, want_large)
        assert all(torch.equal(o, w) for out, ws in zip(outs, want) for o, w in zip(out, ws))
    assert all(bool((x == 7).all()) for x in fill)
    for graph, run in graphs:
        rt.cudaGraphExecDestroy(run)
        rt.cudaGraphDestroy(graph)
    assert _gone()
    assert pkv.device_errors() == 0


def test_graphs_of_torch_hold_nothing_here():
    """Under torch.cuda.graph the graph's own memory pool serves the calls."""
    b = Batch(131, [900, 300], [1, 40], 8, 2, 128, 16)
    want, out = b.run(out=b.old.clone()), b.old.clone()
    torch.cuda.synchronize()
    assert _gone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(out=out)
        b.run(out=out)
    assert not pkv._graphs_hold
    out.copy_(b.old)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert pkv.device_errors() == 0

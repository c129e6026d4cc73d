"""Which workspace a call without one gets, with the CUDA queries stubbed."""
import threading
import weakref
from types import SimpleNamespace

import pytest
import torch

import paged_kv_cache_236_gb300 as pkv

CPU = torch.device("cpu")


@pytest.fixture
def stubbed(monkeypatch):
    """One device, whose current stream is `stubbed.stream`."""
    state = SimpleNamespace(stream=7, capturing=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: SimpleNamespace(cuda_stream=state.stream))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.capturing)
    return state


def _in_thread(fn):
    got = []
    t = threading.Thread(target=lambda: got.append(fn()))
    t.start()
    t.join()
    return got[0]


def test_a_thread_keeps_its_own_buffer(stubbed):
    mine = pkv._workspace(CPU, 1000)
    assert pkv._workspace(CPU, 10).data_ptr() == mine.data_ptr()
    theirs = _in_thread(lambda: pkv._workspace(CPU, 1000))
    assert theirs.data_ptr() != mine.data_ptr()
    assert pkv._workspace(CPU, 1000).data_ptr() == mine.data_ptr()
    stubbed.stream = 8
    assert pkv._workspace(CPU, 1000).data_ptr() != mine.data_ptr()


def test_a_thread_s_buffers_go_with_it(stubbed):
    gone = _in_thread(lambda: weakref.ref(pkv._workspace(CPU, 1000)))
    assert gone() is None


def test_the_scores_call_asks_about_its_own_device(stubbed, monkeypatch):
    """Whether a call is captured is the state of its device's stream, not of
    the device that is current before the call."""
    from paged_kv_cache_236_gb300 import build
    build.build()
    state = SimpleNamespace(current=0, asked=[])

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, state.current = state.current, self.dev

        def __exit__(self, *a):
            state.current = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.current)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: bool(state.asked.append(state.current)))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    pkv._scores_args(torch.zeros(1, 2, 64), torch.zeros(4, 16, 1, 64), i32(0, 1).view(1, 2), i32(20), i32(0, 1),
                     torch.zeros(1, 1, 32), 0.125, True, 1.0, None, None, None, 0, 1)
    assert state.asked == [1] and state.current == 0


def test_captures_without_a_graph_pool_hold_one_workspace_a_stream(stubbed, monkeypatch):
    """The workspaces of a capture that no memory pool serves are held until
    its graph is gone, one for each stream, the larger ones beside the smaller."""
    state = SimpleNamespace(capture=41, gone=[], watched=[])

    class Lib:
        def pkv_capture_id(self, stream, out):
            out._obj.value = state.capture
            return 0

        def pkv_capture_watch(self, stream):
            state.watched.append(state.capture)
            return 0

        def pkv_capture_gone(self, out):
            out._obj.value = state.gone.pop() if state.gone else 0
            return 0

    monkeypatch.setattr(pkv, "lib", lambda: Lib())
    monkeypatch.setattr(pkv, "_in_graph_pool", lambda t: state.capture == 43)
    stubbed.capturing = True
    first = pkv._workspace(CPU, 1000)
    assert pkv._workspace(CPU, 10).data_ptr() == first.data_ptr()
    kept = weakref.ref(first)
    larger = pkv._workspace(CPU, 5000)
    stubbed.stream = 8
    other = pkv._workspace(CPU, 1000)
    assert len({first.data_ptr(), larger.data_ptr(), other.data_ptr()}) == 3
    state.capture = 42
    again = pkv._workspace(CPU, 1000)
    assert again.data_ptr() != other.data_ptr() and state.watched == [41, 42]
    del first, larger, other, again
    assert kept() is not None and set(pkv._graphs_hold) == {41, 42}
    state.gone, state.capture = [41, 42], 43  # of a graph with a pool of its own nothing is held
    x, y = pkv._workspace(CPU, 1000), pkv._workspace(CPU, 1000)
    assert x.data_ptr() != y.data_ptr() and state.watched == [41, 42]
    assert kept() is None and not pkv._graphs_hold


def test_memory_of_other_allocators(monkeypatch):
    """Allocators without a snapshot: cudaMallocAsync makes nodes of the graph,
    of a pluggable one nothing is known."""
    monkeypatch.setattr(torch.cuda, "memory_snapshot", lambda: pytest.fail("not meaningful"))
    for backend, owned in (("cudaMallocAsync", True), ("pluggable", False)):
        monkeypatch.setattr(torch.cuda, "get_allocator_backend", lambda: backend)
        assert pkv._in_graph_pool(torch.empty(1)) is owned
    t = torch.empty(1)
    monkeypatch.setattr(torch.cuda, "get_allocator_backend", lambda: "native")
    for pool, owned in (((0, 0), False), ((0, 3), True), ((5, 0), True)):
        segments = [{"address": 0, "total_size": 1, "segment_pool_id": (7, 7)},
                    {"address": t.data_ptr() - 64, "total_size": 4096, "segment_pool_id": pool}]
        monkeypatch.setattr(torch.cuda, "memory_snapshot", lambda: segments)
        assert pkv._in_graph_pool(t) is owned

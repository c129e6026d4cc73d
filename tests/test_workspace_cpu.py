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

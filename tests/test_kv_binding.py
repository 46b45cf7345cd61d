"""The cache's Python calls without a GPU: which workspace serves whom."""
import gc
import weakref

import pytest
import torch

import speculative_decoding_verification_63_gb300 as sv


class FakeBuffer:
    def __init__(self, n):
        self.n = n

    def numel(self):
        return self.n

    def data_ptr(self):
        return 256


class FakeGpu:
    """What workspace() asks of torch and the library."""
    stream, capture = 7, 0

    def __init__(self, mp):
        mp.setattr(sv, "_ws_cache", {})
        mp.setattr(torch, "empty", lambda n, **kw: FakeBuffer(n))
        mp.setattr(sv, "sv_workspace_init", lambda buf, stream=None: None)
        mp.setattr(sv, "sv_stream_capture_id", lambda stream: self.capture, raising=False)
        mp.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: self.stream,
                   raising=False)
        mp.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capture != 0)
        mp.setattr(torch.cuda, "current_stream", lambda device=None: self)

    def synchronize(self):
        pass


@pytest.fixture
def gpu(monkeypatch):
    return FakeGpu(monkeypatch)


DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("key", ["kv_attention", "kv", "chain"])
def test_a_replaced_workspace_stays_allocated(gpu, key):
    small = sv.workspace(5_000_000, DEV, key)
    assert sv.workspace(4_000_000, DEV, key) is small
    alive = weakref.ref(small)
    del small
    big = sv.workspace(21_000_000, DEV, key)
    gc.collect()
    assert alive() is not None and alive() is not big
    assert sv.workspace(1, DEV, key) is big


def test_attention_has_one_workspace_a_stream(gpu):
    first, other = sv.workspace(100, DEV, "kv_attention"), sv.workspace(100, DEV, "kv")
    gpu.stream = 8
    second = sv.workspace(100, DEV, "kv_attention")
    assert second is not first and sv.workspace(100, DEV, "kv") is other
    gpu.stream = 7
    assert sv.workspace(100, DEV, "kv_attention") is first


def test_a_capture_has_workspaces_of_its_own(gpu):
    eager, kv = sv.workspace(100, DEV, "kv_attention"), sv.workspace(100, DEV, "kv")
    gpu.capture = 1
    one = sv.workspace(100, DEV, "kv_attention")
    assert one is not eager and sv.workspace(90, DEV, "kv_attention") is one
    assert sv.workspace(100, DEV, "kv") is kv        # only its error word is used
    new = sv.workspace(100, DEV, "tree")
    gpu.capture = 2
    two = sv.workspace(100, DEV, "kv_attention")
    assert two is not one and two is not eager
    gpu.capture = 0
    assert sv.workspace(100, DEV, "kv_attention") is eager
    assert sv.workspace(100, DEV, "tree") is not new  # the graph's stays the graph's

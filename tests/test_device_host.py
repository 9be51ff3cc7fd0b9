"""Calls on tensors of another device than the current one (CPU, with stand-ins for CUDA): every
launch has to go to the tensors' device and its current stream, and a status to be read there."""
import contextlib
import types

import pytest
import torch

import dynamic_sparse_attention_build_b200 as dsa
from dynamic_sparse_attention_build_b200 import api, serving
from dynamic_sparse_attention_build_b200 import _binding as B


class Cuda:
    """The current device, and a current stream with handle 1000 + device on each."""

    def __init__(self, monkeypatch):
        self.now, self.calls = 0, []
        monkeypatch.setattr(torch.cuda, "device", self.device)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.now)
        monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(
            cuda_stream=1000 + (self.now if device is None else torch.device(device).index),
            device=torch.device("cuda", self.now if device is None else torch.device(device).index)))
        for name in ("dsa_build_indices", "dsa_sparse_prefill", "dsa_count_pairs", "dsa_get_device_status"):
            def call(*args, name=name):
                self.calls.append((name, self.now, getattr(args[-1], "value", args[-1])))
                return (B.DSA_OK, 0) if name == "dsa_get_device_status" else B.DSA_OK
            monkeypatch.setattr(B, name, call)

    @contextlib.contextmanager
    def device(self, d):
        was, self.now = self.now, torch.device(d).index if not isinstance(d, int) else d
        try:
            yield
        finally:
            self.now = was


class Tensor:
    """As much of a CUDA tensor as the wrappers look at."""

    def __init__(self, *shape, device=1):
        self.shape, self.device, self.is_cuda = shape, torch.device("cuda", device), True

    def stride(self, i):
        return (self.shape[1] * self.shape[2], self.shape[2], 1)[i]

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return 1 << 20


@pytest.fixture
def cuda(monkeypatch):
    c = Cuda(monkeypatch)
    # (whichever way the package asks for the current device and stream)
    for m in (api, serving):
        for name in ("_current_device", "_raw_stream"):
            if hasattr(m, name):
                monkeypatch.setattr(m, name, {"_current_device": lambda: c.now, "_raw_stream": lambda i: 1000 + i}[name])
    return c


@pytest.fixture
def args():
    Q, K, V, O = Tensor(4, 100, 64), Tensor(2, 100, 64), Tensor(2, 100, 64), Tensor(4, 100, 64)
    idx = types.SimpleNamespace(c=B.dsa_indices(), workspace=Tensor(1, 1, 1), block=64)
    return Q, K, V, O, idx


def test_sparse_calls_go_to_the_tensors_device(cuda, args):
    Q, K, V, O, idx = args
    pats = api.make_patterns([dict(kind="ashape", sink=1, window=4)] * 4)
    dsa.build_indices(Q, K, pats, 64, bufs=idx)
    dsa.sparse_prefill(Q, K, V, idx, O=O)
    assert cuda.calls == [("dsa_build_indices", 1, 1001), ("dsa_sparse_prefill", 1, 1001)]
    assert cuda.now == 0
    stream = types.SimpleNamespace(cuda_stream=77, device=torch.device("cuda", 1))
    dsa.sparse_prefill(Q, K, V, idx, O=O, stream=stream)
    assert cuda.calls[-1] == ("dsa_sparse_prefill", 1, 77)


def test_a_stream_of_another_device_is_refused(cuda, args):
    Q, K, V, O, idx = args
    with pytest.raises(ValueError, match="stream"):
        dsa.sparse_prefill(Q, K, V, idx, O=O, stream=types.SimpleNamespace(cuda_stream=77, device=torch.device("cuda", 0)))
    assert cuda.calls == []


def test_device_status_is_read_on_the_streams_device(cuda):
    dsa.device_status()
    dsa.device_status(types.SimpleNamespace(cuda_stream=77, device=torch.device("cuda", 1)))
    assert cuda.calls == [("dsa_get_device_status", 0, 1000), ("dsa_get_device_status", 1, 77)]


def test_paged_layer_stays_on_its_device(cuda, args, monkeypatch):
    Q, K, V, O, idx = args
    layer = dsa.PagedLayer.__new__(dsa.PagedLayer)
    layer.cache = types.SimpleNamespace(K=Tensor(1, 1, 1))
    layer.lens, layer.requests, layer.page = Tensor(1, 1, 4), 4, 16
    for name in ("_store", "_check"):
        monkeypatch.setattr(layer, name, lambda *a, **k: None)
    monkeypatch.setattr(serving, "_ints", lambda *a: None)
    monkeypatch.setattr(api, "alloc_indices", lambda *a, **k: idx)
    monkeypatch.setattr(torch, "empty_like", lambda t, **k: O)
    layer.prefill(Q, K, V, None, patterns=[dict(kind="ashape", sink=1, window=4)] * 4)
    assert layer.status() == (0, 0)
    assert cuda.calls == [("dsa_build_indices", 1, 1001), ("dsa_sparse_prefill", 1, 1001), ("dsa_get_device_status", 1, 1001)]

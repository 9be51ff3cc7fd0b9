"""What a PagedLayer refuses before it enqueues anything (CPU: no call reaches the library)."""
import pytest
import torch

import dynamic_sparse_attention_build_b200 as dsa
from dynamic_sparse_attention_build_b200 import serving


@pytest.fixture
def layer(monkeypatch):
    layer = dsa.PagedLayer.__new__(dsa.PagedLayer)
    layer.requests, layer.ones, layer.calls = 3, "ones", []
    layer.cache = layer.table = None
    layer.lens = torch.zeros(3, dtype=torch.int32)
    monkeypatch.setattr(serving, "_current_device", lambda: None)  # (as a host tensor's index)
    monkeypatch.setattr(layer, "_check", lambda *a: None)  # (the tensors are the host's)
    monkeypatch.setattr(layer, "_store", lambda K, V, new, **k: layer.calls.append((K.shape[1], new)))
    monkeypatch.setattr(serving, "_attend", lambda Q, cache, table, lens, n_q, **k: layer.calls.append(n_q))
    return layer


def rows(n):
    return torch.zeros(2, n, 64, dtype=torch.bfloat16)


@pytest.mark.parametrize("q, k", [(6, 6), (6, 5), (3, 2), (3, 0), (9, 9)])
def test_decode_without_new_lens_takes_one_row_a_request(layer, q, k):
    """By default each request gets one token, so the rows of K and V are the requests'.  More of them (n_q rows each,
    say) would go to the wrong requests, and fewer leave some without."""
    with pytest.raises(ValueError, match="new_lens"):
        layer.decode(rows(q), rows(k), rows(k))
    assert layer.calls == []


@pytest.mark.parametrize("q, k, new", [(3, 3, None), (6, 3, None), (3, 5, None), (6, 6, "given"), (6, 4, "given"), (3, 2, "given")])
def test_decode_takes(layer, q, k, new):
    """One row a request (padded ones behind them where Q has one row each as well), or any rows with their new_lens."""
    layer.decode(rows(q), rows(k), rows(k), new)
    assert layer.calls == [(k, new or "ones"), q // 3]

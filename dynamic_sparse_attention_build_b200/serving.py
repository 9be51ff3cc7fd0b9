"""Serving calls around the sparse prefill (marshalling only, like ``api``): dense attention
over packed prompts.

Token tensors are bf16 CUDA tensors shaped [heads, tokens, d] as in ``api``.  Arguments are
checked here before the library sees a pointer: a wrong shape, type, device or layout raises
``ValueError`` and enqueues nothing.  Every call runs on ``stream`` (default: the current
stream of the tensors' device); what it allocates belongs to that stream.
"""
from __future__ import annotations

import contextlib

import torch

from . import _binding as B


def _need(ok, what):
    if not ok:
        raise ValueError(what)


@contextlib.contextmanager
def _on(device, stream):
    """The tensors' device and the call's stream made current: launches and allocations follow them."""
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
        else:
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _tokens(name, t, heads=None, tokens=None, d=None, device=None):
    _need(isinstance(t, torch.Tensor) and t.dim() == 3, f"{name} must be a tensor [heads, tokens, d]")
    _need(t.is_cuda, f"{name} must be a CUDA tensor")
    _need(t.dtype == torch.bfloat16, f"{name} must be bfloat16, not {t.dtype}")
    _need(device is None or t.device == device, f"{name} is on {t.device}, the call on {device}")
    for at, want in enumerate((heads, tokens, d)):
        _need(want is None or t.shape[at] == want, f"{name} has shape {tuple(t.shape)}; dimension {at} must be {want}")
    _need(t.shape[2] in (64, 128), f"{name}: d must be 64 or 128, not {t.shape[2]}")
    _need(t.stride(2) == 1, f"{name}: the last dimension must be contiguous")


def _strides(t):
    """(head stride, token stride), with those of dimensions of size 1 made regular."""
    h, n, d = t.shape
    ts = t.stride(1) if n > 1 else d
    return (t.stride(0) if h > 1 else n * ts), ts


def _ints(name, t, shape, device):
    _need(isinstance(t, torch.Tensor) and t.dtype == torch.int32, f"{name} must be an int32 tensor")
    _need(t.device == device, f"{name} is on {t.device}, the call on {device}")
    _need(tuple(t.shape) == tuple(shape), f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    _need(t.is_contiguous(), f"{name} must be contiguous")


def _lse(lse, want, shape, device):
    if lse is None:
        return torch.empty(shape, dtype=torch.float32, device=device) if want else None
    _need(lse.dtype == torch.float32 and lse.device == device and tuple(lse.shape) == tuple(shape)
          and lse.is_contiguous(), f"lse must be a contiguous float32 tensor {tuple(shape)} on {device}")
    return lse


def packed_prefill(Q, K, V, cu_seqlens, O=None, lse=None, want_lse=False, stream=None):
    """Dense causal attention over packed sequences; returns (O, lse or None).

    Q [Hq, T, d], K and V [Hkv, T, d] hold the sequences' rows one after the other;
    ``cu_seqlens`` (int32 [S + 1], on the device) says where each begins.  Short prompts
    that arrive together are prefilled this way, long ones with ``sparse_prefill``.  Rows
    of no sequence are left as they were in ``O`` and ``lse`` (undefined where these are
    allocated here)."""
    _tokens("Q", Q)
    Hq, T, d = Q.shape
    dev = Q.device
    _tokens("K", K, None, T, d, dev)
    Hkv = K.shape[0]
    _tokens("V", V, Hkv, T, d, dev)
    _need(Hkv > 0 and Hq % Hkv == 0, f"{Hq} query heads do not divide into {Hkv} KV heads")
    _need(isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.dim() == 1 and cu_seqlens.numel() > 0,
          "cu_seqlens must be an int32 tensor [sequences + 1]")
    _ints("cu_seqlens", cu_seqlens, cu_seqlens.shape, dev)
    if O is not None:
        _tokens("O", O, Hq, T, d, dev)
    with _on(dev, stream) as st:
        if O is None:
            O = torch.empty_like(Q, memory_format=torch.contiguous_format)
        lse = _lse(lse, want_lse, (Hq, T), dev)
        if T > 0 and Hq > 0:
            p = B.dsa_problem(Hq, Hkv, T, d, 64, 0, *_strides(Q), *_strides(K), *_strides(V), *_strides(O))
            B.check(B.dsa_packed_prefill(p, Q.data_ptr(), K.data_ptr(), V.data_ptr(), cu_seqlens.data_ptr(),
                                         cu_seqlens.numel() - 1, O.data_ptr(), lse.data_ptr() if lse is not None else None,
                                         st), "dsa_packed_prefill")
    return O, lse

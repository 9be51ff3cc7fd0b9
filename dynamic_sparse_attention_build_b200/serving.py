"""Serving calls around the sparse prefill (marshalling only, like ``api``): dense attention
over packed prompts, the page tables of a paged cache, the store of keys and values in 8 bits,
and the attention of new tokens over that cache.

Token tensors are bf16 CUDA tensors shaped [heads, tokens, d] as in ``api``.  Arguments are
checked here before the library sees a pointer: a wrong shape, type, device or a last dimension
that is not contiguous raises ``ValueError`` and enqueues nothing.  What the library itself asks
of pointers, strides and sizes (rows on 16-byte boundaries, say) raises ``DSAError`` and enqueues
nothing either.  Every call runs on ``stream`` (default: the current
stream of the tensors' device); what it allocates belongs to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass, field

import torch

from . import _binding as B
from .api import _current_device, _raw_stream, build_indices, device_status, sparse_prefill


def _refuse(what):
    raise ValueError(what)


@contextlib.contextmanager
def _elsewhere(device, stream):
    """The tensors' device and the call's stream made current: launches and allocations follow them."""
    if stream is not None and stream.device != device:
        _refuse(f"the stream belongs to {stream.device}, the tensors to {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):  # (a stream of None changes nothing)
        yield


# Every message is put together only when it is needed: a call's checks take a few us otherwise.
def _tokens(name, t, heads=None, tokens=None, d=None, device=None):
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        _refuse(f"{name} must be a tensor [heads, tokens, d]")
    if not t.is_cuda:
        _refuse(f"{name} must be a CUDA tensor")
    if t.dtype is not torch.bfloat16:
        _refuse(f"{name} must be bfloat16, not {t.dtype}")
    if device is not None and t.device != device:
        _refuse(f"{name} is on {t.device}, the call on {device}")
    shape = t.shape
    h, n, e = shape
    if (heads is not None and h != heads) or (tokens is not None and n != tokens) or (d is not None and e != d):
        at = 0 if heads is not None and h != heads else 1 if tokens is not None and n != tokens else 2
        _refuse(f"{name} has shape {tuple(shape)}; dimension {at} must be {(heads, tokens, d)[at]}")
    if e != 64 and e != 128:
        _refuse(f"{name}: d must be 64 or 128, not {e}")
    if t.stride(2) != 1:
        _refuse(f"{name}: the last dimension must be contiguous")


def _strides(t):
    """(head stride, token stride), with those of dimensions of size 1 made regular."""
    h, n, d = t.shape
    ts = t.stride(1) if n > 1 else d
    return (t.stride(0) if h > 1 else n * ts), ts


def _apart(row, dims):
    """Whether rows of `row` elements are apart: dims are (size, stride), and with them in order of
    their strides each steps over all that the smaller ones span."""
    span = row
    for n, stride in sorted(dims, key=lambda x: x[1]):
        if n > 1:
            if stride < span:
                return False
            span += (n - 1) * stride
    return True


def _rows(name, t, packed):
    """What the library asks of a tensor's rows: 16-byte pieces, and (packed) rows and heads apart."""
    if t.data_ptr() % 16:
        _refuse(f"{name} must begin at a multiple of 16 bytes")
    hs, ts = _strides(t)
    if hs % 8 or ts % 8:
        _refuse(f"{name}: strides must be a multiple of 8 elements")
    if packed and t.shape[1] > 0 and (ts < t.shape[2] or hs == 0):
        _refuse(f"{name}: rows must not overlap")


def _ints(name, t, shape, device):
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32:
        _refuse(f"{name} must be an int32 tensor")
    if t.device != device:
        _refuse(f"{name} is on {t.device}, the call on {device}")
    if t.shape != shape:
        _refuse(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous():
        _refuse(f"{name} must be contiguous")


def _table(t):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[1] == 0:
        _refuse("block_table must be an int32 tensor [requests, pages of a request]")
    return t.shape


def _lse(lse, want, shape, device):
    if lse is None:
        return torch.empty(shape, dtype=torch.float32, device=device) if want else None
    if (not isinstance(lse, torch.Tensor) or lse.dtype is not torch.float32 or lse.device != device or lse.shape != shape
            or not lse.is_contiguous()):
        _refuse(f"lse must be a contiguous float32 tensor {tuple(shape)} on {device}")
    return lse


def _workspace(workspace, need, device):
    if (not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous()
            or workspace.nbytes < need or workspace.data_ptr() % 16):
        _refuse(f"workspace must hold {need} bytes on {device}, from a multiple of 16 bytes on")


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
    if Hkv == 0 or Hq % Hkv:
        _refuse(f"{Hq} query heads do not divide into {Hkv} KV heads")
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() == 0:
        _refuse("cu_seqlens must be an int32 tensor [sequences + 1]")
    _ints("cu_seqlens", cu_seqlens, cu_seqlens.shape, dev)
    if O is not None:
        _tokens("O", O, Hq, T, d, dev)
    if stream is not None or _current_device() != dev.index:
        with _elsewhere(dev, stream):
            return _prefill(Q, K, V, cu_seqlens, O, lse, want_lse)
    return _prefill(Q, K, V, cu_seqlens, O, lse, want_lse)


# What runs behind a call's checks, on the current device and its current stream.
def _prefill(Q, K, V, cu_seqlens, O=None, lse=None, want_lse=False):
    Hq, T, d = Q.shape
    Hkv, dev = K.shape[0], Q.device
    st = _raw_stream(dev.index)
    if O is None:
        O = torch.empty_like(Q, memory_format=torch.contiguous_format)
    lse = _lse(lse, want_lse, (Hq, T), dev)
    if T > 0 and Hq > 0:
        p = B.dsa_problem(Hq, Hkv, T, d, 64, 0, *_strides(Q), *_strides(K), *_strides(V), *_strides(O))
        B.check(B.dsa_packed_prefill(p, Q.data_ptr(), K.data_ptr(), V.data_ptr(), cu_seqlens.data_ptr(),
                                     cu_seqlens.numel() - 1, O.data_ptr(), lse.data_ptr() if lse is not None else None,
                                     st), "dsa_packed_prefill")
    return O, lse


PAGE_SIZES = (16, 32, 64, 128, 256)
E4M3 = torch.float8_e4m3fn


@dataclass(frozen=True, eq=False)
class PageCache:
    """Keys and values in 8 bits (``dsa_cache`` in include/dsa.h): K and V are float8_e4m3fn
    [pages, Hkv, page, d] with equal strides and a contiguous last dimension (a
    [pages, page, Hkv, d] tensor viewed with ``.transpose(1, 2)`` works too), k_scale and
    v_scale float32 [pages, Hkv]."""
    K: torch.Tensor
    V: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    c: B.dsa_cache = field(init=False, repr=False)

    def __post_init__(self):
        K, V = self.K, self.V
        for name, t in (("K", K), ("V", V)):
            if not isinstance(t, torch.Tensor) or t.dim() != 4:
                _refuse(f"{name} must be a tensor [pages, Hkv, page, d]")
            if not t.is_cuda or t.device != K.device:
                _refuse(f"{name} must be a CUDA tensor on one device with K")
            if t.dtype is not E4M3:
                _refuse(f"{name} must be {E4M3}, not {t.dtype}")
            if t.stride(3) != 1:
                _refuse(f"{name}: the last dimension must be contiguous")
        if K.shape != V.shape or K.stride() != V.stride():
            _refuse("K and V must have one shape and one layout")
        pages, Hkv, page, d = K.shape
        if pages == 0 or Hkv == 0:
            _refuse("the cache is empty")
        if page not in PAGE_SIZES:
            _refuse(f"a page has 16, 32, 64, 128 or 256 tokens, not {page}")
        if d not in (64, 128):
            _refuse(f"d must be 64 or 128, not {d}")
        for name, t in (("k_scale", self.k_scale), ("v_scale", self.v_scale)):
            if (not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.device != K.device
                    or t.shape != (pages, Hkv) or not t.is_contiguous()):
                _refuse(f"{name} must be a contiguous float32 tensor [{pages}, {Hkv}] on {K.device}")
        token = K.stride(2)
        head = K.stride(1) if Hkv > 1 else page * token
        whole = K.stride(0) if pages > 1 else Hkv * page * token
        if token < d or not _apart(d, ((page, token), (Hkv, head), (pages, whole))):
            _refuse("pages, heads and tokens of the cache must not overlap")
        object.__setattr__(self, "c", B.dsa_cache(pages, Hkv, page, d, whole, head, token, K.data_ptr(), V.data_ptr(),
                                                  self.k_scale.data_ptr(), self.v_scale.data_ptr()))

    @classmethod
    def empty(cls, pages, Hkv, page, d, device="cuda"):
        """A cache of zeros, every scale at its smallest."""
        new = lambda: torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device=device).view(E4M3)  # noqa: E731
        scale = lambda: torch.full((pages, Hkv), 2.0 ** -60, dtype=torch.float32, device=device)  # noqa: E731
        return cls(new(), new(), scale(), scale())


@dataclass
class Tables:
    """What ``build_tables`` gives: the slot of each new token (-1 behind the last), where each
    request's new tokens begin, the requests' new lengths and the free pages that are left."""
    slots: torch.Tensor
    cu_seqlens: torch.Tensor
    lens: torch.Tensor
    free_count: torch.Tensor


PROMPTS = {None: (), "packed": (0,), "single": (1,)}


def build_tables(lens, new_lens, free_pages, free_count, block_table, page, max_tokens, out=None, stream=None, prompts=None):
    """Pages and slots for the tokens that each request gets next; returns ``Tables``.

    lens, new_lens: int32 [B], the tokens that each request has and gets (a negative number
    ends it and frees its pages); block_table int32 [B, W] and the stack of free pages
    (free_pages int32 [F], free_count int32 [1]) are updated in place.  ``out`` takes the
    results (its ``lens`` and ``free_count`` may be the call's own).  If the pages, the table's
    width or ``max_tokens`` do not suffice, nothing changes, no token has a slot, and
    ``device_status`` says DSA_ERR_CAPACITY.  With ``prompts="packed"`` a request that gets tokens
    must hold none, with ``prompts="single"`` one request gets all ``max_tokens`` besides (their
    attention sees the new rows alone); otherwise nothing changes either, and the status is
    DSA_ERR_DEVICE."""
    if not isinstance(lens, torch.Tensor) or lens.dim() != 1 or lens.numel() == 0:
        _refuse("lens must be an int32 tensor [requests]")
    if not lens.is_cuda:
        _refuse("lens must be a CUDA tensor")
    dev, n = lens.device, lens.numel()
    _ints("lens", lens, (n,), dev)
    _ints("new_lens", new_lens, (n,), dev)
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1 or free_pages.numel() == 0:
        _refuse("free_pages must be an int32 tensor [pages]")
    _ints("free_pages", free_pages, free_pages.shape, dev)
    _ints("free_count", free_count, (1,), dev)
    width = _table(block_table)[1]
    _ints("block_table", block_table, (n, width), dev)
    if page not in PAGE_SIZES:
        _refuse(f"a page has 16, 32, 64, 128 or 256 tokens, not {page}")
    if max_tokens < 0:
        _refuse("max_tokens must not be negative")
    if prompts not in PROMPTS:
        _refuse(f'prompts must be None, "packed" or "single", not {prompts!r}')
    if out is not None:
        _ints("out.slots", out.slots, (max_tokens,), dev)
        _ints("out.cu_seqlens", out.cu_seqlens, (n + 1,), dev)
        _ints("out.lens", out.lens, (n,), dev)
        _ints("out.free_count", out.free_count, (1,), dev)
    if stream is not None or _current_device() != dev.index:
        with _elsewhere(dev, stream):
            return _build(lens, new_lens, free_pages, free_count, block_table, page, max_tokens, out, prompts)
    return _build(lens, new_lens, free_pages, free_count, block_table, page, max_tokens, out, prompts)


def _build(lens, new_lens, free_pages, free_count, block_table, page, max_tokens, out, prompts):
    dev, (n, width) = lens.device, block_table.shape
    st = _raw_stream(dev.index)
    if out is None:
        new = torch.empty(max_tokens + 2 * n + 2, dtype=torch.int32, device=dev)
        out = Tables(*new.split_with_sizes([max_tokens, n + 1, n, 1]))  # one allocation
    call = B.lib().dsa_build_tables if prompts is None else B.lib().dsa_build_prompt_tables
    B.check(call(
        n, lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), free_pages.numel(), free_count.data_ptr(),
        block_table.data_ptr(), width, page, max_tokens, out.slots.data_ptr(),
        out.cu_seqlens.data_ptr(), out.lens.data_ptr(), out.free_count.data_ptr(), *PROMPTS[prompts], st),
        "dsa_build_tables")
    return out


def cache_write(K, V, slots, cache, stream=None):
    """Stores the rows of K and V [Hkv, T, d] at ``slots`` (int32 [T], from ``build_tables``;
    negative ones are passed over) in the cache, in e4m3 with one power-of-two scale per page
    and head."""
    c = cache.c
    dev = cache.K.device
    _tokens("K", K, c.Hkv, None, c.d, dev)
    T = K.shape[1]
    _tokens("V", V, c.Hkv, T, c.d, dev)
    _ints("slots", slots, (T,), dev)
    if T == 0:
        return
    if stream is not None or _current_device() != dev.index:
        with _elsewhere(dev, stream):
            return _write(K, V, slots, cache)
    _write(K, V, slots, cache)


def _write(K, V, slots, cache):
    B.check(B.lib().dsa_cache_write(ctypes.byref(cache.c), K.data_ptr(), V.data_ptr(), *_strides(K), *_strides(V),
                                    slots.data_ptr(), K.shape[1], _raw_stream(K.device.index)), "dsa_cache_write")


def cache_attention(Q, cache, block_table, lens, n_q=1, O=None, lse=None, want_lse=False, workspace=None, stream=None):
    """Attention of each request's newest ``n_q`` tokens over its cached keys; returns (O, lse or None).

    Q [Hq, B * n_q, d] holds the tokens request by request; lens (int32 [B]) counts the tokens
    that each request has in the cache, the new ones among them (``cache_write`` first), and
    block_table (int32 [B, W]) names their pages.  Token i of a request sees its keys up to
    lens - n_q + i; a token that sees none has O = 0 and lse = -inf.  ``workspace`` (bytes,
    as many as ``dsa_cache_attention_workspace`` says) is allocated here if it is not given."""
    c = cache.c
    dev = cache.K.device
    _tokens("Q", Q, None, None, c.d, dev)
    Hq, T, d = Q.shape
    if Hq == 0 or Hq % c.Hkv:
        _refuse(f"{Hq} query heads do not divide into {c.Hkv} KV heads")
    n, width = _table(block_table)
    _ints("block_table", block_table, (n, width), dev)
    _ints("lens", lens, (n,), dev)
    if n_q < 1 or T != n * n_q:
        _refuse(f"Q has {T} rows, not {n_q} for each of {n} requests")
    if O is not None:
        _tokens("O", O, Hq, T, d, dev)
    if workspace is not None:
        _workspace(workspace, B.lib().dsa_cache_attention_workspace(d), dev)
    if stream is not None or _current_device() != dev.index:
        with _elsewhere(dev, stream):
            return _attend(Q, cache, block_table, lens, n_q, O, lse, want_lse, workspace)
    return _attend(Q, cache, block_table, lens, n_q, O, lse, want_lse, workspace)


def _attend(Q, cache, block_table, lens, n_q, O=None, lse=None, want_lse=False, workspace=None):
    c, dev = cache.c, cache.K.device
    Hq, T, d = Q.shape
    n, width = block_table.shape
    st = _raw_stream(dev.index)
    if O is None:
        O = torch.empty_like(Q, memory_format=torch.contiguous_format)
    lse = _lse(lse, want_lse, (Hq, T), dev)
    if workspace is None:
        workspace = torch.empty(B.lib().dsa_cache_attention_workspace(d), dtype=torch.uint8, device=dev)
    if n > 0:
        B.check(B.lib().dsa_cache_attention(
            ctypes.byref(c), Q.data_ptr(), Hq, *_strides(Q), block_table.data_ptr(), width, lens.data_ptr(), n, n_q,
            O.data_ptr(), *_strides(O), lse.data_ptr() if lse is not None else None, workspace.data_ptr(),
            workspace.nbytes, st), "dsa_cache_attention")
    return O, lse


class PagedLayer:
    """One attention layer as a server keeps it for ``requests`` requests at a time: their page
    tables, lengths and free pages, and the 8-bit cache of ``pages`` pages of ``page`` tokens.
    A request may hold ``width`` pages at most.  ``prefill`` takes prompts, short ones packed or
    one long one with sparse patterns, ``decode`` the tokens that follow.  Both enqueue work on
    the current stream of ``device`` only and update lengths, tables and cache in place; ``decode``, and
    ``prefill`` without patterns, can be captured into a CUDA graph.  Use it on one stream at a
    time.  If pages run out, no token of that call is
    stored and ``status`` says DSA_ERR_CAPACITY."""

    def __init__(self, Hq, Hkv, d, requests, pages, page=64, width=None, device="cuda"):
        # what a call would refuse behind the one that takes pages
        if Hq < 1 or Hkv < 1 or Hq % Hkv or Hq > 4096:
            _refuse(f"{Hq} query heads (4096 at most) do not divide into {Hkv} KV heads")
        if not 1 <= requests <= 4096:
            _refuse(f"1 to 4096 requests at a time, not {requests}")
        most = (width or pages) * page
        if most > 0x7fffff00 or (most // 64 + 5) * requests > 0x7fffffff or pages * page > 0x7fffffff:
            _refuse(f"{requests} requests of a width of {width or pages} pages are too many; give a smaller width")
        self.cache = PageCache.empty(pages, Hkv, page, d, device)
        dev = self.cache.K.device
        ints = dict(dtype=torch.int32, device=dev)
        self.Hq, self.page, self.requests = Hq, page, requests
        self.lens = torch.zeros(requests, **ints)
        self.table = torch.full((requests, width or pages), -1, **ints)
        self.free_pages = torch.arange(pages, **ints)
        self.free_count = torch.full((1,), pages, **ints)
        self.ones = torch.ones(requests, **ints)

    def _check(self, Q, K, V, packed):
        """Refuses what a call behind build_tables would: by then tables and lengths have changed.  (What is checked here
        is not checked there again.)"""
        c, dev = self.cache.c, self.cache.K.device
        if self.lens.device != dev or self.lens.shape != (self.requests,):
            _refuse(f"lens must stay an int32 tensor [{self.requests}] on {dev}")
        _tokens("Q", Q, self.Hq, None, c.d, dev)
        _tokens("K", K, c.Hkv, Q.shape[1] if packed else None, c.d, dev)
        _tokens("V", V, c.Hkv, K.shape[1], c.d, dev)
        for name, t in (("Q", Q), ("K", K), ("V", V)):
            _rows(name, t, packed)

    def _store(self, K, V, new_lens, prompts=None):
        T, n = K.shape[1], self.requests
        new = torch.empty(T + n + 1, dtype=torch.int32, device=self.lens.device)
        out = Tables(new[:T], new[T:], self.lens, self.free_count)
        build_tables(self.lens, new_lens, self.free_pages, self.free_count, self.table, self.page, T, out=out,
                     prompts=prompts)
        if T > 0:
            _write(K, V, out.slots, self.cache)
        return out

    def prefill(self, Q, K, V, new_lens, patterns=None, block=64):
        """Prompts of requests that hold no tokens yet (each row sees the call's rows alone).  Q
        [Hq, T, d], K and V [Hkv, T, d] hold their rows one after the other (T may be larger than
        their sum: the rows behind the last are undefined in O), new_lens (int32 [requests]) says
        how many each gets: 0 for a request that gets none, -1 for one that has ended and gives
        its pages back.  With ``patterns`` (as for ``build_indices``) all T rows are one request's
        prompt.  A request that gets tokens though it holds some, or rows that are not one
        prompt's, are found on the GPU: nothing is stored and ``status`` says DSA_ERR_DEVICE.
        Returns O."""
        self._check(Q, K, V, True)
        if not (0 if patterns is None else 1) <= Q.shape[1] <= 1 << 21:
            _refuse(f"a prefill takes up to {1 << 21} rows, not {Q.shape[1]}")
        if _current_device() != self.lens.device.index:
            with torch.cuda.device(self.lens.device):
                return self.prefill(Q, K, V, new_lens, patterns, block)
        if patterns is None:
            out = self._store(K, V, new_lens, "packed")
            return _prefill(Q, K, V, out.cu_seqlens)[0]
        _ints("new_lens", new_lens, (self.requests,), self.lens.device)
        O = sparse_prefill(Q, K, V, build_indices(Q, K, patterns, block))[0]  # first: it may refuse the patterns
        self._store(K, V, new_lens, "single")
        return O

    def decode(self, Q, K, V, new_lens=None, want_lse=False):
        """The next tokens: Q [Hq, requests * n_q, d] holds n_q rows for each request, K and V
        the rows of the requests that get tokens, one after the other.  new_lens (int32
        [requests], -1 ends a request) defaults to one token for every request, so that K and V
        hold one row each; a request that gets fewer than n_q attends with its newest n_q all the
        same.  Where pages run out (see ``status``), the rows attend over the tokens from before.
        Returns (O, lse or None)."""
        self._check(Q, K, V, False)
        n_q, behind = divmod(Q.shape[1], self.requests)
        if behind or not 1 <= n_q <= 4096:
            _refuse(f"Q has {Q.shape[1]} rows for {self.requests} requests")
        if new_lens is None:
            # row b goes to request b: rows behind the last request's are padding where Q has one row each, too
            if K.shape[1] < self.requests or (K.shape[1] > self.requests and n_q != 1):
                _refuse(f"K has {K.shape[1]} rows; without new_lens each of {self.requests} requests gets one")
            new_lens = self.ones
        if _current_device() != self.lens.device.index:
            with torch.cuda.device(self.lens.device):
                return self.decode(Q, K, V, new_lens, want_lse)
        self._store(K, V, new_lens)
        return _attend(Q, self.cache, self.table, self.lens, n_q, want_lse=want_lse)

    def status(self):
        """(status, detail) of the work on the current stream of the layer's device; synchronises it and clears the
        word."""
        return device_status(torch.cuda.current_stream(self.cache.K.device))

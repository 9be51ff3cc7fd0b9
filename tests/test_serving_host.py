"""Host-side checks of the serving calls (no GPU): the library refuses bad arguments before any
launch, the Python layer refuses tensors that are not on a GPU, and the plain forms that the GPU
tests rely on follow hand-worked examples."""
import ctypes
import os

import pytest
import torch

from tests import _serving as plain


@pytest.fixture(scope="module")
def B():
    from dynamic_sparse_attention_build_b200 import _binding
    if not os.path.exists(_binding.LIB_PATH):
        from dynamic_sparse_attention_build_b200 import build
        build.build()
    _binding.lib()
    return _binding


A = 1 << 20  # an aligned address that is never followed: every call below is refused on the host


def problem(B, **kw):
    v = dict(Hq=4, Hkv=2, N=100, d=128, block=64, reserved=0, q_head_stride=12800, q_token_stride=128,
             k_head_stride=12800, k_token_stride=128, v_head_stride=12800, v_token_stride=128, o_head_stride=12800,
             o_token_stride=128)
    v.update(kw)
    return B.dsa_problem(**v)


@pytest.mark.parametrize("change, args", [
    (dict(Hq=5), {}), (dict(N=0), {}), (dict(q_token_stride=120), {}), (dict(v_token_stride=132), {}),
    (dict(q_head_stride=0), {}), (dict(k_head_stride=0), {}), (dict(v_head_stride=0), {}), (dict(o_head_stride=0), {}),
    ({}, dict(Q=None)), ({}, dict(V=A + 8)), ({}, dict(O=A + 2)), ({}, dict(cu=None)), ({}, dict(n=-1)),
])
def test_packed_prefill_refuses(B, change, args):
    a = dict(Q=A, K=A, V=A, cu=A, n=3, O=A)
    a.update(args)
    got = B.lib().dsa_packed_prefill(ctypes.byref(problem(B, **change)), a["Q"], a["K"], a["V"], a["cu"], a["n"], a["O"],
                                     None, None)
    assert got == B.DSA_ERR_INVALID_ARG


def test_packed_prefill_refuses_unsupported_sizes(B):
    for change in (dict(d=96), dict(N=(1 << 21) + 1), dict(Hq=8192, Hkv=8192)):
        assert B.lib().dsa_packed_prefill(ctypes.byref(problem(B, **change)), A, A, A, A, 1, A, None, None) \
            == B.DSA_ERR_UNSUPPORTED


@pytest.mark.parametrize("change, want", [
    (dict(n=0), 1), (dict(width=0), 1), (dict(cap=0), 1), (dict(tokens=-1), 1), (dict(page=48), 1), (dict(page=512), 1),
    (dict(lens=None), 1), (dict(slots=None), 1), (dict(table=None), 1), (dict(n=4097), 2), (dict(tokens=(1 << 30) + 1), 2),
])
def test_build_tables_refuses(B, change, want):
    a = dict(n=3, lens=A, new=A, free=A, cap=9, count=A, table=A, width=4, page=64, tokens=10, slots=A, cu=A, out=A, left=A)
    a.update(change)
    assert B.lib().dsa_build_tables(*a.values(), None) == want


def cache(B, **kw):
    v = dict(num_pages=9, Hkv=2, page=64, d=128, page_stride=2 * 64 * 128, head_stride=64 * 128, token_stride=128, K=A, V=A,
             k_scale=A, v_scale=A)
    v.update(kw)
    return B.dsa_cache(**v)


BAD_CACHES = [(dict(num_pages=0), 1), (dict(page=24), 1), (dict(d=32), 2), (dict(Hkv=0), 1), (dict(K=None), 1),
              (dict(V=A + 8), 1), (dict(k_scale=None), 1), (dict(token_stride=64), 1), (dict(token_stride=136), 1),
              (dict(head_stride=64), 1), (dict(page_stride=100), 1), (dict(page_stride=0), 1), (dict(Hkv=4097), 2),
              (dict(num_pages=1 << 26), 2)]


@pytest.mark.parametrize("change, want", BAD_CACHES)
def test_bad_caches_are_refused(B, change, want):
    c = cache(B, **change)
    assert B.lib().dsa_cache_write(ctypes.byref(c), A, A, 512, 128, 512, 128, A, 4, None) == want
    assert B.lib().dsa_cache_attention(ctypes.byref(c), A, 4, 512, 128, A, 3, A, 2, 1, A, 512, 128, None, A, 1 << 30, None) == want


@pytest.mark.parametrize("change", [dict(T=-1), dict(K=None), dict(V=A + 8), dict(slots=None), dict(kt=100), dict(vh=4)])
def test_cache_write_refuses(B, change):
    a = dict(K=A, V=A, kh=512, kt=128, vh=512, vt=128, slots=A, T=4)
    a.update(change)
    assert B.lib().dsa_cache_write(ctypes.byref(cache(B)), *a.values(), None) == B.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("change, want", [
    (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(n=-1), 1), (dict(nq=0), 1), (dict(width=0), 1), (dict(Q=None), 1),
    (dict(O=A + 4), 1), (dict(qt=100), 1), (dict(ot=64), 1), (dict(oh=0), 1), (dict(ws=None), 1), (dict(size=100), 3),
    (dict(n=4097), 2), (dict(width=1 << 26), 2), (dict(Hq=8192), 2),
])
def test_cache_attention_refuses(B, change, want):
    a = dict(Q=A, Hq=4, qh=512, qt=128, table=A, width=3, lens=A, n=2, nq=1, O=A, oh=512, ot=128, lse=None, ws=A, size=1 << 30)
    a.update(change)
    assert B.lib().dsa_cache_attention(ctypes.byref(cache(B)), *a.values(), None) == want


def test_nothing_to_do_is_no_error(B):
    assert B.lib().dsa_cache_write(ctypes.byref(cache(B)), None, None, 0, 0, 0, 0, None, 0, None) == B.DSA_OK
    assert B.lib().dsa_packed_prefill(ctypes.byref(problem(B)), A, A, A, None, 0, A, None, None) == B.DSA_OK
    assert B.lib().dsa_cache_attention_workspace(128) > B.lib().dsa_cache_attention_workspace(64) > 0


def test_host_tensors_are_refused(B):
    import dynamic_sparse_attention_build_b200 as dsa
    t = torch.zeros(2, 5, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.packed_prefill(t, t, t, i)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.build_tables(i, i, i, i[:1], i[:, None], 16, 4)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.PageCache.empty(3, 2, 16, 64, device="cpu")


# ---- the plain forms ------------------------------------------------------------------------
def test_plain_tables_hand_example():
    # page 4; request 0 has 3 tokens in page 7 and gets 6 more, request 1 (pages 2, 5) ends, request 2 is new
    got = plain.tables_plain([3, 5, 0], [6, -1, 2], [9, 8, -1, -1, -1], 2, [[7, -1, -1], [2, 5, -1], [-1, -1, -1]], 4, 10)
    # 2 and 5 go on the stack [9, 8, 2, 5]; request 0 takes 5 and 2, request 2 takes 8
    assert got[0] == [31, 20, 21, 22, 23, 8, 32, 33, -1, -1]
    assert got[1] == [0, 6, 6, 8] and got[2] == [9, 0, 2] and got[3] == 1
    assert got[4] == [[7, 5, 2], [2, 5, -1], [8, -1, -1]] and got[6]
    # one page too few: nothing changes
    got = plain.tables_plain([0], [9], [1, 2], 2, [[-1, -1, -1]], 4, 10)
    assert got == ([-1] * 10, [0, 0], [0], 2, [[-1, -1, -1]], [1, 2], False)


def test_plain_e4m3_matches_torch_casts():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    every = every[torch.isfinite(every)]
    assert torch.equal(plain.e4m3_64(every), every)
    mids = (torch.sort(every).values[1:] + torch.sort(every).values[:-1]) / 2
    x = torch.cat([mids, mids * (1 + 2 ** -20), mids * (1 - 2 ** -20), torch.linspace(-448, 448, 999, dtype=torch.float64)])
    x = x.float()
    assert torch.equal(plain.e4m3_64(x.double()), x.to(torch.float8_e4m3fn).double())
    assert plain.power_for(0.0) == 2.0 ** -60 and plain.power_for(448.0) == 1.0 and plain.power_for(449.0) == 2.0
    assert plain.power_for(1e38) == 2.0 ** 60


def test_plain_attention_follows_differences():
    """d lse / d s_j is the weight of key j: the plain form's weights against differences."""
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(n, 8, generator=g, dtype=torch.float64) for n in (1, 5, 5))
    last = torch.tensor([3])
    o, lse, _, _, w = plain.attention64(q, k, v, last)
    h = 1e-6
    for j in range(5):
        k2 = k.clone()
        k2[j] += h * q[0]  # the score grows by h |q|^2 / sqrt(d)
        ds = h * float(q[0] @ q[0]) / 8 ** 0.5
        assert abs((float(plain.attention64(q, k2, v, last)[1]) - float(lse)) / ds - float(w[0, j])) < 1e-5
    assert float(w[0, 4]) == 0 and abs(float(w.sum()) - 1) < 1e-12
    assert torch.allclose(o, w @ v)


@pytest.mark.parametrize("change, want", [
    (dict(n=0), 1), (dict(width=0), 1), (dict(tokens=-1), 1), (dict(page=48), 1), (dict(lens=None), 1), (dict(n=4097), 2),
    (dict(single=2), 1), (dict(single=-1), 1),
])
def test_build_prompt_tables_refuses(B, change, want):
    a = dict(n=3, lens=A, new=A, free=A, cap=9, count=A, table=A, width=4, page=64, tokens=10, slots=A, cu=A, out=A, left=A, single=0)
    a.update(change)
    assert B.lib().dsa_build_prompt_tables(*a.values(), None) == want


def test_import_needs_no_private_names_of_torch():
    """Importing loads nothing: what a torch without CUDA lacks is looked up by the first call."""
    import subprocess
    import sys
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import dynamic_sparse_attention_build_b200 as dsa\n"
            "t, i = torch.zeros(2, 5, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)\n"
            "try:\n    dsa.packed_prefill(t, t, t, i)\n"
            "except ValueError as e:\n    print('refused:', e)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0 and "CUDA" in r.stdout, r.stderr


# (page, head and token stride) of 9 pages of 64 tokens, 2 heads, d 128
@pytest.mark.parametrize("strides, good", [
    ((2 * 64 * 128, 64 * 128, 128), True), ((2 * 64 * 128, 128, 2 * 128), True),  # [pages, heads, page, d], [pages, page, heads, d]
    ((64 * 128, 9 * 64 * 128, 128), True), ((128, 9 * 64 * 128, 9 * 128), True),  # heads in front; pages inside
    ((3 * 64 * 144, 64 * 144, 144), True),                                           # gaps everywhere
    ((64 * 128, 64 * 128, 128), False), ((2 * 64 * 128 - 16, 64 * 128, 128), False), ((2 * 64 * 128, 64 * 128 - 16, 128), False),
    ((2 * 64 * 128, 128, 128), False), ((2 * 64 * 128, 144, 2 * 128), False), ((128, 128, 128), False),
])
def test_caches_whose_pages_overlap_are_refused(B, strides, good):
    c = cache(B, page_stride=strides[0], head_stride=strides[1], token_stride=strides[2], V=1 << 30, v_scale=1 << 29)
    want = B.DSA_OK if good else B.DSA_ERR_INVALID_ARG
    assert B.lib().dsa_cache_write(ctypes.byref(c), None, None, 0, 0, 0, 0, None, 0, None) == want
    assert B.lib().dsa_cache_attention(ctypes.byref(c), A, 4, 512, 128, A, 3, A, 0, 1, A, 512, 128, None, A, 1 << 30, None) == want


@pytest.mark.parametrize("change, good", [
    (dict(V=A), False), (dict(V=A + 64 * 128), False), (dict(V=A - 128), False), (dict(V=A + 9 * 2 * 64 * 128), True),
    (dict(V=A - 9 * 2 * 64 * 128), True), (dict(page_stride=4 * 64 * 128, V=A + 2 * 64 * 128), True),  # K and V of one array
    (dict(token_stride=256, head_stride=64 * 256, page_stride=2 * 64 * 256, V=A + 128), True),
    (dict(k_scale=A, v_scale=A), False), (dict(k_scale=A, v_scale=A + 4 * 9 * 2 - 4), False), (dict(k_scale=A, v_scale=A + 4 * 9 * 2), True),
])
def test_a_store_into_keys_and_values_that_overlap_is_refused(B, change, good):
    """Reading them is fine: keys may be the values."""
    c = cache(B, **{**dict(V=1 << 30, v_scale=1 << 29), **change})
    # a call that passes these checks is refused for its number of tokens
    got = B.lib().dsa_cache_write(ctypes.byref(c), A, A, 512, 128, 512, 128, A, (1 << 30) + 1, None)
    assert got == (B.DSA_ERR_UNSUPPORTED if good else B.DSA_ERR_INVALID_ARG)
    assert B.lib().dsa_cache_attention(ctypes.byref(c), A, 4, 512, 128, A, 3, A, 0, 1, A, 512, 128, None, A, 1 << 30, None) == B.DSA_OK


@pytest.mark.parametrize("oh, ot, good", [(512, 128, True), (128, 512, True), (128, 128, False), (256, 192, False), (200, 400, False)])
def test_outputs_whose_rows_overlap_are_refused(B, oh, ot, good):
    """O of 4 heads and 4 rows, d 128.  (Good strides are refused for the missing workspace or the odd length instead.)"""
    got = B.lib().dsa_cache_attention(ctypes.byref(cache(B)), A, 4, 512, 128, A, 3, A, 4, 1, A, oh, ot, None, A, 10, None)
    assert got == (B.DSA_ERR_CAPACITY if good else B.DSA_ERR_INVALID_ARG)
    p = problem(B, N=4, o_head_stride=oh, o_token_stride=ot)
    assert B.lib().dsa_packed_prefill(ctypes.byref(p), A, A, A, A, 0, A, None, None) == (B.DSA_OK if good else B.DSA_ERR_INVALID_ARG)


def test_cache_layouts_whose_pages_overlap_are_refused_in_python(B, monkeypatch):
    from dynamic_sparse_attention_build_b200 import serving
    assert serving._apart(64, ((9, 8192), (2, 4096), (16, 256))) and serving._apart(64, ((1, 0), (2, 64), (1, 5)))
    assert serving._apart(64, ((9, 64), (2, 64 * 9 * 16), (16, 64 * 9)))
    for bad in (((9, 4096), (2, 4096), (16, 256)), ((9, 8192), (2, 64), (16, 64)), ((9, 0), (2, 64), (16, 128)), ((2, 32),)):
        assert not serving._apart(64, bad)


def test_lse_and_workspace_that_are_no_tensors_are_refused():
    from dynamic_sparse_attention_build_b200 import serving
    dev = torch.device("cpu")
    for bad in ([0.0] * 4, 7, torch.zeros(2, 3), torch.zeros(2, 2, dtype=torch.float64), torch.zeros(2, 4)[:, ::2]):
        with pytest.raises(ValueError, match="lse"):
            serving._lse(bad, False, (2, 2), dev)
    good = torch.zeros(2, 2)
    assert serving._lse(good, False, (2, 2), dev) is good and serving._lse(None, False, (2, 2), dev) is None
    for bad in (1 << 20, [0] * 64, torch.zeros(15), torch.zeros(64)[::2], torch.zeros(65, dtype=torch.uint8)[1:]):
        with pytest.raises(ValueError, match="workspace"):
            serving._workspace(bad, 64, dev)
    for good in (torch.zeros(16), torch.zeros(80, dtype=torch.uint8)):
        serving._workspace(good, 64, dev)


def test_serving_calls_keep_the_order_of_their_arguments():
    """What a caller may pass by place; later arguments stand behind these."""
    import inspect
    import dynamic_sparse_attention_build_b200 as dsa
    for call, names in ((dsa.build_tables, "lens new_lens free_pages free_count block_table page max_tokens out stream"),
                        (dsa.packed_prefill, "Q K V cu_seqlens O lse want_lse stream"), (dsa.cache_write, "K V slots cache stream"),
                        (dsa.cache_attention, "Q cache block_table lens n_q O lse want_lse workspace stream"),
                        (dsa.build_indices, "Q K patterns block bufs stream"), (dsa.device_status, "stream"),
                        (dsa.sparse_prefill, "Q K V idx O lse want_lse stream")):
        assert list(inspect.signature(call).parameters)[:len(names.split())] == names.split()

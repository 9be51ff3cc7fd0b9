"""packed_prefill against 64-bit softmax attention, sequence by sequence."""
import math

import pytest
import torch

from tests import _serving as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import dynamic_sparse_attention_build_b200 as m
    return m


def make(Hq, Hkv, T, d, seed=1, scale=1.0, layout="htd"):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def new(h):
        if layout == "thd":  # [tokens, heads, d] seen as [heads, tokens, d]
            return (torch.randn(T, h, d, generator=g, device="cuda") * scale).bfloat16().transpose(0, 1)
        if layout == "wide":  # rows of a wider projection
            return (torch.randn(h, T, d + 72, generator=g, device="cuda") * scale).bfloat16()[:, :, 8:8 + d]
        return (torch.randn(h, T, d, generator=g, device="cuda") * scale).bfloat16()
    return new(Hq), new(Hkv), new(Hkv)


def cu_of(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(O, lse, Q, K, V, cu):
    G = Q.shape[0] // K.shape[0]
    for a, b in zip(cu, cu[1:]):
        for h in range(Q.shape[0]):
            plain.check_rows(O[h, a:b], None if lse is None else lse[h, a:b], Q[h, a:b], K[h // G, a:b], V[h // G, a:b],
                             torch.arange(b - a, device="cuda"), plain.BF16, what=f"rows {a}..{b}, head {h}")


CASES = [
    (1, 1, 64, [1]), (2, 1, 128, [1, 1, 1]), (2, 1, 128, [127]), (2, 2, 128, [128]), (4, 2, 64, [129]),
    (1, 1, 128, [255, 256, 257]), (3, 1, 64, [128, 384, 5, 640]), (6, 2, 128, [700, 3, 129]),
    (4, 2, 64, [1, 2, 130, 0, 500, 0]), (5, 5, 128, [300]), (8, 1, 128, [1000, 257, 1]), (16, 2, 64, [2049]),
    # long sequences of odd head groups: row tiles of different lengths walk the keys together
    (3, 1, 64, [5000]), (2, 2, 64, [4096, 1, 3000]), (1, 1, 128, [3500, 129]),
]


@pytest.mark.parametrize("Hq, Hkv, d, lens", CASES)
def test_matches_64_bit_attention(dsa, Hq, Hkv, d, lens):
    T = sum(lens)
    Q, K, V = make(Hq, Hkv, T, d)
    O, lse = dsa.packed_prefill(Q, K, V, ints(cu_of(lens)), want_lse=True)
    assert dsa.device_status() == (0, 0)
    check(O, lse, Q, K, V, cu_of(lens))


@pytest.mark.parametrize("layout", ["thd", "wide"])
@pytest.mark.parametrize("G", [1, 2])
def test_layouts(dsa, layout, G):
    lens = [150, 290]
    Q, K, V = make(2 * G, 2, 440, 64, layout=layout)
    O = torch.empty(440, 2 * G, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    got, lse = dsa.packed_prefill(Q, K, V, ints(cu_of(lens)), O=O, want_lse=True)
    assert got is O and dsa.device_status() == (0, 0)
    check(O, lse, Q, K, V, cu_of(lens))


@pytest.mark.parametrize("G", [1, 2])
def test_large_scores_and_growing_maxima(dsa, G):
    """Scores of several hundred: the running maximum moves far, weights underflow."""
    Q, K, V = make(G, 1, 600, 128, scale=6.0)
    K = (K.float() * torch.linspace(0.1, 3, 600, device="cuda")[None, :, None]).bfloat16()
    O, lse = dsa.packed_prefill(Q, K, V, ints([0, 600]), want_lse=True)
    assert dsa.device_status() == (0, 0)
    check(O, lse, Q, K, V, [0, 600])


def test_large_values(dsa):
    Q, K, V = make(2, 1, 300, 64)
    V = (V.float() * 2.0 ** 100).bfloat16()
    K = (K.float() * torch.linspace(0.1, 4, 300, device="cuda")[None, :, None]).bfloat16()
    O, lse = dsa.packed_prefill(Q, K, V, ints([0, 300]), want_lse=True)
    check(O, lse, Q, K, V, [0, 300])


@pytest.mark.parametrize("G", [1, 2])
def test_rows_of_no_sequence_are_left_alone(dsa, G):
    """Rows before the first sequence and behind the last: not read, not written."""
    lens, T = [100, 0, 61], 300
    cu = cu_of(lens, 30)
    Q, K, V = make(2 * G, 2, T, 128)
    for t in (Q, K, V):
        t[:, :30] = math.nan
        t[:, cu[-1]:] = math.inf
    O, lse = torch.full_like(Q, 7.0), torch.full((2 * G, T), 9.0, device="cuda")
    dsa.packed_prefill(Q, K, V, ints(cu), O=O, lse=lse)
    assert dsa.device_status() == (0, 0)
    out = torch.ones(T, dtype=torch.bool, device="cuda")
    out[30:cu[-1]] = False
    assert (O[:, out] == 7.0).all() and (lse[:, out] == 9.0).all()
    check(O, lse, Q, K, V, cu)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("at", [60, 127, 128, 200, 255, 256, 280])
def test_non_finite_values_reach_those_who_see_them(dsa, bad, G, at):
    """A non-finite value of row `at` reaches every later row of its sequence and no earlier one,
    whichever tile holds it; other sequences stay as they are."""
    cu = [0, 300, 420]
    Q, K, V = make(G, 1, 420, 64)
    ref, ref_lse = dsa.packed_prefill(Q, K, V, ints(cu), want_lse=True)
    V2 = V.clone()
    V2[0, at, 17] = bad
    O, lse = dsa.packed_prefill(Q, K, V2, ints(cu), want_lse=True)
    assert dsa.device_status() == (0, 0)
    assert torch.equal(lse, ref_lse)
    want = ref.clone()
    want[:, at:300, 17] = bad
    assert torch.equal(O.nan_to_num(1e30, 2e30, -2e30), want.nan_to_num(1e30, 2e30, -2e30))


@pytest.mark.parametrize("which", ["Q", "K"])
def test_nan_of_a_query_or_key(dsa, which):
    cu = [0, 200, 330]
    Q, K, V = make(2, 1, 330, 128)
    ref, _ = dsa.packed_prefill(Q, K, V, ints(cu))
    t = dict(Q=Q, K=K)[which]
    t[:, 140] = math.nan
    O, _ = dsa.packed_prefill(Q, K, V, ints(cu))
    hit = torch.zeros(330, dtype=torch.bool, device="cuda")
    hit[140:200 if which == "K" else 141] = True
    assert torch.isnan(O[:, hit]).all() and torch.equal(O[:, ~hit], ref[:, ~hit])


def test_many_short_sequences(dsa):
    """More sequences than a warp has lanes, empty ones among them, none longer than a tile."""
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 40, (150,), generator=g).tolist()
    Q, K, V = make(4, 2, sum(lens), 64)
    O, lse = dsa.packed_prefill(Q, K, V, ints(cu_of(lens)), want_lse=True)
    assert dsa.device_status() == (0, 0)
    check(O, lse, Q, K, V, cu_of(lens))


def test_malformed_bounds_are_skipped_and_reported(dsa):
    from dynamic_sparse_attention_build_b200 import _binding as B
    Q, K, V = make(2, 1, 300, 64)
    for cu, good in (([0, 100, 50, 50], [(0, 100)]), ([0, 100, 301], [(0, 100)]), ([-5, 100, 200], [(100, 200)])):
        O = torch.full_like(Q, 7.0)
        dsa.packed_prefill(Q, K, V, ints(cu), O=O)
        assert dsa.device_status() == (B.DSA_ERR_DEVICE, 37)
        seen = torch.zeros(300, dtype=torch.bool, device="cuda")
        for a, b in good:
            seen[a:b] = True
        assert (O[:, ~seen] == 7.0).all() and torch.isfinite(O).all()
        a, b = good[-1]
        check(O, None, Q, K, V, [a, b])
    assert dsa.device_status() == (0, 0)


def test_no_sequences_and_no_rows(dsa):
    Q, K, V = make(2, 1, 5, 64)
    O = torch.full_like(Q, 7.0)
    for cu in ([0], [0, 0], [5, 5, 5]):
        dsa.packed_prefill(Q, K, V, ints(cu), O=O)
    assert (O == 7.0).all() and dsa.device_status() == (0, 0)
    empty = Q[:, :0]
    assert dsa.packed_prefill(empty, K[:, :0], V[:, :0], ints([0, 0]))[0].shape == (2, 0, 64)


def test_agrees_with_the_sparse_prefill_of_a_full_window(dsa):
    """A-shape with a window of the whole prompt is dense attention."""
    Q, K, V = make(4, 2, 777, 128)
    idx = dsa.build_indices(Q, K, [dict(kind="ashape", sink=0, window=777)] * 4, 64)
    a, la = dsa.sparse_prefill(Q, K, V, idx, want_lse=True)
    b, lb = dsa.packed_prefill(Q, K, V, ints([0, 777]), want_lse=True)
    check(a, la, Q, K, V, [0, 777])
    check(b, lb, Q, K, V, [0, 777])


def test_captured_and_replayed_with_other_inputs(dsa):
    Q, K, V = make(4, 2, 500, 64)
    cu = ints([0, 200, 500])
    O, lse = torch.zeros_like(Q), torch.zeros(4, 500, device="cuda")
    dsa.packed_prefill(Q, K, V, cu, O=O, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.packed_prefill(Q, K, V, cu, O=O, lse=lse)
    for seed, now in ((2, [0, 1, 499]), (3, [0, 499, 500])):
        q, k, v = make(4, 2, 500, 64, seed=seed)
        for a, b in ((Q, q), (K, k), (V, v), (cu, ints(now))):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        check(O, lse, q, k, v, now)


def test_two_streams_at_once_give_the_same_bits(dsa):
    Q, K, V = make(8, 2, 1500, 128)
    cu = ints([0, 700, 1500])
    want, _ = dsa.packed_prefill(Q, K, V, cu)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[dsa.packed_prefill(Q, K, V, cu, stream=s)[0] for _ in range(4)] for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for os in got for o in os)
    for s in streams:
        assert dsa.device_status(s) == (0, 0)


def test_waits_that_run_out_leave_the_next_launch_exact(dsa):
    from dynamic_sparse_attention_build_b200 import _binding as B
    Q, K, V = make(8, 2, 6000, 128)
    cu = ints([0, 4000, 6000])
    want, want_lse = dsa.packed_prefill(Q, K, V, cu, want_lse=True)
    assert dsa.device_status() == (0, 0)
    out = 0
    try:
        for limit in (1, 300, 1000, 3000, 10000):
            assert B.dsa_set_wait_limit(limit) == B.DSA_OK
            dsa.packed_prefill(Q, K, V, cu)
            status, _ = dsa.device_status()
            assert status in (B.DSA_OK, B.DSA_ERR_TIMEOUT)
            out += status == B.DSA_ERR_TIMEOUT
    finally:
        assert B.dsa_set_wait_limit(0) == B.DSA_OK
    assert out > 0
    O, lse = dsa.packed_prefill(Q, K, V, cu, want_lse=True)
    assert dsa.device_status() == (0, 0)
    assert torch.equal(O, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("change, match", [
    (dict(Q="float"), "bfloat16"), (dict(K="short"), "dimension 1"), (dict(V="heads"), "dimension 0"),
    (dict(Q="three"), "divide"), (dict(cu="long"), "int32"), (dict(cu="host"), "on cpu"), (dict(Q="d"), "64 or 128"),
    (dict(Q="strided"), "contiguous"), (dict(O="short"), "dimension 1"), (dict(lse="short"), "lse"), (dict(cu="none"), "cu_seqlens"),
])
def test_refusals(dsa, change, match):
    Q, K, V = make(4, 2, 50, 64)
    a = dict(Q=Q, K=K, V=V, cu_seqlens=ints([0, 50]), O=None, lse=None)
    (name, how), = change.items()
    if name == "cu":
        a["cu_seqlens"] = {"long": a["cu_seqlens"].long(), "host": a["cu_seqlens"].cpu(), "none": a["cu_seqlens"][:0]}[how]
    elif name == "lse":
        a["lse"] = torch.empty(4, 49, device="cuda")
    else:
        t = a[name] if a[name] is not None else Q.clone()
        a[name] = {"float": t.float(), "short": t[:, :49], "heads": t[:1], "three": t[[0, 0, 1]], "d": t[:, :, :32],
                   "strided": t.transpose(1, 2).contiguous().transpose(1, 2)}[how]
    with pytest.raises(ValueError, match=match):
        dsa.packed_prefill(a["Q"], a["K"], a["V"], a["cu_seqlens"], O=a["O"], lse=a["lse"])


def test_misaligned_rows_are_refused(dsa):
    from dynamic_sparse_attention_build_b200 import _binding as B
    Q, K, V = make(4, 2, 50, 64)
    with pytest.raises(B.DSAError) as e:
        dsa.packed_prefill(Q, torch.zeros(2, 50, 65, dtype=torch.bfloat16, device="cuda")[:, :, 1:], V, ints([0, 50]))
    assert e.value.status == B.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [128], [200, 250], [60, 1, 256] * 20])
def test_waits_that_run_out_on_short_prompts(dsa, lens, d):
    """Prompts whose loads are all on their way before the first wait ends: the loader never meets a wait of its own,
    so another warp gives up first.  The launches behind the ones that gave up are exact."""
    from dynamic_sparse_attention_build_b200 import _binding as B
    Q, K, V = make(4, 2, sum(lens), d)
    cu = ints(cu_of(lens))
    want, want_lse = dsa.packed_prefill(Q, K, V, cu, want_lse=True)
    assert dsa.device_status() == (0, 0)
    out = 0
    try:
        for limit in (1, 100, 300, 1000, 3000):
            assert B.dsa_set_wait_limit(limit) == B.DSA_OK
            for _ in range(4):
                dsa.packed_prefill(Q, K, V, cu)
            assert B.dsa_set_wait_limit(0) == B.DSA_OK
            O, lse = dsa.packed_prefill(Q, K, V, cu, want_lse=True)  # right behind them
            status, _ = dsa.device_status()
            assert status in (B.DSA_OK, B.DSA_ERR_TIMEOUT)
            out += status == B.DSA_ERR_TIMEOUT
            assert torch.equal(O, want) and torch.equal(lse, want_lse)
    finally:
        assert B.dsa_set_wait_limit(0) == B.DSA_OK
    assert out > 0  # (a bound of 1 ns is shorter than any load)
    assert dsa.device_status() == (0, 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("power", [119, 121])
def test_large_values_under_a_maximum_that_lags(dsa, G, d, power):
    """The row's first keys weigh 1, a later one 2^7.9 with a value near the type's largest: a maximum that is not
    raised for it must not take the sum out of fp32's range, as it would stay in it with an exact maximum."""
    T = 300
    Q, K = torch.zeros(G, T, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, T, d, dtype=torch.bfloat16, device="cuda")
    V = make(G, 1, T, d)[2]
    Q[:, :, 0] = 8.0
    for at in (100, 170):  # in the half tile and in the tile behind the first
        K[0, at, 0] = 5.46875 * d ** 0.5 / 8  # (bf16 rounds the weight for d 128, for both sides alike)
        V[0, at] = V[0, at].sign() * 2.0 ** power
    O, lse = dsa.packed_prefill(Q, K, V, ints([0, T]), want_lse=True)
    assert dsa.device_status() == (0, 0)
    check(O, lse, Q, K, V, [0, T])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("power", [10, 20, 24, 26, 28, 30, 32, 40, 60, 100])
def test_scores_far_beyond_the_exponents_range(dsa, G, d, power):
    """One product a score, so scores are exact: the largest of them (a few equal ones) share the row whatever their
    size.  All that is rounded is P, O and the scores' scale, which is the same for equal scores."""
    T = 300
    Q, K = torch.zeros(G, T, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, T, d, dtype=torch.bfloat16, device="cuda")
    V = make(G, 1, T, d)[2]
    Q[:, :, 0] = 2.0 ** power
    K[0, :, 0] = (torch.arange(T, device="cuda") * 37 % 101 + 1).bfloat16()  # (up to 101: exact)
    O, lse = dsa.packed_prefill(Q, K, V, ints([0, T]), want_lse=True)
    assert dsa.device_status() == (0, 0)
    for h in range(G):
        o, l, a = plain.attention64_far(Q[h].double(), K[0].double(), V[0].double(), torch.arange(T, device="cuda"))
        assert torch.isfinite(O).all()
        assert ((O[h].double() - o).abs() <= plain.BF16 * o.abs() + 1.01 * a * (plain.BF16 + 2.0 ** -20)).all()
        assert ((lse[h].double() - l).abs() <= 4 * plain.FP32 * l.abs() + 2.0 ** -20).all()


@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("lens", [[0] * 40 + [5] + [0] * 70 + [300], [0] * 64, [1] * 32 + [0] * 32 + [129], [300] + [0] * 100])
def test_windows_of_empty_sequences(dsa, lens, G):
    T = sum(lens)
    Q, K, V = make(2 * G, 2, max(T, 1), 64)
    O, lse = torch.full_like(Q, 7.0), torch.full(Q.shape[:2], 9.0, device="cuda")
    dsa.packed_prefill(Q, K, V, ints(cu_of(lens)), O=O, lse=lse)
    assert dsa.device_status() == (0, 0)
    assert T > 0 or (O == 7.0).all()
    check(O, lse, Q, K, V, cu_of(lens))

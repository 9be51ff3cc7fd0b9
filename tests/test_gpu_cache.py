"""The paged 8-bit cache: page tables, store, attention over it, and a run of them together."""
import math
import random

import pytest
import torch

from tests import _serving as plain

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dsa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import dynamic_sparse_attention_build_b200 as m
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# --------------------------------------------------------------------------- page tables
def state(rng, n, longest, page, share_end=0.2):
    """Requests with pages of their own, new lengths, and the stack of the other pages."""
    lens = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, longest)]) for _ in range(n)]
    new = [-1 if rng.random() < share_end else rng.choice([0, 1, 1, page, rng.randint(0, longest)]) for _ in range(n)]
    up = lambda x: -(-x // page)  # noqa: E731
    width = max(1, max(up(x + max(y, 0)) for x, y in zip(lens, new)))
    total = sum(up(x + max(y, 0)) for x, y in zip(lens, new)) + 3
    order = list(range(total))
    rng.shuffle(order)
    table = []
    for x in lens:
        table.append([order.pop() for _ in range(up(x))] + [-1] * (width - up(x)))
    return lens, new, order + [-1] * (total - len(order)), len(order), table


def run_tables(dsa, lens, new, free, count, table, page, tokens, in_place=False):
    d = [ints(x) for x in (lens, new, free, [count], table)]
    out = None
    if in_place:
        out = dsa.Tables(torch.full((tokens,), 5, dtype=torch.int32, device="cuda"), ints([5] * (len(lens) + 1)), d[0], d[3])
    got = dsa.build_tables(d[0], d[1], d[2], d[3], d[4], page, tokens, out=out)
    return (got.slots.tolist(), got.cu_seqlens.tolist(), got.lens.tolist(), got.free_count.item(), d[4].tolist(), d[2].tolist())


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n, longest, page", [(1, 0, 16), (1, 1, 16), (1, 700, 64), (2, 40, 32), (33, 300, 16), (513, 90, 64),
                                              (1500, 20, 256), (4096, 12, 16), (7, 30000, 128)])
def test_tables_match_the_rules(dsa, n, longest, page, in_place):
    args = state(random.Random(n + page), n, longest, page)
    tokens = sum(max(x, 0) for x in args[1]) + (0 if n % 2 else 7)
    want = plain.tables_plain(*args, page, tokens)
    assert want[-1]
    assert run_tables(dsa, *args, page, tokens, in_place) == want[:-1]
    assert dsa.device_status() == (0, 0)


def test_tables_refuse_as_a_whole(dsa):
    from dynamic_sparse_attention_build_b200 import _binding as B
    base = dict(lens=[20, 5, 0], new=[30, -1, 4], free=[3, 4, -1, -1], count=2, table=[[0, 1, -1, -1], [2, -1, -1, -1], [-1] * 4],
                page=16, tokens=40)
    assert plain.tables_plain(*base.values())[-1]
    for change, status, detail in ((dict(count=1, free=[3, -1, -1, -1], new=[30, -1, 20], tokens=60),  # 1 + 1 released, 2 + 2 needed
                                    B.DSA_ERR_CAPACITY, 23),
                                   (dict(tokens=33), B.DSA_ERR_CAPACITY, 24), (dict(new=[45, -1, 4]), B.DSA_ERR_CAPACITY, 25),
                                   (dict(lens=[20, -5, 0]), B.DSA_ERR_DEVICE, 38),
                                   (dict(free=[3, 4], count=2), B.DSA_ERR_CAPACITY, 23)):
        a = {**base, **change}
        want = plain.tables_plain(*a.values())
        assert not want[-1]
        assert run_tables(dsa, *a.values()) == want[:-1], change
        assert dsa.device_status() == (status, detail), change
    assert run_tables(dsa, *base.values()) == plain.tables_plain(*base.values())[:-1]
    assert dsa.device_status() == (0, 0)


def test_tables_report_a_page_that_is_none(dsa):
    from dynamic_sparse_attention_build_b200 import _binding as B
    got = run_tables(dsa, [3, 16], [2, 1], [-1], 1, [[-7, -1], [4, -1]], 16, 4)
    assert got[0] == [-1, -1, -1, -1] and dsa.device_status() == (B.DSA_ERR_DEVICE, 39)


def test_tables_captured_over_many_steps(dsa):
    """A decode step's tables captured once, lengths and count updated in place by every replay."""
    page, n = 16, 5
    lens, new, free, count = ints([0, 15, 16, 31, 3]), ints([1] * n), ints(list(range(40))), ints([34])
    table = torch.full((n, 8), -1, dtype=torch.int32, device="cuda")
    for b, pages in enumerate([[], [34], [35], [36, 37], [38]]):
        for j, p in enumerate(pages):
            table[b, j] = p
    host = [lens.tolist(), free.tolist(), count.item(), table.tolist()]
    out = dsa.Tables(ints([0] * n), ints([0] * (n + 1)), lens, count)
    assert dsa.device_status() == (0, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.build_tables(lens, new, free, count, table, page, n, out=out)
    for step in range(40):
        new.copy_(ints([1, 1, -1 if step == 20 else 1, 0, 2]))
        want = plain.tables_plain(host[0], new.tolist(), host[1], host[2], host[3], page, n + 1)
        graph.replay()
        assert out.slots.tolist() == want[0][:n] and out.cu_seqlens.tolist() == want[1]
        host = [want[2], want[5], want[3], want[4]]
        assert [lens.tolist(), free.tolist(), count.item(), table.tolist()] == host
    assert dsa.device_status() == (0, 0)


# --------------------------------------------------------------------------- store
def filled(dsa, pages, Hkv, page, d, seed=1, layout="phtd"):
    g = gen(seed)

    def data():
        x = torch.randn(pages, Hkv, page, d, generator=g, device="cuda") * 60
        if layout == "pthd":  # [pages, page, Hkv, d] seen as [pages, Hkv, page, d]
            x = x.transpose(1, 2).contiguous().to(E4M3).transpose(1, 2)
            return x
        return x.to(E4M3)

    def scale():
        return torch.ldexp(torch.ones(pages, Hkv, device="cuda"),
                           torch.randint(-9, -3, (pages, Hkv), generator=g, device="cuda"))
    return dsa.PageCache(data(), data(), scale(), scale())


def raw(x):
    return x.double().cpu()


def check_write(dsa, K, V, slots, cache, compare=None):
    ref = [(raw(cache.K), raw(cache.k_scale)), (raw(cache.V), raw(cache.v_scale))]
    for X, (data, scale) in zip((K, V), ref):
        plain.write_plain(X.cpu(), slots, data, scale)
    dsa.cache_write(K, V, ints(slots), cache)
    for (data, scale), got, got_scale in zip(ref, (cache.K, cache.V), (cache.k_scale, cache.v_scale)):
        assert torch.equal(raw(got_scale), scale)
        assert torch.equal(raw(got).nan_to_num(1e6), data.nan_to_num(1e6))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page, Hkv, runs", [
    # runs: (page, first place, tokens)
    (16, 1, [(0, 0, 1)]), (16, 2, [(3, 15, 1), (5, 0, 16), (1, 0, 3)]), (64, 3, [(2, 0, 64), (0, 0, 64), (4, 0, 7), (1, 63, 1)]),
    (256, 2, [(1, 0, 256), (3, 0, 200), (0, 255, 1), (2, 100, 156)]), (128, 8, [(i, 7 * i, 1) for i in range(6)]),
    (32, 2, [(0, 1, 31), (1, 0, 32), (2, 0, 32), (3, 0, 5)]),
])
def test_store_is_exact(dsa, page, Hkv, runs, d):
    cache = filled(dsa, 7, Hkv, page, d)
    slots = []
    for k, (p, first, n) in enumerate(runs):
        slots += [-1] * (k % 3) + [p * page + first + i for i in range(n)]
    slots += [-1, -5]
    g = gen(2)
    K, V = (torch.randn(Hkv, len(slots), d, generator=g, device="cuda").bfloat16() * 3 for _ in range(2))
    K[0] *= 40
    check_write(dsa, K, V, slots, cache)
    assert dsa.device_status() == (0, 0)


def test_store_of_many_tokens(dsa):
    """More tokens than one CTA takes one by one: chunks that begin inside a run."""
    page, Hkv, d, pages = 32, 2, 64, 200
    cache = filled(dsa, pages, Hkv, page, d)
    rng = random.Random(1)
    slots, order = [], list(range(pages))
    rng.shuffle(order)
    while len(slots) < 4500:
        pg, first = order.pop(), rng.choice([0, 0, 0, 5])
        slots += [pg * page + i for i in range(first, rng.choice([page, page, 20]))]
    g = gen(3)
    K, V = (torch.randn(Hkv, len(slots), d, generator=g, device="cuda").bfloat16() for _ in range(2))
    check_write(dsa, K, V, slots, cache)
    assert dsa.device_status() == (0, 0)


@pytest.mark.parametrize("layout", ["pthd", "phtd"])
def test_store_layouts(dsa, layout):
    cache = filled(dsa, 4, 2, 16, 64, layout=layout)
    g = gen(4)
    X = torch.randn(21, 4, 64, generator=g, device="cuda").bfloat16()  # K and V of one projection
    slots = [2 * 16 + 3 + i for i in range(5)] + [i for i in range(16)]
    check_write(dsa, X[:, :2].transpose(0, 1), X[:, 2:].transpose(0, 1), slots, cache)


def test_store_of_extreme_values(dsa):
    """Zeros, the smallest and largest magnitudes, borders of the scale, infinities and NaN."""
    cache = filled(dsa, 8, 1, 16, 64)
    K = torch.zeros(1, 128, 64, dtype=torch.bfloat16, device="cuda")
    K[0, 16:32] = 2.0 ** -133
    K[0, 32:48] = 3.3e38
    K[0, 48] = 448.0
    K[0, 64] = 450.0
    K[0, 80, 5] = math.inf
    K[0, 81, 6] = -math.inf
    K[0, 82, 7] = 3.0
    K[0, 96, 5] = math.nan
    K[0, 97, 5] = -2.0
    K[0, 112:128] = math.nan
    check_write(dsa, K, -K, list(range(128)), cache)
    assert dsa.device_status() == (0, 0)


def test_append_token_by_token(dsa):
    """Tokens appended one at a time, growing and shrinking: the scale only grows."""
    cache = dsa.PageCache.empty(2, 2, 16, 64)
    g = gen(5)
    for i in range(20):
        K, V = (torch.randn(2, 1, 64, generator=g, device="cuda").bfloat16() * 2.0 ** ((i * 7) % 11 - 5) for _ in range(2))
        check_write(dsa, K, V, [i if i < 16 else 16 + i - 16], cache)
    assert dsa.device_status() == (0, 0)


def test_store_reports_bad_slots_and_scales(dsa):
    from dynamic_sparse_attention_build_b200 import _binding as B
    cache = filled(dsa, 4, 2, 16, 64)
    before = [x.clone() for x in (cache.K.view(torch.uint8), cache.V.view(torch.uint8), cache.k_scale, cache.v_scale)]
    K = torch.ones(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    dsa.cache_write(K, K, ints([64, 65, 2 ** 31 - 1]), cache)
    assert dsa.device_status() == (B.DSA_ERR_DEVICE, 40)
    for a, b in zip(before, (cache.K.view(torch.uint8), cache.V.view(torch.uint8), cache.k_scale, cache.v_scale)):
        assert torch.equal(a, b)
    for bad in (0.0, math.nan, math.inf, -1.0, 1e30):
        cache.k_scale[1, 1] = bad
        dsa.cache_write(K[:, :1], K[:, :1], ints([20]), cache)
        assert dsa.device_status() == (B.DSA_ERR_DEVICE, 41)
        assert float(cache.k_scale[1, 1]) == 2.0 ** -8  # 1 <= 448 * 2^-8
        assert (cache.K[1, 1, 4].float() == 256).all()
    assert dsa.device_status() == (0, 0)


# --------------------------------------------------------------------------- attention
def attend_inputs(dsa, Hq, Hkv, d, page, lens, n_q, seed=1, layout="phtd", spare=3, big=1.0):
    up = lambda x: -(-x // page)  # noqa: E731
    total = sum(up(n) for n in lens) + spare
    cache = filled(dsa, total, Hkv, page, d, seed, layout)
    order = list(range(total))
    random.Random(seed).shuffle(order)
    width = max(1, max((up(n) for n in lens), default=1)) + 1
    table = [[order.pop() for _ in range(up(n))] for n in lens]
    table = [r + [-1] * (width - len(r)) for r in table]
    Q = torch.randn(Hq, len(lens) * n_q, d, generator=gen(seed + 7), device="cuda") * big
    return cache, ints(table) if lens else torch.zeros(0, 1, dtype=torch.int32, device="cuda"), ints(lens), Q.bfloat16()


def check_attend(O, lse, Q, cache, table, lens, n_q, slack=0.0):
    """Beside the roundings of check_rows (weights in fp16): weights lose what is under 2^-25 of a
    unit that is 2^-10 of the largest weight x value scale; n keys, values up to 448 each."""
    d, Hkv, page = Q.shape[2], cache.K.shape[1], cache.K.shape[2]
    G = Q.shape[0] // Hkv
    for b, n in enumerate(lens):
        pages = table[b, :-(-n // page)].long()
        rows = slice(b * n_q, (b + 1) * n_q)
        last = torch.arange(n - n_q, n, device="cuda")
        for h in range(Hkv):
            k = (cache.K[pages, h].double() * cache.k_scale[pages, h].double()[:, None, None]).reshape(-1, d)[:n]
            v = (cache.V[pages, h].double() * cache.v_scale[pages, h].double()[:, None, None]).reshape(-1, d)[:n]
            vs = cache.v_scale[pages, h].double().repeat_interleave(page)[:n]
            extra = lambda w: n * 448.0 * 2.0 ** -35 * (w * vs).amax(-1, keepdim=True)  # noqa: E731, B023
            for q in range(h * G, (h + 1) * G):
                plain.check_rows(O[q, rows], None if lse is None else lse[q, rows], Q[q, rows], k, v, last, plain.FP16,
                                 extra if n else None, f"request {b}, head {q}", slack)


CASES = [
    # Hq, Hkv, d, page, lens, n_q
    (1, 1, 64, 16, [1], 1), (4, 1, 128, 16, [1, 0, 15, 16, 17], 1), (8, 2, 128, 64, [63, 64, 65, 1000], 1),
    (16, 16, 64, 32, [100, 1], 1), (32, 8, 128, 64, [513], 1), (12, 4, 128, 128, [300, 0, 127, 129], 2),
    (8, 1, 64, 256, [700, 255], 1), (16, 1, 128, 16, [90, 33], 1), (16, 2, 64, 64, [200, 3, 0, 65], 5),
    (32, 1, 128, 64, [130, 20], 3), (2, 2, 64, 16, [4, 2, 9, 0], 7), (32, 8, 128, 64, [2111, 640], 2),
    (6, 2, 128, 32, [5000], 1), (4, 4, 64, 16, [1, 2, 3] * 60, 1), (8, 2, 128, 64, [3000], 40),
    # a unit in as many parts as there are CTAs, rows of several tiles
    (3, 1, 64, 32, [60000], 1), (32, 1, 128, 64, [20000, 5], 3), (2, 2, 128, 16, [1, 70000, 300], 1),
]


@pytest.mark.parametrize("Hq, Hkv, d, page, lens, n_q", CASES)
def test_attention_matches_64_bits(dsa, Hq, Hkv, d, page, lens, n_q):
    cache, table, dl, Q = attend_inputs(dsa, Hq, Hkv, d, page, lens, n_q)
    O, lse = dsa.cache_attention(Q, cache, table, dl, n_q=n_q, want_lse=True)
    assert dsa.device_status() == (0, 0)
    check_attend(O, lse, Q, cache, table, lens, n_q)


@pytest.mark.parametrize("layout", ["pthd", "phtd"])
def test_attention_layouts(dsa, layout):
    lens, n_q = [70, 31, 200], 2
    cache, table, dl, Q = attend_inputs(dsa, 8, 2, 64, 32, lens, n_q, layout=layout)
    Q = Q.transpose(0, 1).contiguous().transpose(0, 1)
    O = torch.empty(6, 8, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    got, lse = dsa.cache_attention(Q, cache, table, dl, n_q=n_q, O=O, want_lse=True)
    assert got is O
    check_attend(O, lse, Q, cache, table, lens, n_q)


@pytest.mark.parametrize("big", [1e-30, 8.0, 1e30])
def test_attention_of_extreme_queries(dsa, big):
    """Queries far from 1: weights that are all alike, or one key's alone."""
    cache, table, dl, Q = attend_inputs(dsa, 4, 2, 128, 64, [300, 77], 1, big=big)
    O, lse = dsa.cache_attention(Q, cache, table, dl, want_lse=True)
    assert torch.isfinite(O).all() and dsa.device_status() == (0, 0)
    if big <= 8:
        check_attend(O, lse, Q, cache, table, [300, 77], 1)


def test_pages_whose_value_scales_differ_widely(dsa):
    lens = [500]
    cache, table, dl, Q = attend_inputs(dsa, 4, 1, 128, 16, lens, 1)
    cache.v_scale.copy_(torch.ldexp(torch.ones_like(cache.v_scale),
                                    torch.randint(-40, 40, cache.v_scale.shape, generator=gen(3), device="cuda")))
    O, lse = dsa.cache_attention(Q, cache, table, dl, want_lse=True)
    # three roundings of exponents below 128 in size (2^-18 each), the value scale among them
    check_attend(O, lse, Q, cache, table, lens, 1, slack=2.0 ** -16)


@pytest.mark.parametrize("n_q", [1, 3])
def test_hidden_values_never_reach_a_row(dsa, n_q):
    """NaN in the rest of the last page, in free pages and under keys that only later tokens see."""
    lens = [37, 90, 16, 2]
    cache, table, dl, Q = attend_inputs(dsa, 4, 2, 64, 16, lens, n_q)
    want, want_lse = dsa.cache_attention(Q, cache, table, dl, n_q=n_q, want_lse=True)
    own = torch.zeros(cache.K.shape[0], 16, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for j in range(n):
            own[int(table[b, j // 16]), j % 16] = True
    for x in (cache.K, cache.V):
        x.view(torch.uint8).transpose(1, 2)[~own] = 0x7f
    O, lse = dsa.cache_attention(Q, cache, table, dl, n_q=n_q, want_lse=True)
    assert dsa.device_status() == (0, 0) and torch.equal(O, want) and torch.equal(lse, want_lse)
    # the newest token's value of request 1 is NaN in one place: its last row sees it, the others do not
    cache.V.view(torch.uint8)[int(table[1, 89 // 16]), 1, 89 % 16, 5] = 0xff
    O, _ = dsa.cache_attention(Q, cache, table, dl, n_q=n_q)
    hit = torch.zeros_like(want, dtype=torch.bool)
    hit[2:, 2 * n_q - 1, 5] = True
    assert torch.isnan(O[hit]).all() and torch.equal(O[~hit], want[~hit])


def test_attention_without_requests(dsa):
    cache, table, dl, Q = attend_inputs(dsa, 4, 2, 64, 16, [], 1)
    O, lse = dsa.cache_attention(Q, cache, table, dl, want_lse=True)
    assert O.shape == (4, 0, 64) and lse.shape == (4, 0) and dsa.device_status() == (0, 0)


def test_attention_reports_bad_pages_lengths_and_scales(dsa):
    from dynamic_sparse_attention_build_b200 import _binding as B
    lens = [100, 60]
    cache, table, dl, Q = attend_inputs(dsa, 4, 2, 64, 16, lens, 1)
    want, _ = dsa.cache_attention(Q, cache, table, dl)
    for bad in (-1, cache.K.shape[0], 2 ** 30):
        t = table.clone()
        t[0, 3] = bad
        O, _ = dsa.cache_attention(Q, cache, t, dl)
        assert dsa.device_status() == (B.DSA_ERR_DEVICE, 39)
        assert torch.equal(O[:, 1], want[:, 1]) and torch.isfinite(O).all()
    for n in (-3, table.shape[1] * 16 + 1, 2 ** 31 - 1):
        O, _ = dsa.cache_attention(Q, cache, table, ints([n, 60]))
        status, detail = dsa.device_status()
        assert status == B.DSA_ERR_DEVICE and detail in (38, 39)
        assert torch.isfinite(O).all()
    cache.v_scale[int(table[0, 2]), 1] = math.nan
    O, _ = dsa.cache_attention(Q, cache, table, dl)
    assert dsa.device_status() == (B.DSA_ERR_DEVICE, 41)
    assert torch.equal(O[:2], want[:2]) and torch.isfinite(O).all()
    assert dsa.device_status() == (0, 0)


def test_offsets_beyond_32_bits(dsa):
    """A cache of more than 2^32 bytes per tensor, its last pages in use."""
    page, Hkv, d = 256, 8, 128
    pages = (1 << 32) // (page * Hkv * d) + 40
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    cache = dsa.PageCache.empty(pages, Hkv, page, d)
    n = 1000
    held = [pages - 1, 0, pages - 17, pages - 3]
    slots = [held[i // page] * page + i % page for i in range(n)]
    g = gen(6)
    K, V = (torch.randn(Hkv, n, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    dsa.cache_write(K, V, ints(slots), cache)
    Q = torch.randn(8, 1, d, generator=g, device="cuda").bfloat16()
    table = ints([held])
    O, lse = dsa.cache_attention(Q, cache, table, ints([n]), want_lse=True)
    assert dsa.device_status() == (0, 0)
    pick = lambda x: x[torch.tensor(held, device="cuda")]  # noqa: E731
    small = dsa.PageCache(pick(cache.K.view(torch.uint8)).view(E4M3), pick(cache.V.view(torch.uint8)).view(E4M3),
                          pick(cache.k_scale), pick(cache.v_scale))
    back = small.K[:, 3].float() * small.k_scale[:, 3, None, None]
    near = back.reshape(-1, d)[:n] - K[3].float()
    # e4m3: half a step is 2^-4 of a normal value, 2^-10 below 2^-6 times the scale
    assert (near.abs() <= 2.0 ** -4 * K[3].float().abs() + 2.0 ** -10 * small.k_scale[:, 3].max()).all()
    check_attend(O, lse, Q, small, ints([[0, 1, 2, 3]]), [n], 1)


def test_attention_gives_the_same_bits_each_time(dsa):
    lens = [3000, 17, 900]
    cache, table, dl, Q = attend_inputs(dsa, 32, 8, 128, 64, lens, 1)
    want, want_lse = dsa.cache_attention(Q, cache, table, dl, want_lse=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [dsa.cache_attention(Q, cache, table, dl, want_lse=True, stream=s) for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    for O, lse in got:
        assert torch.equal(O, want) and torch.equal(lse, want_lse)


def test_waits_that_run_out_leave_the_next_launch_exact(dsa):
    from dynamic_sparse_attention_build_b200 import _binding as B
    lens = [60000, 17, 50000, 70000]
    cache, table, dl, Q = attend_inputs(dsa, 8, 8, 128, 64, lens, 1)
    src, side = torch.zeros(1 << 30, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    dst = torch.empty_like(src)  # copies beside the calls below, so that loads take long
    want, want_lse = dsa.cache_attention(Q, cache, table, dl, want_lse=True)
    assert dsa.device_status() == (0, 0)
    out = 0
    try:
        for limit in (1, 100, 300, 1000) * 5:
            if out > 1:
                break
            assert B.dsa_set_wait_limit(limit) == B.DSA_OK
            with torch.cuda.stream(side):
                for _ in range(4):
                    dst.copy_(src)
            for _ in range(3):
                dsa.cache_attention(Q, cache, table, dl)
            status, _ = dsa.device_status()
            assert status in (B.DSA_OK, B.DSA_ERR_TIMEOUT)
            out += status == B.DSA_ERR_TIMEOUT
            torch.cuda.synchronize()
    finally:
        assert B.dsa_set_wait_limit(0) == B.DSA_OK
    assert out > 0
    O, lse = dsa.cache_attention(Q, cache, table, dl, want_lse=True)
    assert dsa.device_status() == (0, 0)
    assert torch.equal(O, want) and torch.equal(lse, want_lse)


# --------------------------------------------------------------------------- together
def test_serving_steps_together(dsa):
    """Prompts arrive, are prefilled and stored; decode steps follow, captured in one graph; one
    request ends and another takes its pages.  Every step against 64 bits over what the cache holds."""
    Hq, Hkv, d, page, n = 8, 2, 128, 16, 4
    pages, width = 40, 12
    cache = dsa.PageCache.empty(pages, Hkv, page, d)
    lens, free, count = ints([0] * n), ints(list(range(pages))), ints([pages])
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    g = gen(11)
    new = lambda h, t: torch.randn(h, t, d, generator=g, device="cuda").bfloat16()  # noqa: E731
    host = [0] * n

    def admit(prompt):
        T = sum(max(x, 0) for x in prompt) + 6
        got = dsa.build_tables(lens, ints(prompt), free, count, table, page, T)
        lens.copy_(got.lens)
        count.copy_(got.free_count)
        for b, x in enumerate(prompt):
            host[b] = 0 if x < 0 else host[b] + x
        assert lens.tolist() == host
        Q, K, V = new(Hq, T), new(Hkv, T), new(Hkv, T)
        dsa.cache_write(K, V, got.slots, cache)
        O, lse = dsa.packed_prefill(Q, K, V, got.cu_seqlens, want_lse=True)
        cu = got.cu_seqlens.tolist()
        for a, b in zip(cu, cu[1:]):
            for h in range(Hq):
                plain.check_rows(O[h, a:b], lse[h, a:b], Q[h, a:b], K[h // 4, a:b], V[h // 4, a:b],
                                 torch.arange(b - a, device="cuda"), plain.BF16, what="prefill")

    admit([33, 70, 1, 0])
    one = ints([1, 1, 1, 0])
    Q, K, V = new(Hq, n), new(Hkv, n), new(Hkv, n)
    out = dsa.Tables(ints([0] * n), ints([0] * (n + 1)), lens, count)
    O, lse = torch.zeros_like(Q), torch.zeros(Hq, n, device="cuda")

    def step():
        dsa.build_tables(lens, one, free, count, table, page, n, out=out)
        dsa.cache_write(K, V, out.slots, cache)
        dsa.cache_attention(Q, cache, table, lens, O=O, lse=lse)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(40):
        if i == 25:  # request 1 ends, another prompt takes row 3
            admit([0, -1, 0, 50])
            one.copy_(ints([1, 0, 1, 1]))
        # rows of the new tokens follow each other; a request without one keeps its place in Q
        Q.copy_(new(Hq, n))
        K.copy_(new(Hkv, n))
        V.copy_(new(Hkv, n))
        graph.replay()
        for b in range(n):
            host[b] += int(one[b])
        assert lens.tolist() == host
        check_attend(O, lse, Q, cache, table, host, 1)
        last = (host[0] - 1) // page
        assert torch.equal(cache.K[int(table[0, last]), :, (host[0] - 1) % page].float() *
                           cache.k_scale[int(table[0, last])][:, None],
                           plain.e4m3_64(K[:, 0].double() / cache.k_scale[int(table[0, last])].double()[:, None]).float() *
                           cache.k_scale[int(table[0, last])][:, None])
    assert dsa.device_status() == (0, 0)


def test_paged_layer(dsa):
    """Short prompts packed, one long prompt with sparse patterns, decode steps of one and of two
    tokens, a request that ends, and a prompt for which no pages are left."""
    from dynamic_sparse_attention_build_b200 import _binding as B
    Hq, Hkv, d, n = 4, 2, 64, 3
    layer = dsa.PagedLayer(Hq, Hkv, d, n, pages=60, page=16, width=40)
    g = gen(21)
    new = lambda h, t: torch.randn(h, t, d, generator=g, device="cuda").bfloat16()  # noqa: E731
    host = [0] * n

    def check(O, lse, Q, n_q):
        assert layer.lens.tolist() == host and layer.status() == (0, 0)
        check_attend(O, lse, Q, layer.cache, layer.table, host, n_q)

    Q, K, V = new(Hq, 50), new(Hkv, 50), new(Hkv, 50)
    O = layer.prefill(Q, K, V, ints([20, 0, 27]))
    host = [20, 0, 27]
    for a, b in ((0, 20), (20, 47)):
        for h in range(Hq):
            plain.check_rows(O[h, a:b], None, Q[h, a:b], K[h // 2, a:b], V[h // 2, a:b], torch.arange(b - a, device="cuda"),
                             plain.BF16, what="packed")
    Q, K, V = new(Hq, 400), new(Hkv, 400), new(Hkv, 400)
    pats = [dict(kind="ashape", sink=16, window=64)] * Hq
    O = layer.prefill(Q, K, V, ints([0, 400, 0]), patterns=pats)
    host[1] = 400
    want, _ = dsa.sparse_prefill(Q, K, V, dsa.build_indices(Q, K, pats, 64))
    assert torch.equal(O, want)
    for _ in range(3):
        Q = new(Hq, n)
        O, lse = layer.decode(Q, new(Hkv, n), new(Hkv, n), want_lse=True)
        host = [x + 1 for x in host]
        check(O, lse, Q, 1)
    Q = new(Hq, 2 * n)
    O, lse = layer.decode(Q, new(Hkv, 4), new(Hkv, 4), ints([2, -1, 2]), want_lse=True)  # drafted tokens; request 1 ends
    host = [host[0] + 2, 0, host[2] + 2]
    check(O, lse, Q, 2)
    assert host == [25, 0, 32] and layer.free_count.item() == 60 - 2 - 2
    free = layer.free_pages.clone(), layer.table.clone()
    layer.prefill(new(Hq, 1000), new(Hkv, 1000), new(Hkv, 1000), ints([0, 1000, 0]))
    assert layer.status()[0] == B.DSA_ERR_CAPACITY
    assert layer.lens.tolist() == host and torch.equal(free[0], layer.free_pages) and torch.equal(free[1], layer.table)
    with pytest.raises(ValueError, match="rows"):
        layer.decode(new(Hq, 4), new(Hkv, 3), new(Hkv, 3))


@pytest.mark.parametrize("change, match", [
    (dict(Q="float"), "bfloat16"), (dict(Q="d"), "must be 64"), (dict(Q="rows"), "rows"), (dict(Q="heads"), "divide"),
    (dict(table="long"), "int32"), (dict(table="flat"), "block_table"), (dict(table="wide"), "contiguous"),
    (dict(lens="short"), "shape"), (dict(lens="host"), "on cpu"), (dict(n_q=0), "rows"), (dict(n_q=2), "rows"),
    (dict(O="rows"), "dimension 1"), (dict(workspace="small"), "workspace"), (dict(lse="long"), "lse"),
])
def test_attention_refusals(dsa, change, match):
    cache, table, dl, Q = attend_inputs(dsa, 4, 2, 64, 16, [20, 30], 1)
    a = dict(Q=Q, table=table, lens=dl, n_q=1, O=None, lse=None, workspace=None)
    (name, how), = change.items()
    made = {"float": lambda: Q.float(), "d": lambda: torch.cat([Q, Q], 2), "rows": lambda: Q[:, :1], "heads": lambda: Q[:3],
            "flat": lambda: table[0], "wide": lambda: torch.cat([table, table], 1)[:, :table.shape[1]],
            "short": lambda: dl[:1], "host": lambda: dl.cpu(), "small": lambda: torch.empty(64, dtype=torch.uint8, device="cuda")}
    if how == "long":
        a[name] = (table if name == "table" else torch.zeros(4, 2, device="cuda")).long()
    else:
        a[name] = made[how]() if isinstance(how, str) else how
    with pytest.raises(ValueError, match=match):
        dsa.cache_attention(a["Q"], cache, a["table"], a["lens"], n_q=a["n_q"], O=a["O"], lse=a["lse"], workspace=a["workspace"])


def test_cache_refusals(dsa):
    c = filled(dsa, 3, 2, 16, 64)
    for args, match in (((c.K.float(), c.V, c.k_scale, c.v_scale), "float8"),
                        ((c.K, c.V.transpose(1, 2).contiguous().transpose(1, 2), c.k_scale, c.v_scale), "layout"),
                        ((c.K, c.V[:2], c.k_scale, c.v_scale), "shape"), ((c.K, c.V, c.k_scale[:2], c.v_scale), "k_scale"),
                        ((c.K, c.V, c.k_scale, c.v_scale.double()), "v_scale"),
                        ((c.K[:, :, :8], c.V[:, :, :8], c.k_scale, c.v_scale), "tokens"),
                        ((c.K[:, :1].expand(3, 2, 16, 64), c.V[:, :1].expand(3, 2, 16, 64), c.k_scale, c.v_scale), "overlap")):
        with pytest.raises(ValueError, match=match):
            dsa.PageCache(*args)
    K = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    for K2, V2, s, match in ((K[:1], K, ints([0] * 4), "dimension 0"), (K, K[:, :3], ints([0] * 4), "dimension 1"),
                             (K, K, ints([0] * 3), "shape"), (K, K, ints([0] * 4).long(), "int32"), (K.half(), K, ints([0] * 4), "bfloat16")):
        with pytest.raises(ValueError, match=match):
            dsa.cache_write(K2, V2, s, c)


def test_table_refusals(dsa):
    a = dict(lens=ints([1, 2]), new_lens=ints([1, 1]), free_pages=ints([0, 1]), free_count=ints([2]), block_table=ints([[5], [6]]),
             page=16, max_tokens=3)
    for change, match in ((dict(lens=ints([1, 2]).long()), "int32"), (dict(new_lens=ints([1])), "shape"),
                          (dict(free_count=ints([1, 2])), "shape"), (dict(block_table=ints([[1]])), "shape"),
                          (dict(page=20), "page"), (dict(max_tokens=-1), "max_tokens"), (dict(free_pages=ints([])), "free_pages"),
                          (dict(out=dsa.Tables(ints([0] * 2), ints([0] * 3), ints([0] * 2), ints([0]))), "out.slots")):
        with pytest.raises(ValueError, match=match):
            dsa.build_tables(**{**a, **change})


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G, n_q", [(4, 1), (4, 3)])
@pytest.mark.parametrize("power", [10, 18, 20, 22, 24, 25, 26, 27, 28, 29, 30, 40, 60])
def test_scores_far_beyond_the_exponents_range(dsa, d, G, n_q, power):
    """One product a score, so scores are exact: the largest of them (equal ones) share the row whatever their size.
    Weights are 0 or alike, so all that is rounded is O and the scores' scale, the same for equal scores."""
    page, n = 16, 300
    cache = dsa.PageCache.empty(20, 1, page, d)
    at = torch.arange(20 * page, device="cuda")
    cache.K.zero_()
    cache.K[:, 0, :, 0] = (at * 7 % 13 + 1).float().view(20, page).to(E4M3)  # (up to 13: exact)
    cache.V.copy_((torch.randn(20, 1, page, d, generator=gen(4), device="cuda") * 60).to(E4M3))
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    Q = torch.zeros(G, n_q, d, dtype=torch.bfloat16, device="cuda")
    Q[:, :, 0] = 2.0 ** power
    O, lse = dsa.cache_attention(Q, cache, ints([list(range(20))]), ints([n]), n_q=n_q, want_lse=True)
    assert dsa.device_status() == (0, 0)
    k, v = (x.double().view(20 * page, d)[:n] for x in (cache.K, cache.V))
    for h in range(G):
        o, l, a = plain.attention64_far(Q[h].double(), k, v, torch.arange(n - n_q, n, device="cuda"))
        assert torch.isfinite(O).all()
        assert ((O[h].double() - o).abs() <= plain.BF16 * o.abs() + 1.01 * a * (plain.FP16 + 2.0 ** -20)).all()
        assert ((lse[h].double() - l).abs() <= 4 * plain.FP32 * l.abs() + 2.0 ** -20).all()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("room", [1, 3])
def test_tables_of_prompts_refuse_requests_that_hold_tokens(dsa, in_place, room):
    """prompts: a request that gets tokens must hold none; "single": one request gets all of them.  Nothing changes
    otherwise, and the status says so."""
    from dynamic_sparse_attention_build_b200 import _binding as B
    lens, free, table, page = [20, 0, 5], [3, 4, 6] + [-1] * room, [[0, 1, -1], [-1] * 3, [2, -1, -1]], 16

    def run(new, tokens, prompts):
        d = [ints(x) for x in (lens, new, free, [3], table)]
        out = dsa.Tables(ints([5] * tokens), ints([5] * 4), d[0], d[3]) if in_place else None
        got = dsa.build_tables(d[0], d[1], d[2], d[3], d[4], page, tokens, out=out, prompts=prompts)
        return (got.slots.tolist(), got.cu_seqlens.tolist(), got.lens.tolist(), got.free_count.item(), d[4].tolist(), d[2].tolist())

    for new, tokens, prompts, good in (
            ([0, 17, 0], 17, "packed", True), ([-1, 17, 0], 20, "packed", True), ([0, 0, 0], 3, "packed", True),
            ([1, 0, 0], 5, "packed", False), ([0, 4, 1], 5, "packed", False), ([0, 17, 0], 17, "single", True),
            ([-1, 17, -1], 17, "single", True), ([0, 16, 0], 17, "single", False), ([0, 0, 0], 4, "single", False),
            ([3, 0, 0], 3, "single", False), ([1, 0, 0], 5, None, True)):
        want = plain.tables_plain(lens, new, free, 3, table, page, tokens)
        status = (0, 0) if want[-1] else (B.DSA_ERR_CAPACITY, 23)  # (no room for the pages of those that end)
        assert want[-1] or room == 1
        if not good:
            want, status = ([-1] * tokens, [0] * 4, lens, 3, table, free, False), (B.DSA_ERR_DEVICE, 42)
        assert run(new, tokens, prompts) == tuple(want[:-1]), (new, tokens, prompts)
        assert dsa.device_status() == status, (new, tokens, prompts)


def test_paged_layer_refuses_a_prompt_behind_tokens(dsa):
    """prefill attends over the new rows alone, so a request that holds tokens already is reported, and neither its
    tokens nor the others' are stored; with patterns all rows are one request's."""
    from dynamic_sparse_attention_build_b200 import _binding as B
    layer = dsa.PagedLayer(4, 2, 64, 3, pages=60, page=16, width=40)
    g = gen(22)
    new = lambda h, t: torch.randn(h, t, 64, generator=g, device="cuda").bfloat16()  # noqa: E731
    layer.prefill(new(4, 50), new(2, 50), new(2, 50), ints([20, 0, 30]))
    assert layer.status() == (0, 0)
    pats = [dict(kind="ashape", sink=16, window=64)] * 4
    for lens, p in (([0, 9, 1], None), ([0, 10, 9], pats), ([10, 0, 0], pats), ([0, 9, 0], pats)):
        layer.prefill(new(4, 10), new(2, 10), new(2, 10), ints(lens), patterns=p)
        assert layer.status() == (B.DSA_ERR_DEVICE, 42)
        assert layer.lens.tolist() == [20, 0, 30] and layer.free_count.item() == 60 - 4
    layer.prefill(new(4, 10), new(2, 10), new(2, 10), ints([0, 10, 0]), patterns=pats)
    assert layer.status() == (0, 0) and layer.lens.tolist() == [20, 10, 30]
    layer.prefill(new(4, 8), new(2, 8), new(2, 8), ints([-1, 0, -1]))
    layer.prefill(new(4, 8), new(2, 8), new(2, 8), ints([3, 0, 5]))
    assert layer.status() == (0, 0) and layer.lens.tolist() == [3, 10, 5]


@pytest.mark.parametrize("call", ["prefill", "sparse", "decode"])
@pytest.mark.parametrize("name, how, match", [
    ("Q", "float", "bfloat16"), ("Q", "heads", "dimension 0"), ("Q", "d", "dimension 2"), ("K", "float", "bfloat16"),
    ("K", "heads", "dimension 0"), ("V", "rows", "dimension 1"), ("V", "host", "CUDA"), ("Q", "shifted", "16 bytes"),
    ("K", "shifted", "16 bytes"), ("V", "odd", "multiple of 8"), ("new_lens", "long", "int32"), ("new_lens", "short", "shape"),
    ("Q", "none", " has "), ("patterns", "kind", None),
])
def test_paged_layer_refuses_before_it_changes_anything(dsa, call, name, how, match):
    layer = dsa.PagedLayer(4, 2, 64, 3, pages=60, page=16, width=40)
    g = gen(23)
    new = lambda h, t: torch.randn(h, t, 64, generator=g, device="cuda").bfloat16()  # noqa: E731
    layer.prefill(new(4, 50), new(2, 50), new(2, 50), ints([20, 0, 30]))
    rows = 3 if call == "decode" else 40
    a = dict(Q=new(4, rows), K=new(2, rows), V=new(2, rows), new_lens=ints([1, 1, 1] if call == "decode" else [0, rows, 0]))
    if call == "sparse":
        a["patterns"] = [dict(kind="ashape", sink=16, window=64)] * 4
    if name == "patterns":
        if call != "sparse":
            pytest.skip("patterns are the sparse prefill's")
        a["patterns"] = [dict(kind="ashape", sink=-1, window=64)] * 4
    else:
        t = a[name]
        wide = torch.zeros(*t.shape[:-1], 72, dtype=torch.bfloat16, device="cuda") if name != "new_lens" else None
        a[name] = {"float": lambda: t.float(), "heads": lambda: t[:1], "d": lambda: torch.cat([t, t], 2), "rows": lambda: t[:, :2],
                   "host": lambda: t.cpu(), "shifted": lambda: wide[:, :, 1:65], "odd": lambda: torch.zeros(2, rows, 68, dtype=torch.bfloat16, device="cuda")[:, :, :64],
                   "long": lambda: t.long(), "short": lambda: t[:2], "none": lambda: t[:, :0]}[how]()
    held = [x.clone() for x in (layer.lens, layer.table, layer.free_pages, layer.free_count, layer.cache.K.view(torch.uint8),
                                layer.cache.V.view(torch.uint8), layer.cache.k_scale, layer.cache.v_scale)]
    with pytest.raises(Exception) as e:
        (layer.decode if call == "decode" else layer.prefill)(**a)
    if match:
        assert e.type is ValueError and match in str(e.value)
    assert layer.status() == (0, 0)
    for x, y in zip(held, (layer.lens, layer.table, layer.free_pages, layer.free_count, layer.cache.K.view(torch.uint8),
                           layer.cache.V.view(torch.uint8), layer.cache.k_scale, layer.cache.v_scale)):
        assert torch.equal(x, y)


def test_paged_layer_refuses_sizes(dsa):
    for change, match in ((dict(Hq=3), "divide"), (dict(requests=0), "requests"), (dict(requests=4097), "requests"),
                          (dict(Hq=8192, Hkv=8192), "heads"), (dict(width=1 << 27), "width")):
        a = dict(Hq=4, Hkv=2, d=64, requests=3, pages=4, page=16)
        with pytest.raises(ValueError, match=match):
            dsa.PagedLayer(**{**a, **change})


@pytest.mark.parametrize("n", [3, 700])
@pytest.mark.parametrize("tokens", [0, 40, 9000])
def test_tables_whose_lengths_overlap_in_part(dsa, n, tokens):
    """lens_out one place behind lens in the same memory: refused as a whole, the lengths still come out right."""
    from dynamic_sparse_attention_build_b200 import _binding as B
    lens = [(i * 7) % 50 for i in range(n)]
    buf = ints(lens + [0])
    out = dsa.Tables(ints([5] * tokens), ints([5] * (n + 1)), buf[1:], ints([5]))
    table = torch.full((n, 4), 1, dtype=torch.int32, device="cuda")
    dsa.build_tables(buf[:n], ints([1000] * n), ints([0] * 9), ints([2]), table, 16, tokens, out=out)
    assert dsa.device_status() == (B.DSA_ERR_CAPACITY, 25)
    assert out.lens.tolist() == lens and out.free_count.item() == 2 and (out.slots == -1).all() and (out.cu_seqlens == 0).all()


@pytest.mark.parametrize("Hq, Hkv, d, n, n_q", [(4, 2, 128, 1500, 1), (8, 8, 64, 4096, 1), (16, 2, 128, 4096, 2), (4, 1, 64, 2000, 3)])
def test_attention_of_many_requests(dsa, Hq, Hkv, d, n, n_q):
    """More requests than keep the planned CTAs on an SM (their lengths lie in shared memory), a third without keys."""
    rng = random.Random(n)
    lens = [rng.choice([0, rng.randint(0, 5), rng.randint(0, 200)]) for _ in range(n)]
    cache, table, dl, Q = attend_inputs(dsa, Hq, Hkv, d, 16, lens, n_q)
    O, lse = dsa.cache_attention(Q, cache, table, dl, n_q=n_q, want_lse=True)
    assert dsa.device_status() == (0, 0)
    # all at once: what check_attend takes request by request, at 200 keys each
    page, G, W = 16, Hq // Hkv, 200
    at = torch.arange(W, device="cuda")
    pages = table.clamp(min=0).long().gather(1, (at // page).clamp(max=table.shape[1] - 1).expand(n, W))
    live = at[None] < dl[:, None]
    worst = 0.0
    for h in range(Hkv):
        k, v = (torch.where(live[..., None], x[pages, h, at % page].double() * s[pages, h].double()[..., None], 0.0)
                for x, s in ((cache.K, cache.k_scale), (cache.V, cache.v_scale)))
        vs = cache.v_scale[pages, h].double()
        for q in range(h * G, (h + 1) * G):
            x = Q[q].view(n, n_q, d).double()
            s = x @ k.mT / math.sqrt(d)
            s = s.masked_fill(at > (dl[:, None] - n_q + torch.arange(n_q, device="cuda"))[..., None], -math.inf)
            l = torch.logsumexp(s, -1)
            empty = l == -math.inf
            w = torch.where(s == -math.inf, 0.0, torch.exp(s - l.masked_fill(empty, 0.0)[..., None]))
            o, a = w @ v, w @ v.abs()
            e = (d + 8) * plain.FP32 * (x.abs() @ k.abs().amax(1)[..., None])[..., 0] / math.sqrt(d) + 2.0 ** -19
            tol = plain.BF16 * o.abs() + 1.01 * a * (plain.FP16 + 4.2 * e[..., None] + 2.0 ** -20) + 2.0 ** -126 \
                + W * 448.0 * 2.0 ** -35 * (w * vs[:, None]).amax(-1, keepdim=True)
            got, got_l = O[q].view(n, n_q, d).double(), lse[q].view(n, n_q).double()
            assert ((got - o).abs() <= tol).all() and torch.equal(got_l == -math.inf, empty)
            err = (got_l - l).masked_fill(empty, 0.0).abs()
            assert (err <= e + 4 * plain.FP32 * l.masked_fill(empty, 0.0).abs() + 2.0 ** -20).all()
            worst = max(worst, float(err.max()))
    assert (O.view(Hq, n, n_q, d)[:, (dl == 0)] == 0).all()


@pytest.mark.parametrize("Hq, Hkv, d, lens, n_q", [(16, 2, 128, [100, 0, 299, 300, 301], 300), (1, 1, 64, [700, 3], 600),
                                                   (4, 2, 64, [5, 1000], 129)])
def test_attention_of_more_tokens_than_keys(dsa, Hq, Hkv, d, lens, n_q):
    cache, table, dl, Q = attend_inputs(dsa, Hq, Hkv, d, 32, lens, n_q)
    O, lse = dsa.cache_attention(Q, cache, table, dl, n_q=n_q, want_lse=True)
    assert dsa.device_status() == (0, 0)
    check_attend(O, lse, Q, cache, table, lens, n_q)

"""Plain 64-bit forms of the serving calls, and the errors that their kernels may make.

Rounding to nearest is off by at most half a step: 2^-8 of the value for bf16, 2^-11 for fp16,
2^-24 for fp32."""
import math

import torch

BF16, FP16, FP32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24


def score_error(q, k):
    """How far q.k / sqrt(d), summed in fp32 over exact products, and the exponent made of it may
    be off: d additions and a few more operations, each 2^-24 of at most |q||k| / sqrt(d), and
    three roundings of exponents below 16 in size (2^-21 each)."""
    d = q.shape[-1]
    if k.shape[0] == 0:
        return torch.zeros(q.shape[0], dtype=torch.float64, device=q.device)
    return (d + 8) * FP32 * (q.abs() @ k.abs().amax(0)) / math.sqrt(d) + 2.0 ** -19


def attention64(q, k, v, last):
    """Rows of q over the keys j <= last[i]: (o, lse, sums of weight x |value|, score errors, weights)."""
    n = k.shape[0]
    if n == 0:
        z = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device=q.device)
        return z, torch.full_like(z[:, 0], -math.inf), z, z[:, 0], torch.zeros(q.shape[0], 0, device=q.device)
    s = q @ k.mT / math.sqrt(q.shape[-1])
    s = s.masked_fill(torch.arange(n, device=q.device)[None] > last[:, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.where(s == -math.inf, 0.0, torch.exp(s - lse.masked_fill(lse == -math.inf, 0.0)[:, None]))
    return w @ v, lse, w @ v.abs(), score_error(q, k), w


def check_rows(O, lse, q, k, v, last, p_round, extra=None, what="", slack=0.0):
    """O and lse rows of the kernel against 64 bits.  O is off by the rounding of the output, of
    each weight (p_round of it) and by the weights' own error: e^(2 x) - 1 <= 2.1 x for a score off
    by x, in the numerator and in the sum."""
    q, k, v = q.double(), k.double(), v.double()
    o, l, a, e, w = attention64(q, k, v, last)
    e = e + slack
    tol = BF16 * o.abs() + 1.01 * a * (p_round + 4.2 * e[:, None] + 2.0 ** -20) + 2.0 ** -126
    if extra is not None:
        tol = tol + extra(w)
    err = (O.double() - o).abs()
    assert torch.isfinite(O).all(), what
    assert (err <= tol).all(), f"{what}: {float((err - tol).max())} over the tolerance, error {float(err.max())}"
    if lse is not None:
        got = lse.double()
        empty = l == -math.inf
        assert torch.equal(got == -math.inf, empty), what
        err = (got - l).masked_fill(empty, 0.0).abs()
        assert (err <= e + 4 * FP32 * l.masked_fill(empty, 0.0).abs() + 2.0 ** -20).all(), f"{what}: lse {float(err.max())}"


def attention64_far(q, k, v, last):
    """(o, lse, sums of weight x |value|) like attention64, for scores of any size: differences to the row's largest are
    taken before anything is added to them (2^60 + log 3 is 2^60 in 64 bits)."""
    s = q @ k.mT / math.sqrt(q.shape[-1])
    s = s.masked_fill(torch.arange(k.shape[0], device=q.device)[None] > last[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    w = torch.exp(s - m)
    total = w.sum(-1, keepdim=True)
    w = w / total
    return w @ v, (m + total.log())[:, 0], w @ v.abs()


# ---- page tables, one request after the other ----------------------------------------------
def tables_plain(lens, new, free, count, table, page, max_tokens):
    """The rules of dsa_build_tables, on lists: (slots, cu, lens, count, table, free, ok)."""
    lens, new, free = list(lens), list(new), list(free)
    table = [list(r) for r in table]
    before = [r[:] for r in table], free[:], count
    up = lambda x: -(-x // page)  # noqa: E731

    def refuse():
        return [-1] * max_tokens, [0] * (len(lens) + 1), lens, before[2], before[0], before[1], False

    width = len(table[0])
    if any(x < 0 or up(x) > width for x in lens):
        return refuse()
    for b, n in enumerate(new):
        if n < 0:
            for j in range(up(lens[b])):
                if count >= len(free):
                    return refuse()
                free[count] = table[b][j]
                count += 1
    cu, slots, out = [0], [], []
    for b, n in enumerate(new):
        old = 0 if n < 0 else lens[b]
        n = max(n, 0)
        if up(old + n) > width:
            return refuse()
        for j in range(up(old), up(old + n)):
            if count == 0:
                return refuse()
            count -= 1
            table[b][j] = free[count]
        slots += [table[b][i // page] * page + i % page for i in range(old, old + n)]
        cu.append(len(slots))
        out.append(old + n)
    if len(slots) > max_tokens:
        return refuse()
    return slots + [-1] * (max_tokens - len(slots)), cu, out, count, table, free, True


# ---- the 8-bit store -----------------------------------------------------------------------
def e4m3_64(x):
    """x rounded to the nearest e4m3 value, ties to even, larger ones to 448."""
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** -6))
    step = torch.ldexp(torch.ones_like(x), e - 4)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def power_for(amax):
    """The smallest power of two s in 2^-60 .. 2^60 with amax <= 448 s."""
    s = 2.0 ** -60
    while amax > 448.0 * s and s < 2.0 ** 60:
        s *= 2.0
    return s


def write_plain(X, slots, data, scale):
    """X [H, T, d] stored at its slots, page by page, on CPU in 64 bits; data and scale are updated."""
    page = data.shape[2]
    runs = {}
    for t, s in enumerate(slots):
        if s >= 0:
            runs.setdefault(s // page, []).append((s % page, t))
    for pg, got in runs.items():
        first = got[0][0]
        for h in range(X.shape[0]):
            x = X[h, [t for _, t in got]].double()
            fin = x[torch.isfinite(x)].abs()
            s = power_for(float(fin.max()) if fin.numel() else 0.0)
            if first > 0:
                was = float(scale[pg, h])
                s = max(s, 2.0 ** math.ceil(math.log2(was)))
                if s != was:
                    data[pg, h, :first] = e4m3_64(data[pg, h, :first] * (was / s))
            scale[pg, h] = s
            y = torch.where(torch.isnan(x), x, e4m3_64((x / s).clamp(-1e30, 1e30)))
            data[pg, h, first:first + len(got)] = y

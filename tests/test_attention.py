"""The cache and attention calls against plain 64-bit implementations.

Tolerances are bounds, computed from each case's own numbers:
  - rounding to a type t is off by at most finfo(t).eps / 2 of the value (plus half the smallest step near zero);
  - a dot product of d fp32 products is off by at most d 2^-24 sum |a b| (each product and sum rounded once);
  - a weight exp2(x) with x off by e is off by ln(2) e of itself, and the hardware's exp2 by 2^-22;
  - a weight that enters a product as two bf16 terms is off by 2^-17 of itself at most, as one 16-bit term by eps / 2;
  - the weighted mean of v is then off by at most (twice the weights' relative error + n 2^-24) sum p |v|: once in
    the sum of products, once in the sum of weights; sums of n fp32 terms add n 2^-24.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import synth
import ternary_weight_ptq1_amd as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16, I8 = torch.float32, torch.float16, torch.bfloat16, torch.int8
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=F32)


def half_step(y, t):
    """The largest rounding error of values y (fp64) in type t."""
    info = torch.finfo(t)
    return y.abs() * (info.eps / 2) + info.smallest_normal * info.eps / 2


# --------------------------------------------------------------- the cache ----

def rope_table(n, rot):
    half = rot // 2
    a = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * 10000.0 ** (
        -torch.arange(half, dtype=torch.float64, device=DEV) / half)
    return torch.cat([a.cos(), a.sin()], 1).float()


def turned(x, pos, table):
    """(rotated rows in fp64, a bound on the fp32 rotation's error)."""
    x = x.double()
    if table is None:
        return x, torch.zeros_like(x)
    half = table.shape[1] // 2
    row = table[pos.long()].double()[:, None]
    c, s = row[..., :half], row[..., half:]
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    y = torch.cat([a * c - b * s, b * c + a * s, rest], -1)
    e = torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs(), 0 * rest], -1) * (2 * U)
    return y, e


def cache_values(c):
    """K and V [pages, heads, slots, d] in fp64 of a cache (NaN steps included)."""
    k, v = c.k_pages.double(), c.v_pages.double().transpose(-1, -2)
    if c.k_steps is not None:
        k, v = k * c.k_steps.double()[..., None], v * c.v_steps.double()[..., None]
    return k, v


def check_rows(got, want, slack, t, amax=None):
    """got against want (fp64) with `slack` of fp32 error and one rounding to t (int8: half a step of the row)."""
    if t == I8:
        top = want.abs().amax(-1, keepdim=True)
        tol = (top / 127) * 0.5 * (1 + 2.0 ** -15) + slack.amax(-1, keepdim=True) * 2
    else:
        tol = half_step(want.abs() + slack, t) + slack
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"worst error over its bound: {(err / tol.clamp_min(1e-300)).max().item():.3f}"


@pytest.mark.parametrize("src", [F32, F16, BF16])
@pytest.mark.parametrize("ctype", [F16, BF16, I8])
@pytest.mark.parametrize("n,hq,hkv,d,page,rot", [
    (1, 5, 1, 64, 16, 64),
    (3, 0, 2, 128, 32, 32),
    (33, 6, 3, 64, 64, 8),
    (70, 8, 2, 256, 16, 64),
    (129, 4, 4, 128, 256, 128),
    (40, 3, 1, 128, 128, 0),
])
def test_kv_write(src, ctype, n, hq, hkv, d, page, rot):
    g = gen(n + d + rot)
    pages = -(-2 * n // page) + 2
    qt = {F16: F16, BF16: BF16, I8: F32}[ctype]
    x = randn(g, n, hq + 2 * hkv + 1, d).to(src)  # one head more: the rows lie apart
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:n]
    slots[n // 2] = -1
    if n > 8:  # a run of neighbours and one past the end
        slots[:8] = pages * page - 8 + torch.arange(8, device=DEV)
        slots[8:] = torch.randperm(pages * page - 8, generator=g, device=DEV)[:n - 8]
        slots[9], slots[10] = -5, pages * page
    pos = torch.randint(0, 50, (n,), generator=g, device=DEV, dtype=torch.int32)
    table = rope_table(50, rot) if rot else None
    c = P.ptq1_kv_cache(pages, page, hkv, d, ctype, DEV)
    for t in (c.k_pages, c.v_pages):
        t.fill_(3)
    if ctype == I8:
        c.k_steps.fill_(0.5), c.v_steps.fill_(0.5)
    out = P.ptq1_kv_write(q if hq else None, k, v, slots, c, positions=pos, cos_sin=table, q_dtype=qt if hq else None)
    torch.cuda.synchronize()
    if hq:
        y, e = turned(q, pos, table)
        assert out.dtype == qt and out.shape == (n, hq, d)
        check_rows(out, y, e, qt)
    else:
        assert out is None
    kc, vc = cache_values(c)
    ok = (slots >= 0) & (slots < pages * page)
    at, off = slots[ok] // page, slots[ok] % page
    y, e = turned(k, pos, table)
    check_rows(kc[at, :, off], y[ok], e[ok], ctype)
    check_rows(vc[at, :, off], v[ok].double(), torch.zeros_like(y[ok]), ctype)
    kept = torch.ones(pages * page, dtype=torch.bool, device=DEV)
    kept[slots[ok]] = False
    other = 1.5 if ctype == I8 else 3.0
    for t in (kc, vc):  # everything else as it was
        assert bool((t.transpose(1, 2).reshape(pages * page, hkv, d)[kept] == other).all())


def test_kv_write_awkward_rows():
    """Zeros, tiny rows, a NaN, an infinity and a position outside the table."""
    d, page = 128, 16
    for ctype in (I8, BF16):
        c = P.ptq1_kv_cache(2, page, 1, d, ctype, DEV)
        k = torch.ones((6, 1, d), device=DEV)
        k[0] = 0.0
        k[1] = 2.0 ** -120
        k[2, 0, 5] = float("nan")
        k[3, 0, 7] = float("inf")
        k[4] = 3e38
        pos = torch.zeros(6, dtype=torch.int32, device=DEV)
        pos[5] = 9
        table = rope_table(9, 64)
        slots = torch.arange(6, device=DEV)
        q = P.ptq1_kv_write(k, k, k, slots, c, positions=pos, cos_sin=table)
        kc, vc = cache_values(c)
        kc, vc = kc[0, 0], vc[0, 0]
        assert bool((kc[0] == 0).all()) and bool((vc[0] == 0).all())
        assert bool((vc[1] == (0.0 if ctype == I8 else 2.0 ** -120)).all())
        if ctype == I8:
            assert bool(vc[2].isnan().all()) and bool(vc[3].isnan().all())
            assert bool(kc[5].isnan().all())
        else:
            assert bool(vc[2, 5].isnan()) and vc[3, 7].item() == float("inf") and int(vc[2:4].isnan().sum()) == 1
            assert bool(kc[5, :64].isnan().all()) and bool((kc[5, 64:] == 1).all())
        assert bool(((vc[4] - 3e38).abs() <= 3e38 * 2.0 ** -8).all())
        # int8: 127 times fl(1 / 127), whose relative error is at most half a step of fp32
        assert bool(((vc[5] - 1).abs() <= (U if ctype == I8 else 0.0)).all())
        assert bool(q[5, 0, :64].isnan().all()) and bool((q[5, 0, 64:] == 1).all())


def filled_cache(g, pages, page, hkv, d, ctype):
    c = P.ptq1_kv_cache(pages, page, hkv, d, ctype, DEV)
    if ctype == I8:
        c.k_pages.copy_(torch.randint(-127, 128, c.k_pages.shape, generator=g, device=DEV))
        c.v_pages.copy_(torch.randint(-127, 128, c.v_pages.shape, generator=g, device=DEV))
        c.k_steps.copy_(0.01 + 0.02 * torch.rand(c.k_steps.shape, generator=g, device=DEV))
        c.v_steps.copy_(0.01 + 0.02 * torch.rand(c.v_steps.shape, generator=g, device=DEV))
    else:
        c.k_pages.copy_(randn(g, *c.k_pages.shape))
        c.v_pages.copy_(randn(g, *c.v_pages.shape))
    return c


def tables(g, lens, page, width=None):
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    t = torch.full((len(lens), max(1, *need) if width is None else width), -7, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t, pages


def poison_unused(c, table, lens):
    """Everything in the pages that no sequence's length covers: NaN (int8: NaN steps)."""
    page = c.page_size
    used = torch.zeros((c.n_pages, page), dtype=torch.bool, device=DEV)
    for i, n in enumerate(lens):
        for j in range(-(-n // page)):
            used[table[i, j].item(), :min(page, n - j * page)] = True
    hid = ~used[:, None, :].expand(-1, c.n_kv_heads, -1)
    if c.k_steps is not None:
        c.k_steps[hid] = float("nan")
        c.v_steps[hid] = float("nan")
    else:
        c.k_pages[hid] = float("nan")
        c.v_pages[hid[:, :, None, :].expand_as(c.v_pages)] = float("inf")


def sequence(c, values, table, b, n):
    """K or V [heads, n, d] of sequence b in fp64."""
    page = c.page_size
    rows = table[b, :-(-n // page)].long()
    return values[rows].transpose(0, 1).reshape(c.n_kv_heads, -1, c.head_dim)[:, :n]


@pytest.mark.parametrize("ctype,out", [(F16, F16), (BF16, BF16), (BF16, F32), (I8, BF16), (I8, F32), (I8, F16)])
@pytest.mark.parametrize("hkv,d,page,lens", [
    (1, 64, 16, [1]),
    (3, 128, 32, [5, 0, 64, 130]),
    (2, 256, 64, [63, 200, 1]),
    (8, 128, 256, [300, 17]),
])
def test_kv_read(ctype, out, hkv, d, page, lens):
    g = gen(sum(lens) + d)
    table, pages = tables(g, lens, page)
    c = filled_cache(g, pages, page, hkv, d, ctype)
    poison_unused(c, table, lens)
    cu = torch.tensor(np.cumsum([2] + lens), dtype=torch.int32, device=DEV)  # two rows ahead of the first sequence
    total = int(cu[-1]) + 3                                                  # and three behind the last
    ko = torch.full((total, hkv, d), 9.0, dtype=out, device=DEV)
    vo = torch.full((total, hkv, d), 9.0, dtype=out, device=DEV)
    P.ptq1_kv_read(c, table, cu, total, dtype=out, out=(ko, vo))
    kc, vc = cache_values(c)
    for got, val in ((ko, kc), (vo, vc)):
        want = torch.full((total, hkv, d), 9.0, dtype=torch.float64, device=DEV)
        for b, n in enumerate(lens):
            want[int(cu[b]):int(cu[b]) + n] = sequence(c, val, table, b, n).transpose(0, 1)
        # step * code is one fp32 product, then one rounding
        tol = half_step(want, out) + want.abs() * (U if ctype == I8 else 0.0)
        tol[got.double() == want] = 0
        assert bool(((got.double() - want).abs() <= tol).all())
        assert bool((got[:2] == 9).all()) and bool((got[int(cu[-1]):] == 9).all())


def test_kv_read_bad_pages_and_short_output():
    g = gen(5)
    c = filled_cache(g, 4, 16, 2, 64, BF16)
    table = torch.tensor([[1, 99], [-1, 2]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 40, 60], dtype=torch.int32, device=DEV)  # 40 tokens: page 99 is bad, tokens 32.. have none
    k, v = P.ptq1_kv_read(c, table, cu, 50, dtype=F32)             # the last ten rows do not fit
    kc, vc = cache_values(c)
    for got, val in ((k, kc), (v, vc)):
        assert bool((got[:16].double() == val[1].transpose(0, 1)).all())
        assert bool(got[16:50].isnan().all())


# ------------------------------------------------------------------ decode ----

def attention_bounds(q, k, v, scale, wterm, mask=None):
    """(rows, bound on the kernels' error before the rounding of the result) of one kv head in fp64: q [n, d],
    k, v [m, d]; wterm: relative error of a weight as it enters the second product; mask [n, m] (True: seen)."""
    d = q.shape[1]
    logits = scale * (q @ k.T.contiguous())
    size = scale * (q.abs() @ k.abs().T.contiguous())
    if mask is not None:
        logits = logits.masked_fill(~mask, -math.inf)
        size = size.masked_fill(~mask, 0.0)
    top = logits.amax(1, keepdim=True)
    w = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(1, keepdim=True)
    p = torch.where(total > 0, w / total, 0.0)
    # scores: d products and sums, then a few more roundings of the score and its maximum
    score = (d + 8) * U * size.amax(1, keepdim=True) + 4 * U * torch.where(top == -math.inf, 0.0, top.abs())
    weight = score + 2.0 ** -22
    n = (p > 0).sum(1, keepdim=True).double()
    return p @ v, (2 * weight + wterm + 2 * n * U) * (p @ v.abs())


WEIGHT_TERM = {(F32, BF16): 2.0 ** -24, (BF16, BF16): 2.0 ** -17, (F32, F16): 2.0 ** -21, (F16, F16): 2.0 ** -21,
               (F32, I8): 2.0 ** -24, (BF16, I8): 2.0 ** -17, (F16, I8): 2.0 ** -17}


def check_decode(q, c, table, lens, got, scale=None):
    hq, d = q.shape[1:]
    group = hq // c.n_kv_heads
    scale = d ** -0.5 if scale is None else scale
    kc, vc = cache_values(c)
    term = WEIGHT_TERM[(q.dtype, c.dtype)]
    for b, n in enumerate(lens):
        if n == 0:
            assert bool((got[b] == 0).all())
            continue
        k, v = sequence(c, kc, table, b, n), sequence(c, vc, table, b, n)
        for h in range(c.n_kv_heads):
            rows = slice(h * group, (h + 1) * group)
            want, tol = attention_bounds(q[b, rows].double(), k[h], v[h], scale, term)
            tol = tol + half_step(want.abs() + tol, q.dtype)
            err = (got[b, rows].double() - want).abs()
            assert bool((err <= tol).all()), f"b={b} h={h}: {(err / tol).max().item():.3f} of the bound"


PAIRS = [(F32, BF16), (BF16, BF16), (F32, F16), (F16, F16), (F32, I8), (BF16, I8), (F16, I8)]


@pytest.mark.parametrize("qt,ctype", PAIRS)
@pytest.mark.parametrize("hq,hkv,d,page,lens", [
    (1, 1, 64, 16, [1]),
    (5, 1, 128, 16, [31, 0, 33, 64, 7]),
    (6, 2, 256, 32, [129, 1, 255]),
    (32, 8, 128, 64, [257, 511, 512, 1030]),
    (20, 1, 64, 256, [300, 0, 2]),      # more than 16 query heads of one kv head
    (33, 1, 128, 128, [700, 128]),
    (7, 7, 128, 16, [100, 2049]),
])
def test_attn_decode(qt, ctype, hq, hkv, d, page, lens):
    g = gen(hq * d + sum(lens))
    table, pages = tables(g, lens, page)
    c = filled_cache(g, pages, page, hkv, d, ctype)
    poison_unused(c, table, lens)
    q = randn(g, len(lens), hq, d).to(qt)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got = P.ptq1_attn_decode(q, c, table, sl)
    assert got.dtype == qt and got.shape == q.shape
    check_decode(q, c, table, lens, got)
    # a bound on the lengths changes the split, not what is computed
    check_decode(q, c, table, lens, P.ptq1_attn_decode(q, c, table, sl, max_len=max(lens)))
    # the same call gives the same bits
    assert torch.equal(got, P.ptq1_attn_decode(q, c, table, sl))


@pytest.mark.parametrize("ctype", [BF16, I8])
def test_attn_decode_long(ctype):
    """Long enough for many chunks, larger scores than the softmax's first ones, and a scale of the caller's."""
    g = gen(11)
    lens = [40000, 3]
    table, pages = tables(g, lens, 64)
    c = filled_cache(g, pages, 64, 2, 128, ctype)
    q = randn(g, 2, 8, 128) * 3
    got = P.ptq1_attn_decode(q, c, table, torch.tensor(lens, dtype=torch.int32, device=DEV), scale=0.3)
    check_decode(q, c, table, lens, got, scale=0.3)


def test_attn_decode_every_weight_is_exact_to_its_terms():
    """fp32 queries over an int8 cache: no single token's weight may be off by a rounding of its first 16-bit term
    (2^-11).  The tolerance of a whole row hides one such token among a thousand; here each token has a dimension
    of its own, 128 at a time, with steps that are no powers of two."""
    g = gen(15)
    n, d = 1024, 128
    table, pages = tables(g, [n], 64)
    c = filled_cache(g, pages, 64, 1, d, I8)
    c.k_pages.copy_((randn(g, *c.k_pages.shape) * 40).clamp(-127, 127).round())
    q = randn(g, 1, 16, d)
    sl = torch.tensor([n], dtype=torch.int32, device=DEV)
    rows = table[0].long()
    k = sequence(c, cache_values(c)[0], table, 0, n)[0]
    steps = c.v_steps[rows, 0].reshape(-1).double()
    logits = q[0].double() @ k.T.contiguous() * d ** -0.5
    size = q[0].double().abs() @ k.T.contiguous().abs() * d ** -0.5
    w = torch.softmax(logits, 1)
    for first in range(0, n, 128):
        v = torch.zeros((n, d), dtype=I8, device=DEV)
        v[torch.arange(first, first + 128, device=DEV), torch.arange(128, device=DEV)] = 127
        c.v_pages[rows, 0] = v.view(-1, 64, d).transpose(1, 2)
        got = P.ptq1_attn_decode(q, c, table, sl)[0].double()
        want = w[:, first:first + 128] * 127 * steps[first:first + 128]
        # score and exp2 as in attention_bounds (d + 8 roundings, twice: weight and sum), the sum of n weights, the
        # product with the step and the last division
        tol = (2 * (d + 8) * U * size.amax(1, keepdim=True) + 8 * U * logits.abs().amax(1, keepdim=True) + 2 * 2.0 ** -22
               + n * U + 8 * U) * want
        assert bool(((got - want).abs() <= tol).all()), ((got - want).abs() / want).max().item()
        assert bool((((got - want).abs() / want) < 2.0 ** -13).all())


def test_attn_decode_large_and_small_queries():
    """fp32 queries outside fp16's range over an fp16 cache, and zeros."""
    g = gen(12)
    lens = [70, 70, 70]
    table, pages = tables(g, lens, 32)
    c = filled_cache(g, pages, 32, 1, 64, F16)
    q = randn(g, 3, 4, 64)
    q[0] *= 1e7
    q[1] *= 1e-9
    q[2] = 0
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for scale in (1e-7, 1e-2):
        check_decode(q[1:], c, table[1:], lens[1:], P.ptq1_attn_decode(q[1:].contiguous(), c, table[1:], sl[1:],
                                                                        scale=scale), scale)
    check_decode(q[:1], c, table[:1], lens[:1], P.ptq1_attn_decode(q[:1].contiguous(), c, table[:1], sl[:1],
                                                                    scale=1e-8), 1e-8)


def test_attn_decode_refused_sequences():
    """Bad lengths and pages make their own sequence NaN and no other."""
    g = gen(13)
    lens = [100, 100, 100, 100, 100]
    table, pages = tables(g, lens, 16, width=20)
    c = filled_cache(g, pages, 16, 2, 64, BF16)
    good = table.clone()
    table[1, 6] = pages      # the last page of its length
    table[2, 0] = -1
    table[3, 7] = -1         # not covered by the length: never read
    sl = torch.tensor([100, 100, 100, 100, -3], dtype=torch.int32, device=DEV)
    q = randn(g, 5, 4, 64).to(BF16)
    for max_len in (100, 320):
        got = P.ptq1_attn_decode(q, c, table, sl, max_len=max_len)
        assert bool(got[[1, 2, 4]].isnan().all())
        check_decode(q[[0, 3]], c, good[[0, 3]], [100, 100], got[[0, 3]])
    got = P.ptq1_attn_decode(q, c, good, torch.tensor([100, 101, 0, 99, 400], dtype=torch.int32, device=DEV), max_len=100)
    assert bool(got[[1, 4]].isnan().all())
    check_decode(q[[0, 2, 3]], c, good[[0, 2, 3]], [100, 0, 99], got[[0, 2, 3]])


def test_attn_decode_non_finite_values():
    """A NaN key makes the rows of its heads NaN; an infinite value reaches only its dimension (as an infinity or, where
    a weight's second 16-bit term is zero or negative, as a NaN: the header promises either)."""
    g = gen(14)
    lens = [50, 50]
    table, pages = tables(g, lens, 16)
    c = filled_cache(g, pages, 16, 2, 64, BF16)
    c.k_pages[table[0, 1].item(), 1, 3, 5] = float("nan")
    c.v_pages[table[1, 2].item(), 0, 9, 4] = float("inf")
    q = randn(g, 2, 4, 64)
    got = P.ptq1_attn_decode(q, c, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    assert bool(got[0, 2:].isnan().all()) and bool(got[0, :2].isfinite().all())
    assert not bool(got[1, :2, 9].isfinite().any()) and int((~got[1].isfinite()).sum()) == 2


# ------------------------------------------------------------------ prompt ----

def check_prompt(q, k, v, lq, lk, got, causal, scale=None, at_q=0, at_k=0):
    hq, d = q.shape[1:]
    hkv = k.shape[1]
    group = hq // hkv
    scale = d ** -0.5 if scale is None else scale
    term = torch.finfo(q.dtype).eps / 2
    for nq, nk in zip(lq, lk):
        mask = None
        if causal:
            mask = torch.arange(nk, device=DEV)[None] <= torch.arange(nq, device=DEV)[:, None] + (nk - nq)
        for h in range(hq):
            qq = q[at_q:at_q + nq, h].double()
            kk, vv = (t[at_k:at_k + nk, h // group].double() for t in (k, v))
            if nk == 0:
                assert bool((got[at_q:at_q + nq, h] == 0).all())
                continue
            want, tol = attention_bounds(qq, kk, vv, scale, term, mask)
            tol = tol + half_step(want.abs() + tol, q.dtype)
            err = (got[at_q:at_q + nq, h].double() - want).abs()
            assert bool((err <= tol).all()), f"head {h} of {nq} x {nk}: {(err / tol).nan_to_num(9e9).max().item():.3f}"
            if causal and nq > nk:
                assert bool((got[at_q:at_q + nq - nk, h] == 0).all())
        at_q += nq
        at_k += nk


def cumulated(lens, first=0):
    return torch.tensor(np.cumsum([first] + list(lens)), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d,lq,lk", [
    (1, 1, 64, [1], [1]),
    (5, 1, 128, [1, 33, 0, 64], [1, 33, 5, 64]),
    (4, 2, 256, [40, 31], [40, 95]),
    (8, 8, 128, [129, 3], [129, 700]),
    (7, 1, 64, [200, 10, 9], [200, 3, 0]),     # queries that see no key
    (32, 8, 128, [65, 127, 66], [65, 256, 1025]),
    (3, 3, 256, [150], [333]),
    (40, 1, 64, [7, 20], [64, 20]),            # a large group
])
def test_attn_prompt(dtype, causal, hq, hkv, d, lq, lk):
    g = gen(hq + d + sum(lq))
    q, k, v = randn(g, sum(lq), hq, d).to(dtype), randn(g, sum(lk), hkv, d).to(dtype), randn(g, sum(lk), hkv, d).to(dtype)
    got = P.ptq1_attn_prompt(q, k, v, cumulated(lq), cumulated(lk), max_q=max(lq), max_k=max(lk), causal=causal)
    assert got.dtype == dtype and got.shape == q.shape
    check_prompt(q, k, v, lq, lk, got, causal)
    # without the bounds, and the same bits again
    assert torch.equal(got, P.ptq1_attn_prompt(q, k, v, cumulated(lq), cumulated(lk), max_q=max(lq), max_k=max(lk),
                                               causal=causal))
    check_prompt(q, k, v, lq, lk, P.ptq1_attn_prompt(q, k, v, cumulated(lq), cumulated(lk), causal=causal), causal)


def test_attn_prompt_stacked_rows_and_gaps():
    """q, k and v as parts of one stacked projection; rows ahead of the first sequence and behind the last stay."""
    g = gen(21)
    lens = [70, 45]
    x = randn(g, 120, 4 + 2 * 2, 128).to(BF16)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    out = torch.full((120, 4, 128), 7.0, dtype=BF16, device=DEV)
    cu = cumulated(lens, 3)
    P.ptq1_attn_prompt(q, k, v, cu, cu, max_q=70, max_k=70, out=out)
    check_prompt(q, k, v, lens, lens, out, True, at_q=3, at_k=3)
    assert bool((out[:3] == 7).all()) and bool((out[118:] == 7).all())


def test_attn_prompt_bounds_and_ranges():
    """A sequence past its bound, or with rows out of range, gets NaN rows; the others are right."""
    g = gen(22)
    lens = [30, 200, 17]
    q, k, v = (randn(g, 247, 2, 64).to(F16) for _ in range(3))
    cu = cumulated(lens)
    got = P.ptq1_attn_prompt(q, k, v, cu, cu, max_q=100, max_k=247)
    assert bool(got[30:230].isnan().all())
    check_prompt(q, k, v, [30], [30], got[:30], True)
    check_prompt(q[230:], k[230:], v[230:], [17], [17], got[230:], True)
    for bound in (dict(max_q=0), dict(max_k=0)):  # exceeded by all
        assert bool(P.ptq1_attn_prompt(q, k, v, cu, cu, **bound).isnan().all())
    far = cumulated([30, 200, 18])  # the last one's keys end behind the last row
    got = P.ptq1_attn_prompt(q, k, v, cu, far, max_q=247, max_k=247)
    assert bool(got[230:].isnan().all()) and bool(got[:230].isfinite().all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attn_prompt_large_scores(d):
    """Scores whose maximum grows along the keys by more than fp16 or bf16 weights span."""
    g = gen(23)
    n = 300
    q, k, v = (randn(g, n, 1, d).to(BF16) for _ in range(3))
    k = (k.float() * torch.linspace(0.1, 8, n, device=DEV)[:, None, None]).to(BF16)
    for scale in (d ** -0.5, 1.0):
        got = P.ptq1_attn_prompt(q, k, v, cumulated([n]), cumulated([n]), scale=scale)
        check_prompt(q, k, v, [n], [n], got, True, scale)


# ---------------------------------------------------------------- together ----

def folded(seed, n, k):
    t = synth.trits(seed, synth.S_GATE_TRITS, n, k)
    s = synth.scales(seed, synth.S_GATE_SCALES, n, k // 128)
    blocks = oracle.pack(t, s)
    return P.ptq1_tile(torch.from_numpy(blocks).to(DEV), n, k), \
        torch.from_numpy(oracle.dequant(blocks, n, k).astype(np.float64)).to(DEV)


def test_layer_half_prompt_then_token():
    """A layer's attention half as a program runs it: stacked q, k, v projection of a prompt (ptq1_gemm), rotary
    positions and the cache write, the sequence read back, prompt attention, output projection; then one more token
    through the decode calls over the same cache.  Each stage against fp64 from that stage's own inputs."""
    dm, hq, hkv, d, n, page = 1024, 8, 2, 128, 77, 32
    wqkv, dense_qkv = folded(1, (hq + 2 * hkv) * d, dm)
    wo, dense_o = folded(2, dm, hq * d)
    signs = torch.from_numpy(synth.signs(3)).to(DEV)
    x = torch.from_numpy(synth.activations(4, n + 1, dm)).to(DEV)
    rope = rope_table(200, d)
    c = P.ptq1_kv_cache(5, page, hkv, d, BF16, DEV)
    table = torch.tensor([[3, 0, 4]], dtype=torch.int32, device=DEV)
    place = torch.arange(n + 1, device=DEV)
    slots = table[0, place // page].long() * page + place % page
    pos = place.to(torch.int32)
    # prompt
    qkv = P.ptq1_gemm(wqkv, (hq + 2 * hkv) * d, dm, x[:n].contiguous(), signs).view(n, hq + 2 * hkv, d)
    rot = P.hadamard_rotate(x, signs).double()
    want = rot[:n] @ dense_qkv.T.contiguous()
    assert (qkv.double().view(n, -1) - want).norm() <= 3e-3 * want.norm()
    q = P.ptq1_kv_write(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], slots[:n], c, positions=pos[:n],
                        cos_sin=rope, q_dtype=BF16)
    y, e = turned(qkv[:, :hq], pos[:n], rope)
    check_rows(q, y, e, BF16)
    cu = cumulated([n])
    k, v = P.ptq1_kv_read(c, table, cu, n, dtype=BF16)
    y, e = turned(qkv[:, hq:hq + hkv], pos[:n], rope)
    check_rows(k, y, e, BF16)
    assert torch.equal(v, qkv[:, hq + hkv:].to(BF16))
    o = P.ptq1_attn_prompt(q, k, v, cu, cu)
    check_prompt(q, k, v, [n], [n], o, True)
    P.ptq1_gemm(wo, dm, hq * d, o.float().view(n, hq * d), signs)
    # one more token
    qkv1 = P.ptq1_matvec(wqkv, (hq + 2 * hkv) * d, dm, x[n].contiguous(), signs).view(1, hq + 2 * hkv, d)
    q1 = P.ptq1_kv_write(qkv1[:, :hq], qkv1[:, hq:hq + hkv], qkv1[:, hq + hkv:], slots[n:], c, positions=pos[n:],
                         cos_sin=rope)
    assert q1.dtype == F32
    o1 = P.ptq1_attn_decode(q1, c, table, torch.tensor([n + 1], dtype=torch.int32, device=DEV))
    check_decode(q1, c, table, [n + 1], o1)
    out = P.ptq1_matvec(wo, dm, hq * d, o1.view(-1), signs, residual=x[n].contiguous())
    want = x[n].double() + dense_o @ P.hadamard_rotate(o1.view(1, -1), signs).double()[0]
    assert (out.double() - want).norm() <= 1e-5 * want.norm()
    # the decode call on the prompt's last position agrees with the prompt call (16-bit weights there)
    last = P.ptq1_attn_decode(q[-1:].contiguous(), c, table, torch.tensor([n], dtype=torch.int32, device=DEV))
    # both are within their own bounds of the same exact rows
    check_decode(q[-1:], c, table, [n], last)


def decode_state(seed, lens, ctype=BF16, qt=F32):
    g = gen(seed)
    table, pages = tables(g, lens, 32)
    c = filled_cache(g, pages, 32, 2, 128, ctype)
    return randn(g, len(lens), 8, 128).to(qt), c, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


def test_captured_step_replays_with_new_contents():
    """The token step (write, attend) captured once and replayed with the lengths, slots and rows that the program
    puts into the same buffers, its own eager work in between."""
    lens = [300, 700]
    q, c, table, sl = decode_state(31, [n + 8 for n in lens], BF16)
    sl.copy_(torch.tensor(lens, dtype=torch.int32))
    g = gen(32)
    rows = randn(g, 2, 12, 128)
    rope = rope_table(1000, 128)
    slots = torch.zeros(2, dtype=torch.int64, device=DEV)
    ws = torch.empty(P.workspace_bytes("attn_decode", 2, 8, 2, 128, 736), dtype=torch.uint8, device=DEV)
    q_out, out = torch.empty(2, 8, 128, device=DEV), torch.empty(2, 8, 128, device=DEV)

    def step():
        P.ptq1_kv_write(rows[:, :8], rows[:, 8:10], rows[:, 10:], slots, c, positions=sl, cos_sin=rope, out=q_out)
        P.ptq1_attn_decode(q_out, c, table, sl, max_len=736, out=out, ws=ws)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(4):
        rows.copy_(randn(g, 2, 12, 128))
        sl.add_(1)
        place = (sl - 1).long()
        slots.copy_(table[torch.arange(2, device=DEV), place // 32].long() * 32 + place % 32)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        assert torch.equal(got, out)
        check_decode(q_out, c, table, [n + i + 1 for n in lens], out)


def test_other_stream():
    """Calls on a stream of the caller's, with workspaces and results of their own allocated meanwhile."""
    q, c, table, sl = decode_state(33, [2000, 900], I8)
    want = P.ptq1_attn_decode(q, c, table, sl)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = P.ptq1_attn_decode(q, c, table, sl, stream=side)
        torch.empty(1 << 20, device=DEV).fill_(float("nan"))  # the allocator may hand out a freed workspace
        side.synchronize()
        assert torch.equal(got, want)


def test_two_streams_with_a_workspace_each():
    states = [decode_state(40 + i, [1500 + 100 * i, 64]) for i in range(2)]
    want = [P.ptq1_attn_decode(q, c, t, sl) for q, c, t, sl in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [[], []]
    for _ in range(6):
        for i, (q, c, t, sl) in enumerate(states):
            with torch.cuda.stream(streams[i]):
                got[i].append(P.ptq1_attn_decode(q, c, t, sl))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


# -------------------------------------------------- masks, splits, many sequences ----

def prompt_state(g, lq, lk, hq, hkv, d, dtype=BF16):
    return (randn(g, sum(lq), hq, d).to(dtype), randn(g, sum(lk), hkv, d).to(dtype), randn(g, sum(lk), hkv, d).to(dtype))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq,hkv,d,lq,lk", [
    (4, 2, 64, [200, 60], [200, 150]),
    (4, 1, 128, [70, 5, 33], [200, 5, 64]),
    (2, 2, 256, [130, 9], [190, 40]),
    (4, 2, 128, [3, 2], [9000, 700]),      # few rows over many keys: the keys are cut into parts
    (2, 1, 256, [2], [6000]),
    (2, 1, 64, [5], [8100]),
])
def test_attn_prompt_non_finite_hidden(dtype, hq, hkv, d, lq, lk):
    """NaN and infinities in keys and values that a row does not see leave that row as it is: later positions,
    other sequences, rows between sequences."""
    g = gen(sum(lk) + d)
    q, k, v = prompt_state(g, lq, lk, hq, hkv, d, dtype)
    args = dict(max_q=max(lq), max_k=max(lk))
    cq, ck = cumulated(lq), cumulated(lk)
    want = P.ptq1_attn_prompt(q, k, v, cq, ck, **args)
    check_prompt(q, k, v, lq, lk, want, True)
    k2, v2 = k.clone(), v.clone()
    spoiled = torch.zeros(sum(lq), dtype=torch.bool, device=DEV)
    at_q = at_k = 0
    for i, (nq, nk) in enumerate(zip(lq, lk)):
        if nq > 1:  # the last two keys: seen by the last two rows, one of them by the last alone
            v2[at_k + nk - 1, :, 3] = float("inf")
            k2[at_k + nk - 1, :, 1] = float("nan")
            v2[at_k + nk - 1, :, 7] = float("nan")
            spoiled[at_q + nq - 1] = True
        if i == 1:  # one whole sequence of NaN
            k2[at_k:at_k + nk], v2[at_k:at_k + nk] = float("nan"), float("-inf")
            spoiled[at_q:at_q + nq] = True
        at_q, at_k = at_q + nq, at_k + nk
    got = P.ptq1_attn_prompt(q, k2, v2, cq, ck, **args)
    assert torch.equal(got[~spoiled], want[~spoiled])
    # a NaN key makes the whole row NaN
    assert bool(got[spoiled].isnan().all())
    # the rows of one sequence between two others are hidden from both
    gap_q, gap_k = torch.cat([q, q, q]), torch.cat([k, k2, k])
    gap_v = torch.cat([v, torch.full_like(v, float("nan")), v])
    nq, nk = sum(lq), sum(lk)
    if len(lq) == 1:
        cu_q = torch.tensor([0, nq], dtype=torch.int32, device=DEV)
        cu_k = torch.tensor([2 * nk, 3 * nk], dtype=torch.int32, device=DEV)
        got = P.ptq1_attn_prompt(gap_q, gap_k, gap_v, cu_q, cu_k, **args)
        assert torch.equal(got[:nq], want)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attn_prompt_hidden_infinity_of_a_visible_key(d):
    """An infinite value that a row sees reaches that row's dimension alone."""
    g = gen(50 + d)
    n = 150
    q, k, v = prompt_state(g, [n], [n], 2, 1, d)
    want = P.ptq1_attn_prompt(q, k, v, cumulated([n]), cumulated([n]))
    v2 = v.clone()
    v2[77, 0, 5] = float("inf")
    got = P.ptq1_attn_prompt(q, k, v2, cumulated([n]), cumulated([n]))
    seen = torch.arange(n, device=DEV) >= 77
    assert not bool(got[seen][:, :, 5].isfinite().any())
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[77:, :, 5] = True
    assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d,lq,lk", [
    (4, 2, 64, [1], [20000]),
    (8, 2, 128, [16, 3], [12345, 1]),
    (2, 2, 256, [5], [9001]),
    (6, 1, 128, [20, 4, 0, 9], [7000, 2, 50, 0]),   # queries that see nothing beside a cut sequence
    (16, 1, 256, [33, 1], [4100, 4096]),
])
def test_attn_prompt_cut_along_the_keys(dtype, causal, hq, hkv, d, lq, lk):
    g = gen(hq + d + sum(lk))
    q, k, v = prompt_state(g, lq, lk, hq, hkv, d, dtype)
    assert P.workspace_bytes("attn_prompt", len(lq), sum(lq), max(lk), hq, hkv, d) > 0
    out = torch.full((sum(lq) + 2, hq, d), 7.0, dtype=dtype, device=DEV)
    qq = torch.cat([q, q[:1], q[:1]])
    P.ptq1_attn_prompt(qq, k, v, cumulated(lq), cumulated(lk), max_q=max(lq), max_k=max(lk), causal=causal, out=out)
    check_prompt(q, k, v, lq, lk, out, causal)
    assert bool((out[sum(lq):] == 7).all())   # rows behind the last sequence
    again = P.ptq1_attn_prompt(qq, k, v, cumulated(lq), cumulated(lk), max_q=max(lq), max_k=max(lk), causal=causal)
    assert torch.equal(out[:sum(lq)], again[:sum(lq)])
    # a refused sequence beside them
    bad = cumulated(lk)
    bad[-1] = sum(lk) + 1
    got = P.ptq1_attn_prompt(q, k, v, cumulated(lq), bad, max_q=max(lq), max_k=max(lk) + 1, causal=causal)
    first = sum(lq[:-1])
    check_prompt(q, k, v, lq[:-1], lk[:-1], got, causal)
    assert bool(got[first:].isnan().all())


@pytest.mark.parametrize("batch", [65, 200, 1000])
def test_many_sequences(batch):
    """More sequences than lanes, with empty ones among them, through read-back, prompt and decode."""
    g = gen(batch)
    lens = [int(n) for n in np.random.default_rng(batch).integers(0, 40, batch)]
    lens[0], lens[64], lens[-1] = 0, 100, 0
    table, pages = tables(g, lens, 16)
    c = filled_cache(g, pages, 16, 2, 64, BF16)
    poison_unused(c, table, lens)
    cu = cumulated(lens)
    k, v = P.ptq1_kv_read(c, table, cu, sum(lens), dtype=BF16)
    kc, vc = cache_values(c)
    order = [sequence(c, kc, table, b, n).transpose(0, 1) for b, n in enumerate(lens) if n]
    assert torch.equal(k.double(), torch.cat(order))
    order = [sequence(c, vc, table, b, n).transpose(0, 1) for b, n in enumerate(lens) if n]
    assert torch.equal(v.double(), torch.cat(order))
    q = randn(g, sum(lens), 4, 64).to(BF16)
    o = P.ptq1_attn_prompt(q, k, v, cu, cu, max_q=100, max_k=100)
    some = [b for b in range(batch) if b < 3 or b in (63, 64, 65, batch - 2) or b % 50 == 7]
    for b in some:
        a, z = int(cu[b]), int(cu[b + 1])
        check_prompt(q[a:z], k[a:z], v[a:z], [z - a], [z - a], o[a:z], True)
    last = torch.stack([q[int(cu[b + 1]) - 1] if n else q[0] for b, n in enumerate(lens)])
    got = P.ptq1_attn_decode(last, c, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    check_decode(last, c, table, lens, got)


@pytest.mark.parametrize("ctype", [F16, BF16, I8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_kv_write_runs_across_pages(ctype, d):
    """A prompt's neighbouring slots from an odd place on, over pages that lie apart, with holes; the same in one call
    or in two."""
    g = gen(60 + d)
    n, page, hkv = 203, 32, 2
    order = torch.randperm(9, generator=g, device=DEV)
    place = torch.arange(5, 5 + n, device=DEV)
    slots = order[place // page] * page + place % page
    slots[torch.tensor([17, 90, 91, 92], device=DEV)] = -1
    k, v = randn(g, n, hkv, d).to(BF16), randn(g, n, hkv, d).to(BF16)
    caches = [P.ptq1_kv_cache(9, page, hkv, d, ctype, DEV) for _ in range(2)]
    for c in caches:
        for t in (c.k_pages, c.v_pages, c.k_steps, c.v_steps):
            if t is not None:
                t.fill_(1)
    P.ptq1_kv_write(None, k, v, slots, caches[0])
    P.ptq1_kv_write(None, k[:101], v[:101], slots[:101], caches[1])
    P.ptq1_kv_write(None, k[101:], v[101:], slots[101:], caches[1])
    for name in ("k_pages", "v_pages", "k_steps", "v_steps"):
        a, b = (getattr(c, name) for c in caches)
        assert a is None or torch.equal(a, b)
    kc, vc = cache_values(caches[0])
    ok = slots >= 0
    at, off = slots[ok] // page, slots[ok] % page
    zero = torch.zeros((int(ok.sum()), hkv, d), dtype=torch.float64, device=DEV)
    check_rows(kc[at, :, off], k[ok].double(), zero, ctype)
    check_rows(vc[at, :, off], v[ok].double(), zero, ctype)
    kept = torch.ones(9 * page, dtype=torch.bool, device=DEV)
    kept[slots[ok]] = False
    for t in (kc, vc):
        assert bool((t.transpose(1, 2).reshape(9 * page, hkv, d)[kept] == 1).all())


def test_nothing_to_do():
    c = P.ptq1_kv_cache(2, 16, 2, 64, I8, DEV)
    k = torch.empty((0, 2, 64), device=DEV)
    i64, i32 = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV)
    assert P.ptq1_kv_write(None, k, k, i64, c) is None
    assert P.ptq1_kv_write(k, k, k, i64, c, q_dtype=BF16).shape == (0, 2, 64)
    cu0 = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.empty((0, 3), dtype=torch.int32, device=DEV)
    kr, vr = P.ptq1_kv_read(c, table, cu0, 0, dtype=BF16)
    assert kr.shape == vr.shape == (0, 2, 64)
    q = torch.empty((0, 4, 64), dtype=BF16, device=DEV)
    assert P.ptq1_attn_decode(q, c, table, i32).shape == (0, 4, 64)
    kb = k.to(BF16)
    assert P.ptq1_attn_prompt(q, kb, kb, cu0, cu0).shape == (0, 4, 64)
    # sequences without a token, and a table without columns
    q = torch.ones((3, 4, 64), dtype=BF16, device=DEV)
    zero = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert bool((P.ptq1_attn_decode(q, c, torch.empty((3, 0), dtype=torch.int32, device=DEV), zero) == 0).all())
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    kr, vr = P.ptq1_kv_read(c, torch.zeros((3, 1), dtype=torch.int32, device=DEV), cu, 5, dtype=BF16)
    assert kr.shape == (5, 2, 64)
    o = P.ptq1_attn_prompt(q, kb, kb, torch.tensor([0, 1, 1, 3], dtype=torch.int32, device=DEV), cu)
    assert bool((o == 0).all())
    torch.cuda.synchronize()


def test_captured_prompt_and_read_back():
    """Two graphs, a workspace each, replayed in turn and together with eager calls between them."""
    g = gen(70)
    page, lens, new = 32, [5000, 900], [6, 11]
    table, pages = tables(g, lens, page)
    c = filled_cache(g, pages, page, 2, 128, BF16)
    cu_k, cu_q = cumulated(lens), cumulated(new)
    need = P.workspace_bytes("attn_prompt", 2, sum(new), max(lens), 8, 2, 128)
    assert need > 0
    parts = []
    for _ in range(2):
        kv = [torch.empty((sum(lens), 2, 128), dtype=BF16, device=DEV) for _ in range(2)]
        parts.append((randn(g, sum(new), 8, 128).to(BF16), kv, torch.empty((sum(new), 8, 128), dtype=BF16, device=DEV),
                      torch.empty(need, dtype=torch.uint8, device=DEV)))

    def step(q, kv, out, ws):
        P.ptq1_kv_read(c, table, cu_k, sum(lens), dtype=BF16, out=kv)
        P.ptq1_attn_prompt(q, *kv, cu_q, cu_k, max_q=max(new), max_k=max(lens), out=out, ws=ws)

    torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream() for _ in parts], []
    for part, s in zip(parts, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step(*part)
        graphs.append(graph)
    for i in range(3):
        for q, _, out, _ in parts:
            q.copy_(randn(g, *q.shape))
            out.fill_(float("nan"))
        c.k_pages.mul_(0.9)
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for q, kv, out, ws in parts:
            got = out.clone()
            check_prompt(q, *kv, new, lens, got, True)
            step(q, kv, out, ws)
            assert torch.equal(out, got)


@pytest.mark.parametrize("ctype", [BF16, I8])
def test_cache_past_32_bit_offsets(ctype):
    """Pages whose elements lie past 2^32."""
    g = gen(80)
    page, hkv, d, pages = 256, 8, 128, 16400
    assert pages * page * hkv * d > 1 << 32
    c = P.ptq1_kv_cache(pages, page, hkv, d, ctype, DEV)
    table = torch.tensor([[16399, 3, 16397], [16398, 8200, 0]], dtype=torch.int32, device=DEV)
    lens = [600, 515]
    cu = cumulated(lens)
    k, v = (randn(g, sum(lens), hkv, d).to(BF16) for _ in range(2))
    place = torch.cat([torch.arange(n, device=DEV) for n in lens])
    seq = torch.repeat_interleave(torch.arange(2, device=DEV), torch.tensor(lens, device=DEV))
    slots = table[seq, place // page].long() * page + place % page
    P.ptq1_kv_write(None, k, v, slots, c)
    kr, vr = P.ptq1_kv_read(c, table, cu, sum(lens), dtype=F32)
    zero = torch.zeros(kr.shape, dtype=torch.float64, device=DEV)
    check_rows(kr, k.double(), zero + (half_step(k.double(), F32) if ctype == I8 else 0), ctype)
    check_rows(vr, v.double(), zero + (half_step(v.double(), F32) if ctype == I8 else 0), ctype)
    q = randn(g, 2, 16, d)
    got = P.ptq1_attn_decode(q, c, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    kr, vr = kr.double(), vr.double()
    for b in range(2):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        for h in range(hkv):
            want, tol = attention_bounds(q[b, 2 * h:2 * h + 2].double(), kr[rows, h], vr[rows, h], d ** -0.5,
                                         WEIGHT_TERM[(F32, ctype)])
            tol = tol + 4 * U * want.abs() + 4 * U  # kr and vr are rounded products of code and step
            assert bool(((got[b, 2 * h:2 * h + 2].double() - want).abs() <= tol).all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attn_prompt_rows_far_apart(d):
    """Rows at the largest stride, their offsets past 2^32 bytes."""
    g = gen(81)
    n, stride = 200, 1 << 24
    room = torch.empty((n, stride), dtype=BF16, device=DEV)
    q, k, v = (room.as_strided((n, h, d), (stride, d, 1), i * 4096) for i, h in enumerate((4, 2, 2)))
    for t in (q, k, v):
        t.copy_(randn(g, *t.shape))
    got = P.ptq1_attn_prompt(q, k, v, cumulated([n]), cumulated([n]))
    check_prompt(q, k, v, [n], [n], got, True)


# --------------------------------------------- weights far below the largest ----

def ramp_sequence(kind, n):
    """Scores in units of log2: one token that takes nearly everything, first or last, or a ramp up or down."""
    s = torch.full((n,), -27.3, dtype=torch.float64, device=DEV)
    if kind in ("first", "last"):
        s[0 if kind == "first" else n - 1] = 0
        return s
    s = torch.linspace(-60, 0, n, dtype=torch.float64, device=DEV)
    return s if kind == "up" else s.flip(0)


@pytest.mark.parametrize("qt,ctype", PAIRS)
@pytest.mark.parametrize("kind", ["first", "last", "up", "down"])
def test_attn_decode_many_small_weights(qt, ctype, kind):
    """A token that takes nearly the whole weight and has no value, beside thousands that have: what they add must not
    vanish.  int8: that token's step is 2^20 times the others'.  A weight (int8: weight times step) enters as 16-bit
    terms down to 2^-24 of a unit of which the largest has 2^13 at least, so it is off by its relative error or by
    2^-38 of the largest, whichever is more."""
    g = gen(90)
    n, d = 3000, 64
    table, pages = tables(g, [n], 64)
    c = filled_cache(g, pages, 64, 1, d, ctype)
    s = ramp_sequence(kind, n)
    heavy = {"first": 0, "last": n - 1, "up": 0, "down": n - 1}[kind]  # ramps: the token that weighs least
    rows = table[0].long()
    place = torch.arange(n, device=DEV)
    at, off = rows[place // 64], place % 64
    # score = scale q0 k0 in log2 units: q0 = 1, scale ln 2, k0 = s (16-bit types round it: the stored value counts)
    k0 = s.clone()
    c.k_pages.zero_()
    if ctype == I8:
        c.k_steps.fill_(0.5)
        k0 = (k0 * 2).round().clamp(-127, 127)
    c.k_pages[at, 0, off, 0] = k0.to(c.dtype)
    if ctype == I8:
        c.v_steps.fill_(2.0 ** -7)
        c.v_steps[at[heavy], 0, off[heavy]] = 2.0 ** 13
    if kind in ("first", "last"):
        c.v_pages[at[heavy], 0, :, off[heavy]] = 0
    q = torch.zeros((1, 2, d), device=DEV, dtype=qt)
    q[0, :, 0] = 1
    scale = math.log(2.0)
    got = P.ptq1_attn_decode(q, c, table, torch.tensor([n], dtype=torch.int32, device=DEV), scale=scale)[0].double()
    kc, vc = cache_values(c)
    k, v = sequence(c, kc, table, 0, n)[0], sequence(c, vc, table, 0, n)[0]
    want, tol = attention_bounds(q[0].double(), k, v, scale, WEIGHT_TERM[(qt, ctype)])
    p = torch.softmax(scale * (q[0].double() @ k.T.contiguous()), 1)
    if ctype != BF16:
        step = c.v_steps[at, 0, off].double()[None] if ctype == I8 else torch.ones_like(p)
        floor = 2.0 ** -38 * (p * step).amax(1, keepdim=True)
        tol = tol + floor * (v / step[0][:, None]).abs().sum(0)
    tol = tol + half_step(want.abs() + tol, qt)
    err = (got - want).abs()
    assert bool((err <= tol).all()), f"{(err / tol).max().item():.3f} of the bound, {(err / want.abs()).max().item()}"


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["first", "last", "up", "down"])
@pytest.mark.parametrize("rows", [2, 300])
def test_attn_prompt_many_small_weights(dtype, d, kind, rows):
    """The same through the prompt call, cut along the keys (few rows) or not.  fp16 weights have 11 bits, down to
    2^-24 of a unit of which the largest weight has 2^7 at least: off by 2^-32 of it at most."""
    g = gen(91)
    n = 3000
    s = ramp_sequence(kind, n)
    q = torch.zeros((rows, 8, d), device=DEV, dtype=dtype)
    q[:, :, 0] = 1
    k = torch.zeros((n, 8, d), device=DEV, dtype=dtype)
    k[:, :, 0] = s[:, None].to(dtype)
    v = (randn(g, n, 8, d) + 2).to(dtype)  # (a mean that is not zero: the small weights add up)
    if kind in ("first", "last"):
        v[0 if kind == "first" else n - 1] = 0
    scale = math.log(2.0)
    got = P.ptq1_attn_prompt(q, k, v, cumulated([rows]), cumulated([n]), causal=False, scale=scale)
    for h in (0, 7):
        qq, kk, vv = (t[:, h].double() for t in (q, k, v))
        want, tol = attention_bounds(qq, kk, vv, scale, torch.finfo(dtype).eps / 2)
        if dtype == F16:
            p = torch.softmax(scale * (qq @ kk.T.contiguous()), 1)
            tol = tol + 2.0 ** -32 * p.amax(1, keepdim=True) * vv.abs().sum(0)
        tol = tol + half_step(want.abs() + tol, dtype)
        err = (got[:, h].double() - want).abs()
        assert bool((err <= tol).all()), f"{(err / tol).max().item():.3f} of the bound"


def test_attn_decode_small_queries_beside_a_large_one():
    """fp32 queries over fp16: a large element that meets keys of zero takes no precision from the others that the
    bound does not allow (three terms down to 2^-24 of a unit of which the head's largest has 2^14 at least)."""
    g = gen(92)
    n, d = 300, 128
    table, pages = tables(g, [n], 16)
    c = filled_cache(g, pages, 16, 1, d, F16)
    c.k_pages[..., 5] = 0
    q = randn(g, 1, 4, d)
    q[..., 5] = 4096.0
    got = P.ptq1_attn_decode(q, c, table, torch.tensor([n], dtype=torch.int32, device=DEV))
    check_decode(q, c, table, [n], got)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d,lq,lk", [
    (128, 16, 256, [150, 126], [2400, 2300]),
    (128, 16, 128, [300, 40, 196], [3000, 2900, 1000]),
    (64, 32, 64, [400, 1, 666], [2700, 2800, 2600]),
])
def test_attn_prompt_last_tiles_cut(dtype, causal, hq, hkv, d, lq, lk):
    """More tiles than the GPU holds at once: those behind the last full round are cut along the keys."""
    g = gen(hq + d + sum(lk))
    assert P.workspace_bytes("attn_prompt", len(lq), sum(lq), max(lk), hq, hkv, d) > 0
    q, k, v = prompt_state(g, lq, lk, hq, hkv, d, dtype)
    args = dict(max_q=max(lq), max_k=max(lk), causal=causal)
    got = P.ptq1_attn_prompt(q, k, v, cumulated(lq), cumulated(lk), **args)
    check_prompt(q, k, v, lq, lk, got, causal)
    assert torch.equal(got, P.ptq1_attn_prompt(q, k, v, cumulated(lq), cumulated(lk), **args))
    # one sequence refused: the others as they were within their bounds
    bad = cumulated(lk)
    bad[-1] += 1
    args["max_k"] += 1
    got = P.ptq1_attn_prompt(q, k, v, cumulated(lq), bad, **args)
    first = sum(lq[:-1])
    assert bool(got[first:].isnan().all())
    check_prompt(q, k, v, lq[:-1], lk[:-1], got, causal)


@pytest.mark.parametrize("batch", [65, 130, 1000, 5000])
def test_many_sequences_of_unlike_lengths(batch):
    """Large batches with a few long sequences: tiles and pieces of one sequence among those of many."""
    g = gen(100 + batch)
    rng = np.random.default_rng(batch)
    lens = [int(n) for n in rng.integers(0, 9, batch)]
    long = [0, batch // 3, 63, 64, batch - 1]
    for b in long:
        lens[b] = int(rng.integers(700, 3000))
    table, pages = tables(g, lens, 16)
    c = filled_cache(g, pages, 16, 2, 64, BF16)
    cu = cumulated(lens, 5)  # five rows ahead of the first sequence
    total = sum(lens) + 9
    k, v = P.ptq1_kv_read(c, table, cu, total, dtype=BF16)
    kc, vc = cache_values(c)
    some = sorted(set(long + [1, 2, batch // 2, 62, batch - 2]))
    q = randn(g, total, 4, 64).to(BF16)
    o = P.ptq1_attn_prompt(q, k, v, cu, cu, max_q=3000, max_k=3000)
    last = q[:batch].contiguous() if total >= batch else randn(g, batch, 4, 64).to(BF16)
    got = P.ptq1_attn_decode(last, c, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    for b in some:
        a, z = int(cu[b]), int(cu[b + 1])
        for have, val in ((k, kc), (v, vc)):
            assert torch.equal(have[a:z].double(), sequence(c, val, table, b, lens[b]).transpose(0, 1))
        check_prompt(q[a:z], k[a:z], v[a:z], [z - a], [z - a], o[a:z], True)
        check_decode(last[b:b + 1], c, table[b:b + 1], [lens[b]], got[b:b + 1])
    # every row of every sequence was written, with the same numbers as alone
    assert bool(o[5:5 + sum(lens)].isfinite().all()) and bool(got.isfinite().all())
    few = [i for i in range(batch) if lens[i] > 0][:40]
    alone = P.ptq1_attn_decode(last[few].contiguous(), c, table[few].contiguous(),
                               torch.tensor([lens[i] for i in few], dtype=torch.int32, device=DEV))
    small = [j for j, i in enumerate(few) if lens[i] < 256]  # (one piece in either call)
    assert torch.equal(alone[small], got[[few[j] for j in small]])
    # a sequence out of bounds and one of a bad length leave the others as they were
    bad = cu.clone()
    bad[-1] += 100
    o2 = P.ptq1_attn_prompt(q, k, v, cu, bad, max_q=3000, max_k=3100)
    edge = int(cu[batch - 1])
    assert torch.equal(o2[5:edge], o[5:edge]) and bool(o2[edge:5 + sum(lens)].isnan().all())


# -------------------------------------------------- magnitudes at the limits ----

@pytest.mark.parametrize("ctype", [F16, BF16, I8])
@pytest.mark.parametrize("size,scale", [(1e-28, 1e28), (1e-30, 2e29), (2.0 ** -118, 2.0 ** 116), (2.0 ** -124, 2.0 ** 123),
                                        (2.0 ** -131, 2.0 ** 126)])
def test_attn_decode_tiny_queries(ctype, size, scale):
    """fp32 queries near the smallest fp32 values, under a scale that makes ordinary scores of them: their fp16 terms
    (int8: digits) follow the head's magnitude, bf16 terms go down to 2^-133 (half a step of that, times the keys and
    the scale, is what a score may be off by then; twice, since the weights' sum has it too)."""
    g = gen(111)
    lens = [90, 33]
    table, pages = tables(g, lens, 16)
    c = filled_cache(g, pages, 16, 2, 64, ctype)
    q = randn(g, 2, 6, 64) * size
    got = P.ptq1_attn_decode(q, c, table, torch.tensor(lens, dtype=torch.int32, device=DEV), scale=scale)
    if ctype != BF16:
        check_decode(q, c, table, lens, got, scale)
        return
    kc, vc = cache_values(c)
    for b, n in enumerate(lens):
        k, v = sequence(c, kc, table, b, n), sequence(c, vc, table, b, n)
        for h in range(2):
            qq = q[b, 3 * h:3 * h + 3].double()
            want, tol = attention_bounds(qq, k[h], v[h], scale, WEIGHT_TERM[(F32, BF16)])
            p = torch.softmax(scale * (qq @ k[h].T.contiguous()), 1)
            off = scale * 2.0 ** -134 * k[h].abs().sum(1).max()
            tol = tol + 2 * off * (p @ v[h].abs()) + half_step(want.abs() + tol, F32)
            err = (got[b, 3 * h:3 * h + 3].double() - want).abs()
            assert bool((err <= tol).all()), f"b={b} h={h}: {(err / tol).max().item():.3f} of the bound"


@pytest.mark.parametrize("ctype", [F16, BF16, I8])
def test_attn_decode_large_queries_over_zero_keys(ctype):
    """Keys of zero give scores of zero, and the mean of the values, whatever the query and the scale are."""
    g = gen(112)
    lens = [70, 5]
    table, pages = tables(g, lens, 16)
    c = filled_cache(g, pages, 16, 1, 64, ctype)
    c.k_pages.zero_()
    q = randn(g, 2, 4, 64) * 2.0 ** 110
    got = P.ptq1_attn_decode(q, c, table, torch.tensor(lens, dtype=torch.int32, device=DEV), scale=2.0 ** 126)
    check_decode(q, c, table, lens, got, 2.0 ** 126)


@pytest.mark.parametrize("qt", [F32, BF16])
@pytest.mark.parametrize("size,step,scale", [
    (2.0 ** -90, 2.0 ** 90, 0.1),
    (2.0 ** -121, 2.0 ** 121, 0.125),         # the largest steps
    (2.0 ** -60, 2.0 ** 121, 2.0 ** -60),
    (2.0 ** -20, 2.0 ** 121, 2.0 ** -100),
    (2.0 ** 121, 2.0 ** -126, 1.0),           # the smallest steps that ptq1_kv_write makes
    (2.0 ** 100, 2.0 ** -45, 2.0 ** -57),
    (2.0 ** -115, 2.0 ** -2, 2.0 ** 116),
])
def test_attn_decode_large_and_small_steps(qt, size, step, scale):
    """int8 keys of any step that a cache may hold, with queries and scales that make ordinary scores of them: no
    product on the way may leave fp32's range."""
    g = gen(110)
    lens = [300, 70, 1]
    table, pages = tables(g, lens, 32)
    c = filled_cache(g, pages, 32, 2, 128, I8)
    c.k_steps.mul_(50).clamp_(0.5, 1.0).mul_(step / 127)
    c.k_pages[table[1, 1].item(), :, 3] = 0   # a key of zeros among them
    q = (randn(g, 3, 8, 128) * size).to(qt)
    got = P.ptq1_attn_decode(q, c, table, torch.tensor(lens, dtype=torch.int32, device=DEV), scale=scale)
    check_decode(q, c, table, lens, got, scale)


@pytest.mark.parametrize("qt", [F32, BF16])
@pytest.mark.parametrize("step", [2.0 ** 121, 2.0 ** 60, 2.0 ** -60, 2.0 ** -110])
def test_attn_decode_large_and_small_value_steps(qt, step):
    """int8 values of any step, ordinary keys; one token's step is 2^10 times smaller than the others'."""
    g = gen(113)
    lens = [300, 70]
    table, pages = tables(g, lens, 32)
    c = filled_cache(g, pages, 32, 2, 128, I8)
    c.v_pages.copy_((c.v_pages.float() / 2).round())   # (the largest step's results stay below 2^128)
    c.v_steps.mul_(50).clamp_(0.5, 1.0).mul_(step)
    c.v_steps[table[0, 2].item(), :, 5] *= 2.0 ** -10
    q = randn(g, 2, 8, 128).to(qt)
    got = P.ptq1_attn_decode(q, c, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    check_decode(q, c, table, lens, got)


# ------------------------------------------------------ values near fp32's end ----

def largest_values(g, *shape):
    """bf16 values up to 2^127.98, all of them large: sums of a few are past fp32's range."""
    return ((0.9 + 0.09 * torch.rand(shape, generator=g, device=DEV)) * 3.4e38).to(BF16)


@pytest.mark.parametrize("qt", [F32, BF16])
@pytest.mark.parametrize("lens", [[300, 5], [9000, 700]])
def test_attn_decode_largest_values(qt, lens):
    """bf16 values whose mean is in fp32's range and whose sum is not."""
    g = gen(120)
    table, pages = tables(g, lens, 32)
    c = filled_cache(g, pages, 32, 2, 128, BF16)
    c.v_pages.copy_(largest_values(g, *c.v_pages.shape))
    q = randn(g, 2, 8, 128).to(qt)
    got = P.ptq1_attn_decode(q, c, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    check_decode(q, c, table, lens, got)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lq,lk", [([300], [300]), ([3, 2], [9000, 700])])
def test_attn_prompt_largest_values(d, lq, lk):
    g = gen(121)
    q, k, _ = prompt_state(g, lq, lk, 4, 2, d)
    v = largest_values(g, *k.shape)
    got = P.ptq1_attn_prompt(q, k, v, cumulated(lq), cumulated(lk), max_q=max(lq), max_k=max(lk))
    check_prompt(q, k, v, lq, lk, got, True)


# ------------------------------------------------------------ memory of two streams ----

def busy(x):
    """Some milliseconds of ordinary work on the current stream."""
    for _ in range(20):
        x = torch.mm(x, x).mul_(1e-3)
    return x


def side_state(seed):
    q, c, table, sl = decode_state(seed, [2000, 900], I8)
    need = P.workspace_bytes("attn_decode", 2, 8, 2, 128, table.shape[1] * 32)
    assert 0 < need < 1 << 20    # (a block of the allocator's small pool)
    want = P.ptq1_attn_decode(q, c, table, sl)
    return q, c, table, sl, need, want, torch.full((4096, 4096), 1e-3, device=DEV)


def test_side_stream_while_its_work_is_pending():
    """The scratch of a call that waits on a side stream is not handed to the current stream's next tensors of that
    size, nor is its result's memory when the caller drops it."""
    q, c, table, sl, need, want, x = side_state(130)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            busy(x)
        got = P.ptq1_attn_decode(q, c, table, sl, stream=side)
        P.ptq1_attn_decode(q, c, table, sl, stream=side)                     # dropped at once
        taken = [torch.empty(n, dtype=torch.uint8, device=DEV).fill_(255)    # NaN in fp32
                 for n in (need, want.numel() * 4) for _ in range(6)]
        torch.cuda.current_stream().synchronize()
        side.synchronize()
        assert torch.equal(got, want)
        assert all(bool((t == 255).all()) for t in taken)


def test_side_stream_beside_pending_work_of_the_current_stream():
    """Blocks that the current stream has freed, with its own writes still pending on them, do not become the scratch
    or the result of a call on a side stream."""
    q, c, table, sl, need, want, x = side_state(131)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (need, want.numel() * 4) for _ in range(6)]
        torch.cuda.synchronize()
        busy(x)
        for b in blocks:
            b.fill_(255)
        del blocks, b
        got = P.ptq1_attn_decode(q, c, table, sl, stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_side_stream_every_call():
    """The four calls, one behind the other on a side stream, give what they give on the current one."""
    g = gen(132)
    page, n = 32, 150
    rows, rope = randn(g, n, 12, 128), rope_table(200, 128)
    table = torch.arange(5, dtype=torch.int32, device=DEV).view(1, 5)
    slots, pos = torch.arange(n, device=DEV), torch.arange(n, dtype=torch.int32, device=DEV)
    cu, sl = cumulated([n]), torch.tensor([n], dtype=torch.int32, device=DEV)

    def chain(stream):
        c = P.ptq1_kv_cache(5, page, 2, 128, BF16, DEV)
        torch.cuda.synchronize()
        q = P.ptq1_kv_write(rows[:, :8], rows[:, 8:10], rows[:, 10:], slots, c, positions=pos, cos_sin=rope, q_dtype=BF16,
                            stream=stream)
        k, v = P.ptq1_kv_read(c, table, cu, n, dtype=BF16, stream=stream)
        o = P.ptq1_attn_prompt(q, k, v, cu, cu, stream=stream)
        d = P.ptq1_attn_decode(q[-1:], c, table, sl, stream=stream)
        torch.cuda.synchronize()
        return q, k, v, o, d

    for a, b in zip(chain(None), chain(torch.cuda.Stream())):
        assert torch.equal(a, b)


def test_projections_on_a_side_stream_beside_pending_work():
    """The same for a projection: its scratch and result are none of the current stream's freed blocks."""
    n, k = 1024, 1024
    w, _ = folded(3, n, k)
    signs = torch.from_numpy(synth.signs(3)).to(DEV)
    x = torch.from_numpy(synth.activations(5, 64, k)).to(DEV)
    want = P.ptq1_gemm(w, n, k, x, signs)
    sizes = [P.workspace_bytes("gemm", 64, n, k), want.numel() * 4]
    side, work = torch.cuda.Stream(), torch.full((4096, 4096), 1e-3, device=DEV)
    torch.cuda.synchronize()
    for _ in range(3):
        blocks = [torch.empty(size, dtype=torch.uint8, device=DEV) for size in sizes if size for _ in range(6)]
        torch.cuda.synchronize()
        busy(work)
        for b in blocks:
            b.fill_(255)
        del blocks, b
        got = P.ptq1_gemm(w, n, k, x, signs, stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("ctype", [BF16, I8])
def test_kv_write_position_outside_the_table(ctype):
    """Only the elements that would turn are NaN; an int8 row, which has one step, is NaN throughout."""
    g = gen(141)
    n, d, rot = 5, 128, 32
    c = P.ptq1_kv_cache(1, 16, 1, d, ctype, DEV)
    x = randn(g, n, 4, d)
    pos = torch.tensor([0, -1, 3, 8, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    out = P.ptq1_kv_write(x[:, :2], x[:, 2:3], x[:, 3:], torch.arange(n, device=DEV), c, positions=pos,
                          cos_sin=rope_table(8, rot))
    kc, vc = cache_values(c)
    for t in range(n):
        outside = not 0 <= pos[t].item() < 8
        assert bool(out[t, :, :rot].isnan().all()) == outside and torch.equal(out[t, :, rot:], x[t, :2, rot:])
        key = kc[0, 0, t]
        if ctype == I8:
            assert bool(key.isnan().all()) == outside and bool(key.isnan().any()) == outside
        else:
            assert bool(key[:rot].isnan().all()) == outside and torch.equal(key[rot:], x[t, 2, rot:].to(BF16).double())
        assert bool(vc[0, 0, t].isfinite().all())


@pytest.mark.parametrize("qt,ctype", [(BF16, BF16), (F32, BF16), (F16, F16), (F32, F16)])
def test_attn_decode_infinite_key(qt, ctype):
    """An infinite element of a key: rows whose score of it is +infinity are NaN; at -infinity the key has weight
    zero (fp32 queries, which meet it as several terms: that, or NaN); the other head's rows are as they were."""
    g = gen(140)
    n = 50
    table, pages = tables(g, [n], 16)
    c = filled_cache(g, pages, 16, 2, 64, ctype)
    sl = torch.tensor([n], dtype=torch.int32, device=DEV)
    q = randn(g, 1, 8, 64).to(qt)
    q[0, :, 5] = torch.tensor([1.3, -0.7, 2.1, -1.9] * 2, device=DEV).to(qt)
    want = P.ptq1_attn_decode(q, c, table, sl)
    c.k_pages[table[0, 1].item(), 1, 3, 5] = float("inf")    # token 19 of head 1
    got = P.ptq1_attn_decode(q, c, table, sl)
    assert torch.equal(got[0, :4], want[0, :4])
    assert bool(got[0, [4, 6]].isnan().all())
    kc, vc = cache_values(c)
    kept = torch.arange(n, device=DEV) != 19
    k, v = sequence(c, kc, table, 0, n)[1][kept], sequence(c, vc, table, 0, n)[1][kept]
    exact, tol = attention_bounds(q[0, [5, 7]].double(), k, v, 64 ** -0.5, WEIGHT_TERM[(qt, ctype)])
    tol = tol + half_step(exact.abs() + tol, qt)
    without = ((got[0, [5, 7]].double() - exact).abs() <= tol).all(1)
    assert bool((without | (got[0, [5, 7]].isnan().all(1) if qt == F32 else without)).all())


def test_layer_half_output_projection_and_both_paths():
    """What test_layer_half_prompt_then_token leaves out: the prompt's output projection (ptq1_gemm) against 64 bits
    from its own input, and the decode call at the prompt's last position against the prompt call: both are within
    their bounds of the same rows, so they differ by the sum of the bounds at most."""
    g = gen(150)
    dm, hq, hkv, d, n, page = 1024, 8, 2, 128, 77, 32
    wo, dense = folded(2, dm, hq * d)
    signs = torch.from_numpy(synth.signs(3)).to(DEV)
    x = randn(g, n, hq + 2 * hkv, d)
    c = P.ptq1_kv_cache(3, page, hkv, d, BF16, DEV)
    table, place = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV), torch.arange(n, device=DEV)
    slots = table[0, place // page].long() * page + place % page
    q = P.ptq1_kv_write(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], slots, c, positions=place.to(torch.int32),
                        cos_sin=rope_table(n, d), q_dtype=BF16)
    cu = cumulated([n])
    k, v = P.ptq1_kv_read(c, table, cu, n, dtype=BF16)
    o = P.ptq1_attn_prompt(q, k, v, cu, cu)
    check_prompt(q, k, v, [n], [n], o, True)
    rows = o.float().view(n, hq * d)
    y = P.ptq1_gemm(wo, dm, hq * d, rows, signs)
    rot = P.hadamard_rotate(rows, signs).double()
    want = rot @ dense.T.contiguous()
    # bf16 rounds every rotated element by 2^-8 of itself at most, the weights are exact, the sums fp32
    tol = (2.0 ** -8 + hq * d * U) * (rot.abs() @ dense.abs().T.contiguous())
    assert bool(((y.double() - want).abs() <= tol).all())
    last = P.ptq1_attn_decode(q[-1:].contiguous(), c, table, torch.tensor([n], dtype=torch.int32, device=DEV))[0]
    for h in range(hkv):
        heads = slice(h * hq // hkv, (h + 1) * hq // hkv)
        args = (q[-1, heads].double(), k[:, h].double(), v[:, h].double(), d ** -0.5)
        exact, one = attention_bounds(*args, WEIGHT_TERM[(BF16, BF16)])
        _, other = attention_bounds(*args, torch.finfo(BF16).eps / 2)
        tol = one + other + half_step(exact.abs() + one, BF16) + half_step(exact.abs() + other, BF16)
        assert bool(((last[heads].double() - o[-1, heads].double()).abs() <= tol).all())


def test_attn_prompt_ragged_prompts_are_not_cut():
    """Whole prompts of unlike lengths in more tiles than the GPU holds: the last tiles are the shortest and stay whole,
    so the call needs no scratch; chunks behind contexts of about one length, as many tiles, are cut and need it."""
    g = gen(160)
    hq, hkv, d = 20, 4, 64
    lens = [1235, 43, 45, 70, 37, 208, 392, 229, 366, 62, 56, 233, 790, 133, 26, 28]
    chunks, context = [245] * 16, 4000

    def call(lq, lk, ws):
        q, k, v = prompt_state(g, lq, lk, hq, hkv, d)
        cq, ck, out = cumulated(lq), cumulated(lk), torch.empty_like(q)
        size = 0 if ws is None else ws.numel()
        status = P.lib().ptq1_attn_prompt(q.data_ptr(), hq * d, k.data_ptr(), hkv * d, v.data_ptr(), hkv * d, 2,
                                          cq.data_ptr(), ck.data_ptr(), len(lq), sum(lq), sum(lk), max(lq), max(lk), hq,
                                          hkv, d, 1, d ** -0.5, out.data_ptr(), 0 if ws is None else ws.data_ptr(), size,
                                          torch.cuda.current_stream().cuda_stream)
        if status == 0:
            check_prompt(q, k, v, lq, lk, out, True)
        return status

    assert call(lens, lens, None) == 0
    behind = [n + context for n in chunks]
    assert call(chunks, behind, None) == 6
    need = P.workspace_bytes("attn_prompt", 16, sum(chunks), max(behind), hq, hkv, d)
    assert call(chunks, behind, torch.empty(need, dtype=torch.uint8, device=DEV)) == 0


# ------------------------------------------------------------------ large scores ----

def winners(q, k, v, scale, mask=None):
    """(rows, which of them count) of one kv head where a row's largest score is so far ahead that its value is the
    result: by more than 100 and four times what fp32 scores of this size can be off by."""
    logits = scale * (q @ k.T.contiguous())
    size = (scale * (q.abs() @ k.abs().T.contiguous())).amax(1)
    if mask is not None:
        logits = logits.masked_fill(~mask, -math.inf)
    best = logits.topk(min(2, logits.shape[1]), 1)
    ahead = best.values[:, 0] - (best.values[:, -1] if logits.shape[1] > 1 else -math.inf)
    return v[best.indices[:, 0]], ahead > 100 + 4 * (q.shape[1] + 8) * U * size


@pytest.mark.parametrize("qt,ctype", PAIRS)
@pytest.mark.parametrize("size", [1e4, 1e6, 1e8, 1e12])
def test_attn_decode_large_scores(qt, ctype, size):
    """Scores of 10^4 to 10^12 and above: a softmax that picks one token, and no NaN or infinity from what the
    weights are lifted or lowered by."""
    g = gen(170)
    lens = [700, 40, 2]
    table, pages = tables(g, lens, 32)
    c = filled_cache(g, pages, 32, 2, 128, ctype)
    q = randn(g, 3, 8, 128)
    scale = 128 ** -0.5
    if qt == F16:   # the rest of the size in the scale
        q, scale = (q * min(size, 1e3)).to(qt), scale * size / min(size, 1e3)
    else:
        q = (q * size).to(qt)
    got = P.ptq1_attn_decode(q, c, table, torch.tensor(lens, dtype=torch.int32, device=DEV), scale=scale).double()
    kc, vc = cache_values(c)
    counted = 0
    for b, n in enumerate(lens):
        k, v = sequence(c, kc, table, b, n), sequence(c, vc, table, b, n)
        assert bool((got[b].abs() <= v.abs().max() * 1.01).all())       # (a NaN fails too)
        for h in range(2):
            want, ok = winners(q[b, 4 * h:4 * h + 4].double(), k[h], v[h], scale)
            counted += int(ok.sum())
            off = (got[b, 4 * h:4 * h + 4] - want).abs()[ok]
            assert bool((off <= half_step(want[ok], qt) + 4 * U * want[ok].abs()).all())
    assert counted >= 12


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lq,lk", [([150], [150]), ([3], [9000])])
@pytest.mark.parametrize("size", [1e4, 1e6, 1e8, 1e12])
def test_attn_prompt_large_scores_pick_one(dtype, d, lq, lk, size):
    g = gen(171)
    q, k, v = prompt_state(g, lq, lk, 4, 2, d, dtype)
    some = min(size, 1e3)
    q, scale = (q.float() * some).to(dtype), d ** -0.5 * size / some
    got = P.ptq1_attn_prompt(q, k, v, cumulated(lq), cumulated(lk), scale=scale).double()
    assert bool((got.abs() <= v.abs().max().double() * 1.01).all())
    mask = torch.arange(lk[0], device=DEV)[None] <= torch.arange(lq[0], device=DEV)[:, None] + (lk[0] - lq[0])
    counted = 0
    for h in range(4):
        vv = v[:, h // 2].double()
        want, ok = winners(q[:, h].double(), k[:, h // 2].double(), vv, scale, mask)
        counted += int(ok.sum())
        # (its weight is rounded to dtype, their sum is not)
        off, tol = (got[:, h] - want).abs()[ok], half_step(want[ok], dtype) * 2 + 4 * U * want[ok].abs()
        assert bool((off <= tol).all())
    assert counted >= 4


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power", [20, 23, 24, 25, 31])
def test_attn_prompt_scores_around_powers_of_two(dtype, d, power):
    """Exact scores that grow along the keys from just below to just above (minus) a power of two, where the size of
    the last place changes: no weight may leave the type's range, a row's mean stays within its values."""
    g = gen(172 + power)
    n = 200
    v = randn(g, n, 2, d).to(dtype)
    for sign in (1, -1):
        # score in log2 units: sign 2^power + rising small terms, as two exact products
        q = torch.zeros((3, 2, d), device=DEV, dtype=dtype)
        k = torch.zeros((n, 2, d), device=DEV, dtype=dtype)
        half = 2.0 ** min(power // 2, 10)
        q[..., 0], q[..., 1] = half, 1
        k[..., 0] = sign * 2.0 ** min(power - math.log2(half), 15)
        k[..., 1] = torch.arange(-n // 2, n // 2, device=DEV)[:, None] % 64 - 32 + torch.arange(n, device=DEV)[:, None] // 40 * 8
        scale = math.log(2.0) * 2.0 ** (power - math.log2(half) - min(power - math.log2(half), 15))
        for lq in (1, 3):
            got = P.ptq1_attn_prompt(q[:lq], k, v, cumulated([lq]), cumulated([n]), scale=scale, causal=False).double()
            assert bool(got.isfinite().all()) and bool((got.abs() <= 1.02 * v.abs().amax(0).double()).all())


def test_kv_write_largest_rows():
    """int8 rows up to the largest finite value read back finite, within the step's bound."""
    d = 64
    c = P.ptq1_kv_cache(1, 16, 1, d, I8, DEV)
    top = torch.finfo(F32).max
    x = torch.full((16, 1, d), top, device=DEV)
    for i in range(1, 16):
        x[i] = torch.nextafter(x[i - 1], torch.zeros_like(x[i]))
    x[:, :, 1::2] *= -0.5
    P.ptq1_kv_write(None, x, x, torch.arange(16, device=DEV), c)
    table, cu = torch.zeros((1, 1), dtype=torch.int32, device=DEV), cumulated([16])
    for got in P.ptq1_kv_read(c, table, cu, 16, dtype=F32):
        assert bool(got.isfinite().all())
        check_rows(got, x.double(), x.double().abs() * U, I8)


# ------------------------------------------------- weights that make up one ----

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [3, 700])
def test_attn_prompt_rounded_weights_make_up_one(dtype, d, rows):
    """Each weight is rounded to 16 bits, and the rounded ones are summed.  One key of score 0 and value 0 comes first,
    then 500 of score 5 + x (in log2) and one value: the reference stays at the first, and each of the 500 is 2^x
    times a power of two, which is rounded by 0.45 of a step.  Summed unrounded, that would take the row a step away from
    its value (1.98, where half a step is 2^-9 of it, fp16 2^-12); so only what the first key weighs is off, 2^-8 / 16000
    and the fp32 sums, 2 * 600 * 2^-24: neither moves the rounding of the result."""
    n, step = 564, torch.finfo(dtype).eps
    q, k, v = (torch.zeros((m, 4, d), device=DEV, dtype=dtype) for m in (rows, n, n))
    q[..., 0], q[..., 1] = 1, 1
    k[1:64, :, 0] = -100
    k[64:, :, 0], k[64:, :, 1] = 5, math.log2(1 + 0.45 * step)
    v[64:] = 1.98
    got = P.ptq1_attn_prompt(q, k, v, cumulated([rows]), cumulated([n]), causal=False, scale=math.log(2.0))
    w = torch.exp(math.log(2.0) * (q[0, 0].double() @ k[:, 0].double().T.contiguous()))
    exact = (w / w.sum()) @ v[:, 0].double()
    assert bool((exact - exact.to(dtype).double()).abs().max() < 0.4 * step)    # (far from a border of the rounding)
    assert torch.equal(got, exact.to(dtype).expand(rows, 4, d))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [2, 300])
@pytest.mark.parametrize("below", [22, 26, 30])
def test_attn_prompt_small_weights_count_in_the_sum(dtype, d, rows, below):
    """One key of score 0 and value 0, then 65536 of weight 2^-22 to 2^-30 and one value: fp16's subnormal weights are
    multiplied and summed alike.  (They are exact: powers of two, down to 2^-31 of the largest in fp16.)"""
    n = 65537
    q, k, v = (torch.zeros((m, 2, d), device=DEV, dtype=dtype) for m in (rows, n, n))
    q[..., 0], k[1:, :, 0], v[1:] = 1, -below, 1000
    got = P.ptq1_attn_prompt(q, k, v, cumulated([rows]), cumulated([n]), causal=False, scale=math.log(2.0)).double()
    total = 65536 * 2.0 ** -below
    want = torch.tensor(1000 * total / (1 + total), dtype=torch.float64)
    # scale log2(e) is off by 2^-24 of itself, twice: the scores by that times `below`; the sums by 2^-24 for each term
    tol = want * (below * 2.0 ** -22 + 65536 * U)
    assert bool(((got - want).abs() <= tol + half_step(want + tol, dtype)).all()), (got.flatten()[0].item(), want.item())

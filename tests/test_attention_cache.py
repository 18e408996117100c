"""Norms in the cache write, and attention over the cache with a sliding window and by chunks, against plain 64-bit
implementations.

Tolerances are bounds computed from each case's own numbers, as in test_attention.py; beside those:
  - the root mean square of d fp32 values: each square and the sums of a tree of at most 9 levels round once, so the mean
    is off by 10 U of itself (U = 2^-24; the division by d is exact), with eps 11 U; its reciprocal root by half of that
    and the hardware's 2 U; with the products by it and by the gain a normed value is off by 10 U of itself at most.
"""
import math

import numpy as np
import pytest
import torch

import ternary_weight_ptq1_amd as P
from test_attention import (BF16, DEV, F16, F32, I8, PAIRS, U, WEIGHT_TERM, attention_bounds, cache_values, check_rows,
                            cumulated, filled_cache, gen, half_step, randn, rope_table, sequence, tables)

pytestmark = pytest.mark.gpu
NORM = 10 * U


# ------------------------------------------------------ norms in the write ----

def normed(x, gain, eps):
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if gain is None else y * gain.double()


def turned_norm(x, gain, eps, pos, table):
    """(normed and rotated rows in fp64, a bound on the fp32 arithmetic's error)."""
    y = normed(x, gain, eps)
    if table is None:
        return y, y.abs() * NORM
    half = table.shape[1] // 2
    row = table[pos.long()].double()[:, None]
    c, s = row[..., :half], row[..., half:]
    a, b, rest = y[..., :half], y[..., half:2 * half], y[..., 2 * half:]
    size = torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1)
    return torch.cat([a * c - b * s, b * c + a * s, rest], -1), torch.cat([size * (NORM + 2 * U), rest.abs() * NORM], -1)


@pytest.mark.parametrize("src", [F32, F16, BF16])
@pytest.mark.parametrize("ctype", [F16, BF16, I8])
@pytest.mark.parametrize("n,hq,hkv,d,page,rot,eps", [
    (1, 5, 1, 64, 16, 64, 1e-6),
    (3, 0, 2, 128, 32, 32, 1e-5),
    (33, 6, 3, 64, 64, 8, 1e-6),
    (70, 8, 2, 256, 16, 64, 0.5),
    (129, 4, 4, 128, 256, 128, 1e-12),
    (40, 3, 1, 128, 128, 0, 1e-6),
])
def test_kv_write_norm(src, ctype, n, hq, hkv, d, page, rot, eps):
    g = gen(n + d + rot)
    pages = -(-2 * n // page) + 2
    qt = {F16: F16, BF16: BF16, I8: F32}[ctype]
    x = randn(g, n, hq + 2 * hkv + 1, d) * torch.exp(randn(g, n, hq + 2 * hkv + 1, 1))  # one head more: the rows lie apart
    x = x.to(src)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]
    q_gain, k_gain = 1 + 0.5 * randn(g, d), None if n == 33 else 1 + 0.5 * randn(g, d)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:n]
    slots[n // 2] = -1
    pos = torch.randint(0, 50, (n,), generator=g, device=DEV, dtype=torch.int32)
    table = rope_table(50, rot) if rot else None
    c = P.ptq1_kv_cache(pages, page, hkv, d, ctype, DEV)
    for t in (c.k_pages, c.v_pages):
        t.fill_(3)
    if ctype == I8:
        c.k_steps.fill_(0.5), c.v_steps.fill_(0.5)
    out = P.ptq1_kv_write_norm(q if hq else None, k, v, slots, c, q_gain=q_gain if hq else None, k_gain=k_gain, eps=eps,
                               positions=pos, cos_sin=table, q_dtype=qt if hq else None)
    if hq:
        assert out.dtype == qt and out.shape == (n, hq, d)
        check_rows(out, *turned_norm(q, q_gain, eps, pos, table), qt)
    else:
        assert out is None
    kc, vc = cache_values(c)
    ok = slots >= 0
    at, off = slots[ok] // page, slots[ok] % page
    y, e = turned_norm(k, k_gain, eps, pos, table)
    check_rows(kc[at, :, off], y[ok], e[ok], ctype)
    check_rows(vc[at, :, off], v[ok].double(), torch.zeros_like(y[ok]), ctype)
    kept = torch.ones(pages * page, dtype=torch.bool, device=DEV)
    kept[slots[ok]] = False
    other = 1.5 if ctype == I8 else 3.0
    for t in (kc, vc):  # everything else as it was
        assert bool((t.transpose(1, 2).reshape(pages * page, hkv, d)[kept] == other).all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_kv_write_norm_magnitudes(d):
    """Rows from 2^-140 to fp32's largest, zeros among them: what eps leaves of the small ones, and no overflow."""
    g = gen(d)
    sizes = [0.0, 2.0 ** -140, 2.0 ** -70, 2.0 ** -10, 1.0, 2.0 ** 40, 2.0 ** 58, 2.0 ** 60, 2.0 ** 62, 2.0 ** 64,
             2.0 ** 100, 2.0 ** 127]
    x = (randn(g, len(sizes), 3, d).clamp(-1.9, 1.9) * torch.tensor(sizes, dtype=torch.float64, device=DEV)[:, None, None]
         ).clamp(-3.4e38, 3.4e38).float()
    x[-1, 0] = torch.finfo(F32).max
    c = P.ptq1_kv_cache(1, 16, 3, d, BF16, DEV)
    slots = torch.arange(len(sizes), device=DEV)
    for eps in (1e-6, 2.0 ** -100):
        out = P.ptq1_kv_write_norm(x, x, x, slots, c, eps=eps)
        y = normed(x, None, eps)
        # (squares below fp32's normal numbers, which are nothing beside eps, may be lost: mean / eps of the value)
        lost = torch.where(x.double() ** 2 < 2.0 ** -126, 2.0 ** -126 / eps, 0.0)
        check_rows(out, y, y.abs() * (NORM + lost), F32)
        check_rows(cache_values(c)[0][0].transpose(0, 1)[:len(sizes)], y, y.abs() * (NORM + lost), BF16)


def test_kv_write_norm_non_finite():
    """A NaN takes its head, an infinity makes its own element NaN and the others zero; other heads and V stay."""
    for ctype in (BF16, I8):
        c = P.ptq1_kv_cache(1, 16, 2, 64, ctype, DEV)
        x = torch.ones((3, 2, 64), device=DEV)
        x[0, 0, 5] = float("nan")
        x[1, 1, 7] = float("-inf")
        q = P.ptq1_kv_write_norm(x, x, x, torch.arange(3, device=DEV), c)
        assert bool(q[0, 0].isnan().all()) and bool(q[1, 1, 7].isnan()) and int(q.isnan().sum()) == 65
        assert bool((q[1, 1, :7] == 0).all()) and bool((q[1, 1, 8:] == 0).all())
        kc, _ = cache_values(c)
        assert bool(kc[0, 0, 0].isnan().all()) and bool((kc[0, 1, 1].isnan()).sum() == (64 if ctype == I8 else 1))
        one = 1 / math.sqrt(1 + 1e-6)
        assert bool(((q[2] - one).abs() <= NORM).all()) and bool(((kc[0, :, 2] - one).abs() <= 2.0 ** -8).all())


# ------------------------------------------------- single tokens, windowed ----

def window_mask(n_q, n, window, sinks):
    """[n_q, n]: which tokens the last n_q of n see."""
    p = torch.arange(n - n_q, n, device=DEV)[:, None]
    j = torch.arange(n, device=DEV)[None]
    seen = j <= p
    if window:
        seen &= (j > p - window) | (j < sinks)
    return seen


def keep_window(c, table, new, lens, window, sinks):
    """What no query sees is poisoned (NaN values, or steps), and pages that hold nothing else are taken away."""
    page = c.page_size
    used = torch.zeros((c.n_pages, page), dtype=torch.bool, device=DEV)
    for b, (m, n) in enumerate(zip(new, lens)):
        if n == 0:
            continue
        seen = torch.nn.functional.pad(window_mask(min(m, n), n, window, sinks).any(0), (0, -n % page)).view(-1, page)
        for j, row in enumerate(seen):
            if bool(row.any()):
                used[table[b, j].item()] |= row
            else:
                table[b, j] = -1 if j % 2 else c.n_pages + 5
    hid = ~used[:, None, :].expand(-1, c.n_kv_heads, -1)
    if c.k_steps is not None:
        c.k_steps[hid] = float("nan")
        c.v_steps[hid] = float("nan")
    else:
        c.k_pages[hid] = float("nan")
        c.v_pages[hid[:, :, None, :].expand_as(c.v_pages)] = float("inf")


def gathered(c, values, table, b, n):
    """K or V [heads, n, d] of sequence b in fp64, zeros where its page is not there."""
    rows = table[b, :-(-n // c.page_size)].long()
    there = ((rows >= 0) & (rows < c.n_pages))
    x = torch.where(there[:, None, None, None], values[torch.where(there, rows, 0)], 0.0)
    return x.transpose(0, 1).reshape(c.n_kv_heads, -1, c.head_dim)[:, :n]


def check_attention(q, c, table, new, lens, got, term, window=0, sinks=0, scale=None, at=0):
    hq, d = q.shape[1:]
    group = hq // c.n_kv_heads
    scale = d ** -0.5 if scale is None else scale
    kc, vc = cache_values(c)
    for b, (m, n) in enumerate(zip(new, lens)):
        none = max(0, m - n)  # queries ahead of the first token
        assert bool((got[at:at + none] == 0).all())
        if m > none:
            mask = window_mask(m - none, n, window, sinks)
            any_sees = mask.any(0)[None, :, None]
            k, v = (torch.where(any_sees, gathered(c, t, table, b, n), 0.0) for t in (kc, vc))
            for h in range(c.n_kv_heads):
                rows = slice(h * group, (h + 1) * group)
                qq = q[at + none:at + m, rows].double().reshape(-1, d)
                want, tol = attention_bounds(qq, k[h], v[h], scale, term, mask.repeat_interleave(group, 0))
                tol = tol + half_step(want.abs() + tol, q.dtype)
                err = (got[at + none:at + m, rows].double().reshape(-1, d) - want).abs()
                assert bool((err <= tol).all()), f"b={b} h={h}: {(err / tol).nan_to_num(9e9).max().item():.3f} of the bound"
        at += m


@pytest.mark.parametrize("qt,ctype", PAIRS)
@pytest.mark.parametrize("hq,hkv,d,page,lens,window,sinks", [
    (1, 1, 64, 16, [1, 40], 1, 0),
    (5, 1, 128, 16, [31, 0, 33, 64, 7, 300], 32, 4),
    (6, 2, 256, 32, [129, 1, 1255], 100, 17),
    (32, 8, 128, 64, [257, 511, 3512, 6030], 1024, 4),
    (20, 1, 64, 256, [300, 0, 2, 2000], 77, 300),    # more than 16 query heads of one kv head
    (7, 7, 128, 128, [100, 5049], 2000, 0),
    (4, 2, 128, 16, [40, 70, 99], 33, 16),           # the gap is smaller than what two runs of 16 leave
    (4, 2, 64, 16, [500, 64], 10000, 10000),         # everything is seen
])
def test_attn_decode_window(qt, ctype, hq, hkv, d, page, lens, window, sinks):
    g = gen(hq * d + sum(lens))
    table, pages = tables(g, lens, page)
    c = filled_cache(g, pages, page, hkv, d, ctype)
    keep_window(c, table, [1] * len(lens), lens, window, sinks)
    q = randn(g, len(lens), hq, d).to(qt)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got = P.ptq1_attn_decode_window(q, c, table, sl, window, sinks)
    assert got.dtype == qt and got.shape == q.shape
    args = ([1] * len(lens), lens)
    check_attention(q, c, table, *args, got, WEIGHT_TERM[(qt, ctype)], window, sinks)
    # a bound on the lengths changes the split, not what is computed
    check_attention(q, c, table, *args, P.ptq1_attn_decode_window(q, c, table, sl, window, sinks, max_len=max(lens)),
                    WEIGHT_TERM[(qt, ctype)], window, sinks)
    assert torch.equal(got, P.ptq1_attn_decode_window(q, c, table, sl, window, sinks))


@pytest.mark.parametrize("ctype", [BF16, I8])
def test_attn_decode_window_everything_seen(ctype):
    """A window that covers all tokens gives the bits of the call without one."""
    g = gen(3)
    lens = [700, 33, 2500]
    table, pages = tables(g, lens, 32)
    c = filled_cache(g, pages, 32, 2, 128, ctype)
    q = randn(g, 3, 8, 128)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = P.ptq1_attn_decode(q, c, table, sl)
    for window in (2500, 1 << 40):
        assert torch.equal(want, P.ptq1_attn_decode_window(q, c, table, sl, window))


def test_attn_decode_window_refused_sequences():
    """Lengths that are none, and a page that is not there among those that are needed, or among the others."""
    g = gen(4)
    lens = [100, 200, 300, 400]
    table, pages = tables(g, lens, 16)
    c = filled_cache(g, pages, 16, 2, 64, BF16)
    q = randn(g, 4, 4, 64).to(BF16)
    table[1, 0], table[2, 5], table[3, 24] = -1, pages, -9  # a sink's page, one between, the window's
    sl = torch.tensor([-1, 200, 300, 400], dtype=torch.int32, device=DEV)
    got = P.ptq1_attn_decode_window(q, c, table, sl, 50, 4)
    assert bool(got[0].isnan().all()) and bool(got[1].isnan().all()) and bool(got[3].isnan().all())
    check_attention(q[2:3], c, table[2:3], [1], [300], got[2:3], WEIGHT_TERM[(BF16, BF16)], 50, 4)
    got = P.ptq1_attn_decode_window(q, c, table, sl, 50, 0, max_len=350)
    assert bool(got[3].isnan().all())
    check_attention(q[1:2], c, table[1:2], [1], [200], got[1:2], WEIGHT_TERM[(BF16, BF16)], 50, 0)


@pytest.mark.parametrize("batch", [65, 1000])
def test_attn_decode_window_many_sequences(batch):
    g = gen(batch)
    rng = np.random.default_rng(batch)
    lens = [int(n) for n in rng.integers(0, 900, batch)]
    lens[7] = 9000
    table, pages = tables(g, lens, 64)
    c = filled_cache(g, pages, 64, 1, 64, BF16)
    q = randn(g, batch, 2, 64).to(BF16)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got = P.ptq1_attn_decode_window(q, c, table, sl, 600, 3, max_len=9000)
    check_attention(q, c, table, [1] * batch, lens, got, WEIGHT_TERM[(BF16, BF16)], 600, 3)


# ------------------------------------------------- chunks over the cache ----

CHUNK_PAIRS = [(BF16, BF16), (F16, F16), (BF16, I8), (F16, I8)]
# a weight enters rounded to the 16-bit type of the products (int8 caches: fp16, times its step)
CHUNK_TERM = {(BF16, BF16): 2.0 ** -8, (F16, F16): 2.0 ** -11, (BF16, I8): 2.0 ** -11, (F16, I8): 2.0 ** -11}


def chunk_state(seed, new, lens, hq, hkv, d, page, qt, ctype, window=0, sinks=0):
    g = gen(seed)
    table, pages = tables(g, lens, page)
    c = filled_cache(g, pages, page, hkv, d, ctype)
    keep_window(c, table, new, lens, window, sinks)
    q = randn(g, sum(new), hq, d).to(qt)
    return q, c, table, cumulated(new), torch.tensor(lens, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("qt,ctype", CHUNK_PAIRS)
@pytest.mark.parametrize("hq,hkv,d,page,new,lens,window,sinks", [
    (1, 1, 64, 16, [1], [1], 0, 0),
    (5, 1, 128, 16, [5], [77], 0, 0),
    (6, 2, 256, 32, [3, 1], [129, 1], 0, 0),
    (4, 2, 64, 16, [0, 33, 5, 1], [0, 33, 200, 64], 0, 0),
    (40, 8, 128, 64, [33, 100], [33, 463], 0, 0),
    (6, 1, 256, 256, [70, 65], [400, 65], 0, 0),
    (33, 1, 128, 128, [9], [700], 0, 0),              # rows of a token in two tiles
    (200, 1, 64, 32, [3], [90], 0, 0),                # a token's heads are more than a tile
    (2, 2, 128, 16, [10, 7], [4, 7], 0, 0),           # more queries than tokens: the first ones see nothing
    (8, 2, 64, 16, [20, 300], [500, 300], 50, 0),
    (8, 2, 128, 16, [20, 300, 1], [500, 300, 999], 64, 5),
    (6, 2, 256, 32, [130, 2], [930, 700], 100, 17),
    (4, 4, 128, 64, [200], [1500], 1, 0),
    (4, 4, 128, 64, [64], [700], 500, 130),
    (4, 1, 64, 128, [150], [400], 10000, 10000),
])
def test_attn_chunk(qt, ctype, hq, hkv, d, page, new, lens, window, sinks):
    s = chunk_state(hq + sum(lens), new, lens, hq, hkv, d, page, qt, ctype, window, sinks)
    got = P.ptq1_attn_chunk(*s, window=window, sinks=sinks)
    assert got.dtype == qt and got.shape == s[0].shape
    check_attention(*s[:3], new, lens, got, CHUNK_TERM[(qt, ctype)], window, sinks)
    # bounds change the split, not what is computed; the same call gives the same bits
    tight = dict(max_q=max(new), max_len=max(lens))
    once = P.ptq1_attn_chunk(*s, window=window, sinks=sinks, **tight)
    check_attention(*s[:3], new, lens, once, CHUNK_TERM[(qt, ctype)], window, sinks)
    assert torch.equal(once, P.ptq1_attn_chunk(*s, window=window, sinks=sinks, **tight))


@pytest.mark.parametrize("qt,ctype", CHUNK_PAIRS)
@pytest.mark.parametrize("hq,hkv,d,page,new,lens,window,sinks", [
    (8, 2, 64, 16, [4, 1, 90], [9000, 30, 5000], 0, 0),
    (5, 1, 128, 64, [6, 700], [20000, 700], 0, 0),
    (8, 2, 128, 16, [8, 3], [7000, 12000], 4000, 4),
    (6, 2, 256, 32, [5, 40], [6000, 3000], 0, 0),
    (3, 1, 256, 64, [60], [9000], 5000, 100),
])
def test_attn_chunk_cut_along_the_keys(qt, ctype, hq, hkv, d, page, new, lens, window, sinks):
    s = chunk_state(sum(lens), new, lens, hq, hkv, d, page, qt, ctype, window, sinks)
    got = P.ptq1_attn_chunk(*s, window=window, sinks=sinks, max_q=max(new), max_len=max(lens))
    assert P.workspace_bytes("attn_chunk", len(new), sum(new), max(new), hq, hkv, d, max(lens), window, sinks) > 0
    check_attention(*s[:3], new, lens, got, CHUNK_TERM[(qt, ctype)], window, sinks)


@pytest.mark.parametrize("batch", [65, 200, 1000])
@pytest.mark.parametrize("high", [3, 40])
def test_attn_chunk_many_sequences(batch, high):
    rng = np.random.default_rng(batch)
    new = [int(n) for n in rng.integers(0, high, batch)]
    lens = [n + int(m) for n, m in zip(new, rng.integers(0, 500, batch))]
    lens[7] = new[7] + 6000
    s = chunk_state(batch, new, lens, 2, 1, 64, 64, BF16, BF16)
    got = P.ptq1_attn_chunk(*s, max_q=max(new))
    check_attention(*s[:3], new, lens, got, CHUNK_TERM[(BF16, BF16)])


def test_attn_chunk_rows_apart_and_left_as_they_were():
    """Queries that are parts of stacked rows; rows ahead of the first sequence and behind the last stay."""
    g = gen(8)
    new, lens = [20, 3], [150, 90]
    table, pages = tables(g, lens, 16)
    c = filled_cache(g, pages, 16, 2, 128, BF16)
    rows = randn(g, 30, 12, 128).to(BF16)
    q = rows[:, 2:10]
    cu = cumulated(new, 4)
    out = torch.full((30, 8, 128), 7.0, dtype=BF16, device=DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    assert P.ptq1_attn_chunk(q, c, table, cu, sl, out=out) is out
    check_attention(q, c, table, new, lens, out, CHUNK_TERM[(BF16, BF16)], at=4)
    assert bool((out[:4] == 7).all()) and bool((out[27:] == 7).all())


@pytest.mark.parametrize("hq,d", [(4, 64), (4, 128), (4, 256)])
@pytest.mark.parametrize("ctype", [BF16, I8])
def test_attn_chunk_refused_sequences(hq, d, ctype):
    """Lengths that are none, more queries than the bound, rows that are not there, pages that are not there."""
    new, lens = [5, 6, 7, 8, 200, 9], [50, 60, 70, 80, 300, 9]
    q, c, table, cu, sl = chunk_state(9, new, lens, hq, 2, d, 16, BF16, ctype)
    page = table[4, 9].item()
    sl[0], table[2, 1], table[4, 9] = -1, -3, c.n_pages  # tokens 16 .. 31 and 144 .. 159
    got = P.ptq1_attn_chunk(q, c, table, cu, sl, max_q=200)
    at = cu.tolist()
    assert bool(got[at[0]:at[1]].isnan().all()) and bool(got[at[2]:at[3]].isnan().all())
    # queries ahead of the page that is not there do not see it: positions 100 .. 143 of that sequence
    assert bool(got[at[4] + 44:at[5]].isnan().all())
    for b, m, n in ((1, 6, 60), (3, 8, 80), (5, 9, 9)):
        check_attention(q, c, table[b:b + 1], [m], [n], got, CHUNK_TERM[(BF16, ctype)], at=at[b])
    check_attention(q, c, table[4:5], [44], [144], got, CHUNK_TERM[(BF16, ctype)], at=at[4])
    # a bound on the queries; with a window, the missing page is behind most of them
    got = P.ptq1_attn_chunk(q, c, table, cu, sl, max_q=100, window=20)
    assert bool(got[at[4]:at[5]].isnan().all())
    table[4, 9] = page
    table[4, 5] = -1  # tokens 80 .. 95: seen from positions 100 .. 114 (windows from 81 to 95 on)
    got = P.ptq1_attn_chunk(q, c, table, cu, sl, max_q=200, window=20)
    assert bool(got[at[4]:at[4] + 15].isnan().all()) and not bool(got[at[4] + 15:at[5]].isnan().any())
    # rows past the tensor's end, and a length past its bound
    short = P.ptq1_attn_chunk(q[:at[5] + 4], c, table, cu, sl, max_len=79, window=20)
    assert bool(short[at[5]:].isnan().all()) and bool(short[at[3]:at[4]].isnan().all())
    check_attention(q, c, table[1:2], [6], [60], short, CHUNK_TERM[(BF16, ctype)], 20, at=at[1])

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
from test_attention import (BF16, DEV, F16, F32, I8, PAIRS, U, WEIGHT_TERM, attention_bounds, busy, cache_values, check_rows,
                            cumulated, filled_cache, gen, half_step, largest_values, ramp_sequence, randn, rope_table,
                            sequence, tables, winners)

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


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("eps", [2.0 ** 100, 2.0 ** 90, 2.0 ** -100])
def test_kv_write_norm_large_rows_and_eps(d, eps):
    """Rows whose sum of squares is just below and just above fp32's largest, where eps may still count."""
    g = gen(d + 1)
    sizes = [2.0 ** e for e in (48, 50, 52, 56, 58, 59, 60, 61, 62, 63, 64, 65)]
    x = ((1 + torch.rand((12, 2, d), generator=g, device=DEV, dtype=torch.float64)) *
         torch.tensor(sizes, dtype=torch.float64, device=DEV)[:, None, None]).float()
    c = P.ptq1_kv_cache(1, 16, 2, d, BF16, DEV)
    out = P.ptq1_kv_write_norm(x, x, x, torch.arange(12, device=DEV), c, eps=eps)
    y = normed(x, None, eps)
    check_rows(out, y, y.abs() * NORM, F32)


@pytest.mark.parametrize("ctype", [BF16, I8])
def test_kv_write_norm_position_outside_the_table(ctype):
    """Only the elements that would turn are NaN; an int8 row, which has one step, is NaN throughout."""
    g = gen(141)
    n, d, rot = 5, 128, 32
    c = P.ptq1_kv_cache(1, 16, 1, d, ctype, DEV)
    x = randn(g, n, 4, d)
    pos = torch.tensor([0, -1, 3, 8, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    out = P.ptq1_kv_write_norm(x[:, :2], x[:, 2:3], x[:, 3:], torch.arange(n, device=DEV), c, positions=pos,
                               cos_sin=rope_table(8, rot))
    y = normed(x, None, 1e-6)
    kc, vc = cache_values(c)
    for t in range(n):
        outside = not 0 <= pos[t].item() < 8
        assert bool(out[t, :, :rot].isnan().all()) == outside
        check_rows(out[t, :, rot:], y[t, :2, rot:], y[t, :2, rot:].abs() * NORM, F32)
        if ctype == I8:
            assert bool(kc[0, 0, t].isnan().all()) == outside and bool(kc[0, 0, t].isnan().any()) == outside
        else:
            assert bool(kc[0, 0, t, :rot].isnan().all()) == outside
            check_rows(kc[0, 0, t, rot:], y[t, 2, rot:], y[t, 2, rot:].abs() * NORM, ctype)
        assert bool(vc[0, 0, t].isfinite().all())


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


def check_attention(q, c, table, new, lens, got, term, window=0, sinks=0, scale=None, at=0, floor=0.0):
    """floor: what a weight (int8: weight times step) may be off by beside its term, of the row's largest one."""
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
                if floor:
                    weights = torch.softmax((scale * (qq @ k[h].T.contiguous())).masked_fill(~mask.repeat_interleave(group, 0), -math.inf), 1)
                    places = table[b, torch.arange(n, device=DEV) // c.page_size].long(), torch.arange(n, device=DEV) % c.page_size
                    step = c.v_steps[places[0], h, places[1]].double() if c.dtype == I8 else torch.ones(n, dtype=torch.float64, device=DEV)
                    tol = tol + floor * (weights * step).amax(1, keepdim=True) * (v[h].abs() / step[:, None]).sum(0)
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


# Where no sequence may have more than 32 rows of a kv head, a weight enters as two 16-bit terms: what the first leaves,
# half a step of it at most, is rounded once more, by half a step of a value that is at most that (bf16: 2^-8 of a weight
# leaves 2^-17, fp16: 2^-11 leaves 2^-23; int8: a weight times its step in fp32 first, 2^-24, and the step's unit is exact).
FEW_TERM = {(BF16, BF16): 2.0 ** -17, (F16, F16): 2.0 ** -23, (BF16, I8): 2.0 ** -22, (F16, I8): 2.0 ** -22}


@pytest.mark.parametrize("qt,ctype", CHUNK_PAIRS)
@pytest.mark.parametrize("hq,hkv,d,page,new,lens,window,sinks", [
    (1, 1, 64, 16, [32, 1, 0, 7], [40, 1, 9, 700], 0, 0),
    (32, 1, 128, 64, [1, 1], [2, 333], 0, 0),
    (6, 2, 256, 32, [10, 3], [200, 1000], 0, 0),
    (15, 3, 128, 16, [6, 4, 6], [6, 3, 300], 0, 0),       # more queries than tokens
    (8, 2, 128, 16, [8, 3, 1], [300, 5000, 65], 60, 5),
    (4, 4, 64, 256, [9, 30], [5000, 31], 1000, 300),
    (5, 1, 256, 64, [5], [7000], 0, 0),
])
def test_attn_chunk_few_rows(qt, ctype, hq, hkv, d, page, new, lens, window, sinks):
    assert max(new) * hq // hkv <= 32
    s = chunk_state(hq + sum(lens), new, lens, hq, hkv, d, page, qt, ctype, window, sinks)
    got = P.ptq1_attn_chunk(*s, window=window, sinks=sinks, max_q=max(new))
    check_attention(*s[:3], new, lens, got, FEW_TERM[(qt, ctype)], window, sinks)


def chunk_term(qt, ctype, rows):
    return (FEW_TERM if rows <= 32 else CHUNK_TERM)[(qt, ctype)]


def set_token(c, table, b, j, k=None, v=None, heads=slice(None)):
    """Token j of sequence b: K's dimension 1 and V's dimension 3 (int8 caches: their steps) become k and v."""
    at, off = table[b, j // c.page_size].long(), j % c.page_size
    for x, pages, steps in ((k, c.k_pages, c.k_steps), (v, c.v_pages, c.v_steps)):
        if x is None:
            continue
        if steps is not None:
            steps[at, heads, off] = x
        elif pages is c.k_pages:
            pages[at, heads, off, 1] = x
        else:
            pages[at, heads, 3, off] = x


@pytest.mark.parametrize("qt,ctype", CHUNK_PAIRS)
@pytest.mark.parametrize("hq,hkv,d,page,new,lens,window,sinks", [
    (4, 2, 64, 16, [16, 5], [90, 33], 0, 0),
    (8, 2, 128, 16, [8, 6], [700, 30], 100, 4),
    (4, 2, 256, 64, [12, 7], [300, 65], 20, 0),
    (4, 1, 128, 64, [8], [9000], 0, 0),
    (4, 2, 64, 32, [150, 7], [400, 7], 0, 0),
    (4, 2, 128, 16, [100, 9], [300, 200], 64, 3),
    (2, 1, 256, 32, [80], [200], 0, 0),
    (2, 1, 256, 16, [90, 30], [900, 70], 100, 17),
    (2, 1, 64, 64, [130], [9000], 0, 0),
    (2, 1, 128, 64, [70], [8000], 5000, 0),
])
def test_attn_chunk_non_finite(qt, ctype, hq, hkv, d, page, new, lens, window, sinks):
    """NaN and infinities in keys and values: the entries that they enter are not finite, all others are
    the rows without them.  Only kv head 0 holds them."""
    state = chunk_state(sum(new) + d, new, lens, hq, hkv, d, page, qt, ctype, window, sinks)
    q, c, table, cu, sl = state
    args = dict(window=window, sinks=sinks, max_q=max(new))
    group = hq // hkv
    tensors = [t for t in (c.k_pages, c.v_pages, c.k_steps, c.v_steps) if t is not None]
    before = [t.clone() for t in tensors]
    clean = P.ptq1_attn_chunk(*state, **args)
    term = chunk_term(qt, ctype, max(new) * group)
    check_attention(q, c, table, new, lens, clean, term, window, sinks)
    odd = torch.zeros(clean.shape, dtype=torch.bool, device=DEV)       # what must not be finite
    either = torch.zeros(clean.shape, dtype=torch.bool, device=DEV)    # an infinite key's rows: a weight of zero, or NaN
    at = 0
    for b, (m, n) in enumerate(zip(new, lens)):
        mask = window_mask(m, n, window, sinks)
        places = [(n - 1, None, math.inf), (n - 1 - m // 2, None, math.nan), (n - 2, math.inf, None)]
        if window:   # seen by the first queries alone
            places += [(j, math.nan, None) for j in (n - m - window + m // 3 + 1,) if j >= sinks]
        else:
            places += [(n - 1 - m // 3, math.nan, None)]
        if d == 256:  # several in one step, and two kinds in one token
            places += [(n - 1 - m // 2, math.nan, None), (n - 3, None, -math.inf)]
        for j, k, v in places:
            set_token(c, table, b, j, k, v, slice(0, 1))
            rows = mask[:, j]
            if k is not None:
                (odd if math.isnan(k) else either)[at:at + m, :group] |= rows[:, None, None]
            else:
                odd[at:at + m, :group, (slice(None) if ctype == I8 else slice(3, 4))] |= rows[:, None, None]
        at += m
    got = P.ptq1_attn_chunk(*state, **args)
    odd &= ~either
    assert bool(odd.any()) and bool((~odd & ~either).any())
    assert not bool(got[odd].isfinite().any())
    rest = ~odd & ~either
    assert bool(got[rest].isfinite().all())
    # (not the same bits: a row's reference may move because its neighbour's does)
    for t, was in zip(tensors, before):
        t.copy_(was)
    check_attention(q, c, table, new, lens, torch.where(rest, got, clean), term, window, sinks)


@pytest.mark.parametrize("qt,ctype", CHUNK_PAIRS)
def test_attn_chunk_non_finite_queries(qt, ctype):
    """A NaN takes its own row; beside it rows of the same tile stay."""
    for new, lens in (([6], [100]), ([70], [300])):
        state = chunk_state(77, new, lens, 4, 2, 128, 32, qt, ctype)
        clean = P.ptq1_attn_chunk(*state, max_q=new[0])
        state[0][3, 1, 5] = math.nan
        state[0][4, 2, 6] = math.inf
        got = P.ptq1_attn_chunk(*state, max_q=new[0])
        assert bool(got[3, 1].isnan().all()) and not bool(got[4, 2].isfinite().all())
        got[3, 1], got[4, 2] = clean[3, 1], clean[4, 2]
        assert torch.equal(got, clean)


def placed(k, v, page, ctype, steps=None):
    """A cache whose pages hold k and v [n, heads, d] (int8: codes, with steps), in order, and its block table."""
    n, h, d = k.shape
    pages = -(-n // page)
    c = P.ptq1_kv_cache(pages, page, h, d, ctype, DEV)
    pad = torch.zeros((pages * page - n, h, d), dtype=k.dtype, device=DEV)
    kk, vv = (torch.cat([x, pad]).view(pages, page, h, d) for x in (k, v))
    c.k_pages.copy_(kk.transpose(1, 2))
    c.v_pages.copy_(vv.permute(0, 2, 3, 1))
    if ctype == I8:
        c.k_steps.fill_(steps), c.v_steps.fill_(steps)
    return c, torch.arange(pages, dtype=torch.int32, device=DEV).view(1, pages)


@pytest.mark.parametrize("qt,ctype", CHUNK_PAIRS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("m,n", [(150, 150), (3, 9000), (60, 4000)])
@pytest.mark.parametrize("size", [1e4, 1e6, 1e8, 1e12])
def test_attn_chunk_large_scores_pick_one(qt, ctype, d, m, n, size):
    """Scores of 10^4 to 10^12 and above: a softmax that picks one token, and no NaN or infinity on the way."""
    q, c, table, cu, sl = chunk_state(n + d, [m], [n], 4, 2, d, 64, qt, ctype)
    some = min(size, 1e3)
    q, scale = (q.float() * some).to(qt), d ** -0.5 * size / some
    got = P.ptq1_attn_chunk(q, c, table, cu, sl, scale=scale, max_q=m).double()
    kc, vc = cache_values(c)
    k, v = sequence(c, kc, table, 0, n), sequence(c, vc, table, 0, n)
    assert bool((got.abs() <= v.abs().max() * 1.01).all())
    counted = 0
    for h in range(4):
        want, ok = winners(q[:, h].double(), k[h // 2], v[h // 2], scale, window_mask(m, n, 0, 0))
        counted += int(ok.sum())
        # one weight, rounded to the products' type (int8: times its step), over the sum of the rounded ones (int8: of
        # the unrounded ones)
        tol = half_step(want, qt) + chunk_term(qt, ctype, 2 * m) * want.abs() + 4 * U * want.abs()
        assert bool(((got[:, h] - want).abs()[ok] <= tol[ok]).all())
    assert counted >= 4


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power", [20, 23, 24, 25, 31])
def test_attn_chunk_scores_around_powers_of_two(dtype, d, power):
    """Exact scores that grow along the keys across a power of two (or minus it), where the size of the last place
    changes: a row's mean stays within its values."""
    g = gen(172 + power)
    n = 200
    v = randn(g, n, 2, d).to(dtype)
    for sign in (1, -1):
        q = torch.zeros((40, 2, d), device=DEV, dtype=dtype)
        k = torch.zeros((n, 2, d), device=DEV, dtype=dtype)
        half = 2.0 ** min(power // 2, 10)
        q[..., 0], q[..., 1] = half, 1
        k[..., 0] = sign * 2.0 ** min(power - math.log2(half), 15)
        k[..., 1] = torch.arange(-n // 2, n // 2, device=DEV)[:, None] % 64 - 32 + torch.arange(n, device=DEV)[:, None] // 40 * 8
        scale = math.log(2.0) * 2.0 ** (power - math.log2(half) - min(power - math.log2(half), 15))
        c, table = placed(k, v, 64, dtype)
        sl = torch.tensor([n], dtype=torch.int32, device=DEV)
        for m in (1, 3, 40):
            got = P.ptq1_attn_chunk(q[:m], c, table, cumulated([m]), sl, scale=scale, max_q=m).double()
            assert bool(got.isfinite().all()) and bool((got.abs() <= 1.02 * v.abs().amax(0).double()).all())


@pytest.mark.parametrize("qt,ctype", CHUNK_PAIRS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["first", "last", "up", "down"])
@pytest.mark.parametrize("m", [3, 300])
def test_attn_chunk_many_small_weights(qt, ctype, d, kind, m):
    """A token that takes nearly the whole weight and has no value, beside thousands that have.  fp16 terms end at
    2^-24 of a unit of which the largest weight has 2^7 at least (an error of 2^-32 of it), over int8 caches of which the
    largest weight times step has 2^2 at least (2^-27).  The queries' own tokens weigh nothing."""
    g = gen(91)
    n, h = 2700, 4
    s = torch.cat([ramp_sequence(kind, n), torch.full((m,), -100.0, dtype=torch.float64, device=DEV)])
    q = torch.zeros((m, h, d), device=DEV, dtype=qt)
    q[:, :, 0] = 1
    k = torch.zeros((n + m, h, d), device=DEV, dtype=F32)
    v = randn(g, n + m, h, d) + 2
    k[:, :, 0] = s[:, None].float()
    if ctype == I8:
        k, v = (k * 2).round().clamp(-127, 127), (v * 20).round().clamp(-127, 127)
    k, v = k.to(ctype), v.to(ctype)
    if kind in ("first", "last"):
        v[0 if kind == "first" else n - 1] = 0
    c, table = placed(k, v, 64, ctype, 0.5)
    scale = math.log(2.0)
    got = P.ptq1_attn_chunk(q, c, table, cumulated([m]), torch.tensor([n + m], dtype=torch.int32, device=DEV), scale=scale, max_q=m)
    step = 0.5 if ctype == I8 else 1.0
    mask = window_mask(m, n + m, 0, 0)
    for i in (0, h - 1):
        qq, kk, vv = q[:, i].double(), k[:, i].double() * step, v[:, i].double() * step
        want, tol = attention_bounds(qq, kk, vv, scale, chunk_term(qt, ctype, m), mask)
        if ctype != BF16:
            p = torch.softmax((scale * (qq @ kk.T.contiguous())).masked_fill(~mask, -math.inf), 1)
            tol = tol + (2.0 ** -27 if ctype == I8 else 2.0 ** -32) * p.amax(1, keepdim=True) * vv.abs().sum(0)
        tol = tol + half_step(want.abs() + tol, qt)
        err = (got[:, i].double() - want).abs()
        assert bool((err <= tol).all()), f"{(err / tol).max().item():.3f} of the bound"


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("m", [3, 300])
def test_attn_chunk_rounded_weights_make_up_one(dtype, d, m):
    """As for prompts: 500 weights that are rounded by 0.45 of a step, over one value that leaves half a step of room."""
    n, step = 564, torch.finfo(dtype).eps
    q = torch.zeros((m, 2, d), device=DEV, dtype=dtype)
    k, v = (torch.zeros((n + m, 2, d), device=DEV, dtype=dtype) for _ in range(2))
    q[..., 0], q[..., 1] = 1, 1
    k[1:64, :, 0], k[n:, :, 0] = -100, -100
    k[64:n, :, 0], k[64:n, :, 1] = 5, math.log2(1 + 0.45 * step)
    v[64:n] = 1.98
    c, table = placed(k, v, 32, dtype)
    got = P.ptq1_attn_chunk(q, c, table, cumulated([m]), torch.tensor([n + m], dtype=torch.int32, device=DEV), scale=math.log(2.0),
                            max_q=m)
    w = torch.exp(math.log(2.0) * (q[0, 0].double() @ k[:, 0].double().T.contiguous()))
    exact = (w / w.sum()) @ v[:, 0].double()
    assert bool((exact - exact.to(dtype).double()).abs().max() < 0.4 * step)    # (far from a border of the rounding)
    assert torch.equal(got, exact.to(dtype).expand(m, 2, d))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m", [2, 300])
@pytest.mark.parametrize("below", [22, 26, 30])
def test_attn_chunk_small_weights_count_in_the_sum(dtype, m, below):
    """One key of score 0 and value 0, then 65536 of weight 2^-22 to 2^-30 and one value (exact down to 2^-31 of the
    largest in fp16); the queries' own tokens weigh nothing (2^-120)."""
    n, d = 65537, 64
    q = torch.zeros((m, 2, d), device=DEV, dtype=dtype)
    k, v = (torch.zeros((n + m, 2, d), device=DEV, dtype=dtype) for _ in range(2))
    q[..., 0], k[1:n, :, 0], v[1:n], k[n:, :, 0] = 1, -below, 1000, -120
    c, table = placed(k, v, 256, dtype)
    got = P.ptq1_attn_chunk(q, c, table, cumulated([m]), torch.tensor([n + m], dtype=torch.int32, device=DEV), scale=math.log(2.0),
                            max_q=m).double()
    total = 65536 * 2.0 ** -below
    want = torch.tensor(1000 * total / (1 + total), dtype=torch.float64)
    tol = want * (below * 2.0 ** -22 + 65536 * U)
    assert bool(((got - want).abs() <= tol + half_step(want + tol, dtype)).all()), (got.flatten()[0].item(), want.item())


@pytest.mark.parametrize("qt,size,step,scale", [
    (BF16, 2.0 ** -121, 2.0 ** 121, 0.125),
    (BF16, 2.0 ** -60, 2.0 ** 121, 2.0 ** -60),
    (BF16, 2.0 ** -20, 2.0 ** 121, 2.0 ** -100),
    (BF16, 2.0 ** 90, 2.0 ** -90, 0.1),
    (BF16, 2.0 ** 121, 2.0 ** -110, 2.0 ** -11),
    (BF16, 2.0 ** 121, 2.0 ** -100, 2.0 ** -21),
    (BF16, 2.0 ** 100, 2.0 ** -45, 2.0 ** -57),
    (BF16, 2.0 ** -115, 2.0 ** -2, 2.0 ** 116),
    (F16, 2.0 ** 8, 2.0 ** 110, 2.0 ** -118),
    (F16, 2.0 ** -8, 2.0 ** -100, 2.0 ** 108),
])
@pytest.mark.parametrize("new,lens", [([5, 3], [300, 70]), ([70, 40], [300, 70])])
@pytest.mark.parametrize("d", [128, 256])
def test_attn_chunk_large_and_small_steps(qt, size, step, scale, new, lens, d):
    """int8 keys of any step, with queries and scales that make ordinary scores of them: no product on the way leaves
    fp32's range.  (scale times step is a normal number.)  Some rows are nearly one token's, whose code may be zero: beside
    its term a weight times step is off by 2^-27 of the row's largest, as in test_attn_chunk_many_small_weights."""
    g = gen(110)
    table, pages = tables(g, lens, 32)
    c = filled_cache(g, pages, 32, 2, d, I8)
    c.k_steps.mul_(50).clamp_(0.5, 1.0).mul_(step / 127)
    c.k_pages[table[1, 1].item(), :, 3] = 0
    q = (randn(g, sum(new), 8, d) * size).to(qt)
    got = P.ptq1_attn_chunk(q, c, table, cumulated(new), torch.tensor(lens, dtype=torch.int32, device=DEV), scale=scale,
                            max_q=max(new))
    check_attention(q, c, table, new, lens, got, chunk_term(qt, I8, 4 * max(new)), scale=scale, floor=2.0 ** -27)


@pytest.mark.parametrize("step", [2.0 ** 121, 2.0 ** 60, 2.0 ** -60, 2.0 ** -110])
@pytest.mark.parametrize("new,lens", [([5, 3], [300, 70]), ([70, 40], [300, 70]), ([2, 1], [9000, 70])])
@pytest.mark.parametrize("d", [128, 256])
def test_attn_chunk_large_and_small_value_steps(step, new, lens, d):
    """int8 values of any step, ordinary keys; one token's step is 2^10 times smaller than the others'."""
    g = gen(113)
    table, pages = tables(g, lens, 32)
    c = filled_cache(g, pages, 32, 2, d, I8)
    c.v_pages.copy_((c.v_pages.float() / 2).round())   # (the largest step's results stay below 2^128)
    c.v_steps.mul_(50).clamp_(0.5, 1.0).mul_(step)
    c.v_steps[table[0, 2].item(), :, 5] *= 2.0 ** -10
    q = randn(g, sum(new), 8, d).to(BF16)
    got = P.ptq1_attn_chunk(q, c, table, cumulated(new), torch.tensor(lens, dtype=torch.int32, device=DEV), max_q=max(new))
    check_attention(q, c, table, new, lens, got, chunk_term(BF16, I8, 4 * max(new)), floor=2.0 ** -27)


@pytest.mark.parametrize("qt", [BF16, F16])
@pytest.mark.parametrize("m", [3, 100])
def test_attn_chunk_unlike_value_steps(qt, m):
    """Values whose steps differ by 2^40 between tokens, the large ones first, last, or in one page: every row keeps
    the resolution that its own largest product allows (2^-27 of it, beside the terms')."""
    g = gen(114)
    n = 500
    for kind in ("first", "last", "page"):
        table, pages = tables(g, [n], 32)
        c = filled_cache(g, pages, 32, 2, 128, I8)
        rows = table[0].long()
        c.v_steps[rows if kind != "page" else rows[5]] *= 2.0 ** 20
        c.v_steps[rows[1:] if kind == "first" else rows[:-1] if kind == "last" else rows[6]] *= 2.0 ** -40
        q = randn(g, m, 4, 128).to(qt)
        got = P.ptq1_attn_chunk(q, c, table, cumulated([m]), torch.tensor([n], dtype=torch.int32, device=DEV), max_q=m)
        kc, vc = cache_values(c)
        mask = window_mask(m, n, 0, 0)
        for h in range(4):
            k, v = sequence(c, kc, table, 0, n)[h // 2], sequence(c, vc, table, 0, n)[h // 2]
            want, tol = attention_bounds(q[:, h].double(), k, v, 128 ** -0.5, chunk_term(qt, I8, 2 * m), mask)
            p = torch.softmax((128 ** -0.5 * (q[:, h].double() @ k.T.contiguous())).masked_fill(~mask, -math.inf), 1)
            step = c.v_steps[rows[torch.arange(n, device=DEV) // 32], h // 2, torch.arange(n, device=DEV) % 32].double()
            floor = 2.0 ** -27 * (p * step).amax(1, keepdim=True) * (v / step[:, None]).abs().sum(0)
            tol = tol + floor
            if qt == F16:  # (results past fp16 are infinite)
                tol = torch.where(want.abs() > 6e4, math.inf, tol)
            tol = tol + half_step(want.abs() + tol, qt)
            err = (got[:, h].double() - want).abs()
            assert bool(((err <= tol) | (tol == math.inf)).all()), f"{kind} {(err / tol).nan_to_num(9e9).max().item():.3f} of the bound"


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,lens", [([300], [300]), ([3, 2], [9000, 700]), ([60, 9], [9000, 700])])
def test_attn_chunk_largest_values(d, new, lens):
    """bf16 values whose mean is in fp32's range and whose sum is not."""
    g = gen(121)
    table, pages = tables(g, lens, 32)
    c = filled_cache(g, pages, 32, 2, d, BF16)
    c.v_pages.copy_(largest_values(g, *c.v_pages.shape))
    q = randn(g, sum(new), 4, d).to(BF16)
    got = P.ptq1_attn_chunk(q, c, table, cumulated(new), torch.tensor(lens, dtype=torch.int32, device=DEV), max_q=max(new))
    check_attention(q, c, table, new, lens, got, chunk_term(BF16, BF16, 2 * max(new)))


# ------------------------------------------------- together, as a layer has them ----

def positions_of(new, lens):
    return torch.cat([torch.arange(n - m, n, device=DEV) for m, n in zip(new, lens)])


def slots_of(table, new, lens, page):
    seq = torch.repeat_interleave(torch.arange(len(new), device=DEV), torch.tensor(new, device=DEV))
    pos = positions_of(new, lens)
    return table[seq, pos // page].long() * page + pos % page


@pytest.mark.parametrize("qt,ctype", CHUNK_PAIRS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 4)])
def test_layer_half_by_chunks_then_tokens(qt, ctype, window, sinks):
    """Prompts that arrive in chunks of unlike lengths (normed, rotated, written, attended), then single tokens: at
    every step the plain layer over everything so far, and what the chunk call and the single tokens' call give for
    the same token agree."""
    g = gen(200)
    hq, hkv, d, page = 8, 2, 128, 32
    total = [410, 131]
    table, pages = tables(g, total, page)
    c = P.ptq1_kv_cache(pages, page, hkv, d, ctype, DEV)
    rope = rope_table(512, d)
    q_gain, k_gain = 1 + 0.2 * randn(g, d), 1 + 0.2 * randn(g, d)
    lens = [0, 0]
    for new in ([200, 3], [1, 64], [64, 1], [140, 60], [4, 2], [1, 1]):
        lens = [a + b for a, b in zip(lens, new)]
        n = sum(new)
        x = randn(g, n, hq + 2 * hkv, d).to(qt)
        pos = positions_of(new, lens).int()
        q = P.ptq1_kv_write_norm(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], slots_of(table, new, lens, page), c,
                                 q_gain=q_gain, k_gain=k_gain, positions=pos, cos_sin=rope, q_dtype=qt)
        check_rows(q, *turned_norm(x[:, :hq], q_gain, 1e-6, pos, rope), qt)
        sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
        got = P.ptq1_attn_chunk(q, c, table, cumulated(new), sl, window=window, sinks=sinks)
        check_attention(q, c, table, new, lens, got, CHUNK_TERM[(qt, ctype)], window, sinks, floor=2.0 ** -27)
        # the last tokens, once more as single ones
        last = torch.tensor(new, device=DEV).cumsum(0) - 1
        one = (P.ptq1_attn_decode_window(q[last], c, table, sl, window, sinks) if window else
               P.ptq1_attn_decode(q[last], c, table, sl))
        check_attention(q[last], c, table, [1, 1], lens, one, WEIGHT_TERM[(qt, ctype)], window, sinks)
        check_attention(q[last], c, table, [1, 1], lens, got[last], CHUNK_TERM[(qt, ctype)], window, sinks, floor=2.0 ** -27)
    assert lens == total


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_chunks_and_whole_prompts_agree(dtype):
    """A chunk that is a whole prompt, and one behind a context, against the prompt call on the rows read back."""
    g = gen(201)
    new, lens = [300, 90], [300, 700]
    table, pages = tables(g, lens, 64)
    c = filled_cache(g, pages, 64, 2, 128, dtype)
    q = randn(g, sum(new), 8, 128).to(dtype)
    cu, cu_k = cumulated(new), cumulated(lens)
    k, v = P.ptq1_kv_read(c, table, cu_k, sum(lens), dtype=dtype)
    got = P.ptq1_attn_chunk(q, c, table, cu, torch.tensor(lens, dtype=torch.int32, device=DEV))
    want = P.ptq1_attn_prompt(q, k, v, cu, cu_k)
    # (both round: twice the bound on either is two terms of the values' mean magnitude and two results)
    tol = 2 * CHUNK_TERM[(dtype, dtype)] * 4 + 2 * half_step(want.double(), dtype)
    assert bool(((got.double() - want.double()).abs() <= tol).all())


@pytest.mark.parametrize("ctype", [BF16, I8])
def test_captured_chunk_step_replays_with_new_contents(ctype):
    """Write with norms, chunk attention and windowed single tokens captured once and replayed with lengths, slots,
    chunks and rows that the program puts into the same buffers, eager work in between; chunks shrink and grow, and a
    sequence's chunk becomes empty."""
    g = gen(202)
    hq, hkv, d, page, width = 8, 2, 128, 32, 80
    lens = [1500, 700]
    table, pages = tables(g, [width * page] * 2, page)
    c = filled_cache(g, pages, page, hkv, d, ctype)
    rows = randn(g, 12, hq + 2 * hkv, d).to(BF16)
    rope = rope_table(width * page, d)
    slots = torch.zeros(12, dtype=torch.int64, device=DEV)
    pos = torch.zeros(12, dtype=torch.int32, device=DEV)
    cu, sl = cumulated([6, 6]), torch.tensor(lens, dtype=torch.int32, device=DEV)
    gain = 1 + 0.2 * randn(g, d)
    sizes = dict(max_q=8, max_len=width * page)
    need = P.workspace_bytes("attn_chunk", 2, 12, 8, hq, hkv, d, width * page, 1000, 4)
    need_one = P.workspace_bytes("attn_decode_window", 2, hq, hkv, d, width * page, 600, 2)
    assert need > 0
    ws, ws_one = (torch.empty(n, dtype=torch.uint8, device=DEV) for n in (need, max(need_one, 16)))
    q = torch.empty((12, hq, d), dtype=BF16, device=DEV)
    out, one = torch.full_like(q, 7), torch.empty((2, hq, d), dtype=BF16, device=DEV)

    def step():
        P.ptq1_kv_write_norm(rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], slots, c, q_gain=gain, k_gain=gain,
                             positions=pos, cos_sin=rope, out=q)
        P.ptq1_attn_chunk(q, c, table, cu, sl, window=1000, sinks=4, out=out, ws=ws, **sizes)
        P.ptq1_attn_decode_window(q[:2], c, table, sl, 600, 2, max_len=width * page, out=one, ws=ws_one)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step()
    for new in ([6, 6], [4, 8], [8, 0], [1, 1], [7, 5]):
        n = sum(new)
        lens = [a + b for a, b in zip(lens, new)]
        rows.copy_(randn(g, 12, hq + 2 * hkv, d))
        slots.fill_(-1)
        slots[:n] = slots_of(table, new, lens, page)
        pos[:n] = positions_of(new, lens).int()
        cu.copy_(cumulated(new))
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        first = out.clone(), one.clone(), q.clone()
        step()
        assert torch.equal(first[0], out) and torch.equal(first[1], one) and torch.equal(first[2], q)
        check_attention(q[:n], c, table, new, lens, out, CHUNK_TERM[(BF16, ctype)], 1000, 4, floor=2.0 ** -27)
        check_attention(q[:2], c, table, [1, 1], lens, one, WEIGHT_TERM[(BF16, ctype)], 600, 2)
        assert bool((out[n:] == 7).all())


def side_calls():
    g = gen(203)
    lens = [2100, 900]
    table, pages = tables(g, lens, 32)
    c = filled_cache(g, pages, 32, 2, 128, BF16)
    q = randn(g, 100, 8, 128).to(BF16)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    few, many = cumulated([5, 3]), cumulated([60, 40])
    return [lambda **kw: P.ptq1_attn_chunk(q[:8], c, table, few, sl, max_q=5, **kw),
            lambda **kw: P.ptq1_attn_chunk(q, c, table, many, sl, max_q=60, window=1500, sinks=3, **kw),
            lambda **kw: P.ptq1_attn_decode_window(q[:2], c, table, sl, 1700, 3, **kw)]


@pytest.mark.parametrize("which", [0, 1, 2])
def test_window_and_chunk_calls_on_side_streams(which):
    """On a stream of the caller's while its work is pending, beside pending work of the current one: scratch and
    results are nobody else's."""
    call = side_calls()[which]
    want = call()
    x = torch.full((4096, 4096), 1e-3, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            busy(x)
        got = call(stream=side)
        call(stream=side)                                                                      # dropped at once
        taken = [torch.empty(1 << e, dtype=torch.uint8, device=DEV).fill_(255) for e in range(12, 21) for _ in range(3)]
        busy(x)
        torch.cuda.current_stream().synchronize()
        side.synchronize()
        assert torch.equal(got, want)
        assert all(bool((t == 255).all()) for t in taken)


def test_window_and_chunk_calls_on_two_streams():
    """The same calls on two streams at once, with scratch of their own."""
    calls = side_calls()
    want = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(6):
        for s in streams:
            with torch.cuda.stream(s):
                got.append([call() for call in calls])
    torch.cuda.synchronize()
    for results in got:
        assert all(torch.equal(a, b) for a, b in zip(results, want))


@pytest.mark.parametrize("ctype", [BF16, I8])
def test_new_calls_past_32_bit_offsets(ctype):
    """Pages whose elements lie past 2^32: the write with norms, chunks of few and of many rows, windowed tokens."""
    g = gen(204)
    page, hkv, d, pages = 256, 8, 128, 16400
    assert pages * page * hkv * d > 1 << 32
    c = P.ptq1_kv_cache(pages, page, hkv, d, ctype, DEV)
    table = torch.tensor([[16399, 3, 16397], [16398, 8200, 0]], dtype=torch.int32, device=DEV)
    lens = [600, 515]
    k, v = (randn(g, sum(lens), hkv, d).to(BF16) for _ in range(2))
    P.ptq1_kv_write_norm(None, k, v, slots_of(table, lens, lens, page), c)
    small = P.ptq1_kv_cache(6, page, hkv, d, ctype, DEV)     # the same pages, near its beginning
    flat = table.flatten().long()
    small.k_pages.copy_(c.k_pages[flat]), small.v_pages.copy_(c.v_pages[flat])
    if ctype == I8:
        small.k_steps.copy_(c.k_steps[flat]), small.v_steps.copy_(c.v_steps[flat])
    near = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    y, e = turned_norm(k, None, 1e-6, None, None)
    rows, _ = cache_values(small)
    got = torch.cat([sequence(small, rows, near, b, n).transpose(0, 1) for b, n in enumerate(lens)])
    check_rows(got, y, e, ctype)
    for new in ([2, 1], [90, 40]):
        q = randn(g, sum(new), 16, d).to(BF16)
        far = P.ptq1_attn_chunk(q, c, table, cumulated(new), sl, max_q=max(new), window=400, sinks=3)
        check_attention(q, small, near, new, lens, far, chunk_term(BF16, ctype, 2 * max(new)), 400, 3, floor=2.0 ** -27)
    far = P.ptq1_attn_decode_window(q[:2], c, table, sl, 400, 3)
    check_attention(q[:2], small, near, [1, 1], lens, far, WEIGHT_TERM[(BF16, ctype)], 400, 3)


def test_attn_chunk_rows_far_apart():
    """Query rows at the largest stride, their offsets past 2^32 bytes."""
    g = gen(205)
    n, stride = 200, 1 << 24
    room = torch.empty((n, stride), dtype=BF16, device=DEV)
    q = room.as_strided((n, 4, 128), (stride, 128, 1), 4096)
    q.copy_(randn(g, *q.shape))
    table, pages = tables(g, [n], 32)
    c = filled_cache(g, pages, 32, 2, 128, BF16)
    got = P.ptq1_attn_chunk(q, c, table, cumulated([n]), torch.tensor([n], dtype=torch.int32, device=DEV))
    check_attention(q, c, table, [n], [n], got, CHUNK_TERM[(BF16, BF16)])


def test_new_calls_with_nothing_to_do():
    """No tokens, no sequences, no query rows; all lengths zero."""
    c = filled_cache(gen(206), 4, 16, 2, 64, BF16)
    none = torch.empty((0, 4, 64), dtype=BF16, device=DEV)
    kv = torch.empty((0, 2, 64), dtype=BF16, device=DEV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    assert P.ptq1_kv_write_norm(none, kv, kv, torch.empty(0, dtype=torch.int64, device=DEV), c, q_dtype=BF16).shape == none.shape
    assert P.ptq1_attn_decode_window(none, c, i32(0, 4), i32(0), 5).shape == none.shape
    assert P.ptq1_attn_chunk(none, c, i32(0, 4), i32(1), i32(0)).shape == none.shape
    assert P.ptq1_attn_chunk(none, c, i32(2, 4), i32(3), torch.tensor([5, 0], dtype=torch.int32, device=DEV)).shape == none.shape
    q = torch.ones((3, 4, 64), dtype=BF16, device=DEV)
    assert bool((P.ptq1_attn_decode_window(q, c, i32(3, 4), i32(3), 5) == 0).all())
    assert bool((P.ptq1_attn_chunk(q, c, i32(1, 4), cumulated([3]), i32(1)) == 0).all())
    assert bool((P.ptq1_attn_chunk(q, c, i32(1, 4), cumulated([3]), i32(1), window=2, sinks=1) == 0).all())


@pytest.mark.parametrize("qt,ctype", CHUNK_PAIRS)
def test_window_and_chunk_share_pages(qt, ctype):
    """Sequences that share the pages of a common beginning, one of them twice in the batch."""
    g = gen(207)
    table, pages = tables(g, [400], 32)
    c = filled_cache(g, pages, 32, 2, 64, ctype)
    table = table.expand(3, -1).contiguous()
    new, lens = [7, 7, 40], [400, 400, 333]
    q = randn(g, sum(new), 4, 64).to(qt)
    q[7:14] = q[:7]
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got = P.ptq1_attn_chunk(q, c, table, cumulated(new), sl, window=200, sinks=1)
    check_attention(q, c, table, new, lens, got, CHUNK_TERM[(qt, ctype)], 200, 1)
    assert torch.equal(got[:7], got[7:14])
    one = P.ptq1_attn_decode_window(q[[0, 7, 20]], c, table, sl, 200, 1)
    check_attention(q[[0, 7, 20]], c, table, [1] * 3, lens, one, WEIGHT_TERM[(qt, ctype)], 200, 1)
    assert torch.equal(one[0], one[1])


@pytest.mark.parametrize("qt,ctype", PAIRS)
def test_attn_decode_window_non_finite(qt, ctype):
    """NaN and infinities in tokens that are seen enter their heads' rows; those between the first tokens and the
    window do not."""
    g = gen(208)
    lens, window, sinks = [700, 64], 90, 5
    table, pages = tables(g, lens, 32)
    c = filled_cache(g, pages, 32, 2, 128, ctype)
    q = randn(g, 2, 8, 128).to(qt)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for j in (5, 300, 609):                          # beside the window and the first ones
        set_token(c, table, 0, j, math.nan, math.inf)
    got = P.ptq1_attn_decode_window(q, c, table, sl, window, sinks)
    for t in (c.k_pages, c.v_pages, c.k_steps, c.v_steps):
        if t is not None and t.dtype != torch.int8:
            t.copy_(torch.where(t.isfinite(), t, 0))
    check_attention(q, c, table, [1, 1], lens, got, WEIGHT_TERM[(qt, ctype)], window, sinks)
    for j in (4, 610, 699):
        was = [t.clone() for t in (c.k_pages, c.v_pages, c.k_steps, c.v_steps) if t is not None]
        for k, v in ((math.nan, None), (None, math.nan), (None, math.inf)):
            set_token(c, table, 0, j, k, v, slice(0, 1))
            odd = P.ptq1_attn_decode_window(q, c, table, sl, window, sinks)
            dims = slice(None) if k is not None or ctype == I8 else slice(3, 4)
            assert not bool(odd[0, :4, dims].isfinite().any())
            keep = torch.ones_like(odd, dtype=torch.bool)
            keep[0, :4, dims] = False
            assert torch.equal(odd[keep], got[keep])
            for t, w in zip([t for t in (c.k_pages, c.v_pages, c.k_steps, c.v_steps) if t is not None], was):
                t.copy_(w)


@pytest.mark.parametrize("qt", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("m", [3, 150])
@pytest.mark.parametrize("order", ["up", "down", "both"])
@pytest.mark.parametrize("sign", [1, -1])
def test_attn_chunk_scores_of_all_sizes(qt, d, m, order, sign):
    """int8 keys whose steps run from 2^-10 to 2^40 along the sequence (or back, or both), queries of one: the reference
    moves from small scores to those whose products are rounded first.  Rows stay within their values, and where one
    score is far ahead it is that token's value."""
    g = gen(220)
    n = 900
    table, pages = tables(g, [n], 32)
    c = filled_cache(g, pages, 32, 1, d, I8)
    c.k_pages.zero_()
    rows, j = table[0].long(), torch.arange(n, device=DEV)
    c.k_pages[rows[j // 32], 0, j % 32, 0] = sign * 100
    e = torch.linspace(-10, 40, n, device=DEV)
    e = {"up": e, "down": e.flip(0), "both": torch.cat([e[::2], e.flip(0)[::2]])[:n]}[order]
    c.k_steps[rows[j // 32], 0, j % 32] = torch.exp2(e)
    q = torch.zeros((m, 2, d), dtype=qt, device=DEV)
    q[..., 0] = 1
    got = P.ptq1_attn_chunk(q, c, table, cumulated([m]), torch.tensor([n], dtype=torch.int32, device=DEV), scale=0.5, max_q=m).double()
    kc, vc = cache_values(c)
    k, v = sequence(c, kc, table, 0, n)[0], sequence(c, vc, table, 0, n)[0]
    assert bool((got.abs() <= v.abs().amax() * 1.01).all())
    counted = 0
    for h in range(2):
        # a small score's error is its own, not that of the largest among the keys: those have no weight where it has
        logits = (0.5 * (q[:, h].double() @ k.T.contiguous())).masked_fill(~window_mask(m, n, 0, 0), -math.inf)
        best = logits.topk(2, 1)
        ok = best.values[:, 0] - best.values[:, 1] > 100 + 64 * U * best.values[:, 0].abs()
        want = v[best.indices[:, 0]]
        tol = half_step(want, qt) + chunk_term(qt, I8, 2 * m) * want.abs() + 4 * U * want.abs()
        assert bool(((got[:, h] - want).abs()[ok] <= tol[ok]).all())
        counted += int(ok.sum())
        small = best.values[:, 0].abs() < 1024
        if bool(small.any()):
            p = torch.softmax(logits[small], 1)
            err = (got[small, h] - p @ v).abs()
            # scores of up to 1024 and products of 2^-24 of them, four times, weights of one term
            bound = (8 * 1024 * U + chunk_term(qt, I8, 2 * m) + 2 * n * U) * (p @ v.abs()) + 2.0 ** -27 * 127 * n * 0.03 * p.amax(1, keepdim=True)
            assert bool((err <= bound + half_step((p @ v).abs() + bound, qt)).all())
            counted += int(small.sum())
    assert counted > 0


@pytest.mark.parametrize("qt", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("m", [3, 40])
@pytest.mark.parametrize("power,sign", [(17, 1), (17, -1), (19, 1), (19, -1)])
def test_attn_chunk_equal_int8_scores_weigh_the_same(qt, d, m, power, sign):
    """int8 keys of one score, that of three halves of 2^power, over two runs of steps of values 1 and -1: whether the
    reference moves in a step or has been where it is, its keys weigh the same.  The score, 101 codes times a step, lies
    near the middle between two fp32 values, so that no rounded reference is the score less a round number.

    Of a score less a reference near it fp32 leaves 2^-19 at most (both differ by less than 64), and a weight is
    rounded by half a step of fp16: the weights of a run are within 2^-11 + 2^-17 of the other's."""
    run = 128 if m <= 16 else 64                   # (few rows: four waves take 32 keys each in turn)
    copies = 260 if m <= 16 else 1                 # so many sequences of few rows that none is cut: they share their pages
    hkv, page = 8, 64
    log2e = np.float32(math.log2(math.e))
    scale = np.float32(math.log(2.0))
    assert scale * log2e == 1.0                    # (scores in units of log2 are code times step)
    grid = 2.0 ** (power - 23)
    step = np.float32(1.5 * 2.0 ** power / 101)
    while not 0.46 <= 101 * float(step) / grid % 1.0 <= 0.49:
        step = np.nextafter(step, np.float32(math.inf))
    before = np.float32(float(step) - sign * 20 / 101)   # a score that is lower by 20
    n = 3 * run + m
    codes, steps = torch.full((n,), 101.0 * sign), torch.full((n,), float(step))
    steps[:run] = float(before)
    codes[3 * run:], steps[3 * run:] = -127, 2.0 ** power / 40   # the queries' own tokens weigh nothing
    k, v = (torch.zeros((n, hkv, d), dtype=I8, device=DEV) for _ in range(2))
    k[..., 0] = codes.to(I8).to(DEV)[:, None]
    v[run:2 * run], v[2 * run:3 * run] = 1, -1
    c, table = placed(k, v, page, I8, 1.0)
    at = torch.arange(n, device=DEV)
    c.k_steps[table[0, at // page].long(), :, at % page] = steps.to(DEV)[:, None]
    q = torch.zeros((copies * m, 2 * hkv, d), device=DEV, dtype=qt)
    q[..., 0] = 1
    sl = torch.full((copies,), n, dtype=torch.int32, device=DEV)
    got = P.ptq1_attn_chunk(q, c, table.expand(copies, -1).contiguous(), cumulated([m] * copies), sl, scale=float(scale), max_q=m)
    assert P.workspace_bytes("attn_chunk", copies, copies * m, m, 2 * hkv, hkv, d, c.n_pages * page, 0, 0) == 0
    assert got.abs().max().item() <= 2.0 ** -11 + 2.0 ** -17, got.abs().max().item()


def time_of(call):
    """Microseconds of one call among ten, the median of seven times."""
    call()
    times = []
    for _ in range(7):
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(10):
            call()
        stop.record()
        stop.synchronize()
        times.append(start.elapsed_time(stop) * 100)
    return sorted(times)[3]


@pytest.mark.parametrize("dtype,hq,hkv,d,page,new,lens,window,sinks", [
    (BF16, 24, 4, 256, 64, [5] * 4, [2001, 2008, 2015, 2022], 0, 0),
    (BF16, 32, 8, 128, 64, [5] * 4, [2001, 2008, 2015, 2022], 300, 4),
    (F16, 8, 2, 64, 256, [16, 9], [9001, 70], 1001, 2),
    (BF16, 32, 8, 128, 256, [100, 70], [161, 130], 0, 0),
    (F16, 16, 4, 64, 128, [100, 70], [161, 130], 0, 0),
    (F16, 24, 4, 256, 128, [100, 70], [161, 130], 0, 0),
    (BF16, 32, 8, 128, 64, [1500, 1300], [9001, 12003], 1001, 4),
    (F16, 24, 4, 256, 64, [700, 300], [5001, 6003], 501, 4),
])
def test_attn_chunk_takes_no_longer_over_what_no_query_sees(dtype, hq, hkv, d, page, new, lens, window, sinks):
    """Slots that no query sees (behind a sequence's end, ahead of its window) hold NaNs and infinities, as memory that
    was never written to may: the same rows in about the same time.  (Looking for them in the rows at the end takes five
    times as long and more.)"""
    q, c, table, cu, sl = chunk_state(300 + d, new, lens, hq, hkv, d, page, dtype, dtype, window, sinks)
    call = lambda: P.ptq1_attn_chunk(q, c, table, cu, sl, window=window, sinks=sinks, max_q=max(new), max_len=max(lens))
    held = c.v_pages.clone()
    assert not bool(held.isfinite().all())
    c.v_pages.copy_(torch.where(held.isfinite(), held, 0))
    want, clean = call(), time_of(call)
    c.v_pages.copy_(held)
    assert torch.equal(call(), want)
    taken = time_of(call)
    assert taken < 2 * clean, f"{taken:.1f} us for {clean:.1f}"


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,lens", [([300, 90], [300, 700]), ([9, 1], [9, 500])])
def test_chunks_and_whole_prompts_agree_row_by_row(dtype, d, new, lens):
    """The chunk call and the prompt call on the rows read back: either is off from 64 bits by its own row's bound and half
    a step, so the two differ by both at most."""
    g = gen(301)
    table, pages = tables(g, lens, 64)
    c = filled_cache(g, pages, 64, 2, d, dtype)
    q = randn(g, sum(new), 8, d).to(dtype)
    cu, cu_k = cumulated(new), cumulated(lens)
    k, v = P.ptq1_kv_read(c, table, cu_k, sum(lens), dtype=dtype)
    got = P.ptq1_attn_chunk(q, c, table, cu, torch.tensor(lens, dtype=torch.int32, device=DEV), max_q=max(new)).double()
    prompt = P.ptq1_attn_prompt(q, k, v, cu, cu_k).double()
    at_q = at_k = 0
    for m, n in zip(new, lens):
        for h in range(8):
            rows, keys = slice(at_q, at_q + m), slice(at_k, at_k + n)
            qq, kk, vv = q[rows, h].double(), k[keys, h // 4].double(), v[keys, h // 4].double()
            mask = window_mask(m, n, 0, 0)
            bounds = [attention_bounds(qq, kk, vv, d ** -0.5, term, mask) for term in
                      (chunk_term(dtype, dtype, 4 * max(new)), CHUNK_TERM[(dtype, dtype)])]
            tol = sum(t + half_step(want.abs() + t, dtype) for want, t in bounds)
            err = (got[rows, h] - prompt[rows, h]).abs()
            assert bool((err <= tol).all()), f"{(err / tol).max().item():.3f} of the bound"
        at_q, at_k = at_q + m, at_k + n


@pytest.mark.parametrize("qt", [BF16, F16])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("m", [3, 40])
@pytest.mark.parametrize("before", [2.0, -1e3, 134.5, 2.0 ** 18 + 6.5, -2.0 ** 18 + 6.5, 9e5])
@pytest.mark.parametrize("power", [24, 31, 42])
@pytest.mark.parametrize("twice", [False, True])
def test_attn_chunk_int8_scores_that_leap(qt, d, m, before, power, twice):
    """int8 keys whose scores leap within one step from `before` at most to 2^power and more (in units of log2), where
    one is far ahead of the others (twice: it comes again two steps later).  Rows are that key's value.  Its score, 127
    times its step, lies in the middle between two fp32 values, and so does what is left of it above (or below) some of
    the references that the scores before have, 7 less than them."""
    g = gen(320 + power)
    run = 128 if m <= 16 else 64
    n, hkv, page = 4 * run + m, 2, 64
    steps = torch.rand(n, generator=g, device=DEV).double()
    steps[:run] = abs(before) / 64 * (0.9 + 0.1 * steps[:run] if before > 0 else 1 + 0.1 * steps[:run])
    steps[run // 2] = abs(before) / 64
    steps[run:] = 2.0 ** power / 127 * (1 + 0.5 * steps[run:])
    first, again = run + 37, 3 * run + 11
    half = 2.0 ** (power - 24)                       # of the score's last place
    lead = int(1.875 * 2.0 ** power / 127 / half) // 4 * 4 + (1 if before > 0 else 3)
    steps[[first, again] if twice else [first]] = half * lead
    assert 127 * lead % 4 == (3 if before > 0 else 1) and lead < 1 << 24
    codes = torch.full((n,), 127, device=DEV)
    codes[:run] = 64 if before > 0 else -64
    codes[4 * run:], steps[4 * run:] = -127, 2.0 ** power / 64   # the queries' own tokens
    k = torch.zeros((n, hkv, d), dtype=I8, device=DEV)
    v = torch.randint(-127, 128, (n, hkv, d), generator=g, device=DEV).to(I8)
    if twice:
        v[again] = v[first]
    k[..., 0] = codes.to(I8)[:, None]
    c, table = placed(k, v, page, I8, 1.0)
    at = torch.arange(n, device=DEV)
    c.k_steps[table[0, at // page].long(), :, at % page] = steps.float()[:, None]
    q = torch.zeros((m, 2 * hkv, d), device=DEV, dtype=qt)
    q[..., 0] = 1
    scale = float(np.float32(math.log(2.0)))         # (log2(e) times it is one in fp32)
    got = P.ptq1_attn_chunk(q, c, table, cumulated([m]), torch.tensor([n], dtype=torch.int32, device=DEV), scale=scale, max_q=m)
    want = v[first].double().repeat_interleave(2, 0)
    # (the others' scores are lower by a fifth: they weigh nothing)
    tol = chunk_term(qt, I8, 2 * m) * want.abs() + 4 * U * want.abs()
    assert bool(((got.double() - want).abs() <= tol + half_step(want.abs() + tol, qt)).all())

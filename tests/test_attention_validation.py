"""Host-only checks of the cache and attention calls: sizes, refusals of the C entry points before anything is
enqueued (fake device addresses, never dereferenced), and of the binding before the C call."""
import ctypes as C
import os
import subprocess

import pytest
import torch

import ternary_weight_ptq1_amd as P

FAKE = 1 << 24
F32, F16, BF16, I8 = 0, 1, 2, 3


def at(i):
    return FAKE * (i + 1)


def cache(dtype=BF16, page=64, heads=2, d=128, pages=8, **other):
    f = dict(k_pages=at(100), v_pages=at(200), k_steps=at(300) if dtype == I8 else None,
             v_steps=at(400) if dtype == I8 else None, n_pages=pages, page_size=page, n_kv_heads=heads, head_dim=d,
             dtype=dtype)
    f.update(other)
    return P._CacheStruct(*(f[n] for n, _ in P._CacheStruct._fields_))


def err(rc):
    return rc, P.lib().ptq1_last_error().decode()


def write(c=None, **other):
    f = dict(q=at(0), qs=1024, k=at(1), ks=256, v=at(2), vs=256, src=F32, n=4, hq=8, positions=at(3), cos_sin=at(4),
             n_pos=100, rot=128, slots=at(5), out=at(6), qt=BF16)
    f.update(other)
    c = cache() if c is None else c
    return err(P.lib().ptq1_kv_write(f["q"], f["qs"], f["k"], f["ks"], f["v"], f["vs"], f["src"], f["n"], f["hq"],
                                     f["positions"], f["cos_sin"], f["n_pos"], f["rot"], f["slots"], f["out"], f["qt"],
                                     C.byref(c) if c else None, None))


def read(c=None, **other):
    f = dict(table=at(0), max_pages=4, cu=at(1), batch=2, rows=100, k=at(2), v=at(3), dt=BF16)
    f.update(other)
    c = cache() if c is None else c
    return err(P.lib().ptq1_kv_read(C.byref(c), f["table"], f["max_pages"], f["cu"], f["batch"], f["rows"], f["k"],
                                    f["v"], f["dt"], None))


def decode(c=None, **other):
    f = dict(q=at(0), qt=BF16, batch=2, hq=8, table=at(1), max_pages=100, lens=at(2), max_len=6400, scale=0.1,
             out=at(3), ws=at(500), wsb=1 << 40)
    f.update(other)
    c = cache() if c is None else c
    return err(P.lib().ptq1_attn_decode(f["q"], f["qt"], f["batch"], f["hq"], C.byref(c), f["table"], f["max_pages"],
                                        f["lens"], f["max_len"], f["scale"], f["out"], f["ws"], f["wsb"], None))


def prompt(**other):
    f = dict(q=at(0), qs=1024, k=at(20), ks=256, v=at(40), vs=256, dt=BF16, cu_q=at(60), cu_k=at(61), batch=2, nq=300,
             nk=300, max_q=200, max_k=200, hq=8, hkv=2, d=128, causal=1, scale=0.1, out=at(70), ws=at(500),
             wsb=1 << 40)
    f.update(other)
    return err(P.lib().ptq1_attn_prompt(*(f[n] for n in ("q", "qs", "k", "ks", "v", "vs", "dt", "cu_q", "cu_k", "batch",
                                                         "nq", "nk", "max_q", "max_k", "hq", "hkv", "d", "causal",
                                                         "scale", "out", "ws", "wsb")), None))


NULL, SHAPE, ALIGN, OVERFLOW, UNSUPPORTED, WORKSPACE, ALIAS = range(1, 8)


@pytest.mark.parametrize("call", [write, read, decode])
@pytest.mark.parametrize("other,status,word", [
    (dict(dtype=F32), UNSUPPORTED, "cache dtype"),
    (dict(page=48), UNSUPPORTED, "page_size"),
    (dict(page=8), UNSUPPORTED, "page_size"),
    (dict(page=512), UNSUPPORTED, "page_size"),
    (dict(d=96), UNSUPPORTED, "head_dim"),
    (dict(heads=0), SHAPE, "n_kv_heads"),
    (dict(pages=0), SHAPE, "n_pages"),
    (dict(pages=1 << 31), SHAPE, "n_pages"),
    (dict(k_pages=None), NULL, "k_pages"),
    (dict(v_pages=at(200) + 8), ALIGN, "v_pages"),
    (dict(dtype=I8, v_steps=None), NULL, "v_steps"),
])
def test_cache_refused(call, other, status, word):
    rc, msg = call(cache(**other))
    assert rc == status and word in msg


@pytest.mark.parametrize("other,status,word", [
    (dict(n=-1), SHAPE, "n_tokens"),
    (dict(n=(1 << 24) + 1), UNSUPPORTED, "n_tokens"),
    (dict(n=1 << 23), UNSUPPORTED, "n_tokens * heads"),
    (dict(hq=-1), SHAPE, "n_q_heads"),
    (dict(src=I8), UNSUPPORTED, "src_dtype"),
    (dict(qt=I8), UNSUPPORTED, "q_dtype"),
    (dict(rot=12), SHAPE, "rot_dim"),
    (dict(rot=136), SHAPE, "rot_dim"),
    (dict(q=None), NULL, "q is"),
    (dict(k=None), NULL, "k is"),
    (dict(slots=None), NULL, "slots"),
    (dict(positions=None), NULL, "positions"),
    (dict(cos_sin=None), NULL, "cos_sin"),
    (dict(out=None), NULL, "q_out"),
    (dict(qs=1020), SHAPE, "q: row stride"),
    (dict(ks=257), ALIGN, "k: row stride"),
    (dict(v=at(2) + 4), ALIGN, "v is not"),
    (dict(out=at(0) + 4096), ALIAS, "q_out overlaps q"),
    (dict(out=at(100) + 4096), ALIAS, "q_out overlaps the cache"),
    (dict(out=at(5)), ALIAS, "slots"),
    (dict(k=at(200)), ALIAS, "the cache overlaps"),
    (dict(cos_sin=at(100)), ALIAS, "cos_sin"),
    (dict(n_pos=-1), SHAPE, "n_positions"),
    (dict(n_pos=1 << 60), OVERFLOW, "cos_sin"),
    (dict(ks=1 << 61), OVERFLOW, "k: size"),
])
def test_write_refused(other, status, word):
    rc, msg = write(**other)
    assert rc == status and word in msg, msg


def test_write_cache_arrays_overlap():
    rc, msg = write(cache(v_pages=at(100) + 1024))
    assert rc == ALIAS and "overlap one another" in msg
    rc, msg = write(cache(dtype=I8, k_steps=at(200)))
    assert rc == ALIAS
    assert write(n=0, q=None, k=None, v=None, slots=None, out=None)[0] == 0


@pytest.mark.parametrize("other,status,word", [
    (dict(batch=-1), SHAPE, "batch"),
    (dict(max_pages=-1), SHAPE, "max_pages"),
    (dict(rows=-5), SHAPE, "n_rows"),
    (dict(rows=1 << 31), UNSUPPORTED, "n_rows"),
    (dict(batch=1 << 24), UNSUPPORTED, "tiles"),
    (dict(dt=I8), UNSUPPORTED, "out_dtype"),
    (dict(table=None), NULL, "block_table"),
    (dict(cu=None), NULL, "cu_seqlens"),
    (dict(cu=at(1) + 2), ALIGN, "cu_seqlens"),
    (dict(k=None), NULL, "k_out"),
    (dict(v=at(3) + 8), ALIGN, "v_out"),
    (dict(v=at(2) + 1024), ALIAS, "k_out overlaps v_out"),
    (dict(v=at(200)), ALIAS, "overlaps the cache"),
    (dict(k=at(0)), ALIAS, "block_table"),
])
def test_read_refused(other, status, word):
    rc, msg = read(**other)
    assert rc == status and word in msg, msg


def test_read_nothing():
    assert read(batch=0)[0] == 0 and read(rows=0, k=None, v=None)[0] == 0


@pytest.mark.parametrize("other,status,word", [
    (dict(batch=-1), SHAPE, "batch"),
    (dict(batch=65536), UNSUPPORTED, "batch"),
    (dict(hq=7), SHAPE, "multiple"),
    (dict(hq=0), SHAPE, "n_q_heads"),
    (dict(scale=0.0), SHAPE, "scale"),
    (dict(scale=-1.0), SHAPE, "scale"),
    (dict(scale=float("nan")), SHAPE, "scale"),
    (dict(scale=float("inf")), SHAPE, "scale"),
    (dict(scale=1e38), SHAPE, "scale"),
    (dict(max_len=6401), SHAPE, "max_len"),
    (dict(max_len=-1), SHAPE, "max_len"),
    (dict(max_pages=1 << 20, max_len=(1 << 22) + 1), UNSUPPORTED, "max_len"),
    (dict(qt=F16), UNSUPPORTED, "F16 over a BF16 cache"),
    (dict(qt=I8), UNSUPPORTED, "q_dtype"),
    (dict(q=None), NULL, "q is"),
    (dict(q=at(0) + 8), ALIGN, "q is"),
    (dict(lens=None), NULL, "seq_lens"),
    (dict(table=None), NULL, "block_table"),
    (dict(ws=None), WORKSPACE, "ws is NULL"),
    (dict(wsb=16), WORKSPACE, "ws_bytes"),
    (dict(ws=at(500) + 16), ALIGN, "ws"),
    (dict(out=at(0)), ALIAS, "out overlaps q"),
    (dict(out=at(100)), ALIAS, "cache"),
    (dict(out=at(2)), ALIAS, "seq_lens"),
    (dict(ws=at(100)), ALIAS, "ws"),
])
def test_decode_refused(other, status, word):
    rc, msg = decode(**other)
    assert rc == status and word in msg, msg


def test_decode_types_over_each_cache():
    for ctype in (F16, BF16, I8):
        for qt in (F32, F16, BF16):
            rc, msg = decode(cache(ctype), qt=qt, ws=None)
            if ctype == I8 or qt in (F32, ctype):
                assert rc == WORKSPACE  # everything else is in order
            else:
                assert rc == UNSUPPORTED and "q_dtype" in msg
    assert decode(batch=0)[0] == 0


def test_decode_grid_limit():
    """Every launch that is accepted has fewer than 2^24 workgroups of 256 threads (a grid's threads fit 32 bits)."""
    size = P.lib().ptq1_attn_decode_workspace_bytes
    # (out = q: what passes the sizes' checks is refused before a launch)
    for heads, hq, d, batch in ((1024, 1024, 64, 16384), (1, 65536, 64, 4096), (1000, 64000, 128, 65535), (257, 257, 64, 65281)):
        rc, msg = decode(cache(heads=heads, d=d), hq=hq, batch=batch, out=at(0))
        assert rc == UNSUPPORTED and "groups of 16 query heads" in msg, msg
        assert size(batch, hq, heads, d, 6400) == 0
    for heads, hq, d, batch in ((1024, 1024, 64, 16368), (1, 65536, 64, 4092), (256, 256, 64, 65472)):
        rc, msg = decode(cache(heads=heads, d=d), hq=hq, batch=batch, out=at(0))
        assert rc == ALIAS, msg
    # what a refused size would be launched with is what the limit is for: pieces of the plan, as the workspace tells
    for heads, hq, d, batch in ((1024, 1024, 64, 1), (5, 65535, 64, 3), (1, 16, 128, 60000), (1024, 65536, 256, 100)):
        groups = heads * -(-(hq // heads) // 16)
        pieces = size(batch, hq, heads, d, 1 << 22) // (hq * (d + 2) * 4)
        assert pieces * groups <= batch * groups + (1 << 14)


def test_decode_workspace():
    size = P.lib().ptq1_attn_decode_workspace_bytes
    assert size(1, 8, 2, 128, 256) == 0          # one step: nothing to join
    need = size(2, 8, 2, 128, 6400)
    assert need > 0 and need % 256 == 0
    assert decode(wsb=need - 1)[0] == WORKSPACE
    # bounded by the GPU, not by the lengths: 512 workgroups and one more piece for every sequence
    assert size(1, 40, 8, 128, 1 << 22) <= (512 // 8 + 1) * 40 * (128 + 2) * 4 + 256
    assert size(4, 40, 8, 128, 1 << 22) <= (512 // 8 + 4) * 40 * (128 + 2) * 4 + 256
    for bad in ((-1, 8, 2, 128, 100), (1, 7, 2, 128, 100), (1, 8, 2, 96, 100), (1, 8, 2, 128, -1)):
        assert size(*bad) == 0


@pytest.mark.parametrize("other,status,word", [
    (dict(dt=F32), UNSUPPORTED, "dtype"),
    (dict(d=80), UNSUPPORTED, "head_dim"),
    (dict(hq=9), SHAPE, "multiple"),
    (dict(hkv=0), SHAPE, "n_kv_heads"),
    (dict(scale=0.0), SHAPE, "scale"),
    (dict(batch=-1), SHAPE, "batch"),
    (dict(nq=-1), SHAPE, "n_q_rows"),
    (dict(max_k=-1), SHAPE, "max_k"),
    (dict(nq=1 << 31), UNSUPPORTED, "rows of one kv head"),
    (dict(nq=1 << 30, max_q=1 << 30), UNSUPPORTED, "rows of one kv head"),
    (dict(nq=1 << 28, hq=8, hkv=8), UNSUPPORTED, "tiles"),
    (dict(ks=1 << 25), UNSUPPORTED, "k_stride"),
    (dict(q=None), NULL, "q is"),
    (dict(v=None), NULL, "v is"),
    (dict(cu_k=None), NULL, "cu_k"),
    (dict(out=None), NULL, "out"),
    (dict(k=at(20) + 8), ALIGN, "k is"),
    (dict(qs=1028), ALIGN, "q: row stride"),
    (dict(vs=128), SHAPE, "v: row stride"),
    (dict(out=at(0)), ALIAS, "out overlaps q"),
    (dict(out=at(61)), ALIAS, "cu_q or cu_k"),
])
def test_prompt_refused(other, status, word):
    rc, msg = prompt(**other)
    assert rc == status and word in msg, msg


def test_prompt_workspace():
    size = P.lib().ptq1_attn_prompt_workspace_bytes
    assert size(1, 8192, 8192, 32, 8, 128) == 0      # the query rows fill the GPU
    need = size(1, 16, 32768, 8, 2, 128)             # few rows over many keys
    assert need > 0 and need % 256 == 0
    few = dict(batch=1, nq=16, nk=32768, max_q=16, max_k=32768)
    assert prompt(**few, ws=None)[0] == WORKSPACE
    assert prompt(**few, wsb=need - 1)[0] == WORKSPACE
    assert prompt(**few, ws=at(500) + 128)[0] == ALIGN
    assert prompt(**few, ws=at(20))[0] == ALIAS
    for bad in ((-1, 16, 100, 8, 2, 128), (1, 16, 100, 8, 3, 128), (1, 16, 100, 8, 2, 100), (1, -1, 100, 8, 2, 128)):
        assert size(*bad) == 0
    assert prompt(batch=0)[0] == 0 and prompt(nq=0)[0] == 0


# ------------------------------------------------------------- the binding ----

@pytest.fixture
def host_ok(monkeypatch):
    """Host tensors pass for device tensors; a compute entry point that is reached fails the test."""
    real = P.lib()

    class Guard:
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return getattr(real, name)

            def refuse(*a):
                raise AssertionError(f"{name} reached with invalid arguments")
            return refuse

    monkeypatch.setattr(P, "_on_device", lambda t: True)
    monkeypatch.setattr(P, "lib", lambda: Guard())


def kv(dtype=torch.bfloat16, heads=2, d=128):
    return P.ptq1_kv_cache(4, 16, heads, d, dtype, "cpu")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_host_tensors_refused():
    with pytest.raises(ValueError, match="device tensor"):
        P.KvCache(z(4, 2, 16, 128), z(4, 2, 128, 16))
    with pytest.raises(ValueError, match="device tensor"):
        P.ptq1_attn_prompt(z(4, 2, 64), z(4, 2, 64), z(4, 2, 64), i32(0, 4), i32(0, 4))


def test_binding_cache(host_ok):
    with pytest.raises(ValueError, match="k_pages must be"):
        P.KvCache(z(4, 2, 16, 128, dtype=torch.float32), z(4, 2, 128, 16, dtype=torch.float32))
    with pytest.raises(ValueError, match="v_pages must be"):
        P.KvCache(z(4, 2, 16, 128), z(4, 2, 16, 128))
    with pytest.raises(ValueError, match="contiguous"):
        P.KvCache(z(4, 2, 128, 16).transpose(2, 3), z(4, 2, 128, 16))
    with pytest.raises(TypeError, match="k_steps"):
        P.KvCache(z(4, 2, 16, 128, dtype=torch.int8), z(4, 2, 128, 16, dtype=torch.int8))
    with pytest.raises(ValueError, match="v_steps must be"):
        P.KvCache(z(4, 2, 16, 128, dtype=torch.int8), z(4, 2, 128, 16, dtype=torch.int8),
                  z(4, 2, 16, dtype=torch.float32), z(4, 16, 2, dtype=torch.float32))
    with pytest.raises(ValueError, match="int8 cache"):
        P.KvCache(z(4, 2, 16, 128), z(4, 2, 128, 16), z(4, 2, 16, dtype=torch.float32))
    with pytest.raises(ValueError, match="dtype"):
        P.ptq1_kv_cache(4, 16, 2, 128, torch.float32, "cpu")
    c = kv()
    with pytest.raises(AttributeError, match="k_pages cannot be set"):
        c.k_pages = c.k_pages.clone()


def test_binding_write(host_ok):
    c = kv()
    q, k, s = z(3, 8, 128), z(3, 2, 128), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(TypeError, match="KvCache"):
        P.ptq1_kv_write(q, k, k, s, c.k_pages)
    for bad, match in (((q, z(3, 4, 128), k, s, c), "k has 4 heads"), ((q, k, z(2, 2, 128), s, c), "v must be"),
                       ((z(2, 8, 128), k, k, s, c), "q must be"), ((q, k, k, s[:2], c), "slots has"),
                       ((q, k, k, s.int(), c), "slots must be"), ((q.half(), k, k, s, c), "q must be"),
                       ((q, z(3, 128, 2).transpose(1, 2), k, s, c), "heads of a row"),
                       ((q, z(1, 2, 128).expand(3, 2, 128), k, s, c), "rows overlap"),
                       ((z(3, 1024), k, k, s, c), "q must be")):
        with pytest.raises(ValueError, match=match):
            P.ptq1_kv_write(*bad)
    with pytest.raises(ValueError, match="needs positions"):
        P.ptq1_kv_write(q, k, k, s, c, cos_sin=z(9, 64, dtype=torch.float32))
    with pytest.raises(ValueError, match="positions has"):
        P.ptq1_kv_write(q, k, k, s, c, positions=i32(1, 2), cos_sin=z(9, 64, dtype=torch.float32))
    with pytest.raises(ValueError, match="cos_sin must be"):
        P.ptq1_kv_write(q, k, k, s, c, positions=i32(1, 2, 3), cos_sin=z(9, 64))
    with pytest.raises(ValueError, match="q_dtype"):
        P.ptq1_kv_write(q, k, k, s, c, q_dtype=torch.int8)
    with pytest.raises(ValueError, match="out has"):
        P.ptq1_kv_write(q, k, k, s, c, out=z(2, 8, 128))
    with pytest.raises(ValueError, match="out needs q"):
        P.ptq1_kv_write(None, k, k, s, c, out=z(3, 8, 128))


def test_binding_read(host_ok):
    c, t = kv(), torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="block_table must be"):
        P.ptq1_kv_read(c, t, i32(0, 3), 3)
    with pytest.raises(ValueError, match="block_table must be"):
        P.ptq1_kv_read(c, t.long(), i32(0, 3, 4), 4)
    with pytest.raises(ValueError, match="batch \\+ 1"):
        P.ptq1_kv_read(c, t, i32(), 4)
    with pytest.raises(ValueError, match="n_rows"):
        P.ptq1_kv_read(c, t, i32(0, 3, 4), -4)
    with pytest.raises(ValueError, match="dtype"):
        P.ptq1_kv_read(c, t, i32(0, 3, 4), 4, dtype=torch.int8)
    with pytest.raises(ValueError, match="v_out has"):
        P.ptq1_kv_read(c, t, i32(0, 3, 4), 4, out=(z(4, 2, 128), z(3, 2, 128)))


def test_binding_decode(host_ok):
    c, t, q = kv(), torch.zeros((2, 3), dtype=torch.int32), z(2, 8, 128)
    with pytest.raises(ValueError, match="q must be \\[batch"):
        P.ptq1_attn_decode(z(2, 8, 64), c, t, i32(1, 2))
    with pytest.raises(ValueError, match="contiguous"):
        P.ptq1_attn_decode(z(8, 2, 128).transpose(0, 1), c, t, i32(1, 2))
    with pytest.raises(ValueError, match="seq_lens has"):
        P.ptq1_attn_decode(q, c, t, i32(1))
    with pytest.raises(ValueError, match="seq_lens must be"):
        P.ptq1_attn_decode(q, c, t, i32(1, 2).long())
    with pytest.raises(ValueError, match="out must be"):
        P.ptq1_attn_decode(q, c, t, i32(1, 2), out=z(2, 8, 128, dtype=torch.float32))
    long = torch.zeros((2, 300), dtype=torch.int32)
    with pytest.raises(ValueError, match="ws has"):
        P.ptq1_attn_decode(q, c, long, i32(1, 2), ws=z(100, dtype=torch.uint8))


def test_binding_prompt(host_ok):
    q, k, cu = z(9, 8, 128), z(9, 2, 128), i32(0, 4, 9)
    for bad, match in (((q.float(), k, k, cu, cu), "q must be"), ((q, k.half(), k, cu, cu), "k must be"),
                       ((q, k, z(8, 2, 128), cu, cu), "k and v must"), ((q, z(9, 2, 64), z(9, 2, 64), cu, cu), "k and v must"),
                       ((q, k, k, cu, i32(0, 9)), "cu_k has"), ((q, k, k, cu.long(), cu), "cu_q must be"),
                       ((q, k, k, i32(), cu), "batch \\+ 1")):
        with pytest.raises(ValueError, match=match):
            P.ptq1_attn_prompt(*bad)
    with pytest.raises(ValueError, match="out has"):
        P.ptq1_attn_prompt(q, k, k, cu, cu, out=z(8, 8, 128))


def test_prompt_workspace_stays_bounded():
    """A loose bound on the keys must not ask for more than 256 MB."""
    size = P.lib().ptq1_attn_prompt_workspace_bytes
    for batch in (1, 3, 64, 500, 4096):
        for rows in (1, 70, 1000, 20000, 300000):
            for max_k in (300, 5000, 100000, 1 << 24):
                for hq, hkv, d in ((8, 8, 64), (40, 8, 128), (64, 1, 256)):
                    assert size(batch, rows, max_k, hq, hkv, d) <= (1 << 28) + 256


def test_decode_pieces_cover_every_sequence(tmp_path):
    """The split's arithmetic as the kernels have it, at its limits (up to 65535 sequences of 2^22 tokens, two pieces
    wanted, where steps times tokens of a piece would pass 32 bits): the pieces are as many as the host has room for,
    and lie end to end."""
    source = tmp_path / "split.cpp"
    source.write_text(r"""
#include <cstdio>
#include "ptq1_split.h"
int main()
{
    const int64_t batches[] = {1, 2, 3, 64, 257, 1024, 16384, 65535}, shares[] = {1, 2, 13, 64, 512};
    const int lens[] = {-1, 0, 1, 255, 256, 257, 5000, 131071, (1 << 22) - 1, 1 << 22, (1 << 22) + 1};
    const int64_t max_len = 1 << 22;
    for (int64_t batch : batches)
        for (int64_t share : shares)
            for (int most : lens) {      // every sequence but two has this length
                int64_t total = 0;
                for (int64_t i = 0; i < batch; ++i) total += ptq1::decode_steps(i < 2 ? lens[3 + i] : most, max_len);
                const int64_t want = ptq1::wanted_pieces(batch, share);
                const int per = ptq1::steps_per_piece(static_cast<int>(total), want);
                if (per < 1 || per > ptq1::kMaxSteps) return 1;
                int64_t pieces = 0;
                for (int64_t i = 0; i < batch; ++i) {
                    const int len = i < 2 ? lens[3 + i] : most, steps = ptq1::decode_steps(len, max_len);
                    const int n = ptq1::pieces_of(steps, per);
                    pieces += n;
                    int at = 0;
                    for (int k = 0; k < n; ++k) {
                        const ptq1::PieceTokens p = ptq1::piece_tokens(k, per, len);
                        if (p.begin != at) return 2;
                        at = p.end;
                        if (len >= 1 && len <= max_len && p.end <= p.begin) return 3;
                    }
                    if (len >= 0 && len <= max_len && at != len) return 4;
                }
                if (pieces > want + batch) return 5;
            }
    std::puts("covered");
    return 0;
}
""")
    program = tmp_path / "split"
    csrc = os.path.join(os.path.dirname(P.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-I", csrc, str(source), "-o", str(program)], check=True)
    done = subprocess.run([str(program)], capture_output=True, text=True)
    assert done.returncode == 0 and done.stdout == "covered\n", done.returncode


class Streams:
    """A stand-in for torch's current stream: which stream's memory every allocation of a call comes from, and which
    streams its results are tied to."""

    class Stream:
        def __init__(self, name, handle):
            self.name, self.cuda_stream, self.device = name, handle, torch.device("cpu")

    def __init__(self, monkeypatch):
        import contextlib

        self.main, self.side = self.Stream("main", 1), self.Stream("side", 2)
        self.current, self.allocated, self.tied = self.main, [], []

        @contextlib.contextmanager
        def under(s):
            before, self.current = self.current, s
            yield
            self.current = before

        for name in ("empty", "empty_like", "empty_strided"):
            real = getattr(torch, name)

            def make(*a, _real=real, **kw):
                self.allocated.append(self.current.name)
                return _real(*a, **kw)

            monkeypatch.setattr(torch, name, make)
        monkeypatch.setattr(torch.cuda, "stream", under)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.tied.append(s.name))
        monkeypatch.setattr(P, "_on_device", lambda t: True)
        real = P.lib()

        class Launched:
            def __getattr__(_, name):
                return getattr(real, name) if name.endswith("_bytes") else lambda *a: 0

        monkeypatch.setattr(P, "lib", lambda: Launched())


def side_calls():
    """(call, whether it allocates without out) of each cache and attention call, over host tensors."""
    c, t = kv(), torch.zeros((2, 400), dtype=torch.int32)
    q, k, s = z(3, 8, 128), z(3, 2, 128), torch.zeros(3, dtype=torch.int64)
    return {"kv_write": lambda **o: P.ptq1_kv_write(q, k, k, s, c, **o),
            "kv_read": lambda **o: P.ptq1_kv_read(c, t, i32(0, 2, 4), 4, **o),
            "attn_decode": lambda **o: P.ptq1_attn_decode(q[:2], c, t, i32(1, 2), **o),
            "attn_prompt": lambda **o: P.ptq1_attn_prompt(z(16, 8, 128), z(9000, 2, 128), z(9000, 2, 128), i32(0, 16),
                                                          i32(0, 9000), **o)}


@pytest.mark.parametrize("name", ["kv_write", "kv_read", "attn_decode", "attn_prompt"])
def test_side_stream_allocates_its_own_memory(monkeypatch, name):
    """Scratch and results of a call on a stream of the caller's come from that stream's memory (the current stream's
    freed blocks may have pending work of its own), and the results are tied to the current stream, which uses them."""
    streams = Streams(monkeypatch)
    call = side_calls()[name]
    streams.allocated.clear()
    call(stream=streams.side)
    assert streams.allocated and set(streams.allocated) == {"side"}
    assert streams.tied and set(streams.tied) == {"main"} and streams.current is streams.main
    # on the current stream, given or not: its own memory, nothing to tie
    for stream in (None, streams.main):
        streams.allocated.clear(), streams.tied.clear()
        call(stream=stream)
        assert set(streams.allocated) == {"main"} and not streams.tied


def test_stream_of_another_device_refused(monkeypatch):
    streams = Streams(monkeypatch)
    streams.side.device = torch.device("cuda:1")
    for call in side_calls().values():
        with pytest.raises(ValueError, match="the stream is on cuda:1"):
            call(stream=streams.side)


def test_side_stream_of_the_projections(monkeypatch):
    """The calls around the attention (codec, rotation, projections, feed-forward block) alike."""
    streams = Streams(monkeypatch)
    n = k = 1024
    f32 = dict(dtype=torch.float32)
    x, row, signs = z(2, k, **f32), z(k, **f32), z(1024, **f32)
    w, w2 = (torch.zeros(size(n, k), dtype=torch.uint8) for size in (P.ptq1_tiled_bytes, P.pq2_tiled_bytes))
    blocks, blocks2 = (torch.zeros(size(n, k), dtype=torch.uint8) for size in (P.ptq1_packed_bytes, P.pq2_packed_bytes))
    trits, scales = torch.zeros((n, k), dtype=torch.int8), torch.zeros((n, k // 128), dtype=torch.int16)
    calls = [(P.ptq1_pack, trits, scales), (P.ptq1_tile, blocks, n, k), (P.ptq1_dequant, blocks, n, k),
             (P.pq2_pack, trits, scales), (P.pq2_tile, blocks2, n, k), (P.pq2_dequant, blocks2, n, k),
             (P.hadamard_rotate, x, signs), (P.hadamard_unrotate_rows, x, signs), (P.ptq1_swiglu, row, row),
             (P.ptq1_matvec, w, n, k, row, signs), (P.ptq1_matvec_float_peel, w, n, k, row, signs),
             (P.pq2_matvec, w2, n, k, row, signs), (P.ptq1_matvec_w2a8, w, n, k, row),
             (P.ptq1_gate_up, w, w, n, k, row, signs), (P.ptq1_gemm, w, n, k, x, signs), (P.pq2_gemm, w2, n, k, x, signs),
             (P.ptq1_gemm_w2a8, w, n, k, x), (P.ptq1_ffn_block, x, w, w, w, signs, k, n),
             (P.pq2_ffn_block, x, w2, w2, w2, signs, k, n), (P.ptq1_ffn_block_noalloc, x, w, w, w, signs, k, n)]
    for call, *args in calls:
        streams.allocated.clear(), streams.tied.clear()
        call(*args, stream=streams.side)
        assert streams.allocated and set(streams.allocated) == {"side"}, call.__name__
        assert streams.tied and set(streams.tied) == {"main"} and streams.current is streams.main, call.__name__
        streams.allocated.clear(), streams.tied.clear()
        call(*args)
        assert set(streams.allocated) == {"main"} and not streams.tied, call.__name__

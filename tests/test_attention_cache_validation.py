"""Host-only checks of the calls with norms, windows and chunks: sizes, refusals of the C entry points before anything is
enqueued (fake device addresses, never dereferenced), and of the binding before the C call."""
import ctypes as C
import os
import subprocess

import pytest
import torch

import ternary_weight_ptq1_amd as P
from test_attention_validation import (ALIAS, ALIGN, BF16, F16, F32, I8, NULL, OVERFLOW, SHAPE, UNSUPPORTED, WORKSPACE,
                                       Streams, at, cache, err, host_ok, i32, kv, z)  # noqa: F401


def norm(c=None, **other):
    f = dict(q=at(0), qs=1024, k=at(1), ks=256, v=at(2), vs=256, src=F32, n=4, hq=8, qg=at(7), kg=at(8), eps=1e-6,
             positions=at(3), cos_sin=at(4), n_pos=100, rot=128, slots=at(5), out=at(6), qt=BF16)
    f.update(other)
    c = cache() if c is None else c
    return err(P.lib().ptq1_kv_write_norm(f["q"], f["qs"], f["k"], f["ks"], f["v"], f["vs"], f["src"], f["n"], f["hq"],
                                          f["qg"], f["kg"], f["eps"], f["positions"], f["cos_sin"], f["n_pos"], f["rot"],
                                          f["slots"], f["out"], f["qt"], C.byref(c) if c else None, None))


def window(c=None, **other):
    f = dict(q=at(0), qt=BF16, batch=2, hq=8, table=at(1), max_pages=100, lens=at(2), max_len=6400, window=5000, sinks=4,
             scale=0.1, out=at(3), ws=at(500), wsb=1 << 40)
    f.update(other)
    c = cache() if c is None else c
    return err(P.lib().ptq1_attn_decode_window(f["q"], f["qt"], f["batch"], f["hq"], C.byref(c), f["table"],
                                               f["max_pages"], f["lens"], f["max_len"], f["window"], f["sinks"],
                                               f["scale"], f["out"], f["ws"], f["wsb"], None))


@pytest.mark.parametrize("call", [norm, window])
@pytest.mark.parametrize("other,status,word", [
    (dict(dtype=F32), UNSUPPORTED, "cache dtype"),
    (dict(page=48), UNSUPPORTED, "page_size"),
    (dict(page=512), UNSUPPORTED, "page_size"),
    (dict(d=96), UNSUPPORTED, "head_dim"),
    (dict(heads=0), SHAPE, "n_kv_heads"),
    (dict(pages=0), SHAPE, "n_pages"),
    (dict(k_pages=None), NULL, "k_pages"),
    (dict(v_pages=at(200) + 8), ALIGN, "v_pages"),
    (dict(dtype=I8, v_steps=None), NULL, "v_steps"),
])
def test_cache_refused(call, other, status, word):
    rc, msg = call(cache(**other))
    assert rc == status and word in msg


@pytest.mark.parametrize("other,status,word", [
    (dict(n=-1), SHAPE, "n_tokens"),
    (dict(n=1 << 23), UNSUPPORTED, "n_tokens * heads"),
    (dict(src=I8), UNSUPPORTED, "src_dtype"),
    (dict(qt=I8), UNSUPPORTED, "q_dtype"),
    (dict(rot=12), SHAPE, "rot_dim"),
    (dict(eps=0.0), SHAPE, "eps"),
    (dict(eps=-1e-6), SHAPE, "eps"),
    (dict(eps=2.0 ** -101), SHAPE, "eps"),
    (dict(eps=2.0 ** 101), SHAPE, "eps"),
    (dict(eps=float("nan")), SHAPE, "eps"),
    (dict(eps=float("inf")), SHAPE, "eps"),
    (dict(q=None), NULL, "q is"),
    (dict(slots=None), NULL, "slots"),
    (dict(qg=at(7) + 4), ALIGN, "q_gain"),
    (dict(kg=at(8) + 8), ALIGN, "k_gain"),
    (dict(out=at(7)), ALIAS, "q_gain"),
    (dict(out=at(8)), ALIAS, "k_gain"),
    (dict(kg=at(100) + 256), ALIAS, "k_gain"),
    (dict(qs=1020), SHAPE, "q: row stride"),
    (dict(out=at(0) + 4096), ALIAS, "q_out overlaps q"),
    (dict(out=at(100) + 4096), ALIAS, "q_out overlaps the cache"),
    (dict(n_pos=1 << 60), OVERFLOW, "cos_sin"),
])
def test_write_norm_refused(other, status, word):
    rc, msg = norm(**other)
    assert rc == status and word in msg, msg


def test_write_norm_without_anything_to_do():
    assert norm(n=0, q=None, k=None, v=None, slots=None, out=None, qg=None, kg=None)[0] == 0
    rc, msg = norm(cache(v_pages=at(100) + 1024))
    assert rc == ALIAS and "overlap one another" in msg
    # gains that the call does not read are not looked at
    assert norm(n=0, hq=0, qg=at(7) + 4)[0] == 0


@pytest.mark.parametrize("other,status,word", [
    (dict(window=0), SHAPE, "window"),
    (dict(window=-5), SHAPE, "window"),
    (dict(sinks=-1), SHAPE, "sinks"),
    (dict(batch=-1), SHAPE, "batch"),
    (dict(batch=1 << 17), UNSUPPORTED, "batch"),
    (dict(hq=7), SHAPE, "n_q_heads"),
    (dict(scale=0.0), SHAPE, "scale"),
    (dict(max_len=6401), SHAPE, "max_len"),
    (dict(qt=F16), UNSUPPORTED, "q_dtype"),
    (dict(q=None), NULL, "q is"),
    (dict(table=None), NULL, "block_table"),
    (dict(lens=at(2) + 2), ALIGN, "seq_lens"),
    (dict(out=at(0)), ALIAS, "out overlaps q"),
    (dict(out=at(100)), ALIAS, "out overlaps the cache"),
    (dict(wsb=16), WORKSPACE, "ptq1_attn_decode_window"),
    (dict(ws=None), WORKSPACE, "ptq1_attn_decode_window"),
    (dict(ws=at(0)), ALIAS, "ws overlaps"),
])
def test_window_refused(other, status, word):
    rc, msg = window(**other)
    assert rc == status and word in msg, msg


def test_window_workspace():
    """The work is laid out for the tokens that are read: a window smaller than the lengths takes less."""
    size = P.workspace_bytes
    full = size("attn_decode", 4, 32, 8, 128, 100000)
    assert size("attn_decode_window", 4, 32, 8, 128, 100000, 100000, 0) == full
    assert size("attn_decode_window", 4, 32, 8, 128, 100000, 1 << 60, 1 << 60) == full
    assert 0 < size("attn_decode_window", 4, 32, 8, 128, 100000, 2000, 4) < full
    assert size("attn_decode_window", 4, 32, 8, 128, 100000, 100, 4) == 0
    for bad in ((4, 32, 8, 128, 1000, 0, 0), (4, 32, 8, 128, 1000, 5, -1), (-1, 32, 8, 128, 1000, 5, 0)):
        assert size("attn_decode_window", *bad) == 0
    assert window(batch=0, ws=None, wsb=0)[0] == 0


def test_window_arithmetic(tmp_path):
    """window_of (ptq1_split.h) over lengths, windows and sinks: the numbers are those of the tokens that are seen, each
    once and in order, with what is left of two runs of 16 in the hole, and no more of them than the bound."""
    src = tmp_path / "w.cpp"
    src.write_text("""
#include <cstdio>
#include "ptq1_split.h"
using namespace ptq1;
int bad(const char *what, int n, int w, int s) { std::printf("%s: %d %d %d\\n", what, n, w, s); return 1; }
int main()
{
    const int sizes[] = {0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 64, 100, 255, 256, 300};
    for (int n = 1; n < 300; ++n)
        for (int w : sizes)
            for (int s : sizes) {
                if (w == 0) continue;
                const WindowTokens t = window_of(n, w, s);
                if (t.gap % 16 || t.sunk % 16 || t.gap < 0 || t.tokens > window_bound(n, w, s)) return bad("sizes", n, w, s);
                int seen = 0, last = -1;
                for (int v = 0; v < t.tokens; ++v) {
                    const int tok = v >= t.sunk ? v + t.gap : v;
                    if (tok <= last || tok >= n) return bad("order", n, w, s);
                    last = tok;
                    const bool is = tok >= n - w || tok < s, hole = v >= t.hole && v < t.hole_end;
                    if (is == hole) return bad("hole", n, w, s);
                    seen += is;
                    if (hole) {  // its run of 16 holds a token that is seen: its page is there
                        bool near = false;
                        for (int j = tok & ~15; j < (tok & ~15) + 16; ++j) near |= j < n && (j >= n - w || j < s);
                        if (!near) return bad("page", n, w, s);
                    }
                }
                int want = 0;
                for (int j = 0; j < n; ++j) want += j >= n - w || j < s;
                if (seen != want) return bad("count", n, w, s);
            }
    const int big = 1 << 22;
    const WindowTokens t = window_of(big, big + 1, big);
    return t.tokens == big && t.gap == 0 ? 0 : bad("big", big, big + 1, big);
}
""")
    exe = tmp_path / "w"
    csrc = os.path.join(os.path.dirname(P.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", csrc, str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr


def chunk(c=None, **other):
    f = dict(q=at(0), qs=1024, qt=BF16, cu=at(4), batch=2, rows=40, max_q=30, hq=8, table=at(1), max_pages=100, lens=at(2),
             max_len=6400, window=0, sinks=0, scale=0.1, out=at(3), ws=at(500), wsb=1 << 40)
    f.update(other)
    c = cache() if c is None else c
    return err(P.lib().ptq1_attn_chunk(f["q"], f["qs"], f["qt"], f["cu"], f["batch"], f["rows"], f["max_q"], f["hq"],
                                       C.byref(c), f["table"], f["max_pages"], f["lens"], f["max_len"], f["window"],
                                       f["sinks"], f["scale"], f["out"], f["ws"], f["wsb"], None))


@pytest.mark.parametrize("other,status,word", [
    (dict(window=-1), SHAPE, "window"),
    (dict(sinks=-1), SHAPE, "sinks"),
    (dict(batch=-1), SHAPE, "batch"),
    (dict(rows=-1), SHAPE, "n_q_rows"),
    (dict(max_q=-1), SHAPE, "max_q"),
    (dict(hq=7), SHAPE, "n_q_heads"),
    (dict(scale=float("nan")), SHAPE, "scale"),
    (dict(max_pages=-1), SHAPE, "max_pages"),
    (dict(max_len=6401), SHAPE, "max_len"),
    (dict(max_pages=1 << 20, max_len=(1 << 22) + 1), UNSUPPORTED, "max_len"),
    (dict(qt=F32), UNSUPPORTED, "q_dtype"),
    (dict(qt=F16), UNSUPPORTED, "q_dtype"),
    (dict(rows=1 << 31), UNSUPPORTED, "rows"),
    (dict(batch=1 << 23), UNSUPPORTED, "tiles"),
    (dict(q=None), NULL, "q is"),
    (dict(cu=None), NULL, "cu_q"),
    (dict(table=None), NULL, "block_table"),
    (dict(lens=at(2) + 2), ALIGN, "seq_lens"),
    (dict(q=at(0) + 8), ALIGN, "q is not"),
    (dict(qs=1004), SHAPE, "q: row stride"),
    (dict(qs=1028), ALIGN, "q: row stride"),
    (dict(out=None), NULL, "out is"),
    (dict(out=at(0) + 1024), ALIAS, "out overlaps q"),
    (dict(out=at(200)), ALIAS, "out overlaps the cache"),
    (dict(out=at(4)), ALIAS, "cu_q"),
    (dict(wsb=16), WORKSPACE, "ptq1_attn_chunk"),
    (dict(ws=None), WORKSPACE, "ptq1_attn_chunk"),
    (dict(ws=at(100)), ALIAS, "ws overlaps"),
    (dict(ws=at(2)), ALIAS, "ws overlaps"),
])
def test_chunk_refused(other, status, word):
    rc, msg = chunk(**other)
    assert rc == status and word in msg, msg


def test_chunk_cache_refused():
    for other, status, word in ((dict(dtype=F32), UNSUPPORTED, "cache dtype"), (dict(page=8), UNSUPPORTED, "page_size"),
                                (dict(d=80), UNSUPPORTED, "head_dim"), (dict(k_pages=None), NULL, "k_pages"),
                                (dict(dtype=I8, k_steps=None), NULL, "k_steps")):
        rc, msg = chunk(cache(**other))
        assert rc == status and word in msg
    assert chunk(batch=0)[0] == 0 and chunk(rows=0, q=None, out=None)[0] == 0


def test_chunk_workspace():
    size = lambda *a: P.workspace_bytes("attn_chunk", *a)  # noqa: E731
    assert size(1, 5, 5, 40, 8, 128, 100, 0, 0) == 0                 # a few steps: nothing to cut
    few, more = size(1, 5, 5, 40, 8, 128, 8000, 0, 0), size(1, 5, 500, 40, 8, 128, 8000, 0, 0)
    assert 0 < few == more                                           # no sequence has more queries than there are
    assert size(1, 50, 50, 40, 8, 128, 8000, 30, 4) == 0             # a small window: nothing to cut
    assert size(1, 65536, 65536, 40, 8, 128, 65536, 0, 0) == 0       # the tiles fill the GPU
    assert size(-1, 5, 5, 40, 8, 128, 200, 0, 0) == 0 and size(1, 5, 5, 40, 8, 128, 200, -1, 0) == 0


def test_chunk_arithmetic(tmp_path):
    """ptq1_chunk.h over positions, windows and sinks: a tile's steps hold every key that one of its rows sees, each in
    one step; in the steps that every row is said to see whole, every row sees every key; no tile has more steps than the
    bound; the pieces of all tiles fit their number."""
    src = tmp_path / "c.cpp"
    src.write_text("""
#include <cstdio>
#include <initializer_list>
#include "ptq1_chunk.h"
using namespace ptq1;
int bad(const char *what, int a, int b, int w, int s) { std::printf("%s: %d %d %d %d\\n", what, a, b, w, s); return 1; }
int main()
{
    const int windows[] = {1, 2, 15, 63, 64, 65, 100, 128, 200, 400, 5000}, sinks[] = {0, 1, 16, 63, 64, 65, 130, 500};
    for (int first = -70; first < 420; first += first < 140 ? 3 : 17)
        for (int rows : {1, 2, 5, 26, 64, 127, 128})
            for (int w : windows)
                for (int s : sinks) {
                    const int last = first + rows - 1, len = imax(0, last + 1);
                    const ChunkSteps c = chunk_steps(first, last, w, s);
                    if (c.steps > steps_bound(len + 50, w, s, 128 / rows)) return bad("bound", first, rows, w, s);
                    static int in[1000];
                    for (int j = 0; j < 1000; ++j) in[j] = 0;
                    int before = -1;
                    for (int i = 0; i < c.steps; ++i) {
                        const int n0 = step_key(c, i);
                        if (n0 <= before || n0 >= c.reach) return bad("order", first, rows, w, s);
                        before = n0;
                        for (int j = n0; j < n0 + kChunkKeys; ++j) in[j] += 1;
                        // the page of a run that is looked up holds a key that some row sees
                        for (int q = 0; q < 4; ++q) {
                            const int r = n0 + 16 * q, tok = r < c.sunk ? r : imin(imax(r, c.lo), c.reach - 1);
                            bool some = false, near = false;
                            for (int j = tok & ~15; j < (tok & ~15) + 16; ++j) some |= j < c.reach && (j >= c.lo || j < c.sunk);
                            for (int j = r; j < r + 16; ++j) near |= j < c.reach && (j >= c.lo || j < c.sunk);
                            if (tok < 0 || tok >= len || !some || (near && tok >> 4 != r >> 4)) return bad("page", first, rows, w, s);
                        }
                    }
                    for (int p = first; p <= last; p += p + 1 == last ? 1 : 1 + (last - p) / 4) {
                        const SeenKeys k = seen_keys(p, w);
                        for (int j = 0; j < 900; ++j) {
                            const bool sees = j <= p && (j > p - w || j < s);
                            if (sees != (j < k.hi && (j >= k.lo || j < s))) return bad("seen", first, rows, w, s);
                            if (sees && in[j] != 1) return bad("missing", p, j, w, s);
                        }
                        for (int i = imax(0, c.all_from); i < imin(c.steps, c.all_to); ++i)
                            for (int j = step_key(c, i); j < step_key(c, i) + kChunkKeys; ++j)
                                if (!(j <= p && j > p - w)) return bad("whole", p, j, w, s);
                    }
                }
    // pieces: per * wanted covers the total, so the pieces of tiles with these steps are at most wanted + tiles
    for (int wanted : {1, 7, 64, 512})
        for (int tiles : {1, 3, 100})
            for (int steps : {0, 1, 3, 4, 5, 63, 1000, 65536}) {
                const int per = chunk_piece(tiles * steps, wanted);
                if (tiles * chunk_pieces(steps, per) > wanted + tiles || per < kChunkMinSteps) return bad("pieces", wanted, tiles, steps, per);
            }
    // cuts: one piece is always allowed, more while they are long enough and find places
    for (int lane = 0; lane < 64; ++lane) {
        const int n = chunk_cut_of(lane);
        if (n < 1 || n > 960 || (lane > 0 && n < chunk_cut_of(lane - 1)) || (lane < 15 && lane != 8 && n != lane + (lane < 8))) return bad("cut", lane, n, 0, 0);
        for (int wanted : {1, 7, 64, 512})
            for (int tiles : {1, 3, 100, 2048})
                for (int steps : {1, 4, 5, 63, 1000, 65536}) {
                    const float cost = chunk_cost(n, tiles, steps, wanted, 3.0f, 0.1f);
                    const int per = imax(kChunkMinSteps, (steps + n - 1) / n);
                    if (n == 1 ? !(cost > 0) : cost >= 0 && (tiles * chunk_pieces(steps, per) > 2 * wanted || (steps + n - 1) / n < kChunkMinSteps))
                        return bad("cost", n, tiles, steps, wanted);
                }
    }
    const ChunkSteps c = chunk_steps((1 << 22) - 5, (1 << 22) - 1, (1 << 22) + 1, 1 << 22);
    return c.steps == 65536 && c.lo == 0 ? 0 : bad("large", c.steps, c.lo, c.reach, c.gap);
}
""")
    exe = tmp_path / "c"
    csrc = os.path.join(os.path.dirname(P.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", csrc, str(src), "-o",
                    str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr


# ------------------------------------------------------------- the binding ----

def test_binding_write_norm(host_ok):
    c = kv()
    q, k, s = z(3, 8, 128), z(3, 2, 128), torch.zeros(3, dtype=torch.int64)
    gain = torch.ones(128)
    for kw, match in ((dict(q_gain=torch.ones(64)), "q_gain has"), (dict(k_gain=gain.half()), "k_gain must be"),
                      (dict(k_gain=torch.ones(256)[::2]), "k_gain must be contiguous"),
                      (dict(cos_sin=torch.zeros(4, 8)), "needs positions"), (dict(q_dtype=torch.int8), "q_dtype")):
        with pytest.raises(ValueError, match=match):
            P.ptq1_kv_write_norm(q, k, k, s, c, **kw)
    with pytest.raises(TypeError, match="q_gain"):
        P.ptq1_kv_write_norm(q, k, k, s, c, q_gain=[1.0] * 128)
    with pytest.raises(ValueError, match="k has 4 heads"):
        P.ptq1_kv_write_norm(q, z(3, 4, 128), k, s, c, q_gain=gain)


def test_binding_window(host_ok):
    c, t = kv(), torch.zeros((2, 400), dtype=torch.int32)
    q = z(2, 8, 128)
    with pytest.raises(ValueError, match="block_table"):
        P.ptq1_attn_decode_window(q, c, t[:1], i32(1, 2), 10)
    with pytest.raises(ValueError, match="seq_lens has"):
        P.ptq1_attn_decode_window(q, c, t, i32(1, 2, 3), 10)
    with pytest.raises(ValueError, match="ws has"):
        P.ptq1_attn_decode_window(q, c, t, i32(1, 2), 3000, 4, ws=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="out has"):
        P.ptq1_attn_decode_window(q, c, t, i32(1, 2), 10, out=z(2, 4, 128))


def test_binding_chunk(host_ok):
    c, t, cu = kv(), torch.zeros((2, 400), dtype=torch.int32), i32(0, 3, 5)
    q = z(5, 8, 128)
    for bad, match in (((z(5, 8, 64), c, t, cu, i32(3, 3)), "q must be"), ((q.float(), c, t, cu, i32(3, 3)), "q must be"),
                       ((q, c, t[:1], cu, i32(3, 3)), "block_table"), ((q, c, t, cu[:0], i32()), "cu_q must hold"),
                       ((q, c, t, cu.long(), i32(3, 3)), "cu_q must be"), ((q, c, t, cu, i32(3, 3, 3)), "seq_lens has"),
                       ((z(5, 128, 8).transpose(1, 2), c, t, cu, i32(3, 3)), "heads of a row")):
        with pytest.raises(ValueError, match=match):
            P.ptq1_attn_chunk(*bad)
    with pytest.raises(ValueError, match="ws has"):
        P.ptq1_attn_chunk(q, c, t, cu, i32(3, 3), ws=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="out has"):
        P.ptq1_attn_chunk(q, c, t, cu, i32(3, 3), out=z(5, 4, 128))
    with pytest.raises(TypeError, match="KvCache"):
        P.ptq1_attn_chunk(q, c.k_pages, t, cu, i32(3, 3))


def side_calls():
    """The calls of this file over host tensors."""
    c, t = kv(), torch.zeros((2, 400), dtype=torch.int32)
    q, k, s = z(3, 8, 128), z(3, 2, 128), torch.zeros(3, dtype=torch.int64)
    return {"kv_write_norm": lambda **o: P.ptq1_kv_write_norm(q, k, k, s, c, **o),
            "attn_decode_window": lambda **o: P.ptq1_attn_decode_window(q[:2], c, t, i32(1, 2), 3000, **o),
            "attn_chunk": lambda **o: P.ptq1_attn_chunk(q, c, t, i32(0, 1, 3), i32(1, 2), **o)}


@pytest.mark.parametrize("name", ["kv_write_norm", "attn_decode_window", "attn_chunk"])
def test_side_stream_allocates_its_own_memory(monkeypatch, name):
    streams = Streams(monkeypatch)
    call = side_calls()[name]
    streams.allocated.clear()
    call(stream=streams.side)
    assert streams.allocated and set(streams.allocated) == {"side"}
    assert streams.tied and set(streams.tied) == {"main"} and streams.current is streams.main
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


@pytest.mark.parametrize("far", [1 << 63, (1 << 64) + 1, 1 << 200])
def test_bounds_past_64_bits(monkeypatch, far):
    """Windows, first tokens and bounds of any size are as given, not their lowest 64 bits."""
    real, calls = P.lib(), []

    class Seen:
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return getattr(real, name)
            return lambda *a: calls.append(a) or 0

    monkeypatch.setattr(P, "_on_device", lambda t: True)
    monkeypatch.setattr(P, "_current_handle", lambda device: 0)
    monkeypatch.setattr(P, "lib", lambda: Seen())
    c, t, q = kv(), torch.zeros((2, 400), dtype=torch.int32), z(3, 8, 128)
    most = (1 << 63) - 1
    P.ptq1_attn_decode_window(q[:2], c, t, i32(1, 2), far, far)
    P.ptq1_attn_decode_window(q[:2], c, t, i32(1, 2), -far, 0, max_len=far)
    P.ptq1_attn_decode(q[:2], c, t, i32(1, 2), max_len=far)
    P.ptq1_attn_chunk(q, c, t, i32(0, 1, 3), i32(1, 2), window=far, sinks=far, max_q=far, max_len=-far)
    assert calls[0][8:11] == (6400, most, most)
    assert calls[1][8] == most and calls[1][9] < 0
    assert calls[2][8] == most
    assert calls[3][6] == most and calls[3][12] < 0 and calls[3][13:15] == (most, most)
    for kind, shape in (("attn_decode_window", (1, 8, 2, 128, 100000)), ("attn_chunk", (1, 8, 8, 8, 2, 128, 100000))):
        need = P.workspace_bytes(kind, *shape, 100000, 100000)
        assert need > 0 and P.workspace_bytes(kind, *shape, far, far) == need

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
    f = dict(q=at(0), qt=BF16, batch=2, hq=8, table=at(1), max_pages=100, lens=at(2), max_len=6400, window=500, sinks=4,
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


def side_calls():
    """The calls of this file over host tensors."""
    c, t = kv(), torch.zeros((2, 400), dtype=torch.int32)
    q, k, s = z(3, 8, 128), z(3, 2, 128), torch.zeros(3, dtype=torch.int64)
    return {"kv_write_norm": lambda **o: P.ptq1_kv_write_norm(q, k, k, s, c, **o),
            "attn_decode_window": lambda **o: P.ptq1_attn_decode_window(q[:2], c, t, i32(1, 2), 3000, **o)}


@pytest.mark.parametrize("name", ["kv_write_norm", "attn_decode_window"])
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

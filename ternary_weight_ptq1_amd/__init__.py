"""Python binding of ``libptq1.so`` (the C ABI in ``include/ptq1.h``).

Argument marshalling only: every function passes device pointers of torch
tensors and ``torch.cuda.current_stream()`` to the C entry point of the same
name and raises :class:`Ptq1Error` on a non-OK status.  torch supplies device
memory and streams; every step of the computation runs in the HIP kernels.
There is no fallback: if the library is not built, importing the binding's
functions raises.
"""
from __future__ import annotations

import ctypes as C
import functools
import inspect
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# PTQ1_LIB may name another build of the same library (the sanitizer build
# of build.py --sanitize, for host-only test runs)
LIB_PATH = os.environ.get("PTQ1_LIB", os.path.join(_HERE, "libptq1.so"))
HEADER = os.path.join(os.path.dirname(_HERE), "include", "ptq1.h")

BLOCK_WEIGHTS = 128
TRIT_BYTES = 26
BLOCK_BYTES = 28
HADAMARD = 1024
TILE_ROWS = 32
TILE_BLOCKS = 2

STATUS = {0: "PTQ1_OK", 1: "PTQ1_ERR_NULL", 2: "PTQ1_ERR_SHAPE", 3: "PTQ1_ERR_ALIGN",
          4: "PTQ1_ERR_OVERFLOW", 5: "PTQ1_ERR_UNSUPPORTED", 6: "PTQ1_ERR_WORKSPACE",
          7: "PTQ1_ERR_ALIAS", 8: "PTQ1_ERR_HIP"}


class Ptq1Error(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn}: {STATUS.get(status, status)}: {message}")
        self.status = status
        self.message = message


_lib = None
i64, sz, p = C.c_int64, C.c_size_t, C.c_void_p

_SIGS = {
    "ptq1_status_string": ([C.c_int], C.c_char_p),
    "ptq1_last_error": ([], C.c_char_p),
    "ptq1_geometry": ([p, C.c_int32], C.c_int),
    "ptq1_packed_bytes": ([i64, i64], i64),
    "ptq1_tiled_bytes": ([i64, i64], i64),
    "ptq1_tile": ([p, i64, i64, p, p], C.c_int),
    "ptq1_pack": ([p, p, i64, i64, p, p], C.c_int),
    "ptq1_dequant": ([p, i64, i64, p, p], C.c_int),
    "hadamard_rotate": ([p, p, i64, i64, p, p], C.c_int),
    "hadamard_unrotate_rows": ([p, i64, i64, p, i64, p, p, p], C.c_int),
    "ptq1_matvec_workspace_bytes": ([i64, i64], sz),
    "ptq1_matvec": ([p, i64, i64, p, p, p, p, p, sz, p], C.c_int),
    "ptq1_matvec_float_peel": ([p, i64, i64, p, p, p, p, p, sz, p], C.c_int),
    "ptq1_gate_up_workspace_bytes": ([i64, i64], sz),
    "ptq1_gate_up": ([p, p, i64, i64, p, p, p, p, p, sz, p], C.c_int),
    "ptq1_swiglu": ([p, p, p, i64, p], C.c_int),
    "ptq1_gemm_workspace_bytes": ([i64, i64, i64], sz),
    "ptq1_gemm": ([p, i64, i64, p, i64, p, p, p, sz, p], C.c_int),
    "ptq1_ffn_workspace_bytes": ([i64, i64, i64], sz),
    "ptq1_ffn_block": ([p, p, i64, i64, i64, p, p, p, p, C.c_float, p, p, sz, p], C.c_int),
    "pq2_packed_bytes": ([i64, i64], i64),
    "pq2_pack": ([p, p, i64, i64, p, p], C.c_int),
    "pq2_dequant": ([p, i64, i64, p, p], C.c_int),
    "pq2_tiled_bytes": ([i64, i64], i64),
    "pq2_tile": ([p, i64, i64, p, p], C.c_int),
    "pq2_matvec_workspace_bytes": ([i64, i64], sz),
    "pq2_matvec": ([p, i64, i64, p, p, p, p, p, sz, p], C.c_int),
    "pq2_gemm_workspace_bytes": ([i64, i64, i64], sz),
    "pq2_gemm": ([p, i64, i64, p, i64, p, p, p, sz, p], C.c_int),
    "pq2_ffn_workspace_bytes": ([i64, i64, i64], sz),
    "ptq1_matvec_w2a8_workspace_bytes": ([i64, i64], sz),
    "ptq1_gemm_w2a8_workspace_bytes": ([i64, i64, i64], sz),
    "ptq1_gemm_w2a8": ([p, i64, i64, p, i64, p, p, sz, p], C.c_int),
    "ptq1_matvec_w2a8": ([p, i64, i64, p, p, p, p, sz, p], C.c_int),
    "pq2_ffn_block": ([p, p, i64, i64, i64, p, p, p, p, C.c_float, p, p, sz, p], C.c_int),
    "ptq1_ffn_workspace_offsets": ([i64, i64, i64, p], C.c_int),
    "ptq1_ffn_block_noalloc": ([p, p, i64, i64, i64, p, p, p, p, C.c_float, p, p], C.c_int),
    "pq2_ffn_workspace_offsets": ([i64, i64, i64, p], C.c_int),
    "ptq1_kv_write": ([p, i64, p, i64, p, i64, C.c_int32, i64, C.c_int32, p, p, i64, C.c_int32, p, p, C.c_int32, p, p],
                      C.c_int),
    "ptq1_kv_write_norm": ([p, i64, p, i64, p, i64, C.c_int32, i64, C.c_int32, p, p, C.c_float, p, p, i64, C.c_int32, p, p,
                            C.c_int32, p, p], C.c_int),
    "ptq1_kv_read": ([p, p, i64, p, i64, i64, p, p, C.c_int32, p], C.c_int),
    "ptq1_attn_decode_workspace_bytes": ([i64, C.c_int32, C.c_int32, C.c_int32, i64], sz),
    "ptq1_attn_decode": ([p, C.c_int32, i64, C.c_int32, p, p, i64, p, i64, C.c_float, p, p, sz, p], C.c_int),
    "ptq1_attn_decode_window_workspace_bytes": ([i64, C.c_int32, C.c_int32, C.c_int32, i64, i64, i64], sz),
    "ptq1_attn_decode_window": ([p, C.c_int32, i64, C.c_int32, p, p, i64, p, i64, i64, i64, C.c_float, p, p, sz, p],
                                C.c_int),
    "ptq1_attn_chunk_workspace_bytes": ([i64, i64, i64, C.c_int32, C.c_int32, C.c_int32, i64, i64, i64], sz),
    "ptq1_attn_chunk": ([p, i64, C.c_int32, p, i64, i64, i64, C.c_int32, p, p, i64, p, i64, i64, i64, C.c_float, p, p, sz,
                         p], C.c_int),
    "ptq1_attn_prompt_workspace_bytes": ([i64, i64, i64, C.c_int32, C.c_int32, C.c_int32], sz),
    "ptq1_attn_prompt": ([p, i64, p, i64, p, i64, C.c_int32, p, p, i64, i64, i64, i64, i64, C.c_int32, C.c_int32,
                          C.c_int32, C.c_int32, C.c_float, p, p, sz, p], C.c_int),
    "ptq1_profile_arm": ([C.c_char_p, p, p, C.c_int32], C.c_int),
    "ptq1_profile_count": ([C.c_char_p], C.c_int32),
}


def lib():
    """The loaded C library.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m ternary_weight_ptq1_amd.build`")
        L = C.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/ptq1.h."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"\b([a-z_0-9]+)\s*\(", text.split('extern "C" {', 1)[1])


def _check(fn: str, status: int):
    if status != 0:
        raise Ptq1Error(fn, status, lib().ptq1_last_error().decode())


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


# ------------------------------------------------------------- validation ----
# The C library sees only pointers and sizes, so every tensor is checked here
# against the sizes the call will read or write before anything is enqueued:
# a host tensor or a short one would become an out-of-range device access.

def _on_device(t: torch.Tensor) -> bool:
    return t.is_cuda


def _dev(t: torch.Tensor, name: str, dtype=None, numel: int | None = None, min_numel: int | None = None,
         device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not _on_device(t):
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, the call uses {numel}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} has {t.numel()} elements, the call reads or writes {min_numel}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")
    return t


def _opt(t, name, dtype, numel=None, device=None):
    return None if t is None else _dev(t, name, dtype, numel=numel, device=device)


def _signs(s, device, required=True):
    if s is None:
        if required:
            raise ValueError("signs1024 is required")
        return None
    return _dev(s, "signs1024", torch.float32, numel=HADAMARD, device=device)


def _rows_of(x: torch.Tensor, k: int, name: str = "x") -> int:
    """Rows of an activation tensor of width k (its element count must be a multiple of k)."""
    if k <= 0:
        raise ValueError(f"k = {k} must be positive")
    if x.numel() % k != 0:
        raise ValueError(f"{name} has {x.numel()} elements, not a multiple of k = {k}")
    return x.numel() // k


def _mat(w: torch.Tensor, name: str, nbytes: int, device):
    """A weight matrix of nbytes bytes (a negative nbytes is a bad shape, refused by the library)."""
    return _dev(w, name, torch.uint8, min_numel=nbytes if nbytes > 0 else None, device=device)


def _ws(nbytes: int, device, ws):
    if nbytes == 0:
        return None, 0
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes
    _dev(ws, "ws", torch.uint8, min_numel=nbytes, device=device)
    return ws, ws.numel()


def _out(out, name, shape, device, dtype=torch.float32):
    count = 1
    for s in shape:
        count *= s
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _dev(out, name, dtype, numel=count, device=device)


def _tied(result, stream):
    """result, its tensors' memory kept from other uses until what `stream` does with them is done."""
    for t in result if isinstance(result, tuple) else (result,):
        if t is not None:
            t.record_stream(stream)
    return result


def _on_its_stream(call):
    """A call whose stream= is not the current one is made with that stream as the current one, so that its scratch and
    results come from that stream's memory: a block that the current stream has freed may still have work of that
    stream pending on it."""
    at = list(inspect.signature(call).parameters).index("stream")

    @functools.wraps(call)
    def run(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None or stream == torch.cuda.current_stream():
            return call(*args, **kw)
        here = torch.cuda.current_stream(stream.device)
        with torch.cuda.stream(stream):
            return _tied(call(*args, **kw), here)

    return run


# ------------------------------------------------------------------ codec ----

def ptq1_geometry() -> tuple[int, int, int, int, int, int]:
    """(weights per block, trit bytes, block bytes, Hadamard width, tile rows, tile blocks)."""
    out = (C.c_int32 * 6)()
    _check("ptq1_geometry", lib().ptq1_geometry(C.cast(out, p), 6))
    return tuple(out)


def ptq1_packed_bytes(n: int, k: int) -> int:
    return lib().ptq1_packed_bytes(n, k)


def _trits_scales(trits, scales_f16):
    _dev(trits, "trits", torch.int8)
    if trits.dim() != 2:
        raise ValueError("trits must be [n, k]")
    n, k = trits.shape
    if k % BLOCK_WEIGHTS != 0:
        raise ValueError(f"k = {k} is not a multiple of {BLOCK_WEIGHTS}")
    _dev(scales_f16, "scales_f16", (torch.int16, torch.float16, torch.uint16), numel=n * (k // BLOCK_WEIGHTS),
         device=trits.device)
    return n, k


@_on_its_stream
def ptq1_pack(trits: torch.Tensor, scales_f16: torch.Tensor, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """int8 trits [n, k] + binary16 bit patterns [n, k/128] (int16 or float16) -> uint8 [n, k/128*28]."""
    n, k = _trits_scales(trits, scales_f16)
    out = _out(out, "blocks", (n, (k // BLOCK_WEIGHTS) * BLOCK_BYTES), trits.device, torch.uint8)
    _check("ptq1_pack", lib().ptq1_pack(_ptr(trits), _ptr(scales_f16), n, k, _ptr(out), _stream(stream)))
    return out


def ptq1_tiled_bytes(n: int, k: int) -> int:
    return lib().ptq1_tiled_bytes(n, k)


@_on_its_stream
def ptq1_tile(blocks: torch.Tensor, n: int, k: int, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """Packed [n, k/128*28] uint8 -> the tiled device layout (flat uint8) the
    matvec, gate/up, GEMM and feed-forward calls read."""
    nbytes = ptq1_tiled_bytes(n, k)
    if nbytes < 0:
        raise ValueError(f"bad shape [{n}][{k}]")
    _mat(blocks, "blocks", ptq1_packed_bytes(n, k), None)
    out = _out(out, "tiled", (nbytes,), blocks.device, torch.uint8)
    _check("ptq1_tile", lib().ptq1_tile(_ptr(blocks), n, k, _ptr(out), _stream(stream)))
    return out


@_on_its_stream
def ptq1_dequant(blocks: torch.Tensor, n: int, k: int, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    _mat(blocks, "blocks", ptq1_packed_bytes(n, k), None)
    out = _out(out, "w", (n, k), blocks.device)
    _check("ptq1_dequant", lib().ptq1_dequant(_ptr(blocks), n, k, _ptr(out), _stream(stream)))
    return out


# --------------------------------------------------------------- rotation ----

@_on_its_stream
def hadamard_rotate(x: torch.Tensor, signs1024: torch.Tensor, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Rotate the rows of x [m, k] (or [k]); out may be x."""
    _dev(x, "x", torch.float32)
    _signs(signs1024, x.device)
    k = x.shape[-1] if x.dim() > 0 else 0
    m = _rows_of(x, k)
    if out is None:
        out = torch.empty_like(x)
    _dev(out, "y", torch.float32, numel=x.numel(), device=x.device)
    _check("hadamard_rotate", lib().hadamard_rotate(_ptr(x), _ptr(out), m, k, _ptr(signs1024),
                                                    _stream(stream)))
    return out


@_on_its_stream
def hadamard_unrotate_rows(table: torch.Tensor, signs1024: torch.Tensor, ids: torch.Tensor | None = None,
                           n_rows: int | None = None, out: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
    _dev(table, "table", torch.float32)
    if table.dim() != 2:
        raise ValueError("table must be [n_table, d]")
    _signs(signs1024, table.device)
    n_table, d = table.shape
    if ids is not None:
        _dev(ids, "ids", torch.int32, device=table.device)
        n_rows = ids.numel()
    elif n_rows is None:
        n_rows = n_table
    out = _out(out, "out", (n_rows, d), table.device)
    _check("hadamard_unrotate_rows",
           lib().hadamard_unrotate_rows(_ptr(table), n_table, d, _ptr(ids), n_rows, _ptr(signs1024),
                                        _ptr(out), _stream(stream)))
    return out


# ----------------------------------------------------------------- decode ----

@_on_its_stream
def ptq1_matvec(blocks: torch.Tensor, n: int, k: int, x: torch.Tensor, signs1024: torch.Tensor | None,
                residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                ws: torch.Tensor | None = None, stream=None, fn: str = "ptq1_matvec") -> torch.Tensor:
    """y = residual + W R x, W tiled (ptq1_tile).  ws: optional scratch of
    at least workspace_bytes("matvec", n, k) bytes."""
    _dev(x, "x", torch.float32, numel=k)
    dv = x.device
    _mat(blocks, "blocks", ptq1_tiled_bytes(n, k), dv)
    _signs(signs1024, dv, required=False)
    _opt(residual, "residual", torch.float32, numel=n, device=dv)
    out = _out(out, "y", (n,), dv)
    ws, wsb = _ws(lib().ptq1_matvec_workspace_bytes(n, k), dv, ws)
    _check(fn, getattr(lib(), fn)(_ptr(blocks), n, k, _ptr(x), _ptr(signs1024), _ptr(residual),
                                  _ptr(out), _ptr(ws), wsb, _stream(stream)))
    return out


@_on_its_stream
def ptq1_matvec_float_peel(blocks, n, k, x, signs1024, residual=None, out=None, ws=None, stream=None):
    """The same matvec with every trit peeled on the float pipeline, eight lanes per block (tiled layout)."""
    return ptq1_matvec(blocks, n, k, x, signs1024, residual, out, ws, stream, fn="ptq1_matvec_float_peel")


@_on_its_stream
def ptq1_gate_up(w_gate: torch.Tensor, w_up: torch.Tensor, f: int, d: int, x: torch.Tensor,
                 signs1024: torch.Tensor | None, g: torch.Tensor | None = None,
                 u: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    _dev(x, "x", torch.float32, numel=d)
    dv = x.device
    tb = ptq1_tiled_bytes(f, d)
    _mat(w_gate, "w_gate", tb, dv)
    _mat(w_up, "w_up", tb, dv)
    _signs(signs1024, dv, required=False)
    g = _out(g, "g", (f,), dv)
    u = _out(u, "u", (f,), dv)
    ws, wsb = _ws(lib().ptq1_gate_up_workspace_bytes(f, d), dv, ws)
    _check("ptq1_gate_up", lib().ptq1_gate_up(_ptr(w_gate), _ptr(w_up), f, d, _ptr(x), _ptr(signs1024),
                                              _ptr(g), _ptr(u), _ptr(ws), wsb, _stream(stream)))
    return g, u


@_on_its_stream
def ptq1_swiglu(g: torch.Tensor, u: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    _dev(g, "g", torch.float32)
    _dev(u, "u", torch.float32, numel=g.numel(), device=g.device)
    if out is None:
        out = torch.empty_like(g)
    _dev(out, "h", torch.float32, numel=g.numel(), device=g.device)
    _check("ptq1_swiglu", lib().ptq1_swiglu(_ptr(g), _ptr(u), _ptr(out), g.numel(), _stream(stream)))
    return out


# ---------------------------------------------------------------- prefill ----

@_on_its_stream
def ptq1_gemm(blocks: torch.Tensor, n: int, k: int, x: torch.Tensor, signs1024: torch.Tensor | None,
              out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _dev(x, "x", torch.float32)
    dv = x.device
    m = _rows_of(x, k)
    _mat(blocks, "blocks", ptq1_tiled_bytes(n, k), dv)
    _signs(signs1024, dv, required=False)
    out = _out(out, "y", (m, n), dv)
    ws, wsb = _ws(lib().ptq1_gemm_workspace_bytes(m, n, k), dv, ws)
    _check("ptq1_gemm", lib().ptq1_gemm(_ptr(blocks), n, k, _ptr(x), m, _ptr(signs1024), _ptr(out),
                                        _ptr(ws), wsb, _stream(stream)))
    return out


@_on_its_stream
def ptq1_ffn_block(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                   signs1024: torch.Tensor, d: int, f: int, rms_eps: float = 0.0,
                   out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                   stream=None, rms_gain: torch.Tensor | None = None, fn: str = "ptq1_ffn_block") -> torch.Tensor:
    """x [m, d] -> x + W_down R(silu(W_gate R xn) * (W_up R xn)), xn = a * rms_gain * x (a = RMS
    scale of x when rms_eps > 0; rms_gain [d] or None); out may be x.  fn = "pq2_ffn_block" takes
    PQ2_0 tiled matrices (pq2_tile)."""
    _dev(x, "x", torch.float32)
    dv = x.device
    m = _rows_of(x, d)
    tiled = pq2_tiled_bytes if fn == "pq2_ffn_block" else ptq1_tiled_bytes
    _mat(w_gate, "w_gate", tiled(f, d), dv)
    _mat(w_up, "w_up", tiled(f, d), dv)
    _mat(w_down, "w_down", tiled(d, f), dv)
    _signs(signs1024, dv)
    _opt(rms_gain, "rms_gain", torch.float32, numel=d, device=dv)
    if out is None:
        out = torch.empty_like(x)
    _dev(out, "x_out", torch.float32, numel=m * d, device=dv)
    wsfn = "pq2_ffn_workspace_bytes" if fn == "pq2_ffn_block" else "ptq1_ffn_workspace_bytes"
    ws, wsb = _ws(getattr(lib(), wsfn)(m, d, f), dv, ws)
    _check(fn, getattr(lib(), fn)(_ptr(x), _ptr(out), m, d, f, _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                  _ptr(signs1024), float(rms_eps), _ptr(rms_gain) if rms_gain is not None else None,
                                  _ptr(ws), wsb, _stream(stream)))
    return out


@_on_its_stream
def ptq1_ffn_block_noalloc(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                           signs1024: torch.Tensor, d: int, f: int, rms_eps: float = 0.0,
                           out: torch.Tensor | None = None, stream=None,
                           rms_gain: torch.Tensor | None = None) -> torch.Tensor:
    """ptq1_ffn_block on the library's own static scratch buffer (no workspace argument; calls on one GPU
    must not overlap).  `out` must be given by a caller that cannot allocate."""
    _dev(x, "x", torch.float32)
    dv = x.device
    m = _rows_of(x, d)
    _mat(w_gate, "w_gate", ptq1_tiled_bytes(f, d), dv)
    _mat(w_up, "w_up", ptq1_tiled_bytes(f, d), dv)
    _mat(w_down, "w_down", ptq1_tiled_bytes(d, f), dv)
    _signs(signs1024, dv)
    _opt(rms_gain, "rms_gain", torch.float32, numel=d, device=dv)
    if out is None:
        out = torch.empty_like(x)
    _dev(out, "x_out", torch.float32, numel=m * d, device=dv)
    _check("ptq1_ffn_block_noalloc",
           lib().ptq1_ffn_block_noalloc(_ptr(x), _ptr(out), m, d, f, _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                        _ptr(signs1024), float(rms_eps),
                                        _ptr(rms_gain) if rms_gain is not None else None, _stream(stream)))
    return out


@_on_its_stream
def pq2_ffn_block(x, w_gate, w_up, w_down, signs1024, d, f, rms_eps=0.0, out=None, ws=None, stream=None,
                  rms_gain=None):
    """ptq1_ffn_block over PQ2_0 tiled matrices."""
    return ptq1_ffn_block(x, w_gate, w_up, w_down, signs1024, d, f, rms_eps, out, ws, stream, rms_gain,
                          fn="pq2_ffn_block")


# ------------------------------------------------------------------ PQ2_0 ----

PQ2_BLOCK_BYTES = 34


def pq2_packed_bytes(n: int, k: int) -> int:
    return lib().pq2_packed_bytes(n, k)


@_on_its_stream
def pq2_pack(trits: torch.Tensor, scales_f16: torch.Tensor, out: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """int8 trits [n, k] + binary16 bit patterns [n, k/128] -> uint8 [n, k/128*34]."""
    n, k = _trits_scales(trits, scales_f16)
    out = _out(out, "blocks", (n, (k // BLOCK_WEIGHTS) * PQ2_BLOCK_BYTES), trits.device, torch.uint8)
    _check("pq2_pack", lib().pq2_pack(_ptr(trits), _ptr(scales_f16), n, k, _ptr(out), _stream(stream)))
    return out


@_on_its_stream
def pq2_dequant(blocks: torch.Tensor, n: int, k: int, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    _mat(blocks, "blocks", pq2_packed_bytes(n, k), None)
    out = _out(out, "w", (n, k), blocks.device)
    _check("pq2_dequant", lib().pq2_dequant(_ptr(blocks), n, k, _ptr(out), _stream(stream)))
    return out


def pq2_tiled_bytes(n: int, k: int) -> int:
    return lib().pq2_tiled_bytes(n, k)


@_on_its_stream
def pq2_tile(blocks: torch.Tensor, n: int, k: int, out: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """Packed PQ2_0 [n, k/128*34] uint8 -> the tiled layout pq2_matvec reads (flat uint8)."""
    nbytes = pq2_tiled_bytes(n, k)
    if nbytes < 0:
        raise ValueError(f"bad shape [{n}][{k}]")
    _mat(blocks, "blocks", pq2_packed_bytes(n, k), None)
    out = _out(out, "tiled", (nbytes,), blocks.device, torch.uint8)
    _check("pq2_tile", lib().pq2_tile(_ptr(blocks), n, k, _ptr(out), _stream(stream)))
    return out


@_on_its_stream
def pq2_matvec(tiled: torch.Tensor, n: int, k: int, x: torch.Tensor, signs1024: torch.Tensor | None,
               residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
               ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = residual + W R x over a PQ2_0 tiled matrix (pq2_tile)."""
    _dev(x, "x", torch.float32, numel=k)
    dv = x.device
    _mat(tiled, "tiled", pq2_tiled_bytes(n, k), dv)
    _signs(signs1024, dv, required=False)
    _opt(residual, "residual", torch.float32, numel=n, device=dv)
    out = _out(out, "y", (n,), dv)
    ws, wsb = _ws(lib().pq2_matvec_workspace_bytes(n, k), dv, ws)
    _check("pq2_matvec", lib().pq2_matvec(_ptr(tiled), n, k, _ptr(x), _ptr(signs1024), _ptr(residual),
                                          _ptr(out), _ptr(ws), wsb, _stream(stream)))
    return out


@_on_its_stream
def pq2_gemm(tiled: torch.Tensor, n: int, k: int, x: torch.Tensor, signs1024: torch.Tensor | None,
             out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [m, n] = bf16(R X) . W^T over a PQ2_0 tiled matrix (pq2_tile)."""
    _dev(x, "x", torch.float32)
    dv = x.device
    m = _rows_of(x, k)
    _mat(tiled, "tiled", pq2_tiled_bytes(n, k), dv)
    _signs(signs1024, dv, required=False)
    out = _out(out, "y", (m, n), dv)
    ws, wsb = _ws(lib().pq2_gemm_workspace_bytes(m, n, k), dv, ws)
    _check("pq2_gemm", lib().pq2_gemm(_ptr(tiled), n, k, _ptr(x), m, _ptr(signs1024), _ptr(out), _ptr(ws), wsb,
                                      _stream(stream)))
    return out


@_on_its_stream
def ptq1_matvec_w2a8(tiled: torch.Tensor, n: int, k: int, x: torch.Tensor, residual: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = residual + W q * step with x quantised to 8-bit integers (per call, absmax)."""
    _dev(x, "x", torch.float32, numel=k)
    dv = x.device
    _mat(tiled, "tiled", ptq1_tiled_bytes(n, k), dv)
    _opt(residual, "residual", torch.float32, numel=n, device=dv)
    out = _out(out, "y", (n,), dv)
    ws, wsb = _ws(lib().ptq1_matvec_w2a8_workspace_bytes(n, k), dv, ws)
    _check("ptq1_matvec_w2a8", lib().ptq1_matvec_w2a8(_ptr(tiled), n, k, _ptr(x), _ptr(residual), _ptr(out),
                                                      _ptr(ws), wsb, _stream(stream)))
    return out


@_on_its_stream
def ptq1_gemm_w2a8(tiled: torch.Tensor, n: int, k: int, x: torch.Tensor, out: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [m, n] with each row of x quantised to 8-bit integers (its own absmax)."""
    _dev(x, "x", torch.float32)
    dv = x.device
    m = _rows_of(x, k)
    _mat(tiled, "tiled", ptq1_tiled_bytes(n, k), dv)
    out = _out(out, "y", (m, n), dv)
    ws, wsb = _ws(lib().ptq1_gemm_w2a8_workspace_bytes(m, n, k), dv, ws)
    _check("ptq1_gemm_w2a8", lib().ptq1_gemm_w2a8(_ptr(tiled), n, k, _ptr(x), m, _ptr(out), _ptr(ws), wsb,
                                                  _stream(stream)))
    return out


# -------------------------------------------------------------- attention ----

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int8: 3}
_FLOATS = (torch.float32, torch.float16, torch.bfloat16)
_CACHE_TYPES = (torch.float16, torch.bfloat16, torch.int8)
_SIXTEEN = (torch.float16, torch.bfloat16)


class _CacheStruct(C.Structure):
    _fields_ = [("k_pages", p), ("v_pages", p), ("k_steps", p), ("v_steps", p), ("n_pages", i64),
                ("page_size", C.c_int32), ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32), ("dtype", C.c_int32)]


class KvCache:
    """A paged key-value cache over tensors that it keeps: k_pages [n_pages, n_kv_heads, page_size, head_dim],
    v_pages [n_pages, n_kv_heads, head_dim, page_size] (fp16, bf16 or int8) and, for int8, k_steps and v_steps
    [n_pages, n_kv_heads, page_size] fp32.  Its attributes cannot be set: the calls use the tensors it was made of."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, k_steps: torch.Tensor | None = None,
                 v_steps: torch.Tensor | None = None):
        _dev(k_pages, "k_pages", _CACHE_TYPES)
        if k_pages.dim() != 4:
            raise ValueError("k_pages must be [n_pages, n_kv_heads, page_size, head_dim]")
        n, h, page, d = k_pages.shape
        _dev(v_pages, "v_pages", k_pages.dtype, device=k_pages.device)
        if tuple(v_pages.shape) != (n, h, d, page):
            raise ValueError(f"v_pages must be [n_pages, n_kv_heads, head_dim, page_size] = {[n, h, d, page]}")
        if k_pages.dtype == torch.int8:
            for name, s in (("k_steps", k_steps), ("v_steps", v_steps)):
                _dev(s, name, torch.float32, device=k_pages.device)
                if tuple(s.shape) != (n, h, page):
                    raise ValueError(f"{name} must be [n_pages, n_kv_heads, page_size] = {[n, h, page]}")
        elif k_steps is not None or v_steps is not None:
            raise ValueError("k_steps and v_steps belong to an int8 cache")
        self.k_pages, self.v_pages, self.k_steps, self.v_steps = k_pages, v_pages, k_steps, v_steps
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = n, h, page, d
        self.dtype, self.device = k_pages.dtype, k_pages.device
        self._struct = _CacheStruct(*(None if t is None else t.data_ptr()
                                      for t in (k_pages, v_pages, k_steps, v_steps)),
                                    n, page, h, d, _DTYPES[k_pages.dtype])
        self._ref = C.byref(self._struct)

    def __setattr__(self, name, value):
        if "_ref" in self.__dict__:
            raise AttributeError(f"a KvCache's {name} cannot be set: make a new one over other tensors")
        object.__setattr__(self, name, value)


def ptq1_kv_cache(n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, dtype=torch.bfloat16,
                  device="cuda") -> KvCache:
    """A cache of its own memory (uninitialised: only what was written is ever used)."""
    if dtype not in _CACHE_TYPES:
        raise ValueError(f"dtype must be one of {_CACHE_TYPES}, got {dtype}")
    k = torch.empty((n_pages, n_kv_heads, page_size, head_dim), dtype=dtype, device=device)
    v = torch.empty((n_pages, n_kv_heads, head_dim, page_size), dtype=dtype, device=device)
    steps = [torch.empty((n_pages, n_kv_heads, page_size), dtype=torch.float32, device=device) for _ in range(2)] \
        if dtype == torch.int8 else (None, None)
    return KvCache(k, v, *steps)


def _elsewhere(device) -> bool:
    """The operands' device is not the current one (the call is then made under it)."""
    index = device.index
    return index is not None and index != torch._C._cuda_getDevice()


def _beside(device, stream) -> bool:
    """A stream is given that is not the operands' device's current one (the call is then made under it, _under)."""
    if stream is None:
        return False
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the call runs on {device}")
    return stream != torch.cuda.current_stream(device)


def _under(stream, device, fresh: bool, call, *args):
    """call(*args) with `stream` as the current one (as _on_its_stream does); fresh: the results are new tensors."""
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        result = call(*args)
    return _tied(result, here) if fresh else result


def _current_handle(device):
    return None if device.index is None else torch._C._cuda_getCurrentRawStream(device.index)


def _plain(t, dtype, numel: int, device) -> bool:
    """A contiguous tensor of exactly this type, size and device (_dev says what is wrong with any other)."""
    return type(t) is torch.Tensor and t.dtype is dtype and t.numel() == numel and t.device == device \
        and t.is_contiguous() and t.is_cuda


def _rows3(t: torch.Tensor, name: str, dtype, device) -> tuple[int, int, int, int]:
    """(rows, heads, head_dim, row stride) of a [rows, heads, head_dim] tensor whose rows may lie apart."""
    if type(t) is torch.Tensor and t.is_cuda and t.dtype in dtype and t.device == device and t.dim() == 3:
        rows, heads, d = t.shape
        sr, sh, sd = t.stride()
        if sd == 1 and sh == d and (sr >= heads * d or rows < 2):
            return rows, heads, d, sr if rows > 1 else heads * d
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not _on_device(t):
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows, heads, head_dim]")
    if t.dtype not in dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")
    rows, heads, d = t.shape
    sr, sh, sd = t.stride()
    if ((d > 1 and sd != 1) or (heads > 1 and sh != d)) and rows > 0 and heads > 0 and d > 0:
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if rows > 1:
        if sr < heads * d:
            raise ValueError(f"{name}: rows overlap one another (stride {sr})")
        return rows, heads, d, sr
    return rows, heads, d, heads * d


def _kv(cache) -> KvCache:
    if not isinstance(cache, KvCache):
        raise TypeError("cache must be a KvCache")
    return cache


def _table(block_table, batch, device):
    if type(block_table) is torch.Tensor and block_table.dtype is torch.int32 and block_table.is_cuda \
            and block_table.device == device and block_table.dim() == 2 and block_table.is_contiguous():
        rows, width = block_table.shape
        if rows == batch:
            return width
    _dev(block_table, "block_table", torch.int32, device=device)
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError(f"block_table must be [{batch}, max_pages]")
    return block_table.shape[1]


def _kv_write(q, k, v, slots, cache, positions, cos_sin, q_dtype, out, stream, norm):
    """Both writes; norm: None or (q_gain, k_gain, eps)."""
    kv = _kv(cache)
    dv = kv.device
    if _elsewhere(dv):
        with torch.cuda.device(dv):
            return _kv_write(q, k, v, slots, cache, positions, cos_sin, q_dtype, out, stream, norm)
    if _beside(dv, stream):
        return _under(stream, dv, out is None, _kv_write, q, k, v, slots, cache, positions, cos_sin, q_dtype, out, None, norm)
    n, h, d, ks = _rows3(k, "k", _FLOATS, dv)
    if h != kv.n_kv_heads or d != kv.head_dim:
        raise ValueError(f"k has {h} heads of {d}, the cache {kv.n_kv_heads} of {kv.head_dim}")
    src = k.dtype
    nv, hv, d2, vs = _rows3(v, "v", (src,), dv)
    if nv != n or hv != h or d2 != d:
        raise ValueError(f"v must be {[n, h, d]}")
    hq = qs = 0
    if q is not None:
        nq, hq, d3, qs = _rows3(q, "q", (src,), dv)
        if nq != n or d3 != d:
            raise ValueError(f"q must be [{n}, n_q_heads, {d}]")
        if q_dtype is None:
            q_dtype = src
        elif q_dtype not in _FLOATS:
            raise ValueError(f"q_dtype must be one of {_FLOATS}, got {q_dtype}")
    elif out is not None:
        raise ValueError("out needs q")
    if not _plain(slots, torch.int64, n, dv):
        _dev(slots, "slots", torch.int64, numel=n, device=dv)
    rot = n_pos = 0
    if cos_sin is not None:
        _dev(cos_sin, "cos_sin", torch.float32, device=dv)
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [n_positions, rot_dim]")
        n_pos, rot = cos_sin.shape
        if positions is None:
            raise ValueError("cos_sin needs positions")
    if positions is not None and not _plain(positions, torch.int32, n, dv):
        _dev(positions, "positions", torch.int32, numel=n, device=dv)
    if norm is not None:
        for name, gain in (("q_gain", norm[0]), ("k_gain", norm[1])):
            if gain is not None and not _plain(gain, torch.float32, d, dv):
                _dev(gain, name, torch.float32, numel=d, device=dv)
    handle = _current_handle(dv)
    if q is not None:
        if out is None:
            out = torch.empty_like(q, dtype=q_dtype, memory_format=torch.contiguous_format)
        else:
            _dev(out, "out", q_dtype, numel=n * hq * d, device=dv)
    rows = 0 if q is None else q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, _DTYPES[src], n, hq
    rest = (positions.data_ptr() if rot else 0, cos_sin.data_ptr() if rot else 0, n_pos, rot, slots.data_ptr(),
            0 if out is None else out.data_ptr(), _DTYPES[src if q is None else q_dtype], kv._ref, handle)
    if norm is None:
        status = lib().ptq1_kv_write(*rows, *rest)
    else:
        q_gain, k_gain, eps = norm
        status = lib().ptq1_kv_write_norm(*rows, 0 if q_gain is None else q_gain.data_ptr(),
                                          0 if k_gain is None else k_gain.data_ptr(), eps, *rest)
    if status:
        _check("ptq1_kv_write" if norm is None else "ptq1_kv_write_norm", status)
    return out


def ptq1_kv_write(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: KvCache,
                  positions: torch.Tensor | None = None, cos_sin: torch.Tensor | None = None, q_dtype=None,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Writes fresh tokens k, v [n, n_kv_heads, head_dim] into the cache at slots (int64 [n]; page * page_size +
    place, -1: not written), turning k and q [n, n_q_heads, head_dim] by the rows positions (int32 [n]) of
    cos_sin [n_positions, rot_dim] (rot_dim / 2 cosines, then sines) if it is given.  q, k and v may be parts of
    the rows of one stacked projection.  Returns the turned queries in q_dtype (q's own by default), or None
    without q."""
    return _kv_write(q, k, v, slots, cache, positions, cos_sin, q_dtype, out, stream, None)


def ptq1_kv_write_norm(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: KvCache,
                       q_gain: torch.Tensor | None = None, k_gain: torch.Tensor | None = None, eps: float = 1e-6,
                       positions: torch.Tensor | None = None, cos_sin: torch.Tensor | None = None, q_dtype=None,
                       out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """ptq1_kv_write with an RMS norm of every head of q and k ahead of the rotation: (mean(x^2) + eps)^(-1/2) * gain *
    x, gains fp32 [head_dim] (None: ones).  The other arguments and the result are ptq1_kv_write's."""
    return _kv_write(q, k, v, slots, cache, positions, cos_sin, q_dtype, out, stream, (q_gain, k_gain, eps))


def ptq1_kv_read(cache: KvCache, block_table: torch.Tensor, cu_seqlens: torch.Tensor, n_rows: int,
                 dtype=torch.bfloat16, out: tuple[torch.Tensor, torch.Tensor] | None = None, stream=None):
    """The first cu_seqlens[b + 1] - cu_seqlens[b] tokens of every sequence b (pages block_table[b], int32),
    packed: k and v [n_rows, n_kv_heads, head_dim] of dtype.  cu_seqlens int32 [batch + 1]."""
    kv = _kv(cache)
    dv = kv.device
    if _elsewhere(dv):
        with torch.cuda.device(dv):
            return ptq1_kv_read(cache, block_table, cu_seqlens, n_rows, dtype, out, stream)
    if _beside(dv, stream):
        return _under(stream, dv, out is None, ptq1_kv_read, cache, block_table, cu_seqlens, n_rows, dtype, out)
    _dev(cu_seqlens, "cu_seqlens", torch.int32, device=dv)
    batch = cu_seqlens.numel() - 1
    if batch < 0:
        raise ValueError("cu_seqlens must hold batch + 1 offsets")
    max_pages = _table(block_table, batch, dv)
    if dtype not in _FLOATS:
        raise ValueError(f"dtype must be one of {_FLOATS}, got {dtype}")
    if n_rows < 0:
        raise ValueError(f"n_rows = {n_rows} is negative")
    handle = _current_handle(dv)
    if out is None:
        h, d = kv.n_kv_heads, kv.head_dim
        k, v = torch.empty_strided((2, n_rows, h, d), (n_rows * h * d, h * d, d, 1), dtype=dtype, device=dv).unbind(0)
    else:
        k, v = out
        count = n_rows * kv.n_kv_heads * kv.head_dim
        _dev(k, "k_out", dtype, numel=count, device=dv)
        _dev(v, "v_out", dtype, numel=count, device=dv)
    status = lib().ptq1_kv_read(kv._ref, block_table.data_ptr(), max_pages, cu_seqlens.data_ptr(), batch, n_rows,
                                k.data_ptr(), v.data_ptr(), _DTYPES[dtype], handle)
    if status:
        _check("ptq1_kv_read", status)
    return k, v


def _bound(n: int) -> int:
    """A bound of the caller's as the C calls take it: past 64 bits (where ctypes would keep the lowest ones) the largest
    there is."""
    return n if -1 << 63 <= n < 1 << 63 else (1 << 63) - 1 if n > 0 else -1


def _attn_decode(q, cache, block_table, seq_lens, scale, max_len, out, ws, stream, seen):
    """Both calls of single tokens; seen: () or (window, sinks)."""
    kv = _kv(cache)
    dv = kv.device
    if _elsewhere(dv):
        with torch.cuda.device(dv):
            return _attn_decode(q, cache, block_table, seq_lens, scale, max_len, out, ws, stream, seen)
    if _beside(dv, stream):
        return _under(stream, dv, out is None, _attn_decode, q, cache, block_table, seq_lens, scale, max_len, out, ws, None,
                      seen)
    _dev(q, "q", _FLOATS, device=dv)
    if q.dim() != 3 or q.shape[2] != kv.head_dim:
        raise ValueError(f"q must be [batch, n_q_heads, {kv.head_dim}]")
    batch, hq, d = q.shape
    max_pages = _table(block_table, batch, dv)
    if not _plain(seq_lens, torch.int32, batch, dv):
        _dev(seq_lens, "seq_lens", torch.int32, numel=batch, device=dv)
    max_len = max_pages * kv.page_size if max_len is None else _bound(max_len)
    handle = _current_handle(dv)
    if seen:
        if (seen[0] | seen[1]) >> 63:  # (cheaper than two calls)
            seen = _bound(seen[0]), _bound(seen[1])
        name, call, size = "ptq1_attn_decode_window", lib().ptq1_attn_decode_window, lib().ptq1_attn_decode_window_workspace_bytes
    else:
        name, call, size = "ptq1_attn_decode", lib().ptq1_attn_decode, lib().ptq1_attn_decode_workspace_bytes
    wsb = size(batch, hq, kv.n_kv_heads, d, max_len, *seen)
    if ws is None:
        if wsb:
            ws = torch.empty_strided((wsb,), (1,), dtype=torch.uint8, device=dv)
    else:
        ws, wsb = _ws(wsb, dv, ws)
    if out is None:
        out = torch.empty_like(q)
    else:
        _dev(out, "out", q.dtype, numel=q.numel(), device=dv)
    status = call(q.data_ptr(), _DTYPES[q.dtype], batch, hq, kv._ref, block_table.data_ptr(), max_pages,
                  seq_lens.data_ptr(), max_len, *seen, d ** -0.5 if scale is None else scale, out.data_ptr(),
                  0 if ws is None else ws.data_ptr(), wsb, handle)
    if status:
        _check(name, status)
    return out


def ptq1_attn_decode(q: torch.Tensor, cache: KvCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                     scale: float | None = None, max_len: int | None = None, out: torch.Tensor | None = None,
                     ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of one new token per sequence, q [batch, n_q_heads, head_dim], over the first seq_lens[b] (int32)
    tokens of its pages block_table[b] (int32 [batch, max_pages]).  scale: 1 / sqrt(head_dim) by default; max_len: a
    bound on seq_lens (the table's by default).  ws: optional scratch of at least workspace_bytes("attn_decode",
    batch, n_q_heads, n_kv_heads, head_dim, max_len) bytes."""
    return _attn_decode(q, cache, block_table, seq_lens, scale, max_len, out, ws, stream, ())


def ptq1_attn_decode_window(q: torch.Tensor, cache: KvCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                            window: int, sinks: int = 0, scale: float | None = None, max_len: int | None = None,
                            out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """ptq1_attn_decode over the last `window` tokens of every sequence (the new one among them) and its first `sinks`
    alone.  Pages that hold neither are not read: their entries of block_table may be anything.  ws: optional scratch of
    at least workspace_bytes("attn_decode_window", batch, n_q_heads, n_kv_heads, head_dim, max_len, window, sinks)
    bytes."""
    return _attn_decode(q, cache, block_table, seq_lens, scale, max_len, out, ws, stream, (window, sinks))


def ptq1_attn_chunk(q: torch.Tensor, cache: KvCache, block_table: torch.Tensor, cu_q: torch.Tensor,
                    seq_lens: torch.Tensor, window: int = 0, sinks: int = 0, scale: float | None = None,
                    max_q: int | None = None, max_len: int | None = None, out: torch.Tensor | None = None,
                    ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of the last tokens of every sequence over the cache that holds them already (ptq1_kv_write first): rows
    cu_q[b] .. cu_q[b + 1] (int32 [batch + 1]) of q [n_q_rows, n_q_heads, head_dim] (the cache's own 16-bit type, fp16 or
    bf16 over an int8 cache; rows may lie apart) are the last of sequence b's seq_lens[b] (int32) tokens, whose pages are
    block_table[b] (int32 [batch, max_pages]).  Causal; window > 0: over the last `window` tokens (the query's own among
    them) and the first `sinks` alone; pages that no query sees are not read.  scale: 1 / sqrt(head_dim) by default;
    max_q, max_len: bounds on the sequences' queries and tokens (all rows, the table's by default); where max_q * n_q_heads
    / n_kv_heads is at most 32 a kernel for few rows runs, whose weights have 16 bits and more (of many rows' 8 in bf16, 11
    in fp16), so give max_q where a batch has few queries a sequence.  ws: optional scratch of at least
    workspace_bytes("attn_chunk", batch, n_q_rows, max_q, n_q_heads, n_kv_heads, head_dim, max_len, window,
    sinks) bytes."""
    kv = _kv(cache)
    dv = kv.device
    if _elsewhere(dv):
        with torch.cuda.device(dv):
            return ptq1_attn_chunk(q, cache, block_table, cu_q, seq_lens, window, sinks, scale, max_q, max_len, out, ws,
                                   stream)
    if _beside(dv, stream):
        return _under(stream, dv, out is None, ptq1_attn_chunk, q, cache, block_table, cu_q, seq_lens, window, sinks, scale,
                      max_q, max_len, out, ws)
    rows, hq, d, qs = _rows3(q, "q", _SIXTEEN, dv)
    if d != kv.head_dim:
        raise ValueError(f"q must be [n_q_rows, n_q_heads, {kv.head_dim}]")
    _dev(cu_q, "cu_q", torch.int32, device=dv)
    batch = cu_q.numel() - 1
    if batch < 0:
        raise ValueError("cu_q must hold batch + 1 offsets")
    max_pages = _table(block_table, batch, dv)
    if not _plain(seq_lens, torch.int32, batch, dv):
        _dev(seq_lens, "seq_lens", torch.int32, numel=batch, device=dv)
    max_q = rows if max_q is None else max_q
    max_len = max_pages * kv.page_size if max_len is None else max_len
    if (max_q | max_len | window | sinks) >> 63:
        max_q, max_len, window, sinks = map(_bound, (max_q, max_len, window, sinks))
    handle = _current_handle(dv)
    wsb = lib().ptq1_attn_chunk_workspace_bytes(batch, rows, max_q, hq, kv.n_kv_heads, d, max_len, window, sinks)
    if ws is None:
        if wsb:
            ws = torch.empty_strided((wsb,), (1,), dtype=torch.uint8, device=dv)
    else:
        ws, wsb = _ws(wsb, dv, ws)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _dev(out, "out", q.dtype, numel=rows * hq * d, device=dv)
    status = lib().ptq1_attn_chunk(q.data_ptr(), qs, _DTYPES[q.dtype], cu_q.data_ptr(), batch, rows, max_q, hq, kv._ref,
                                   block_table.data_ptr(), max_pages, seq_lens.data_ptr(), max_len, window, sinks,
                                   d ** -0.5 if scale is None else scale, out.data_ptr(),
                                   0 if ws is None else ws.data_ptr(), wsb, handle)
    if status:
        _check("ptq1_attn_chunk", status)
    return out


def ptq1_attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
                     max_q: int | None = None, max_k: int | None = None, causal: bool = True,
                     scale: float | None = None, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Attention over packed prompts: q [n_q_rows, n_q_heads, head_dim], k and v [n_k_rows, n_kv_heads, head_dim]
    (fp16 or bf16; rows may lie apart), sequence b's rows cu_q[b] .. cu_q[b + 1] and cu_k[b] .. cu_k[b + 1] (int32
    [batch + 1]).  causal: the last query of a sequence sees its last key.  max_q, max_k: bounds on the sequences'
    query and key counts (all rows by default).  scale: 1 / sqrt(head_dim) by default.  ws: optional scratch of at
    least workspace_bytes("attn_prompt", batch, n_q_rows, min(max_k, n_k_rows), n_q_heads, n_kv_heads, head_dim)
    bytes."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dv = q.device
    if _elsewhere(dv):
        with torch.cuda.device(dv):
            return ptq1_attn_prompt(q, k, v, cu_q, cu_k, max_q, max_k, causal, scale, out, ws, stream)
    if _beside(dv, stream):
        return _under(stream, dv, out is None, ptq1_attn_prompt, q, k, v, cu_q, cu_k, max_q, max_k, causal, scale, out, ws)
    nq, hq, d, qs = _rows3(q, "q", _SIXTEEN, dv)
    kind = q.dtype
    nk, hkv, dk, ks = _rows3(k, "k", (kind,), dv)
    nv, hv, d2, vs = _rows3(v, "v", (kind,), dv)
    if dk != d or nv != nk or hv != hkv or d2 != d:
        raise ValueError(f"k and v must both be [n_k_rows, n_kv_heads, {d}]")
    _dev(cu_q, "cu_q", torch.int32, device=dv)
    batch = cu_q.numel() - 1
    if batch < 0:
        raise ValueError("cu_q must hold batch + 1 offsets")
    if not _plain(cu_k, torch.int32, batch + 1, dv):
        _dev(cu_k, "cu_k", torch.int32, numel=batch + 1, device=dv)
    max_q = nq if max_q is None else min(max_q, nq)
    max_k = nk if max_k is None else min(max_k, nk)
    handle = _current_handle(dv)
    wsb = lib().ptq1_attn_prompt_workspace_bytes(batch, nq, max_k, hq, hkv, d)
    if ws is None:
        if wsb:
            ws = torch.empty_strided((wsb,), (1,), dtype=torch.uint8, device=dv)
    else:
        ws, wsb = _ws(wsb, dv, ws)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _dev(out, "out", kind, numel=nq * hq * d, device=dv)
    status = lib().ptq1_attn_prompt(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, _DTYPES[kind], cu_q.data_ptr(),
                                    cu_k.data_ptr(), batch, nq, nk, max_q, max_k, hq, hkv, d, 1 if causal else 0,
                                    d ** -0.5 if scale is None else scale, out.data_ptr(),
                                    0 if ws is None else ws.data_ptr(), wsb, handle)
    if status:
        _check("ptq1_attn_prompt", status)
    return out


def ffn_workspace_offsets(m: int, d: int, f: int, fmt: str = "ptq1") -> tuple[int, int, int]:
    """Byte offsets of (g, u, h) in an FFN block's workspace (-1: not stored on that path)."""
    out = (C.c_int64 * 3)()
    fn = "pq2_ffn_workspace_offsets" if fmt == "pq2" else "ptq1_ffn_workspace_offsets"
    _check(fn, getattr(lib(), fn)(m, d, f, C.cast(out, p)))
    return tuple(out)


def workspace_bytes(kind: str, *shape) -> int:
    fn = {"matvec": "ptq1_matvec_workspace_bytes", "gate_up": "ptq1_gate_up_workspace_bytes",
          "gemm": "ptq1_gemm_workspace_bytes", "ffn": "ptq1_ffn_workspace_bytes",
          "pq2_matvec": "pq2_matvec_workspace_bytes", "pq2_gemm": "pq2_gemm_workspace_bytes",
          "attn_decode": "ptq1_attn_decode_workspace_bytes",
          "attn_decode_window": "ptq1_attn_decode_window_workspace_bytes",
          "attn_chunk": "ptq1_attn_chunk_workspace_bytes",
          "attn_prompt": "ptq1_attn_prompt_workspace_bytes"}[kind]
    return int(getattr(lib(), fn)(*map(_bound, shape)))


# -------------------------------------------------------------- profiling ----

_hip = None


def _hiprt():
    """The HIP runtime (already loaded by torch), for raw events."""
    global _hip
    if _hip is None:
        h = C.CDLL("libamdhip64.so")
        h.hipEventCreate.argtypes = [C.POINTER(C.c_void_p)]
        h.hipEventDestroy.argtypes = [C.c_void_p]
        h.hipEventSynchronize.argtypes = [C.c_void_p]
        h.hipEventElapsedTime.argtypes = [C.POINTER(C.c_float), C.c_void_p, C.c_void_p]
        _hip = h
    return _hip


class KernelTimer:
    """Times the next `count` launches of one kernel family inside any call
    (ptq1_profile_arm): HIP events recorded by the library on the stream of
    each launch.  Use as a context manager around the timed calls, then read
    `durations_ms()` after a device synchronisation."""

    def __init__(self, kernel: str, count: int):
        self.kernel = kernel.encode()
        self.count = count
        hip = _hiprt()
        self._start = (C.c_void_p * count)()
        self._stop = (C.c_void_p * count)()
        for arr in (self._start, self._stop):
            for i in range(count):
                ev = C.c_void_p()
                if hip.hipEventCreate(C.byref(ev)) != 0:
                    raise RuntimeError("hipEventCreate failed")
                arr[i] = ev

    def __enter__(self):
        _check("ptq1_profile_arm", lib().ptq1_profile_arm(self.kernel, C.cast(self._start, p),
                                                          C.cast(self._stop, p), self.count))
        return self

    def __exit__(self, *exc):
        self.launches = lib().ptq1_profile_count(self.kernel)
        _check("ptq1_profile_arm", lib().ptq1_profile_arm(self.kernel, None, None, 0))
        return False

    def durations_ms(self) -> list[float]:
        hip = _hiprt()
        out = []
        for i in range(self.launches):
            if hip.hipEventSynchronize(self._stop[i]) != 0:
                raise RuntimeError("hipEventSynchronize failed")
            ms = C.c_float()
            if hip.hipEventElapsedTime(C.byref(ms), self._start[i], self._stop[i]) != 0:
                raise RuntimeError("hipEventElapsedTime failed")
            out.append(ms.value)
        return out

    def close(self):
        hip = _hiprt()
        for arr in (self._start, self._stop):
            for i in range(self.count):
                if arr[i]:
                    hip.hipEventDestroy(arr[i])
                    arr[i] = None


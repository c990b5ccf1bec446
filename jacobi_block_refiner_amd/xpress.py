"""Thin ctypes binding of ``libxpress.so`` (the C ABI in ``include/xpress.h``).

Argument marshalling only: tensors are passed as device pointers together with the current HIP
stream of PyTorch, and every step of the method runs in the library's HIP kernels. There is no
fallback: if the library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import re
from dataclasses import dataclass
from pathlib import Path

import torch

PKG = Path(__file__).resolve().parent
LIB_PATH = PKG / "libxpress.so"
HEADER = PKG.parent / "include" / "xpress.h"

OK, ERR_ARG, ERR_WORKSPACE, ERR_HIP = 0, 1, 2, 3
LAT_ROWS, LAT_FRAGMENTS = 0, 1
INIT_FROM_BASE = 1
STOP_AT_FIXED_POINT = 2


class XpressError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"xpress status {status}: {message}")
        self.status = status


class _Weights(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("r", ctypes.c_int32), ("H", ctypes.c_int32),
        ("M", ctypes.c_int32), ("V", ctypes.c_int64),
        ("w1", ctypes.c_void_p), ("down_h", ctypes.c_void_p), ("down_g", ctypes.c_void_p),
        ("in_proj", ctypes.c_void_p), ("mix_L", ctypes.c_void_p), ("w_gate", ctypes.c_void_p),
        ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p), ("w2", ctypes.c_void_p),
        ("w1p", ctypes.c_void_p),
    ]


class _Cache(ctypes.Structure):
    _fields_ = [
        ("n_layers", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page", ctypes.c_int32),
        ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("dtype", ctypes.c_uint32),
        ("rows", ctypes.c_int32), ("table_ld", ctypes.c_int32),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("table", ctypes.c_void_p), ("len", ctypes.c_void_p), ("ref", ctypes.c_void_p),
    ]


_lib = None


def declared_symbols() -> list[str]:
    """Function names declared in include/xpress.h."""
    text = HEADER.read_text()
    return re.findall(r"^(?:xpress_status|const char\*)\s+(xpress_\w+)\(", text, flags=re.M)


def lib() -> ctypes.CDLL:
    """The loaded library. Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with jacobi_block_refiner_amd.build.build()")
        L = ctypes.CDLL(str(LIB_PATH))
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        f32, u32 = ctypes.c_float, ctypes.c_uint32
        W, C = ctypes.POINTER(_Weights), ctypes.POINTER(_Cache)
        sig = {
            "xpress_workspace_size": [i32, i32, i32, i64, i32, i32, ctypes.POINTER(sz)],
            "xpress_fold_mixer": [P, i32, i32, P, P],
            "xpress_fold_embedding": [W, P, P],
            "xpress_hidden_cache": [W, P, i32, P, P, sz, P],
            "xpress_initial_block": [P, i64, P, i32, i32, i64, P, P],
            "xpress_latent_pass": [W, P, P, P, i32, P, ctypes.c_uint32, P, sz, P],
            "xpress_readout_argmax": [W, P, ctypes.c_uint32, P, i64, i32, P, P, P, sz, P],
            "xpress_readout_tiles": [i64, i32, ctypes.POINTER(i32)],
            "xpress_readout_partials": [W, P, ctypes.c_uint32, P, i64, i32, P, P],
            "xpress_argmax_reduce": [P, i32, i32, i32, P, P, P],
            "xpress_topc_prepare": [W, P, i64, i32, i32, P, P, P, P, sz, P],
            "xpress_readout_argmax_topc": [P, P, P, P, i32, i32, i32, i32, P, P, P],
            "xpress_readout_argmax_topc_ids": [W, P, P, P, i32, i32, P, P, P],
            "xpress_jacobi_step": [W, P, P, i64, P, P, i32, i32, i32, ctypes.c_uint32, P, P, P,
                                   sz, P],
            "xpress_jacobi_step_noalloc": [W, P, P, i64, P, P, i32, i32, i32, ctypes.c_uint32,
                                           P, P, P],
            "xpress_jacobi_step_graph": [W, P, P, i64, P, P, i32, i32, i32, ctypes.c_uint32, P, P,
                                         P, sz, ctypes.POINTER(ctypes.c_void_p)],
            "xpress_graph_launch": [P, P],
            "xpress_graph_destroy": [P],
            "xpress_cache_workspace_size": [C, i32, ctypes.POINTER(sz)],
            "xpress_cache_fork": [C, P, P, i32, P],
            "xpress_cache_extend": [C, P, i32, P, i32, P, P, sz, P],
            "xpress_cache_append": [C, i32, P, P, i64, P, i32, i32, P],
            "xpress_cache_append_if": [C, P, i32, P, P, i64, P, i32, i32, P],
            "xpress_cache_read": [C, i32, P, i32, P, i32, P, P, i64, P],
            "xpress_cache_trim": [C, P, i32, P, P],
            "xpress_cache_trim_if": [C, P, P, i32, P, P],
            "xpress_cache_compact": [C, P, P, sz, P],
            "xpress_attention_workspace_size": [C, i32, i32, i32, ctypes.POINTER(sz)],
            "xpress_block_attention": [C, i32, P, i64, P, i32, i32, i32, f32, i32, P, i64, P, P,
                                       sz, P],
            "xpress_verify_workspace_size": [i32, i32, i64, ctypes.POINTER(sz)],
            "xpress_verify_draft": [P, u32, i64, P, P, P, u32, i64, P, P, i32, i32, i64, P, P, P,
                                    P, sz, P],
            "xpress_logprobs_workspace_size": [i32, i64, i32, ctypes.POINTER(sz)],
            "xpress_token_logprobs": [P, u32, i64, P, P, i32, i32, i64, i32, P, P, P, P, P, P, sz, P],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.xpress_last_error.restype = ctypes.c_char_p
        L.xpress_last_error.argtypes = []
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != OK:
        msg = lib().xpress_last_error().decode()
        raise XpressError(status, msg)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


# The current stream's handle alone: building torch's Stream object around it takes 2.9 us, this 0.3.
# It is no public function, so a torch without it takes the object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream() -> int:
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _bf16(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    return t


def _at_least(t, n: int, name: str) -> None:
    """The C ABI takes bare pointers and a block count: a tensor shorter than that count implies
    would be read or written past its end, so it is refused here."""
    if t is not None and t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, fewer than the {n} that N implies")


def _base_rows(base, rows: int, V: int) -> None:
    _bf16(base, "base")
    if base.stride(1) != 1 or base.dim() != 2:
        raise ValueError("base must be a [rows, V] view with unit column stride")
    if base.shape[0] < rows or base.shape[1] != V:
        raise ValueError(f"base is {tuple(base.shape)}; the call needs [{rows}, {V}]")


def _step_inputs(w, h, base, anchor, am1, blk) -> int:
    """N from blk [N, B]; h, base, anchor and am1 must cover N blocks."""
    d = w.dims
    N, B = blk.shape
    if B != d["B"]:
        raise ValueError(f"blk has {B} slots per block, the weights {d['B']}")
    _at_least(_bf16(h, "h"), N * B * d["H"], "h")
    _base_rows(base, N * (B - 1), d["V"])
    _at_least(anchor, N, "anchor")
    _at_least(am1, N, "am1")
    return N


@dataclass
class Weights:
    """Device bf16 weights of one refiner head, ``nn.Linear`` layouts; ``mix_L`` is folded and
    stored [B, B, r]."""

    w1: torch.Tensor
    down_h: torch.Tensor
    down_g: torch.Tensor
    in_proj: torch.Tensor
    mix_L: torch.Tensor
    w_gate: torch.Tensor
    w_up: torch.Tensor
    w_down: torch.Tensor
    w2: torch.Tensor
    # optional fp32 [V, r] projected embedding table (fold_embedding); None: not used
    w1p: torch.Tensor | None = None

    @property
    def dims(self):
        V, r = self.w1.shape
        return dict(B=self.mix_L.shape[1], r=r, H=self.down_h.shape[1], M=self.w_gate.shape[0],
                    V=V)

    def struct(self) -> _Weights:
        d = self.dims
        s = _Weights(B=d["B"], r=d["r"], H=d["H"], M=d["M"], V=d["V"])
        for k in ("w1", "down_h", "down_g", "in_proj", "mix_L", "w_gate", "w_up", "w_down", "w2"):
            t = _bf16(getattr(self, k), k)
            if not t.is_contiguous():
                raise ValueError(f"{k} must be contiguous")
            setattr(s, k, t.data_ptr())
        if self.w1p is not None:
            t = self.w1p
            if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
                raise TypeError("w1p must be a contiguous CUDA float32 tensor")
            if tuple(t.shape) != (d["V"], d["r"]):
                raise ValueError(f"w1p shape {tuple(t.shape)} != (V, r) = ({d['V']}, {d['r']})")
            s.w1p = t.data_ptr()
        return s


def workspace_size(n_max: int, B: int, r: int, V: int, C: int, k_max: int) -> int:
    out = ctypes.c_size_t()
    _check(lib().xpress_workspace_size(n_max, B, r, V, C, k_max, ctypes.byref(out)))
    return int(out.value)


def alloc_workspace(n_max: int, B: int, r: int, V: int, C: int, k_max: int, device="cuda"):
    n = workspace_size(n_max, B, r, V, C, k_max)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def fold_mixer(raw: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """raw: [r, B, B] bf16 -> folded mixer [B, B, r] (channel innermost)."""
    raw = _bf16(raw, "raw").contiguous()
    r, B, _ = raw.shape
    out = torch.empty(B, B, r, dtype=raw.dtype, device=raw.device) if out is None else out
    _check(lib().xpress_fold_mixer(_ptr(raw), r, B, _ptr(out), _stream()))
    return out


def fold_embedding(w: Weights, out: torch.Tensor | None = None) -> torch.Tensor:
    """Projected embedding table w1p [V, r] fp32: in_proj's embedding block applied to every row
    of w1 (set it as ``w.w1p`` to run the latent stage as two launches instead of three)."""
    d = w.dims
    s = w.struct()
    out = (torch.empty(d["V"], d["r"], dtype=torch.float32, device=w.w1.device)
           if out is None else out)
    _check(lib().xpress_fold_embedding(ctypes.byref(s), _ptr(out), _stream()))
    return out


def hidden_cache(w: Weights, h: torch.Tensor, xh: torch.Tensor, ws: torch.Tensor) -> torch.Tensor:
    s = w.struct()
    N = h.shape[0]
    _at_least(_bf16(h, "h"), N * w.dims["B"] * w.dims["H"], "h")
    _at_least(xh, N * w.dims["B"] * w.dims["r"], "xh")
    _check(lib().xpress_hidden_cache(ctypes.byref(s), _ptr(_bf16(h, "h")), N, _ptr(xh), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream()))
    return xh


def initial_block(base: torch.Tensor, anchor: torch.Tensor, blk: torch.Tensor) -> torch.Tensor:
    N, B = blk.shape
    _base_rows(base, N * (B - 1), base.shape[1])
    _at_least(anchor, N, "anchor")
    _check(lib().xpress_initial_block(ctypes.c_void_p(base.data_ptr()), base.stride(0),
                                      _ptr(anchor), N, B, base.shape[1], _ptr(blk), _stream()))
    return blk


def lat_buffer(N: int, B: int, r: int, layout: int = LAT_ROWS, device="cuda") -> torch.Tensor:
    """A latent buffer for N blocks in `layout` (fragment order: whole 32-row tiles)."""
    rows = N * (B - 1)
    if layout == LAT_FRAGMENTS:
        rows = (rows + 31) // 32 * 32
    return torch.empty(rows, r, dtype=torch.bfloat16, device=device)


def latent_pass(w: Weights, blk, am1, xh, lat, ws: torch.Tensor, layout: int = LAT_ROWS) -> torch.Tensor:
    s = w.struct()
    N = blk.shape[0]
    _at_least(am1, N, "am1")
    _at_least(xh, N * w.dims["B"] * w.dims["r"], "xh")
    _at_least(lat, N * (w.dims["B"] - 1) * w.dims["r"], "lat")
    _check(lib().xpress_latent_pass(ctypes.byref(s), _ptr(blk), _ptr(am1), _ptr(xh), N,
                                    _ptr(lat), layout, _ptr(ws), ws.numel() * ws.element_size(),
                                    _stream()))
    return lat


def readout_argmax(w: Weights, lat, base, blk, ws, changed=None, layout: int = LAT_ROWS) -> torch.Tensor:
    s = w.struct()
    N = blk.shape[0]
    _base_rows(base, N * (w.dims["B"] - 1), w.dims["V"])
    _at_least(lat, N * (w.dims["B"] - 1) * w.dims["r"], "lat")
    _check(lib().xpress_readout_argmax(ctypes.byref(s), _ptr(lat), layout,
                                       ctypes.c_void_p(base.data_ptr()), base.stride(0), N,
                                       _ptr(blk), _ptr(changed), _ptr(ws),
                                       ws.numel() * ws.element_size(), _stream()))
    return blk


def readout_tiles(V: int, rows: int) -> int:
    out = ctypes.c_int32()
    _check(lib().xpress_readout_tiles(V, rows, ctypes.byref(out)))
    return int(out.value)


def readout_partials(w: Weights, lat, base, part: torch.Tensor, layout: int = LAT_ROWS) -> torch.Tensor:
    """part: int32/uint32-compatible tensor [ntiles, rows, 2] (value bits, id), range-major."""
    s = w.struct()
    rows = part.shape[1]
    N = rows // (w.dims["B"] - 1)
    _base_rows(base, N * (w.dims["B"] - 1), w.dims["V"])
    _at_least(lat, N * (w.dims["B"] - 1) * w.dims["r"], "lat")
    _check(lib().xpress_readout_partials(ctypes.byref(s), _ptr(lat), layout,
                                         ctypes.c_void_p(base.data_ptr()), base.stride(0), N,
                                         _ptr(part), _stream()))
    return part


def argmax_reduce(part: torch.Tensor, blk: torch.Tensor, changed=None) -> torch.Tensor:
    N, B = blk.shape
    ntiles = part.shape[0]
    _check(lib().xpress_argmax_reduce(_ptr(part), ntiles, N, B, _ptr(blk), _ptr(changed),
                                      _stream()))
    return blk


def topc_prepare(w: Weights, base, N: int, C: int, cand, base_c, w2c=None, ws=None):
    """w2c None: candidates and base_c only (for readout_argmax_topc_ids)."""
    s = w.struct()
    _base_rows(base, N * (w.dims["B"] - 1), w.dims["V"])
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().xpress_topc_prepare(ctypes.byref(s), ctypes.c_void_p(base.data_ptr()),
                                     base.stride(0), N, C, _ptr(cand), _ptr(base_c), _ptr(w2c),
                                     _ptr(ws), nbytes, _stream()))
    return cand, base_c, w2c


def readout_argmax_topc(lat, w2c, base_c, cand, blk, changed=None) -> torch.Tensor:
    N, B = blk.shape
    rows, c, r = w2c.shape
    _check(lib().xpress_readout_argmax_topc(_ptr(lat), _ptr(w2c), _ptr(base_c), _ptr(cand), N, B,
                                            r, c, _ptr(blk), _ptr(changed), _stream()))
    return blk


def readout_argmax_topc_ids(w: Weights, lat, base_c, cand, blk, changed=None) -> torch.Tensor:
    """The top-C readout reading w2[cand] through the ids (no gathered copy)."""
    s = w.struct()
    N = blk.shape[0]
    c = cand.shape[-1]
    _check(lib().xpress_readout_argmax_topc_ids(ctypes.byref(s), _ptr(lat), _ptr(base_c),
                                                _ptr(cand), N, c, _ptr(blk), _ptr(changed),
                                                _stream()))
    return blk


def jacobi_step(w: Weights, h, base, anchor, am1, blk, *, K: int, C: int = 0,
                flags: int = INIT_FROM_BASE, ws: torch.Tensor, passes_run=None) -> torch.Tensor:
    s = w.struct()
    N = _step_inputs(w, h, base, anchor, am1, blk)
    _check(lib().xpress_jacobi_step(ctypes.byref(s), _ptr(_bf16(h, "h")),
                                    ctypes.c_void_p(base.data_ptr()), base.stride(0), _ptr(anchor),
                                    _ptr(am1), N, K, C, flags, _ptr(blk), _ptr(passes_run),
                                    _ptr(ws), ws.numel() * ws.element_size(), _stream()))
    return blk


def jacobi_step_noalloc(w: Weights, h, base, anchor, am1, blk, *, K: int, C: int = 0,
                        flags: int = INIT_FROM_BASE, passes_run=None) -> torch.Tensor:
    """``jacobi_step`` on the library's own static per-GPU scratch: no workspace argument and no
    allocation. Calls that overlap on one GPU share that scratch and race."""
    s = w.struct()
    N = _step_inputs(w, h, base, anchor, am1, blk)
    _check(lib().xpress_jacobi_step_noalloc(ctypes.byref(s), _ptr(_bf16(h, "h")),
                                            ctypes.c_void_p(base.data_ptr()), base.stride(0),
                                            _ptr(anchor), _ptr(am1), N, K, C, flags, _ptr(blk),
                                            _ptr(passes_run), _stream()))
    return blk


class StepGraph:
    """A draft step recorded once as a HIP graph (``xpress_jacobi_step_graph``); ``launch()``
    replays the whole step on the current stream with one call. The tensors given at creation are
    kept referenced: the graph reads and writes them in place on every launch."""

    def __init__(self, w: Weights, h, base, anchor, am1, blk, *, K: int, C: int = 0,
                 flags: int = INIT_FROM_BASE, ws: torch.Tensor, passes_run=None):
        s = w.struct()
        N = _step_inputs(w, h, base, anchor, am1, blk)
        self._keep = (w, h, base, anchor, am1, blk, ws, passes_run)
        self._handle = ctypes.c_void_p()
        _check(lib().xpress_jacobi_step_graph(
            ctypes.byref(s), _ptr(_bf16(h, "h")), ctypes.c_void_p(base.data_ptr()),
            base.stride(0), _ptr(anchor), _ptr(am1), N, K, C, flags, _ptr(blk), _ptr(passes_run),
            _ptr(ws), ws.numel() * ws.element_size(), ctypes.byref(self._handle)))

    def launch(self) -> None:
        if not self._handle:
            raise RuntimeError("graph was closed")
        _check(lib().xpress_graph_launch(self._handle, _stream()))

    def close(self) -> None:
        if self._handle:
            _check(lib().xpress_graph_destroy(self._handle))
            self._handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------- the target's side of a draft step

BF16, F16, F32 = 0, 1, 2
MX4 = 16  # of a cache: its values are held in 4 bits
_DTYPES = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}


def _list(t, n: int, dtype, name: str):
    """A device list of at least n elements of one type, as a pointer; None passes as NULL."""
    if t is None:
        return None
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA {dtype} tensor")
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, the call needs {n}")
    return t.data_ptr()


def _tokens(t, n: int, width: int, dtype, name: str) -> int:
    """A [n, width] view with unit column stride; its row stride in elements (of a single row, where
    a view may have any: the width)."""
    if t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA {dtype} tensor")
    shape = t.shape
    if len(shape) != 2 or shape[0] < n or shape[1] != width or (width > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} is {tuple(shape)}; the call needs [{n}, {width}] rows with unit "
                         "column stride")
    return t.stride(0) if n > 1 else width


def _ws(ws):
    if not ws.is_cuda or not ws.is_contiguous():
        raise TypeError("ws must be a contiguous CUDA tensor")
    return ws.data_ptr(), ws.numel() * ws.element_size()


@dataclass
class Cache:
    """A paged K/V cache (``xpress_cache``): pools of pages, one table row a sequence, tokens a
    sequence and holders a page. The caller owns the tensors; the struct is built with the object, and
    anew when one of its tensors is replaced. Pools of bytes hold values of 4 bits."""

    k: torch.Tensor  # [n_layers, n_pages, Hkv, page, D] bf16 or fp16, or
    v: torch.Tensor  # [n_layers, n_pages, Hkv, page/16, 17*D/2] uint8
    table: torch.Tensor  # [rows, table_ld] int32, -1 past a row's pages
    length: torch.Tensor  # [rows] int32
    ref: torch.Tensor  # [n_pages] int32
    dtype: torch.dtype | None = None  # of the values; None: the pools' (bytes: bf16)

    def __post_init__(self):
        if self.k.dim() != 5 or self.v.shape != self.k.shape:
            raise ValueError("k and v must be [n_layers, n_pages, Hkv, page, D]")
        mx4 = self.k.dtype == torch.uint8
        if mx4 and self.k.shape[4] % 17:
            raise ValueError("k and v of 4 bits must be [n_layers, n_pages, Hkv, page/16, 17*D/2]")
        if self.table.dim() != 2 or self.length.shape != self.table.shape[:1]:
            raise ValueError("table must be [rows, table_ld] and length [rows]")
        if self.ref.shape != self.k.shape[1:2]:
            raise ValueError("ref must be [n_pages]")
        if self.k.dtype not in (torch.bfloat16, torch.float16, torch.uint8):
            raise TypeError("k must be bfloat16 or float16, or uint8 for 4 bits")
        values = self.dtype or (torch.bfloat16 if mx4 else self.k.dtype)
        if values not in ((torch.bfloat16, torch.float16) if mx4 else (self.k.dtype,)):
            raise TypeError(f"a cache of {self.k.dtype} pools cannot hold {values}")
        for name, dtype in (("k", self.k.dtype), ("v", self.k.dtype), ("table", torch.int32),
                            ("length", torch.int32), ("ref", torch.int32)):
            t = getattr(self, name)
            if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous CUDA {dtype} tensor")
        n_layers, n_pages, Hkv, page, D = self.k.shape
        if mx4:
            page, D = page * 16, D // 17 * 2
        rows, ld = self.table.shape
        self._struct = _Cache(n_layers, n_pages, page, Hkv, D, _DTYPES[values] + (MX4 if mx4 else 0),
                              rows, ld, self.k.data_ptr(), self.v.data_ptr(), self.table.data_ptr(),
                              self.length.data_ptr(), self.ref.data_ptr())
        self._ref = ctypes.byref(self._struct)
        self._dtype, self._width, self._D, self.page = values, Hkv * D, D, page

    def __setattr__(self, name, value):
        before = self.__dict__.get(name)
        object.__setattr__(self, name, value)
        fields = isinstance(before, torch.Tensor) or name == "dtype"
        if fields and "_ref" in self.__dict__:
            try:
                self.__post_init__()
            except Exception:
                object.__setattr__(self, name, before)
                raise

    @classmethod
    def empty(cls, n_layers: int, n_pages: int, Hkv: int, page: int, D: int, rows: int,
              table_ld: int, dtype=torch.bfloat16, device="cuda", bits: int = 16) -> "Cache":
        """An empty cache: every page free, every row of length 0. The pools are not filled. bits 4:
        values of ``dtype`` go in and come out, and are held in 4 bits and a scale of 8 for 32."""
        if bits not in (4, 16):
            raise ValueError("bits must be 4 or 16")
        if bits == 4 and (page % 16 or D % 32):
            raise ValueError("a cache of 4 bits takes pages of 16 tokens and heads of 32 channels")
        shape = (n_layers, n_pages, Hkv, page, D)
        pool = dtype
        if bits == 4:
            shape, pool = (n_layers, n_pages, Hkv, page // 16, 17 * D // 2), torch.uint8
        return cls(k=torch.empty(shape, dtype=pool, device=device),
                   v=torch.empty(shape, dtype=pool, device=device), dtype=dtype if bits == 4 else None,
                   table=torch.full((rows, table_ld), -1, dtype=torch.int32, device=device),
                   length=torch.zeros(rows, dtype=torch.int32, device=device),
                   ref=torch.zeros(n_pages, dtype=torch.int32, device=device))

    def _rows(self, seq, N, name="seq") -> int:
        if N is None:
            N = self.table.shape[0] if seq is None else seq.numel()
        return N


def cache_workspace(cache: Cache, n_max: int) -> torch.Tensor:
    """Workspace of ``cache_extend`` for up to n_max rows and of ``cache_compact``."""
    out = ctypes.c_size_t()
    _check(lib().xpress_cache_workspace_size(cache._ref, n_max, ctypes.byref(out)))
    return torch.empty(max(out.value, 256), dtype=torch.uint8, device=cache.k.device)


def cache_fork(cache: Cache, src: torch.Tensor, dst: torch.Tensor) -> None:
    """Row dst[i] becomes a copy of row src[i], sharing its pages."""
    n = dst.numel()
    _check(lib().xpress_cache_fork(cache._ref, _list(src, n, torch.int32, "src"),
                                   _list(dst, n, torch.int32, "dst"), n, _stream()))


def cache_extend(cache: Cache, add, *, lacking: torch.Tensor, ws: torch.Tensor, seq=None,
                 N: int | None = None) -> torch.Tensor:
    """Room for add tokens (an int, or an int32 tensor of one count a row) at the end of each row;
    a shared last page is copied first. lacking (int32): 0, or why nothing was changed."""
    N = cache._rows(seq, N)
    each = add if isinstance(add, torch.Tensor) else None
    ws_ptr, ws_bytes = _ws(ws)
    _check(lib().xpress_cache_extend(cache._ref, _list(seq, N, torch.int32, "seq"), N,
                                     _list(each, N, torch.int32, "add"),
                                     0 if each is not None else int(add),
                                     _list(lacking, 1, torch.int32, "lacking"), ws_ptr, ws_bytes,
                                     _stream()))
    return lacking


def cache_append(cache: Cache, layer: int, k_new: torch.Tensor, v_new: torch.Tensor, *, B: int,
                 seq=None, N: int | None = None, lacking: torch.Tensor | None = None) -> None:
    """K and V of one layer for the last B tokens of each row; k_new, v_new: [N*B, Hkv*D] views
    with the same row stride. lacking (as ``cache_extend`` wrote it): nothing is written unless it
    is 0."""
    N = cache._rows(seq, N)
    ld = _tokens(k_new, N * B, cache._width, cache._dtype, "k_new")
    if _tokens(v_new, N * B, cache._width, cache._dtype, "v_new") != ld:
        raise ValueError("k_new and v_new must have the same row stride")
    _check(lib().xpress_cache_append_if(cache._ref, _list(lacking, 1, torch.int32, "lacking"), layer,
                                        k_new.data_ptr(), v_new.data_ptr(), ld,
                                        _list(seq, N, torch.int32, "seq"), N, B, _stream()))


def cache_read(cache: Cache, layer: int, k_out: torch.Tensor, v_out: torch.Tensor, *, B: int,
               first: torch.Tensor | None = None, seq=None, N: int | None = None) -> None:
    """K and V of one layer read back: tokens first[i].. (int32; None: the last B) of each row, into
    k_out, v_out: [N*B, Hkv*D] views with the same row stride. Positions outside a row give 0."""
    N = cache._rows(seq, N)
    ld = _tokens(k_out, N * B, cache._width, cache._dtype, "k_out")
    if _tokens(v_out, N * B, cache._width, cache._dtype, "v_out") != ld:
        raise ValueError("k_out and v_out must have the same row stride")
    _check(lib().xpress_cache_read(cache._ref, layer, _list(seq, N, torch.int32, "seq"), N,
                                   _list(first, N, torch.int32, "first"), B, k_out.data_ptr(),
                                   v_out.data_ptr(), ld, _stream()))


def cache_trim(cache: Cache, drop=None, *, seq=None, N: int | None = None,
               lacking: torch.Tensor | None = None) -> None:
    """Row seq[i] loses its last drop[i] tokens (drop None: all of them). lacking (as
    ``cache_extend`` wrote it): nothing is freed unless it is 0."""
    N = cache._rows(seq, N)
    _check(lib().xpress_cache_trim_if(cache._ref, _list(lacking, 1, torch.int32, "lacking"),
                                      _list(seq, N, torch.int32, "seq"), N,
                                      _list(drop, N, torch.int32, "drop"), _stream()))


def cache_compact(cache: Cache, *, live: torch.Tensor, ws: torch.Tensor) -> torch.Tensor:
    """Moves the live pages to the front of the pools; live (int32) gets their number."""
    ws_ptr, ws_bytes = _ws(ws)
    _check(lib().xpress_cache_compact(cache._ref, _list(live, 1, torch.int32, "live"), ws_ptr,
                                      ws_bytes, _stream()))
    return live


def attention_workspace(cache: Cache, n_max: int, B: int, Hq: int) -> torch.Tensor:
    out = ctypes.c_size_t()
    _check(lib().xpress_attention_workspace_size(cache._ref, n_max, B, Hq, ctypes.byref(out)))
    return torch.empty(max(out.value, 256), dtype=torch.uint8, device=cache.k.device)


def block_attention(cache: Cache, layer: int, q: torch.Tensor, *, B: int, Hq: int,
                    out: torch.Tensor, ws: torch.Tensor, shared: int = 0,
                    scale: float | None = None, seq=None, N: int | None = None,
                    lse: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the last B tokens of each row over one layer; q and out: [N*B, Hq*D] views.
    The first ``shared`` tokens, common to all rows, are read once. scale defaults to D**-0.5."""
    N = cache._rows(seq, N)
    D = cache._D
    q_ld = _tokens(q, N * B, Hq * D, cache._dtype, "q")
    out_ld = _tokens(out, N * B, Hq * D, cache._dtype, "out")
    ws_ptr, ws_bytes = _ws(ws)
    _check(lib().xpress_block_attention(
        cache._ref, layer, q.data_ptr(), q_ld, _list(seq, N, torch.int32, "seq"), N, B, Hq,
        D ** -0.5 if scale is None else scale, shared, out.data_ptr(), out_ld,
        _list(lse, N * B * Hq, torch.float32, "lse"), ws_ptr, ws_bytes, _stream()))
    return out


def verify_workspace(n_max: int, B: int, V: int, device="cuda") -> torch.Tensor:
    out = ctypes.c_size_t()
    _check(lib().xpress_verify_workspace_size(n_max, B, V, ctypes.byref(out)))
    return torch.empty(max(out.value, 256), dtype=torch.uint8, device=device)


def verify_draft(logits: torch.Tensor, blk: torch.Tensor, *, out: torch.Tensor,
                 accepted: torch.Tensor, ws: torch.Tensor, u=None, temperature=None,
                 draft_len=None, q=None, drop=None) -> torch.Tensor:
    """Which drafts of blk [N, B] stand against the target's logits [N*B, V], and the token after
    them; q [N*(B-1), V]: the drafts' probabilities (None: drafts chosen by argmax)."""
    N, B = blk.shape
    V = logits.shape[-1]
    if logits.dtype not in _DTYPES:
        raise TypeError("logits must be bfloat16, float16 or float32")
    ld = _tokens(logits, N * B, V, logits.dtype, "logits")
    q_ptr, q_type, q_ld = None, BF16, V
    if q is not None:
        if q.dtype not in _DTYPES:
            raise TypeError("q must be bfloat16, float16 or float32")
        q_ld = _tokens(q, N * (B - 1), V, q.dtype, "q")
        q_ptr, q_type = q.data_ptr(), _DTYPES[q.dtype]
    ws_ptr, ws_bytes = _ws(ws)
    i64, i32, f32 = torch.int64, torch.int32, torch.float32
    _check(lib().xpress_verify_draft(
        logits.data_ptr(), _DTYPES[logits.dtype], ld, _list(blk, N * B, i64, "blk"),
        _list(draft_len, N, i32, "draft_len"), q_ptr, q_type, q_ld,
        _list(temperature, N, f32, "temperature"), _list(u, N * B, f32, "u"), N, B, V,
        _list(out, N * B, i64, "out"), _list(accepted, N, i32, "accepted"),
        _list(drop, N, i32, "drop"), ws_ptr, ws_bytes, _stream()))
    return out


def logprobs_workspace(rows_max: int, V: int, top: int = 0, device="cuda") -> torch.Tensor:
    out = ctypes.c_size_t()
    _check(lib().xpress_logprobs_workspace_size(rows_max, V, top, ctypes.byref(out)))
    return torch.empty(max(out.value, 256), dtype=torch.uint8, device=device)


def token_logprobs(logits: torch.Tensor, token: torch.Tensor | None = None, *, ws: torch.Tensor,
                   temperature=None, logprob=None, entropy=None, rank=None, top_ids=None,
                   top_logprobs=None) -> None:
    """Of tokens [N, B] (negative: none there) under logits [N*B, V]: their log probabilities, the
    entropy, their ranks, and the most likely alternatives, top_ids and top_logprobs [N*B, top]; each
    is written where it is given. temperature: [N] float32 (None: 1). token None: [N*B, 1] rows."""
    rows, V = logits.shape
    N, B = (rows, 1) if token is None else token.shape
    if logits.dtype not in _DTYPES:
        raise TypeError("logits must be bfloat16, float16 or float32")
    ld = _tokens(logits, N * B, V, logits.dtype, "logits")
    top = 0
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs go together")
    if top_ids is not None:
        top = top_ids.shape[-1]
        if top_ids.shape != top_logprobs.shape or top_ids.dim() != 2:
            raise ValueError("top_ids and top_logprobs must be [N*B, top]")
    ws_ptr, ws_bytes = _ws(ws)
    i64, i32, f32 = torch.int64, torch.int32, torch.float32
    n = N * B
    _check(lib().xpress_token_logprobs(
        logits.data_ptr(), _DTYPES[logits.dtype], ld, _list(token, n, i64, "token"),
        _list(temperature, N, f32, "temperature"), N, B, V, top, _list(logprob, n, f32, "logprob"),
        _list(entropy, n, f32, "entropy"), _list(rank, n, i32, "rank"),
        _list(top_ids, n * top, i64, "top_ids"), _list(top_logprobs, n * top, f32, "top_logprobs"),
        ws_ptr, ws_bytes, _stream()))

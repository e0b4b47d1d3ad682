"""Thin Python binding of libqlin (ctypes).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams.  There is no fallback:
if the library is missing, every call raises.

Calls whose arguments are all contiguous tensors of the right types on the
current device, with nothing to be allocated, take a short way through a small
extension (``csrc/qlin_binding.cpp``) that reads the tensors itself (4 to 7 us a
call less); all others are looked at here, argument by argument, and so are those
of a program whose torch the extension was not built for (a warning says so).

Names follow the C ABI in ``include/qlin.h`` without the ``qlin_`` prefix.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import struct
import threading
import warnings

import torch

from . import build as _build

FORMATS = {"w4a8": 0, "w6a8": 1}
PROLOGUES = {"none": 0, "rmsnorm": 1, "swiglu": 2}
FLAG_PDL = 1

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_DEVICE_TIMEOUT, ERR_WORKSPACE, ERR_BAD_INDEX = range(7)

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # qlin_dtype

_lock = threading.Lock()
_lib = None


class QlinError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """Load libqlin.so from the package's build folder (no implicit build)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(f"libqlin.so is not built ({path}); run __graft_entry__.build() "
                                   "or python -m w6a8_quantized_linear_gb300.build")
            L = ctypes.CDLL(path)
            i64, sz, vp, i32 = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int
            st = ctypes.c_int
            sig = {
                "qlin_version": (ctypes.c_char_p, []),
                "qlin_status_string": (ctypes.c_char_p, [st]),
                "qlin_check_shape": (st, [i32, i64, i64, i64]),
                "qlin_packed_bytes": (sz, [i32, i64, i64, i64]),
                "qlin_repack_workspace_bytes": (st, [i32, i64, i64, i64, ctypes.POINTER(sz), ctypes.POINTER(sz)]),
                "qlin_repack": (st, [i32, i64, i64, i64, vp, vp, sz, vp]),
                "qlin_repack_codebook": (st, [i64, i64, i64, vp, vp, sz, vp]),
                "qlin_forward_workspace_bytes": (st, [i32, i64, i64, i64, ctypes.POINTER(sz)]),
                "qlin_workspace_init": (st, [vp, sz, vp]),
                "qlin_forward": (st, [i32, i32, i32, i64, i64, i64, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, sz,
                                      ctypes.c_uint, vp]),
                "qlin_forward_multi": (st, [i32, i32, i32, i32, vp, i64, i64, vp, vp, vp, vp, vp, ctypes.c_float,
                                            vp, vp, vp, sz, ctypes.c_uint, vp]),
                "qlin_forward_moe": (st, [i32, i32, i32, i32, i64, i64, i64, vp, vp, i32, vp, vp, vp, vp,
                                          ctypes.c_float, vp, vp, vp, sz, ctypes.c_uint, vp]),
                "qlin_forward_codebook": (st, [i32, i32, i32, i64, i64, i64, vp, vp, vp, vp, vp, vp, ctypes.c_float,
                                               vp, vp, vp, sz, ctypes.c_uint, vp]),
                "qlin_forward_launch_info": (st, [i32, i64, i64, i64, ctypes.POINTER(i64), ctypes.POINTER(i64),
                                                  ctypes.POINTER(i64)]),
                "qlin_read_device_status": (st, [vp, vp]),
                "qlin_debug_forward": (st, [i32, i32, i32, i64, i64, i64, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp,
                                            vp, vp, vp, sz, vp]),
                "qlin_debug_forward_fault": (st, [i32, i32, i32, i64, i64, i64, vp, vp, vp, vp, vp, ctypes.c_float, vp,
                                                  vp, sz, i64, vp]),
                "qlin_forward_noalloc": (st, [i32, i32, i32, i64, i64, i64, vp, vp, vp, vp, vp, ctypes.c_float, vp,
                                              ctypes.c_uint, vp]),
                "qlin_debug_plan": (st, [i32, i32, i64, i64, i64, ctypes.POINTER(i32), ctypes.POINTER(i32)]),
                "qlin_debug_repack_tcgen05": (st, [i32, i64, i64, i64, vp, vp, sz, vp]),
                "qlin_debug_forward_tcgen05": (st, [i32, i32, i32, i64, i64, i64, vp, vp, vp, vp, vp, ctypes.c_float,
                                                    vp, vp, vp, vp, vp, sz, ctypes.c_uint, vp]),
                "qlin_rope_turns": (st, [vp, i32, vp]),
                "qlin_kv_append": (st, [vp, vp, i32, i32, vp, i64, vp, i64, vp, i64, vp, vp, ctypes.c_float, vp, i32,
                                        i32, vp, i64, vp, sz, ctypes.c_uint, vp]),
                "qlin_kv_append_at": (st, [vp, vp, i32, i32, vp, i64, vp, i64, vp, i64, vp, vp, ctypes.c_float, vp, i32,
                                           i32, vp, i64, i32, ctypes.c_char_p, vp, i64, vp, sz, ctypes.c_uint, vp]),
                "qlin_tree_attention_workspace_bytes": (st, [vp, i32, i32, i32, ctypes.POINTER(sz)]),
                "qlin_tree_attention": (st, [vp, vp, i32, vp, i64, ctypes.c_float, vp, i64, vp, sz, ctypes.c_uint,
                                             vp]),
                "qlin_tree_attention_stats": (st, [vp, vp, i32, vp, i64, ctypes.c_float, vp, i64, vp, vp, sz, ctypes.c_uint,
                                                   vp]),
                "qlin_kv_weigh": (st, [vp, vp, i32, vp, i64, vp, ctypes.c_float, vp, i64, vp, ctypes.c_float, vp, i64, i64,
                                       vp, vp, i64, i64, i64, vp, vp, sz, ctypes.c_uint, vp]),
                "qlin_debug_kv_weigh_fault": (st, [vp, vp, i32, vp, i64, vp, ctypes.c_float, vp, i64, i64, vp, i64, vp, sz,
                                                   i64, vp]),
                "qlin_debug_tree_attention_fault": (st, [vp, vp, i32, vp, i64, ctypes.c_float, vp, i64, vp, sz, i64, vp]),
                "qlin_kv_keep": (st, [vp, vp, vp, i64, vp, vp, vp, sz, ctypes.c_uint, vp]),
                "qlin_kv_evict_workspace_bytes": (st, [vp, i32, i64, ctypes.POINTER(sz)]),
                "qlin_kv_evict": (st, [vp, vp, vp, vp, i64, i64, vp, vp, i64, i64, i64, vp, i32, vp, vp, vp, sz,
                                       ctypes.c_uint, vp]),
                "qlin_debug_sample_plan": (st, [i64, i64, i32, i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]),
                "qlin_debug_sample_weight": (st, [i32, vp, vp, vp, vp]),
                "qlin_adjust_logits": (st, [i32, i32, i64, i32, vp, i64, vp, i64, ctypes.c_char_p, ctypes.c_uint, vp]),
                "qlin_sample": (st, [i32, i64, i32, vp, i64, vp, vp, vp, vp, vp, vp, vp, ctypes.c_uint, vp]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


_binding = None


class _NoBinding:
    """In the extension's place where it cannot be loaded: no call is for the short way."""
    kv_append = kv_weigh = kv_evict = adjust_logits = staticmethod(lambda *args: None)


def _load_binding():
    """The short way's extension, loaded with the library that it calls."""
    global _binding
    lib()
    with _lock:
        if _binding is None:
            try:
                if not _build.binding_fits():
                    raise ImportError("it was not built for this torch and Python")
                spec = importlib.util.spec_from_file_location("_qlin_binding", _build.BINDING)
                module = importlib.util.module_from_spec(spec)
                spec.loader.exec_module(module)
            except ImportError as e:
                warnings.warn(f"_qlin_binding.so is not loaded, and calls take some microseconds longer: {e}; run "
                              "__graft_entry__.build() or python -m w6a8_quantized_linear_gb300.build", RuntimeWarning,
                              stacklevel=3)
                module = _NoBinding
            _binding = module
    return _binding


def status_string(status: int) -> str:
    return lib().qlin_status_string(int(status)).decode()


def version() -> str:
    return lib().qlin_version().decode()


def _fmt(f) -> int:
    return FORMATS[f] if isinstance(f, str) else int(f)


def _pro(p) -> int:
    return PROLOGUES[p] if isinstance(p, str) else int(p)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != OK:
        raise QlinError(status, where)


def check_shape(fmt, N: int, K: int, G: int) -> int:
    return lib().qlin_check_shape(_fmt(fmt), N, K, G)


def packed_bytes(fmt, N: int, K: int, G: int) -> int:
    return lib().qlin_packed_bytes(_fmt(fmt), N, K, G)


def repack_workspace_bytes(fmt, N: int, K: int, G: int) -> tuple[int, int]:
    lo, rec = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().qlin_repack_workspace_bytes(_fmt(fmt), N, K, G, ctypes.byref(lo), ctypes.byref(rec)),
           "repack_workspace_bytes")
    return lo.value, rec.value


def repack(buf: torch.Tensor, fmt, N: int, K: int, G: int, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rewrite ``buf`` (uint8, checkpoint layout, on the GPU) into the kernel-order stream, in place."""
    if ws is None:
        _, rec = repack_workspace_bytes(fmt, N, K, G)
        ws = torch.empty(rec, dtype=torch.uint8, device=buf.device)
    _check(lib().qlin_repack(_fmt(fmt), N, K, G, _ptr(buf), _ptr(ws), ws.numel(), _stream(stream)), "repack")
    return buf


def repack_codebook(buf: torch.Tensor, N: int, K: int, G: int, ws: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """``repack`` for a W4A8 weight used with a codebook (``forward_codebook``):
    the codebook stream layout, in place."""
    if ws is None:
        _, rec = repack_workspace_bytes("w4a8", N, K, G)
        ws = torch.empty(rec, dtype=torch.uint8, device=buf.device)
    _check(lib().qlin_repack_codebook(N, K, G, _ptr(buf), _ptr(ws), ws.numel(), _stream(stream)), "repack_codebook")
    return buf


def forward_workspace_bytes(fmt, N: int, K: int, G: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().qlin_forward_workspace_bytes(_fmt(fmt), N, K, G, ctypes.byref(n)), "forward_workspace_bytes")
    return n.value


def workspace_init(ws: torch.Tensor, stream=None) -> None:
    _check(lib().qlin_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "workspace_init")


def new_workspace(nbytes: int, device="cuda", stream=None) -> torch.Tensor:
    """A zeroed forward workspace of ``nbytes`` (allocated by torch, zeroed by the library)."""
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    workspace_init(ws, stream)
    return ws


def forward(fmt, prologue, packed: torch.Tensor, N: int, K: int, G: int, x=None, gate=None, up=None, gamma=None,
            eps: float = 1e-6, y: torch.Tensor | None = None, ws: torch.Tensor | None = None, flags: int = 0,
            stream=None) -> torch.Tensor:
    """y[M, N] (fp32) = repacked weight x int8-quantised prologue(activation)."""
    act = gate if _pro(prologue) == 2 else x
    M = act.shape[0]
    if y is None:
        y = torch.empty(M, N, dtype=torch.float32, device=packed.device)
    if ws is None:
        ws = new_workspace(forward_workspace_bytes(fmt, N, K, G), packed.device, stream)
    _check(lib().qlin_forward(_fmt(fmt), _pro(prologue), M, N, K, G, _ptr(packed), _ptr(x), _ptr(gate), _ptr(up),
                              _ptr(gamma), float(eps), _ptr(y), _ptr(ws), ws.numel(), flags, _stream(stream)),
           "forward")
    return y


MAX_MULTI = 8


def forward_multi(fmt, prologue, packed: list, N: list, K: int, G: int, x=None, gate=None, up=None, gamma=None,
                  eps: float = 1e-6, y: list | None = None, bias: list | None = None,
                  ws: torch.Tensor | None = None, flags: int = 0, stream=None) -> list:
    """Several weights on one shared activation in one launch: y[l] = packed[l] x
    quantised prologue(activation) (+ bias[l], fp32 [N[l]], where given).
    Returns the list of fp32 [M, N[l]] outputs."""
    act = gate if _pro(prologue) == 2 else x
    M = act.shape[0]
    n = len(packed)
    if len(N) != n:
        raise ValueError("packed and N differ in length")
    dev = packed[0].device
    if y is None:
        y = [torch.empty(M, Nl, dtype=torch.float32, device=dev) for Nl in N]
    if ws is None:
        ws = new_workspace(forward_workspace_bytes(fmt, max(N), K, G), dev, stream)
    n_arr = (ctypes.c_int64 * n)(*N)
    p_arr = (ctypes.c_void_p * n)(*[_ptr(t) for t in packed])
    y_arr = (ctypes.c_void_p * n)(*[_ptr(t) for t in y])
    b_arr = None if bias is None else (ctypes.c_void_p * n)(*[_ptr(t) for t in bias])
    _check(lib().qlin_forward_multi(_fmt(fmt), _pro(prologue), M, n, ctypes.cast(n_arr, ctypes.c_void_p), K, G,
                                    ctypes.cast(p_arr, ctypes.c_void_p), _ptr(x), _ptr(gate), _ptr(up), _ptr(gamma),
                                    float(eps), ctypes.cast(y_arr, ctypes.c_void_p),
                                    None if b_arr is None else ctypes.cast(b_arr, ctypes.c_void_p), _ptr(ws), ws.numel(), flags,
                                    _stream(stream)), "forward_multi")
    return y


def forward_moe(fmt, prologue, bank: torch.Tensor, E: int, N: int, K: int, G: int, ids: torch.Tensor, x=None,
                gate=None, up=None, gamma=None, eps: float = 1e-6, bias: torch.Tensor | None = None,
                y: torch.Tensor | None = None, ws: torch.Tensor | None = None, flags: int = 0,
                stream=None) -> torch.Tensor:
    """Expert bank: y[m, j] = expert ids[m, j] applied to token m (fp32 [M, topk, N]).
    ``bank`` is the [E * N, K] bank repacked as one weight; ``ids`` int32 [M, topk]
    on the device."""
    act = gate if _pro(prologue) == 2 else x
    M = act.shape[0]
    topk = ids.shape[1]
    if ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 [M, topk] tensor")
    if y is None:
        y = torch.empty(M, topk, N, dtype=torch.float32, device=bank.device)
    if ws is None:
        ws = new_workspace(forward_workspace_bytes(fmt, E * N, K, G), bank.device, stream)
    _check(lib().qlin_forward_moe(_fmt(fmt), _pro(prologue), M, E, N, K, G, _ptr(bank), _ptr(ids), topk, _ptr(x),
                                  _ptr(gate), _ptr(up), _ptr(gamma), float(eps), _ptr(bias), _ptr(y), _ptr(ws),
                                  ws.numel(), flags, _stream(stream)), "forward_moe")
    return y


def forward_codebook(fmt, prologue, packed: torch.Tensor, codebook: torch.Tensor, N: int, K: int, G: int, x=None,
                     gate=None, up=None, gamma=None, eps: float = 1e-6, bias: torch.Tensor | None = None,
                     y: torch.Tensor | None = None, ws: torch.Tensor | None = None, flags: int = 0,
                     stream=None) -> torch.Tensor:
    """``forward`` with the levels of the 4-bit codes read from ``codebook``
    (fp32 [16] on the device) instead of code - 8; optional fp32 [N] bias."""
    if codebook.dtype != torch.float32 or codebook.numel() != 16 or not codebook.is_contiguous():
        raise ValueError("codebook must be a contiguous float32 tensor of 16 levels")
    act = gate if _pro(prologue) == 2 else x
    M = act.shape[0]
    if y is None:
        y = torch.empty(M, N, dtype=torch.float32, device=packed.device)
    if ws is None:
        ws = new_workspace(forward_workspace_bytes(fmt, N, K, G), packed.device, stream)
    _check(lib().qlin_forward_codebook(_fmt(fmt), _pro(prologue), M, N, K, G, _ptr(packed), _ptr(codebook), _ptr(x),
                                       _ptr(gate), _ptr(up), _ptr(gamma), float(eps), _ptr(bias), _ptr(y), _ptr(ws),
                                       ws.numel(), flags, _stream(stream)), "forward_codebook")
    return y


def forward_noalloc(fmt, prologue, packed: torch.Tensor, N: int, K: int, G: int, x=None, gate=None, up=None,
                    gamma=None, eps: float = 1e-6, y: torch.Tensor | None = None, flags: int = 0,
                    stream=None) -> torch.Tensor:
    """``forward`` for callers that cannot allocate device memory: the library
    uses its own fixed 64 KiB device array as the workspace (see qlin.h)."""
    act = gate if _pro(prologue) == 2 else x
    M = act.shape[0]
    if y is None:
        y = torch.empty(M, N, dtype=torch.float32, device=packed.device)
    _check(lib().qlin_forward_noalloc(_fmt(fmt), _pro(prologue), M, N, K, G, _ptr(packed), _ptr(x), _ptr(gate),
                                      _ptr(up), _ptr(gamma), float(eps), _ptr(y), flags, _stream(stream)),
           "forward_noalloc")
    return y


def launch_info(fmt, N: int, K: int, G: int) -> dict:
    c, u, b = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().qlin_forward_launch_info(_fmt(fmt), N, K, G, ctypes.byref(c), ctypes.byref(u), ctypes.byref(b)),
           "launch_info")
    return {"ctas": c.value, "units": u.value, "stream_bytes": b.value}


def read_device_status(ws: torch.Tensor, stream=None) -> int:
    return lib().qlin_read_device_status(_ptr(ws), _stream(stream))


def debug_forward(fmt, prologue, packed: torch.Tensor, N: int, K: int, G: int, x=None, gate=None, up=None,
                  gamma=None, eps: float = 1e-6, ws: torch.Tensor | None = None, stream=None) -> dict:
    """qlin_forward with its test exports: y, exact group sums, activation codes, row scales."""
    act = gate if _pro(prologue) == 2 else x
    M = act.shape[0]
    dev = packed.device
    out = {"y": torch.empty(M, N, dtype=torch.float32, device=dev),
           "acc": torch.empty(M, N, K // G, dtype=torch.int32, device=dev),
           "q": torch.empty(M, K, dtype=torch.int8, device=dev),
           "s": torch.empty(M, dtype=torch.float32, device=dev)}
    if ws is None:
        ws = new_workspace(forward_workspace_bytes(fmt, N, K, G), dev, stream)
    _check(lib().qlin_debug_forward(_fmt(fmt), _pro(prologue), M, N, K, G, _ptr(packed), _ptr(x), _ptr(gate),
                                    _ptr(up), _ptr(gamma), float(eps), _ptr(out["y"]), _ptr(out["acc"]),
                                    _ptr(out["q"]), _ptr(out["s"]), _ptr(ws), ws.numel(), _stream(stream)),
           "debug_forward")
    return out


def debug_forward_fault(fmt, prologue, packed: torch.Tensor, N: int, K: int, G: int, unit: int, x=None, gate=None,
                        up=None, gamma=None, eps: float = 1e-6, y=None, ws: torch.Tensor | None = None,
                        stream=None) -> int:
    """Enqueue a forward whose GEMV never issues the copy of ``unit``; returns the enqueue status."""
    act = gate if _pro(prologue) == 2 else x
    M = act.shape[0]
    if y is None:
        y = torch.empty(M, N, dtype=torch.float32, device=packed.device)
    return lib().qlin_debug_forward_fault(_fmt(fmt), _pro(prologue), M, N, K, G, _ptr(packed), _ptr(x), _ptr(gate),
                                          _ptr(up), _ptr(gamma), float(eps), _ptr(y), _ptr(ws), ws.numel(), unit,
                                          _stream(stream))


def debug_repack_tcgen05(buf: torch.Tensor, fmt, N: int, K: int, G: int, ws: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """``repack`` into the row layout of the tcgen05 main loop (test export; G >= 32)."""
    if ws is None:
        _, rec = repack_workspace_bytes(fmt, N, K, G)
        ws = torch.empty(rec, dtype=torch.uint8, device=buf.device)
    _check(lib().qlin_debug_repack_tcgen05(_fmt(fmt), N, K, G, _ptr(buf), _ptr(ws), ws.numel(), _stream(stream)),
           "debug_repack_tcgen05")
    return buf


def debug_forward_tcgen05(fmt, prologue, packed: torch.Tensor, N: int, K: int, G: int, x=None, gate=None, up=None,
                          gamma=None, eps: float = 1e-6, y: torch.Tensor | None = None, exports: bool = False,
                          ws: torch.Tensor | None = None, flags: int = 0, stream=None) -> dict:
    """The tcgen05 main loop on a weight from ``debug_repack_tcgen05`` (test
    export): y, and with ``exports`` the exact group sums, codes and row scales."""
    act = gate if _pro(prologue) == 2 else x
    M = act.shape[0]
    dev = packed.device
    out = {"y": y if y is not None else torch.empty(M, N, dtype=torch.float32, device=dev)}
    if exports:
        out["acc"] = torch.empty(M, N, K // G, dtype=torch.int32, device=dev)
        out["q"] = torch.empty(M, K, dtype=torch.int8, device=dev)
        out["s"] = torch.empty(M, dtype=torch.float32, device=dev)
    if ws is None:
        ws = new_workspace(forward_workspace_bytes(fmt, N, K, G), dev, stream)
    _check(lib().qlin_debug_forward_tcgen05(_fmt(fmt), _pro(prologue), M, N, K, G, _ptr(packed), _ptr(x), _ptr(gate),
                                            _ptr(up), _ptr(gamma), float(eps), _ptr(out["y"]), _ptr(out.get("acc")),
                                            _ptr(out.get("q")), _ptr(out.get("s")), _ptr(ws), ws.numel(), flags,
                                            _stream(stream)), "debug_forward_tcgen05")
    return out


def debug_plan(fmt, M: int, N: int, K: int, G: int) -> dict:
    """The plan qlin_forward uses for this shape on the current device (test export)."""
    c, st = ctypes.c_int(), ctypes.c_int()
    _check(lib().qlin_debug_plan(_fmt(fmt), M, N, K, G, ctypes.byref(c), ctypes.byref(st)), "debug_plan")
    return {"cluster": c.value, "stages": st.value}


# ---- the rest of a decode / verification step ---------------------------------


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("heads", ctypes.c_int32), ("width", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class _StepStruct(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("len", ctypes.c_void_p), ("count", ctypes.c_void_p),
                ("depth", ctypes.c_void_p), ("mask", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("tree_stride", ctypes.c_int64), ("B", ctypes.c_int32), ("T", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


class KVCache:
    """A paged cache: ``k`` and ``v`` are [pages, heads, page_size, width] tensors
    (bf16 or fp16) of equal strides, the last dimension contiguous; a permuted
    view of a [pages, page_size, heads, width] pool is one too."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must be [pages, heads, page_size, width] tensors of one shape, type and device")
        if k.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("the cache holds bfloat16 or float16")
        if k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must have the same strides and contiguous rows")
        self.k, self.v, self.device, self.dtype = k, v, k.device, k.dtype
        self.pages, self.heads, self.page_size, self.width = k.shape
        self._index = k.get_device()  # -1: not on a GPU
        # a dimension of one has no stride that matters
        step = [st if n > 1 else 8 for st, n in zip(k.stride()[:2], k.shape[:2])]
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), self.pages, step[0], step[1], k.stride(2),
                                    DTYPES[k.dtype], self.heads, self.width, self.page_size)
        self._ref = ctypes.addressof(self._struct)
        self._code = DTYPES[k.dtype]


class KVStep:
    """One step of B sequences, T rows each (``qlin_kv_step``): ``page_table``
    int32 [B, max_pages], ``len`` int32 [B], optional ``count`` int32 [B], and
    ``depth`` / ``mask`` int32 [T] (one tree for all sequences) or [B, T].  The
    tensors are kept, and read by the calls that use the step."""

    def __init__(self, page_table: torch.Tensor, len: torch.Tensor, T: int, count=None, depth=None, mask=None):
        B = len.shape[0]
        for name, t in (("page_table", page_table), ("len", len), ("count", count), ("depth", depth), ("mask", mask)):
            if t is not None and (t.dtype != torch.int32 or t.device != len.device):
                raise ValueError(f"{name} must be an int32 tensor on the device of len")
        if len.dim() != 1 or page_table.dim() != 2 or page_table.shape[0] != B:
            raise ValueError("page_table must be [B, max_pages] and len [B]")
        if B and page_table.stride(1) != 1 and page_table.shape[1] > 1:
            raise ValueError("the rows of page_table must be contiguous")
        if not len.is_contiguous() or (count is not None and (count.shape != (B,) or not count.is_contiguous())):
            raise ValueError("len and count must be contiguous [B] tensors")
        tree = [t for t in (depth, mask) if t is not None]
        for t in tree:
            if t.shape not in ((T,), (B, T)) or not t.is_contiguous() or t.dim() != tree[0].dim():
                raise ValueError("depth and mask must be contiguous [T] or [B, T] tensors of one shape")
        self.page_table, self.len, self.count, self.depth, self.mask = page_table, len, count, depth, mask
        self.B, self.T, self.device = B, T, len.device
        n = page_table.shape[1]
        self._struct = _StepStruct(_ptr(page_table), _ptr(len), _ptr(count), _ptr(depth), _ptr(mask),
                                   page_table.stride(0) if B > 1 else n, T if tree and tree[0].dim() == 2 else 0, B, T, n)
        self._ref = ctypes.addressof(self._struct)
        self._index = len.get_device()


_fns: dict = {}
_F32, _I32 = torch.float32, torch.int32
# Bound once, as each costs a call some host time; the public forms where a torch has no such names (built without CUDA).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


def _fn(name: str):
    fn = _fns.get(name)
    if fn is None or _lib is None:
        fn = _fns[name] = getattr(lib(), name)
    return fn


def _same_device(index: int, *tensors) -> None:
    """All tensors on GPU ``index``, and that device current (the library launches on the current one)."""
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"a tensor is on {t.device}, another of the call's tensors on "
                             + (f"cuda:{index}" if index >= 0 else "the CPU, not on a GPU"))
    if index < 0:
        raise ValueError("the tensors are on the CPU, not on a GPU")
    if index != _current_device():
        raise ValueError(f"the tensors are on cuda:{index}, but cuda:{_current_device()} is the current device")


def _raw_stream(stream, index: int) -> int:
    if stream is None:
        return _current_stream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """Memory for an output of a call on ``stream``, owned by that stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(t, n: int, width: int, dtype, what: str) -> int:
    """Row stride of a [n, width] (or [n, heads, D]) tensor of ``dtype``."""
    if t.dtype is dtype:
        if t.is_contiguous():
            if t.shape == (n, width):
                return width
            if t.dim() == 3 and t.shape[0] == n and t.numel() == n * width:
                return width
        elif t.dim() == 2 and t.shape == (n, width) and t.stride(1) == 1:
            return t.stride(0) if n > 1 else width
        elif t.dim() == 3 and t.shape[0] == n and t.shape[1] * t.shape[2] == width and t.stride(2) == 1 and (
                t.stride(1) == t.shape[2]):
            return t.stride(0) if n > 1 else width
    raise ValueError(f"{what} must be a [{n}, {width}] tensor of {dtype} with contiguous rows")


def _heads(t, width: int, what: str) -> int:
    n = t.shape[1] if t.dim() == 2 else t.shape[1] * t.shape[2] if t.dim() == 3 else 0
    if n < 1 or n % width:
        raise ValueError(f"{what} must be [rows, heads * {width}], whole heads in each row")
    return n // width


def _floats(t, n: int, what: str):
    if t is None:
        return None
    if t.dtype is not _F32 or t.numel() != n or (n > 1 and not t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous float32 tensor of {n} values")
    return t.data_ptr()


def _ints(t, n: int, what: str):
    if t is None:
        return None
    if t.dtype is not _I32 or t.numel() != n or (n > 1 and not t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous int32 tensor of {n} values")
    return t.data_ptr()


def rope_turns(theta: float = 1e4, rot: int = 0, radians=None, device="cuda") -> torch.Tensor:
    """Rotation frequencies for ``kv_append`` (int64 [rot / 2], 64-bit fractions of
    a turn per position): theta ** (-2i / rot), or the given ``radians`` per
    position."""
    if radians is None:
        if rot < 0 or rot % 2 or not theta > 0:
            raise ValueError("rot must be even and not negative, theta above 0")
        radians = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    n = len(radians)
    out = torch.empty(n, dtype=torch.int64)
    src = torch.tensor(list(radians), dtype=torch.float64)
    _check(_fn("qlin_rope_turns")(src.data_ptr(), n, out.data_ptr()), "rope_turns")
    return out.to(device)


def rope_axes(sections, dealt: bool = False) -> bytes:
    """Which axis of a row's positions turns each pair, for ``kv_append``: ``sections[a]``
    pairs on axis a (up to four axes), one section behind the other, or ``dealt``
    in turn to the axes that still have some."""
    left = [int(n) for n in sections]
    if not 1 <= len(left) <= 4 or min(left) < 0:
        raise ValueError("sections must be one to four counts, none negative")
    if not dealt:
        return bytes(a for a, n in enumerate(left) for _ in range(n))
    axis = bytearray()
    while any(left):
        for a, n in enumerate(left):
            if n:
                left[a] -= 1
                axis.append(a)
    return bytes(axis)


def kv_append(cache: KVCache, step: KVStep, q=None, k=None, v=None, q_gamma=None, k_gamma=None, eps: float = 1e-6,
              turns=None, pairs: bool = False, q_out=None, ws=None, flags: int = 0, stream=None, position=None,
              axis: bytes | None = None):
    """Head norms and rotation of a step's projected q and k ([B * T, heads * width],
    fp32 or bf16); k and v are stored behind the sequences' committed tokens.
    Returns the normed and rotated q in the cache's type (or None without q).
    ``ws`` (256 bytes): its status word gets ``ERR_BAD_INDEX`` for a page out of
    range; without one nothing is reported.  A row's position is the committed
    length plus its depth, unless ``position`` gives it: int32 [B * T], or
    [B * T, axes] with ``axis`` (``rope_axes``) naming the axis of each pair."""
    n, D, dev = step.B * step.T, cache.width, cache._index
    if stream is None and 0 <= dev == step._index and dev == _current_device():
        status = (_binding or _load_binding()).kv_append(
            dev, cache._ref, step._ref, n, D, cache.heads, cache._code, q, k, v, q_gamma, k_gamma, eps, turns, pairs, q_out, ws,
            flags, _current_stream(dev), position, axis)
        if status is not None:
            if status:
                _check(status, "kv_append")
            return q_out
    _same_device(dev, step.len, q, k, v, q_gamma, k_gamma, turns, q_out, ws, position)
    if (k is None) != (v is None):
        raise ValueError("k and v are given together")
    src = q if q is not None else k
    if src is None:
        raise ValueError("nothing to append: neither q nor k and v are given")
    dtype = src.dtype
    Hq = qs = ks = vs = os_ = 0
    if q is not None:
        Hq = _heads(q, D, "q")
        qs = _rows(q, n, Hq * D, dtype, "q")
        if q_out is None:
            q_out = _empty((n, Hq * D), cache.dtype, cache.device, stream)
        os_ = _rows(q_out, n, Hq * D, cache.dtype, "q_out")
    if k is not None:
        ks, vs = _rows(k, n, cache.heads * D, dtype, "k"), _rows(v, n, cache.heads * D, dtype, "v")
    nt = 0
    if turns is not None:
        nt = turns.numel()
        if turns.dtype is not torch.int64 or not turns.is_contiguous():
            raise ValueError("turns must come from rope_turns")
    head = (cache._ref, step._ref, Hq, DTYPES.get(dtype, -1), None if q is None else q.data_ptr(), qs,
            None if k is None else k.data_ptr(), ks, None if v is None else v.data_ptr(), vs,
            _floats(q_gamma, D, "q_gamma"), _floats(k_gamma, D, "k_gamma"), eps, turns.data_ptr() if nt else None, nt,
            1 if pairs else 0)
    tail = (None if q is None else q_out.data_ptr(), os_, None if ws is None else ws.data_ptr(),
            0 if ws is None else ws.numel(), flags, _current_stream(dev) if stream is None else _raw_stream(stream, dev))
    if position is None:
        if axis is not None:
            raise ValueError("axis names axes of position, which is not given")
        status = _fn("qlin_kv_append")(*head, *tail)
    else:
        shape = position.shape
        axes = shape[1] if len(shape) == 2 else 1
        whole = position.is_contiguous()
        if position.dtype is not _I32 or not 1 <= len(shape) <= 2 or shape[0] != n or (
                not whole and axes > 1 and position.stride(1) != 1):
            raise ValueError(f"position must be an int32 tensor of [{n}] or [{n}, axes] with contiguous rows")
        if axis is not None and (type(axis) is not bytes or len(axis) != nt):
            raise ValueError("axis must come from rope_axes, one entry for each of turns")
        status = _fn("qlin_kv_append_at")(*head, position.data_ptr(), axes if whole or n < 2 else position.stride(0), axes,
                                          axis, *tail)
    if status:
        _check(status, "kv_append")
    return q_out


def tree_attention_workspace_bytes(cache: KVCache, B: int, T: int, Hq: int) -> int:
    n = ctypes.c_size_t()
    _check(_fn("qlin_tree_attention_workspace_bytes")(cache._ref, B, T, Hq, ctypes.byref(n)),
           "tree_attention_workspace_bytes")
    return n.value


def tree_attention(cache: KVCache, step: KVStep, q: torch.Tensor, scale: float | None = None, out=None, ws=None,
                   flags: int = 0, stream=None, stats=None) -> torch.Tensor:
    """Attention of a step's rows (q of ``kv_append``, [B * T, Hq * width]) over the
    cache: every row sees the committed tokens of its sequence and the step's
    rows that its mask names.  Returns bf16 [B * T, Hq * width].  ``scale``:
    width ** -0.5 unless given.  Without ``ws`` the call takes memory of its own,
    and what its status word gets (``ERR_BAD_INDEX``, ``ERR_DEVICE_TIMEOUT``) is
    lost with it: a caller that reads ``read_device_status`` gives one.  ``stats``
    (fp32 [B * T, Hq, 2], optional) gets the rows' softmax references (log2 units)
    and sums, for ``kv_weigh``."""
    n, D, dev = step.B * step.T, cache.width, cache._index
    _same_device(dev, step.len, q, out, ws, stats)
    Hq = _heads(q, D, "q")
    qs = _rows(q, n, Hq * D, cache.dtype, "q")
    if out is None:
        out = _empty((n, Hq * D), torch.bfloat16, cache.device, stream)
    os_ = _rows(out, n, Hq * D, torch.bfloat16, "out")
    raw = _raw_stream(stream, dev)
    if ws is None:
        ws = _empty(tree_attention_workspace_bytes(cache, step.B, step.T, Hq), torch.uint8, cache.device, stream)
        workspace_init(ws, raw)
    head = (cache._ref, step._ref, Hq, q.data_ptr(), qs, D ** -0.5 if scale is None else scale, out.data_ptr(), os_)
    tail = (ws.data_ptr(), ws.numel(), flags, raw)
    if stats is None:
        status = _fn("qlin_tree_attention")(*head, *tail)
    else:
        status = _fn("qlin_tree_attention_stats")(*head, _stats(stats, n, Hq), *tail)
    if status:
        _check(status, "tree_attention")
    return out


def _stats(t, n: int, Hq: int) -> int:
    if t.dtype is not _F32 or t.shape != (n, Hq, 2) or not t.is_contiguous():
        raise ValueError(f"stats must be a contiguous float32 tensor of [{n}, {Hq}, 2]")
    return t.data_ptr()


def debug_tree_attention_fault(cache: KVCache, step: KVStep, q: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                               copy: int, stream=None) -> int:
    """Test export: ``tree_attention`` (scale width ** -0.5) whose first CTA never issues its
    ``copy``-th copy of a tile; returns the launch status (the device status word is read
    separately)."""
    n, D, dev = step.B * step.T, cache.width, cache._index
    _same_device(dev, step.len, q, out, ws)
    Hq = _heads(q, D, "q")
    return _fn("qlin_debug_tree_attention_fault")(
        cache._ref, step._ref, Hq, q.data_ptr(), _rows(q, n, Hq * D, cache.dtype, "q"), D ** -0.5, out.data_ptr(),
        _rows(out, n, Hq * D, torch.bfloat16, "out"), ws.data_ptr(), ws.numel(), copy, _raw_stream(stream, dev))


def kv_keep(cache: KVCache, step: KVStep, keep: torch.Tensor, n_keep: torch.Tensor, len_out=None, ws=None,
            flags: int = 0, stream=None) -> None:
    """Move the accepted rows ``keep[b, :n_keep[b]]`` (int32 [B, T], increasing) of each
    sequence up behind its committed tokens; ``len_out`` (int32 [B], may be the
    step's ``len``) gets the new lengths.  ``ws`` (256 bytes): its status word gets
    ``ERR_BAD_INDEX`` for a bad list or page; without one nothing is reported."""
    _same_device(cache._index, step.len, keep, n_keep, len_out, ws)
    B, T = step.B, step.T
    if keep.shape != (B, T) or keep.dtype is not torch.int32 or (T > 1 and keep.stride(1) != 1):
        raise ValueError("keep must be an int32 [B, T] tensor with contiguous rows")
    _check(_fn("qlin_kv_keep")(cache._ref, step._ref, keep.data_ptr(), keep.stride(0) if B > 1 else T,
                               _ints(n_keep, B, "n_keep"), _ints(len_out, B, "len_out"), _ptr(ws),
                               0 if ws is None else ws.numel(), flags, _raw_stream(stream, cache._index)), "kv_keep")


def _scores(t, shape, dtype, what: str) -> tuple[int, int]:
    """Strides of a [B, heads, room] tensor of ``dtype``, its tokens contiguous."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{what} must be a {dtype} tensor of {list(shape)}")
    if t.is_contiguous():
        return shape[1] * shape[2], shape[2]
    if shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"the tokens of {what} must be contiguous")
    return t.stride(0) if shape[0] > 1 else shape[1] * shape[2], t.stride(1) if shape[1] > 1 else shape[2]


def _score_pair(score, position, shape, what: str) -> tuple[int, int]:
    strides = _scores(score, shape, _F32, what)
    if position is not None and _scores(position, shape, _I32, "position" + what[5:]) != strides:
        raise ValueError(f"position{what[5:]} must have the strides of {what}")
    return strides


def kv_weigh(cache: KVCache, step: KVStep, q: torch.Tensor, stats: torch.Tensor, score: torch.Tensor, keep=None,
             n_keep=None, decay: float = 1.0, scale: float | None = None, score_out=None, position_out=None, at=None, ws=None,
             flags: int = 0, stream=None) -> torch.Tensor:
    """Add to ``score`` (fp32 [B, heads, room]) the attention weight that each token
    of the cache got from a step's rows (``q`` and ``stats`` as ``tree_attention``
    took and gave them): decay * score + the weights of the kept rows.  ``keep``,
    ``n_keep`` as in ``kv_keep`` (call this before it): the accepted path; without
    them all rows are kept.  The kept rows' own tokens get theirs at the places
    that ``kv_keep`` gives them, and ``position_out`` (int32, like score, optional)
    their positions: ``at`` (int32 [B * T]), or len + depth.  A row whose statistics
    are not finite weighs nothing.  Returns ``score_out`` (in place unless given)."""
    n, D, dev = step.B * step.T, cache.width, cache._index
    if stream is None and 0 <= dev == step._index and dev == _current_device():
        status = (_binding or _load_binding()).kv_weigh(
            dev, cache._ref, step._ref, step.B, step.T, D, cache.heads, cache._code, q, stats, score, keep, n_keep, decay,
            D ** -0.5 if scale is None else scale, score_out, position_out, at, ws, flags, _current_stream(dev))
        if status is not None:
            if status:
                _check(status, "kv_weigh")
            return score if score_out is None else score_out
    _same_device(dev, step.len, q, stats, score, keep, n_keep, score_out, position_out, at, ws)
    Hq = _heads(q, D, "q")
    qs = _rows(q, n, Hq * D, cache.dtype, "q")
    B, T = step.B, step.T
    ks = 0
    if keep is not None:
        if keep.shape != (B, T) or keep.dtype is not _I32 or (T > 1 and keep.stride(1) != 1):
            raise ValueError("keep must be an int32 [B, T] tensor with contiguous rows")
        ks = keep.stride(0) if B > 1 else T
    if score.dim() != 3:
        raise ValueError("score must be [B, heads, room]")
    shape = (B, cache.heads, score.shape[2])
    seq, head = _scores(score, shape, _F32, "score")
    if score_out is None:
        score_out = score
    out_seq, out_head = _score_pair(score_out, position_out, shape, "score_out")
    status = _fn("qlin_kv_weigh")(
        cache._ref, step._ref, Hq, q.data_ptr(), qs, _stats(stats, n, Hq), D ** -0.5 if scale is None else scale, _ptr(keep),
        ks, _ints(n_keep, B, "n_keep"), decay, score.data_ptr(), seq, head, score_out.data_ptr(), _ptr(position_out), out_seq,
        out_head, shape[2], _ints(at, n, "at"), _ptr(ws), 0 if ws is None else ws.numel(), flags,
        _current_stream(dev) if stream is None else _raw_stream(stream, dev))
    if status:
        _check(status, "kv_weigh")
    return score_out


def debug_kv_weigh_fault(cache: KVCache, step: KVStep, q: torch.Tensor, stats: torch.Tensor, score: torch.Tensor,
                         ws: torch.Tensor, copy: int, stream=None) -> int:
    """Test export: ``kv_weigh`` of all rows in place whose first CTA never issues its ``copy``-th copy of a panel of
    keys; returns the launch status (the device status word is read separately)."""
    n, D, dev = step.B * step.T, cache.width, cache._index
    _same_device(dev, step.len, q, stats, score, ws)
    Hq = _heads(q, D, "q")
    seq, head = _scores(score, (step.B, cache.heads, score.shape[2]), _F32, "score")
    return _fn("qlin_debug_kv_weigh_fault")(
        cache._ref, step._ref, Hq, q.data_ptr(), _rows(q, n, Hq * D, cache.dtype, "q"), _stats(stats, n, Hq), D ** -0.5,
        score.data_ptr(), seq, head, score.data_ptr(), score.shape[2], ws.data_ptr(), ws.numel(), copy, _raw_stream(stream, dev))


def kv_evict_workspace_bytes(cache: KVCache, step: KVStep, room: int) -> int:
    n = ctypes.c_size_t()
    _check(_fn("qlin_kv_evict_workspace_bytes")(cache._ref, step.B, room, ctypes.byref(n)), "kv_evict_workspace_bytes")
    return n.value


def kv_evict(cache: KVCache, step: KVStep, score: torch.Tensor, n_keep: torch.Tensor, first: int = 0, since=None,
             position=None, score_out=None, position_out=None, len_out=None, ws=None, flags: int = 0, stream=None) -> None:
    """Keep, head by head, the ``n_keep[b]`` committed tokens of the highest ``score``
    (fp32 [B, heads, room]; equal ones by index) of each sequence; those of
    positions below ``first`` or from ``since[b]`` on before all others.  Kept tokens
    behind place n_keep move into the places that empty before it: keys, values,
    scores and ``position`` (int32, like score; a token's place unless given).
    ``score_out`` and ``position_out``: where the scores and positions left go, in
    place unless given.  ``len_out`` (int32 [B], may be the step's ``len``) gets
    the new lengths.  Without ``ws`` the call takes memory of its own, and what its
    status word gets (``ERR_BAD_INDEX``) is lost with it."""
    dev = cache._index
    if stream is None and 0 <= dev == step._index and dev == _current_device():
        status = (_binding or _load_binding()).kv_evict(
            dev, cache._ref, step._ref, step.B, cache.heads, score, n_keep, first, since, position, score_out, position_out, len_out,
            ws, flags, _current_stream(dev))
        if status is not None:
            if status:
                _check(status, "kv_evict")
            return
    _same_device(dev, step.len, score, n_keep, since, position, score_out, position_out, len_out, ws)
    B = step.B
    if score.dim() != 3:
        raise ValueError("score must be [B, heads, room]")
    shape = (B, cache.heads, score.shape[2])
    seq, head = _score_pair(score, position, shape, "score")
    if score_out is None:
        score_out = score
    if position_out is None:
        position_out = position
    out_seq, out_head = _score_pair(score_out, position_out, shape, "score_out")
    raw = _raw_stream(stream, cache._index)
    if ws is None:
        ws = _empty(kv_evict_workspace_bytes(cache, step, shape[2]), torch.uint8, cache.device, stream)
        workspace_init(ws, raw)
    status = _fn("qlin_kv_evict")(
        cache._ref, step._ref, score.data_ptr(), _ptr(position), seq, head, score_out.data_ptr(), _ptr(position_out),
        out_seq, out_head, shape[2], _ints(n_keep, B, "n_keep"), first, _ints(since, B, "since"),
        _ints(len_out, B, "len_out"), ws.data_ptr(), ws.numel(), flags, raw)
    if status:
        _check(status, "kv_evict")


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=None, top_k=None, top_p=None, min_p=None, token=None,
           prob=None, flags: int = 0, stream=None) -> torch.Tensor:
    """One token per row of ``logits`` ([M, V], fp32 or bf16) from the uniform numbers
    ``u`` (fp32 [M]); temperature, top_p, min_p fp32 [M], top_k int32 [M], each
    optional.  Returns int32 [M]; ``prob`` (fp32 [M], optional) gets each
    token's probability among the kept ones."""
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be [M, V] with contiguous rows")
    M, V = logits.shape
    dev = logits.get_device()
    _same_device(dev, u, temperature, top_k, top_p, min_p, token, prob)
    if token is None:
        token = _empty((M,), torch.int32, logits.device, stream)
    _check(_fn("qlin_sample")(M, V, DTYPES.get(logits.dtype, -1), logits.data_ptr(), logits.stride(0) if M > 1 else V,
                              _floats(u, M, "u"), _floats(temperature, M, "temperature"), _ints(top_k, M, "top_k"),
                              _floats(top_p, M, "top_p"), _floats(min_p, M, "min_p"), _ints(token, M, "token"),
                              _floats(prob, M, "prob"), flags, _raw_stream(stream, dev)), "sample")
    return token


_MAX_SEQUENCES = 65535  # of a call of adjust_logits
# qlin_adjustments: eleven addresses, four strides, L and n_bias; packed, as that costs a call less than setting fields
_ADJUSTMENTS = struct.Struct("@11P4q2i")


def _table(t, rows: int, dtype, what: str) -> tuple[int, int]:
    """Width and row stride of a [rows, width] tensor of ``dtype``, or of [width] for all rows (stride 0)."""
    shape = t.shape
    if t.dtype is dtype and len(shape) == 2 and shape[0] == rows and t.is_contiguous():
        return shape[1], shape[1]
    if t.dtype is not dtype or not 1 <= len(shape) <= 2 or (len(shape) == 2 and shape[0] != rows) or (
            shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{what} must be a {dtype} tensor of {rows} contiguous rows, or of one row for all")
    n = shape[-1]
    return n, 0 if len(shape) == 1 else t.stride(0) if rows > 1 else n


def adjust_logits(logits: torch.Tensor, out=None, history=None, history_len=None, prompt_len=None, draft=None, mask=None,
                  repetition=None, presence=None, frequency=None, bias_token=None, bias=None, allowed=None,
                  flags: int = 0, stream=None) -> torch.Tensor:
    """Penalties for repeated tokens, biases and a grammar's mask on ``logits``
    ([B * T, V], fp32 or bf16, T rows per sequence), before ``sample``.  Returns
    ``out`` (new unless given; ``logits`` itself: in place).

    ``history`` int32 [B, L]: the sequences' tokens, ``history_len`` int32 [B] of
    them in use, the first ``prompt_len`` int32 [B] the prompt's; ``draft`` int32
    [B, T] and ``mask`` (as in ``KVStep``): the step's tokens, of which a row
    sees its own path's.  Tokens seen: divided (multiplied, where not above 0)
    by ``repetition``; tokens generated n times: less frequency * n + presence
    (fp32 [B] each).  ``bias_token`` int32 and ``bias`` fp32 [B, n] or [n]: added
    (those of one token to one another first, in order).  ``allowed`` int32
    [B * T, ceil(V / 32)] or [ceil(V / 32)]: a bit per token, the others become
    -inf.  B is the rows of history, draft, or a penalty; else of bias_token;
    without any of these, each row is its own sequence."""
    dev = logits.get_device()
    if stream is None and 0 <= dev == _current_device():
        status = (_binding or _load_binding()).adjust_logits(
            dev, logits, out, history, history_len, prompt_len, draft, mask, repetition, presence, frequency, bias_token, bias,
            allowed, flags, _current_stream(dev))
        if status is not None:
            if status:
                _check(status, "adjust_logits")
            return out
    if logits.dim() != 2:
        raise ValueError("logits must be [B * T, V]")
    M, V = logits.shape
    ld = V
    if not logits.is_contiguous():
        if logits.stride(1) != 1 and V > 1:
            raise ValueError("logits must have contiguous rows")
        ld = logits.stride(0) if M > 1 else V
    _same_device(dev, *[t for t in (out, history, history_len, prompt_len, draft, mask, repetition, presence, frequency, bias_token,
                                    bias, allowed) if t is not None])
    B = M
    for t in (history, draft, history_len, prompt_len, repetition, presence, frequency):
        if t is not None:
            B = len(t) if t.dim() else 0
            break
    else:
        if bias_token is not None and bias_token.dim() == 2:
            B = len(bias_token)
        elif M > _MAX_SEQUENCES:  # rows that nothing tells apart
            B = 1
    if (B < 1 or M % B) if M else B != 0:
        raise ValueError(f"{M} rows of logits do not belong to {B} sequences")
    T = M // B if B else 0
    L = history_stride = tree_stride = n_bias = bias_stride = allowed_stride = 0
    at_history = at_draft = at_mask = at_token = at_bias = at_allowed = 0
    if history is not None:
        if history.dim() != 2:
            raise ValueError("history must be [B, L]")
        L, history_stride = _table(history, B, _I32, "history")
        at_history = history.data_ptr()
    if draft is not None:
        if draft.shape != (B, T):
            raise ValueError("draft must be [B, T]")
        at_draft = _ints(draft, M, "draft")
        if mask is not None:
            if mask.dtype is not _I32 or mask.shape not in ((T,), (B, T)) or not mask.is_contiguous():
                raise ValueError("mask must be a contiguous int32 [T] or [B, T] tensor")
            at_mask, tree_stride = mask.data_ptr(), T if mask.dim() == 2 else 0
    elif mask is not None:
        raise ValueError("mask names rows of draft, which is not given")
    if (bias_token is None) != (bias is None):
        raise ValueError("bias_token and bias are given together")
    if bias is not None:
        n_bias, bias_stride = _table(bias_token, B, _I32, "bias_token")
        if bias.shape != bias_token.shape or _table(bias, B, _F32, "bias") != (n_bias, bias_stride):
            raise ValueError("bias must have the shape and strides of bias_token")
        at_token, at_bias = bias_token.data_ptr(), bias.data_ptr()
    if allowed is not None:
        words, allowed_stride = _table(allowed, M, _I32, "allowed")
        if words < (V + 31) // 32:
            raise ValueError("allowed must have a bit for each token")
        at_allowed = allowed.data_ptr()
    packed = _ADJUSTMENTS.pack(
        at_history, _ints(history_len, B, "history_len") or 0, _ints(prompt_len, B, "prompt_len") or 0, at_draft, at_mask,
        _floats(repetition, B, "repetition") or 0, _floats(presence, B, "presence") or 0,
        _floats(frequency, B, "frequency") or 0, at_token, at_bias, at_allowed, history_stride, tree_stride, bias_stride,
        allowed_stride, L, n_bias)
    out_ld = V
    if out is None:
        out = _empty((M, V), logits.dtype, logits.device, stream)
    elif out is logits:
        out_ld = ld
    else:
        if out.dtype is not logits.dtype or out.shape != (M, V):
            raise ValueError("out must have the shape and type of logits")
        if not out.is_contiguous():
            if out.stride(1) != 1 and V > 1:
                raise ValueError("out must have contiguous rows")
            out_ld = out.stride(0) if M > 1 else V
    status = _fn("qlin_adjust_logits")(B, T, V, DTYPES.get(logits.dtype, -1), logits.data_ptr(), ld,
                                       out.data_ptr(), out_ld, packed, flags, _current_stream(dev) if stream is None else _raw_stream(stream, dev))
    if status:
        _check(status, "adjust_logits")
    return out


def debug_sample_weight(x: torch.Tensor, max: torch.Tensor, temperature: torch.Tensor) -> torch.Tensor:
    """Test export: the weights that ``sample`` gives to logits ``x`` under their rows' largest ``max`` (fp32, on the
    CPU), as int64 multiples of 2^-42."""
    x, max, temperature = (t.to("cpu", torch.float32).contiguous() for t in torch.broadcast_tensors(x, max, temperature))
    out = torch.empty(x.shape, dtype=torch.int64)
    _check(_fn("qlin_debug_sample_weight")(x.numel(), x.data_ptr(), max.data_ptr(), temperature.data_ptr(),
                                           out.data_ptr()), "debug_sample_weight")
    return out


def debug_sample_plan(M: int, V: int, dtype, top_k: bool, most: int) -> tuple[int, bool]:
    """Test export: (CTAs per row, whether they read it where it is) of ``sample`` for M rows of V logits on a device
    whose clusters hold at most ``most`` CTAs (8 or 16)."""
    ctas, in_place = ctypes.c_int(), ctypes.c_int()
    _check(_fn("qlin_debug_sample_plan")(M, V, DTYPES.get(dtype, -1), int(top_k), most, ctypes.byref(ctas),
                                         ctypes.byref(in_place)), "debug_sample_plan")
    return ctas.value, bool(in_place.value)

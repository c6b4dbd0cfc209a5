"""Python binding of libqgemv (ctypes). Argument marshalling only: every step of the
quantize / pack / dequant-GEMV path runs in the C++ host library or in the HIP kernels.

PyTorch supplies device memory and streams: device arguments are torch tensors on a ROCm
device, and work is enqueued on torch's current stream unless ``stream`` is given.
Importing this module fails if the shared library has not been built
(``python dequant_gemv_q4g32_amd/build.py``); there is no fallback implementation.

QGEMV_HOST_ONLY_LIBRARY=<path> loads a build of the host code alone instead (the sanitizer
build of ``build.build_host_sanitized``): only the host functions are bound then, and every
device entry point is absent, so calling one raises instead of running anywhere else.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import re
import sys
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
HOST_ONLY_LIB = os.environ.get("QGEMV_HOST_ONLY_LIBRARY")
LIB_PATH = HOST_ONLY_LIB or os.path.join(_HERE, "libqgemv.so")
# exported by the host code (host.cpp); everything else is device code
HOST_FUNCTIONS = ("qg_abi_version", "qg_strerror", "qg_canonical_bytes", "qg_device_layout",
                  "qg_packed_bytes", "qg_kv_page_bytes", "qg_rope_freqs", "qg_pack_bits", "qg_unpack_bits", "qg_quantize", "qg_to_device_layout",
                  "qg_from_device_layout")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "qgemv.h")

FORMATS = {"q2sb": 2, "q3sb": 3, "q4g32": 4, "q5sb": 5, "q6sb": 6, "q4g16": 7, "q4g64": 8, "q4g128": 9,
           "q4a32": 10, "q4g32h": 11,
           "q2sb_bf16": 12, "q3sb_bf16": 13, "q5sb_bf16": 15, "q6sb_bf16": 16, "q3g32": 17, "q5g32": 18,
           "q3sb_planes": 14}
GROUPWISE_FORMATS = ("q3g32", "q5g32")   # plain group-wise codes, fp32 scale and min per 32
Q4_GROUPS = {"q4g16": 16, "q4g32": 32, "q4g64": 64, "q4g128": 128}   # symmetric INT4 group sizes
SUPERBLOCK_FORMATS = ("q2sb", "q3sb", "q5sb", "q6sb", "q2sb_bf16", "q3sb_bf16", "q5sb_bf16", "q6sb_bf16",
                      "q3sb_planes")
K_MULTIPLE = {"q4g32": 32, "q2sb": 256, "q3sb": 256, "q5sb": 256, "q6sb": 256, "q4g16": 64, "q4g64": 64, "q4g128": 128,
              "q4a32": 64, "q4g32h": 64, "q2sb_bf16": 256, "q3sb_bf16": 256, "q5sb_bf16": 256,
              "q6sb_bf16": 256, "q3g32": 64, "q5g32": 64,
              "q3sb_planes": 256}


class QGError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {_lib.qg_strerror(status).decode()} (status {status})"
        if status == -7:
            msg += f"; HIP: {_lib.qg_last_hip_error().decode()}"
        super().__init__(msg)


class Layout(ctypes.Structure):
    _fields_ = [("total_bytes", ctypes.c_int64), ("algorithmic_bytes", ctypes.c_int64),
                ("nplanes", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("plane_offset", ctypes.c_int64 * 4), ("plane_row_bytes", ctypes.c_int64 * 4)]


class _Pool(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("layers", ctypes.c_int64),
                ("layer_stride", ctypes.c_int64), ("kind", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32)]


class _Rotary(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("factor", ctypes.c_float), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


def _load() -> ctypes.CDLL:
    # torch ships its own HIP runtime under the same soname as ROCm's. Loading torch first
    # makes libqgemv bind to that one runtime; loading libqgemv first would map a second HIP
    # and HSA runtime into the process, which then finds no device, and torch's streams and
    # device pointers would mean nothing to it anyway.
    if not HOST_ONLY_LIB:
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python dequant_gemv_q4g32_amd/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    sig = {
        "qg_abi_version": ([], i32),
        "qg_strerror": ([i32], ctypes.c_char_p),
        "qg_last_hip_error": ([], ctypes.c_char_p),
        "qg_canonical_bytes": ([i32, i64, i64, ctypes.POINTER(i64)], i32),
        "qg_device_layout": ([i32, i64, i64, ctypes.POINTER(Layout)], i32),
        "qg_packed_bytes": ([i32, i64, i64, ctypes.POINTER(i64), ctypes.POINTER(i64)], i32),
        "qg_pack_bits": ([i32, vp, i64, vp], i32),
        "qg_unpack_bits": ([i32, vp, i64, vp], i32),
        "qg_quantize": ([i32, vp, i64, i64, i64, vp], i32),
        "qg_to_device_layout": ([i32, vp, i64, i64, vp], i32),
        "qg_from_device_layout": ([i32, vp, i64, i64, vp], i32),
        "qg_gemv": ([i32, vp, vp, vp, i32, i64, i64, vp], i32),
        "qg_gemv_batched": ([i32, vp, i64, vp, i64, vp, i64, i32, i64, i64, i64, vp], i32),
        "qg_gemm": ([i32, vp, vp, i64, vp, i64, i32, i64, i64, i64, vp], i32),
        "qg_gemm_grouped": ([i32, i32, vp, vp, vp, vp, vp, vp, vp, i64, i32, vp], i32),
        "qg_gemm_act_order": ([i32, vp, vp, i64, vp, vp, i64, i32, i64, i64, i64, vp], i32),
        "qg_kv_quantize": ([vp, i64, i64, i64, vp, vp, vp], i32),
        "qg_kv_dequantize": ([vp, vp, i64, i64, vp, i64, vp], i32),
        "qg_kv_page_bytes": ([i32, i64, i64, i64, ctypes.POINTER(i64)], i32),
        "qg_kv_append": ([vp, i64, vp, i64, i64, i64, vp, i64, vp, i64, vp, vp, i64, vp], i32),
        "qg_kv_gather": ([vp, i64, vp, i64, i64, i64, vp, i64, vp, i64, vp, vp, i64, vp], i32),
        "qg_paged_attention_bytes": ([vp, i64, i64, i64, ctypes.POINTER(i64)], i32),
        "qg_paged_attention": ([vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64, ctypes.c_float, vp, i64, i32, vp,
                                vp, i64, vp], i32),
        "qg_kv_copy_pages": ([vp, vp, vp, i64, vp], i32),
        "qg_kv_fork": ([vp, vp, i64, i64, i64, vp, vp, vp, vp, vp, i64, vp], i32),
        "qg_kv_free": ([vp, vp, i64, i64, i64, vp, vp, vp, i64, vp], i32),
        "qg_kv_compact_bytes": ([vp, ctypes.POINTER(i64)], i32),
        "qg_kv_compact": ([vp, vp, i64, vp, i64, i64, i64, vp, vp, vp, vp, vp, i64, vp], i32),
        "qg_prefix_attention_bytes": ([vp, i64, i64, i64, i64, i64, ctypes.POINTER(i64)], i32),
        "qg_prefix_attention": ([vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, i64, i64, i64, i64, ctypes.c_float, vp, i64, i32,
                                 vp, vp, i64, vp], i32),
        "qg_kv_extend_bytes": ([vp, i64, ctypes.POINTER(i64)], i32),
        "qg_kv_extend": ([vp, vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, i64, vp, i64, vp], i32),
        "qg_kv_trim": ([vp, vp, i64, i64, i64, vp, vp, vp, vp], i32),
        "qg_rope_freqs": ([i32, i64] + [ctypes.c_double] * 5 + [vp], i32),
        "qg_qk_rope": ([vp, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp], i32),
        "qg_kv_append_rope": ([vp, i64, vp, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp], i32),
        "qg_dequantize": ([i32, vp, vp, vp, i64, i64, vp], i32),
        "qg_read_probe": ([vp, i64, vp, vp], i32),
    }
    for f in FORMATS:
        sig[f"quantize_{f}"] = ([vp, i64, i64, i64, vp], i32)
        sig[f"dequant_gemv_{f}"] = ([vp, vp, vp, i64, i64, vp], i32)
        sig[f"dequant_gemm_{f}"] = ([vp, vp, i64, vp, i64, i64, i64, i64, vp], i32)
        sig[f"dequantize_{f}"] = ([vp, vp, vp, i64, i64, vp], i32)
    for name, (args, res) in sig.items():
        if HOST_ONLY_LIB and not (name in HOST_FUNCTIONS or name.startswith("quantize_")):
            continue
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if lib.qg_abi_version() != 1:
        raise ImportError("libqgemv ABI version mismatch")
    return lib


_lib = _load()
lib = _lib


def declared_functions() -> list:
    """Names of the functions include/qgemv.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)))


def _check(status: int, what: str) -> None:
    if status != 0:
        raise QGError(status, what)


def _fmt(fmt) -> int:
    if isinstance(fmt, str):
        return FORMATS[fmt]
    return int(fmt)


def _ptr(a: np.ndarray) -> int:
    return a.ctypes.data


# ---------------------------------------------------------------- host --------------------

def canonical_bytes(fmt, n: int, k: int) -> int:
    out = ctypes.c_int64()
    _check(_lib.qg_canonical_bytes(_fmt(fmt), n, k, ctypes.byref(out)), "qg_canonical_bytes")
    return out.value


def device_layout(fmt, n: int, k: int) -> Layout:
    out = Layout()
    _check(_lib.qg_device_layout(_fmt(fmt), n, k, ctypes.byref(out)), "qg_device_layout")
    return out


def pack_bits(bits: int, codes: np.ndarray) -> np.ndarray:
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    out = np.empty((codes.size * bits + 7) // 8, np.uint8)
    _check(_lib.qg_pack_bits(bits, _ptr(codes), codes.size, _ptr(out)), "qg_pack_bits")
    return out


def unpack_bits(bits: int, buf: np.ndarray, count: int) -> np.ndarray:
    buf = np.ascontiguousarray(buf, dtype=np.uint8)
    if buf.size < (count * bits + 7) // 8:
        raise ValueError("buffer too short")
    out = np.empty(count, np.uint8)
    _check(_lib.qg_unpack_bits(bits, _ptr(buf), count, _ptr(out)), "qg_unpack_bits")
    return out


def quantize(fmt, w: np.ndarray) -> np.ndarray:
    """fp32 W [n, k] -> canonical encoding (uint8, qg_canonical_bytes bytes)."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    n, k = w.shape
    out = np.empty(canonical_bytes(fmt, n, k), np.uint8)
    _check(_lib.qg_quantize(_fmt(fmt), _ptr(w), n, k, k, _ptr(out)), "qg_quantize")
    return out


def to_device_layout(fmt, canonical: np.ndarray, n: int, k: int) -> np.ndarray:
    canonical = np.ascontiguousarray(canonical, dtype=np.uint8)
    if canonical.size != canonical_bytes(fmt, n, k):
        raise ValueError("canonical buffer has the wrong size")
    out = np.empty(device_layout(fmt, n, k).total_bytes, np.uint8)
    _check(_lib.qg_to_device_layout(_fmt(fmt), _ptr(canonical), n, k, _ptr(out)), "qg_to_device_layout")
    return out


def from_device_layout(fmt, dev: np.ndarray, n: int, k: int) -> np.ndarray:
    dev = np.ascontiguousarray(dev, dtype=np.uint8)
    if dev.size != device_layout(fmt, n, k).total_bytes:
        raise ValueError("device-layout buffer has the wrong size")
    out = np.empty(canonical_bytes(fmt, n, k), np.uint8)
    _check(_lib.qg_from_device_layout(_fmt(fmt), _ptr(dev), n, k, _ptr(out)), "qg_from_device_layout")
    return out


# ---------------------------------------------------------------- device -------------------

def _torch():
    import torch
    return torch


def _stream(stream) -> int:
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def upload(fmt, w: np.ndarray, device="cuda") -> "torch.Tensor":
    """Quantize fp32 W on the host, lay it out for the device and copy it to `device`."""
    torch = _torch()
    n, k = w.shape
    dev = to_device_layout(fmt, quantize(fmt, w), n, k)
    return torch.from_numpy(dev).to(device)


def to_device(fmt, canonical: np.ndarray, n: int, k: int, device="cuda") -> "torch.Tensor":
    torch = _torch()
    return torch.from_numpy(to_device_layout(fmt, canonical, n, k)).to(device)


def gemv(fmt, w, x, n: int, k: int, out=None, out_f32: bool = False, stream=None):
    """y = W_hat x. w: uint8 device buffer (device layout), x: fp16 [k] -> y fp16/fp32 [n]."""
    torch = _torch()
    if out is None:
        out = torch.empty(n, dtype=torch.float32 if out_f32 else torch.float16, device=x.device)
    _check(_lib.qg_gemv(_fmt(fmt), w.data_ptr(), x.data_ptr(), out.data_ptr(), int(out.dtype == torch.float32),
                        n, k, _stream(stream)), "qg_gemv")
    return out


def gemv_batched(fmt, w, w_stride: int, x, y, count: int, n: int, k: int, stream=None):
    """count independent GEMVs: W_b at w + b*w_stride bytes, x_b = x[b], y_b = y[b]."""
    torch = _torch()
    _check(_lib.qg_gemv_batched(_fmt(fmt), w.data_ptr(), w_stride, x.data_ptr(), x.stride(0), y.data_ptr(),
                                y.stride(0), int(y.dtype == torch.float32), count, n, k, _stream(stream)),
           "qg_gemv_batched")
    return y


def gemm(fmt, w, X, n: int, k: int, out=None, out_f32: bool = False, stream=None):
    """Y = X W_hat^T. w: uint8 device buffer (device layout), X: fp16 [m, k] (row stride
    X.stride(0)) -> Y fp16/fp32 [m, n]."""
    torch = _torch()
    m = X.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32 if out_f32 else torch.float16, device=X.device)
    _check(_lib.qg_gemm(_fmt(fmt), w.data_ptr(), X.data_ptr(), X.stride(0), out.data_ptr(), out.stride(0),
                        int(out.dtype == torch.float32), m, n, k, _stream(stream)), "qg_gemm")
    return out


def gemm_act_order(fmt, w, X, perm, n: int, k: int, out=None, out_f32: bool = False, stream=None):
    """Y = X[:, perm] W_hat^T for weights quantized with their columns permuted (stored column c
    is original column perm[c]). X: fp16 [m, k] (m <= 8) or [k]; perm: int32 [k] on the device."""
    torch = _torch()
    vec = X.dim() == 1
    m = 1 if vec else X.shape[0]
    if out is None:
        out = torch.empty((n,) if vec else (m, n), dtype=torch.float32 if out_f32 else torch.float16, device=X.device)
    if perm.dtype != torch.int32:
        raise TypeError("perm must be int32")
    _check(_lib.qg_gemm_act_order(_fmt(fmt), w.data_ptr(), X.data_ptr(), k if vec else X.stride(0), perm.data_ptr(),
                                  out.data_ptr(), n if vec else out.stride(0), int(out.dtype == torch.float32), m, n, k,
                                  _stream(stream)), "qg_gemm_act_order")
    return out


def gemm_grouped(fmt, ws, Xs, shapes, outs=None, out_f32: bool = False, stream=None):
    """One launch over several matrices: outs[g] = Xs[g] W_hat_g^T for W_g of shapes[g] = (n, k)
    at ws[g] (device layout). Every Xs[g] is fp16 [m, k_g] (one m, at most 8, row stride
    X.stride(0)) or [k_g] for m = 1; outs[g] is [m, n_g] (or [n_g]), allocated when None."""
    torch = _torch()
    count = len(ws)
    if not (len(Xs) == len(shapes) == count):
        raise ValueError("ws, Xs and shapes must have one entry per matrix")
    vec = Xs[0].dim() == 1
    m = 1 if vec else Xs[0].shape[0]
    dt = torch.float32 if out_f32 else torch.float16
    if outs is None:
        outs = [torch.empty((n,) if vec else (m, n), dtype=dt, device=X.device) for X, (n, _) in zip(Xs, shapes)]
    arr = lambda ctype, vals: (ctype * max(count, 1))(*vals)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    _check(_lib.qg_gemm_grouped(
        _fmt(fmt), count, arr(vp, [w.data_ptr() for w in ws]), arr(vp, [X.data_ptr() for X in Xs]),
        arr(i64, [X.stride(0) if X.dim() == 2 else X.shape[0] for X in Xs]), arr(vp, [y.data_ptr() for y in outs]),
        arr(i64, [y.stride(0) if y.dim() == 2 else y.shape[0] for y in outs]), arr(i64, [n for n, _ in shapes]),
        arr(i64, [k for _, k in shapes]), m, int(outs[0].dtype == torch.float32), _stream(stream)), "qg_gemm_grouped")
    return outs


def kv_quantize(x, codes=None, scales=None, stream=None):
    """8-bit KV-cache groups: fp16 [rows, cols] (row stride x.stride(0), cols % 32 == 0) ->
    (int8 codes [rows, cols], fp16 scales [rows, cols / 32])."""
    torch = _torch()
    rows, cols = x.shape
    if codes is None:
        codes = torch.empty((rows, cols), dtype=torch.int8, device=x.device)
    if scales is None:
        scales = torch.empty((rows, cols // 32), dtype=torch.float16, device=x.device)
    _check(_lib.qg_kv_quantize(x.data_ptr(), x.stride(0), rows, cols, codes.data_ptr(), scales.data_ptr(),
                               _stream(stream)), "qg_kv_quantize")
    return codes, scales


def kv_dequantize(codes, scales, out=None, stream=None):
    """int8 codes [rows, cols] and fp16 scales [rows, cols / 32] -> fp16 [rows, cols]."""
    torch = _torch()
    rows, cols = codes.shape
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float16, device=codes.device)
    _check(_lib.qg_kv_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, out.data_ptr(), out.stride(0),
                                 _stream(stream)), "qg_kv_dequantize")
    return out


# ---------------------------------------------------------------- paged KV cache -----------

KV_KINDS = {"q8": 1, "f16": 2}


def kv_page_bytes(kind: str, kv_heads: int, head_dim: int, page_tokens: int) -> int:
    """Bytes of one page record: page_tokens tokens of K and V for every KV head."""
    out = ctypes.c_int64()
    _check(_lib.qg_kv_page_bytes(KV_KINDS[kind], kv_heads, head_dim, page_tokens, ctypes.byref(out)), "qg_kv_page_bytes")
    return out.value


def _workspace(what: str, c: _Pool, *sizes) -> int:
    out = ctypes.c_int64()
    _check(getattr(_lib, what)(ctypes.addressof(c), *sizes, ctypes.byref(out)), what)
    return out.value


class KVPool:
    """A pool of cache pages: uint8 [num_pages, page_bytes], or [layers, num_pages, page_bytes] for
    several layers that share one page table. kind "q8": int8 groups of 32 with fp16 scales (the
    codec of kv_quantize); "f16": fp16. The record's layout is in include/qgemv.h. The pool keeps
    `pages` alive; every call on it takes its tensors on the pool's device and runs on torch's
    current stream of that device unless `stream` (a torch stream of that device, or a handle of
    one as an int) is given."""

    def __init__(self, pages, kind: str, kv_heads: int, head_dim: int, page_tokens: int):
        torch = _torch()
        size = kv_page_bytes(kind, kv_heads, head_dim, page_tokens)
        if pages.dtype != torch.uint8 or pages.dim() not in (2, 3) or pages.shape[-1] != size:
            raise ValueError(f"pages must be uint8 [.., num_pages, {size}]")
        dense = pages.stride(-1) == 1 and (pages.shape[-2] == 1 or pages.stride(-2) == size)
        if not pages.is_cuda or not dense:
            raise ValueError("pages must be on a GPU, each layer's records dense")
        self.pages, self.kind, self.kv_heads, self.head_dim, self.page_tokens = pages, kind, kv_heads, head_dim, page_tokens
        self.num_pages = pages.shape[-2]
        self.layers = pages.shape[0] if pages.dim() == 3 else 1
        self.device = pages.device
        self._index = pages.get_device()
        self._c = _Pool(pages.data_ptr(), self.num_pages, self.layers, pages.stride(0) if self.layers > 1 else 0,
                        KV_KINDS[kind], kv_heads, head_dim, page_tokens)
        self._ref = ctypes.addressof(self._c)
        # workspace sizes, kept by the sizes they follow from: asking the library takes 1 us of a call's 15
        self._attention_bytes = functools.lru_cache(256)(functools.partial(_workspace, "qg_paged_attention_bytes", self._c))
        self._prefix_bytes = functools.lru_cache(256)(functools.partial(_workspace, "qg_prefix_attention_bytes", self._c))
        self._extend_bytes = functools.lru_cache(256)(functools.partial(_workspace, "qg_kv_extend_bytes", self._c))
        self._compact_bytes = functools.lru_cache(1)(functools.partial(_workspace, "qg_kv_compact_bytes", self._c))

    @classmethod
    def zeros(cls, kind: str, kv_heads: int, head_dim: int, page_tokens: int, num_pages: int, layers: int = 1,
              device="cuda"):
        torch = _torch()
        size = kv_page_bytes(kind, kv_heads, head_dim, page_tokens)
        return cls(torch.zeros((layers, num_pages, size), dtype=torch.uint8, device=device), kind, kv_heads, head_dim,
                   page_tokens)


# torch's own accessors behind torch.cuda.current_device and current_stream, which cost a decode
# step's launch time each; the public ones where a torch does not have them
_th = sys.modules.get("torch")
_device_now = getattr(getattr(_th, "_C", None), "_cuda_getDevice", None) or (lambda: _th.cuda.current_device())
_stream_now = (getattr(getattr(_th, "_C", None), "_cuda_getCurrentRawStream", None)
               or (lambda index: _th.cuda.current_stream(index).cuda_stream))


@contextlib.contextmanager
def _on(pool, stream):
    """The pool's device current and `stream` (None: that device's current one) torch's current
    stream, so that what a call allocates inside belongs to the stream it runs on."""
    if stream is not None and not isinstance(stream, int) and stream.device != pool.device:
        raise ValueError(f"stream must be one of {pool.device}")       # entering it would switch the device
    with _th.cuda.device(pool._index):
        if stream is None:
            yield
            return
        if isinstance(stream, int):
            stream = _th.cuda.ExternalStream(stream) if stream else _th.cuda.default_stream()
        with _th.cuda.stream(stream):
            yield


def _ints(pool, what: str, t, length=None):
    """Address of a dense int32 vector on the pool's device."""
    if (t.dtype is not _th.int32 or t.get_device() != pool._index or t.dim() != 1 or not t.is_contiguous()
            or (length is not None and t.numel() != length)):
        raise ValueError(f"{what} must be a dense int32 vector{'' if length is None else f' of {length}'} on {pool.device}")
    return t.data_ptr()


def _table(pool, t):
    """(address, leading dimension, rows, pages a row) of a page table."""
    if (t.dtype is not _th.int32 or t.get_device() != pool._index or t.dim() != 2
            or not (t.is_contiguous() or t.shape[1] < 2 or t.stride(1) == 1)):
        raise ValueError(f"a page table must be int32 [sequences, pages] with dense rows on {pool.device}")
    rows, pages = t.shape
    return t.data_ptr(), t.stride(0), rows, pages


def _rows16(pool, what: str, t, count: int):
    """(address, leading dimension) of fp16 rows [count, kv_heads * head_dim]."""
    if (t.dtype is not _th.float16 or t.get_device() != pool._index or t.dim() != 2
            or not (t.is_contiguous() or t.stride(1) == 1) or t.shape != (count, pool.kv_heads * pool.head_dim)):
        raise ValueError(f"{what} must be fp16 [{count}, {pool.kv_heads * pool.head_dim}] with dense rows on {pool.device}")
    return t.data_ptr(), t.stride(0)


def kv_append(pool, table, k, v, positions, seqs=None, layer: int = 0, stream=None) -> None:
    """Write token rows into the cache: k, v fp16 [count, kv_heads * head_dim]; row i becomes token
    positions[i] of table row seqs[i] (row i when seqs is None). A row without a place (position
    -1, say) is skipped; the rows of one call must name distinct places."""
    if stream is not None or _device_now() != pool._index:
        with _on(pool, stream):
            return kv_append(pool, table, k, v, positions, seqs, layer)
    count = positions.numel()
    _check(_lib.qg_kv_append(pool._ref, layer, *_table(pool, table), *_rows16(pool, "k", k, count),
                             *_rows16(pool, "v", v, count), None if seqs is None else _ints(pool, "seqs", seqs, count),
                             _ints(pool, "positions", positions), count, _stream_now(pool._index)), "qg_kv_append")


def kv_gather(pool, table, positions, seqs=None, k=None, v=None, layer: int = 0, stream=None):
    """Read token rows back, decoded: (k, v) fp16 [count, kv_heads * head_dim], row i token
    positions[i] of table row seqs[i] (row i when seqs is None), zeros where there is none."""
    if stream is not None or _device_now() != pool._index:
        with _on(pool, stream):
            return kv_gather(pool, table, positions, seqs, k, v, layer)
    count, cols = positions.numel(), pool.kv_heads * pool.head_dim
    if k is None:
        k = positions.new_empty((count, cols), dtype=_th.float16)
    if v is None:
        v = _th.empty_like(k) if k.is_contiguous() else positions.new_empty((count, cols), dtype=_th.float16)
    _check(_lib.qg_kv_gather(pool._ref, layer, *_table(pool, table), *_rows16(pool, "k", k, count),
                             *_rows16(pool, "v", v, count), None if seqs is None else _ints(pool, "seqs", seqs, count),
                             _ints(pool, "positions", positions), count, _stream_now(pool._index)), "qg_kv_gather")
    return k, v


def paged_attention_bytes(pool, batch: int, heads: int, max_len: int) -> int:
    """Workspace bytes of paged_attention for these sizes (0: it needs none)."""
    return pool._attention_bytes(batch, heads, max_len)


def _attention_args(pool, q, table, max_len, scale, out, out_f32, lse, return_lse):
    """What the attentions over the cache take in common, checked, with its defaults and outputs."""
    if q.dtype is not _th.float16 or q.get_device() != pool._index or q.dim() != 3:
        raise ValueError(f"q must be fp16 [batch, heads, head_dim] on {pool.device}")
    shape = batch, heads, dim = q.shape
    if dim != pool.head_dim or not (q.is_contiguous() or (q.stride(2) == 1 and (heads == 1 or q.stride(1) == dim))):
        raise ValueError(f"q must have dense heads of {pool.head_dim}")
    at, ld, rows, pages = _table(pool, table)
    if max_len is None:
        max_len = pages * pool.page_tokens
    if rows != batch or pages * pool.page_tokens < max_len:
        raise ValueError("the table must have a row for each sequence, and pages for max_len tokens")
    if scale is None:
        scale = dim ** -0.5
    if out is None:
        out = q.new_empty(shape, dtype=_th.float32) if out_f32 else q.new_empty(shape)
    elif (out.shape != shape or out.dtype not in (_th.float16, _th.float32) or out.device != pool.device
          or out.stride(2) != 1 or (heads > 1 and out.stride(1) != dim)):
        raise ValueError(f"out must be fp16 or fp32 [{batch}, {heads}, {dim}] with dense heads on {pool.device}")
    if lse is not None:
        if lse.shape != (batch, heads) or lse.dtype != _th.float32 or lse.device != pool.device or not lse.is_contiguous():
            raise ValueError(f"lse must be dense fp32 [{batch}, {heads}] on {pool.device}")
    elif return_lse:
        lse = q.new_empty((batch, heads), dtype=_th.float32)
    return batch, heads, at, ld, max_len, scale, out, lse


def paged_attention(pool, q, table, lens, max_len: Optional[int] = None, scale: Optional[float] = None, window: int = 0,
                    out=None, out_f32: bool = False, lse=None, return_lse: bool = False, workspace=None, layer: int = 0,
                    stream=None):
    """Attention of one new token a sequence over its cached tokens. q: fp16 [batch, heads, head_dim]
    (row stride q.stride(0), heads dense); table: int32 [batch, pages]; lens: int32 [batch], each
    sequence's tokens, the new one's K and V (kv_append) among them. max_len bounds lens (default:
    what the table holds); scale defaults to head_dim ** -0.5; window > 0 sees the last `window`
    tokens only. Returns out [batch, heads, head_dim] (fp16, or fp32 with out_f32), or (out, lse)
    with return_lse or when lse (fp32 [batch, heads]) is given. A sequence without tokens gets zeros and
    lse -inf. workspace: uint8 of paged_attention_bytes(...), used by one call at a time; allocated
    here when None. out, lse and workspace overlap nothing that the call reads, q among it."""
    if stream is not None or _device_now() != pool._index:
        with _on(pool, stream):
            return paged_attention(pool, q, table, lens, max_len, scale, window, out, out_f32, lse, return_lse, workspace, layer)
    batch, heads, at, ld, max_len, scale, out, lse = _attention_args(pool, q, table, max_len, scale, out, out_f32, lse, return_lse)
    if workspace is None:
        need = pool._attention_bytes(batch, heads, max_len)
        workspace = q.new_empty(need, dtype=_th.uint8) if need else None
    elif workspace.dtype != _th.uint8 or workspace.device != pool.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be dense uint8 on {pool.device}")
    _check(_lib.qg_paged_attention(pool._ref, layer, q.data_ptr(), q.stride(0), at, ld, _ints(pool, "lens", lens, batch),
                                   batch, heads, max_len, window, scale, out.data_ptr(), out.stride(0),
                                   out.dtype is _th.float32, None if lse is None else lse.data_ptr(),
                                   *((None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())),
                                   _stream_now(pool._index)), "qg_paged_attention")
    return out if lse is None else (out, lse)


def prefix_attention_bytes(pool, batch: int, heads: int, groups: int, max_len: int, max_tail: int) -> int:
    """Workspace bytes of prefix_attention for these sizes."""
    return pool._prefix_bytes(batch, heads, groups, max_len, max_tail)


def prefix_attention(pool, q, table, lens, starts, prefix, max_len: Optional[int] = None, max_tail: Optional[int] = None,
                     scale: Optional[float] = None, out=None, out_f32: bool = False, lse=None, return_lse: bool = False,
                     workspace=None, layer: int = 0, stream=None):
    """paged_attention of rows that share their first tokens in groups (forks of one prompt, say): the
    shared tokens are read and multiplied once a group where that is less work than for each row. Group g is the rows
    starts[g] to starts[g + 1] - 1 (int32 [groups + 1], ascending); the first prefix[g] tokens (int32 [groups]) of its
    rows are the same, by pages that they share or by equal ones. Rows in no group, and what follows a prefix, are read as by
    paged_attention. max_tail bounds the tokens that a row does not share (default: max_len); more of them are slower,
    no less right. The other arguments and the results are paged_attention's, without a window."""
    if stream is not None or _device_now() != pool._index:
        with _on(pool, stream):
            return prefix_attention(pool, q, table, lens, starts, prefix, max_len, max_tail, scale, out, out_f32, lse, return_lse,
                                    workspace, layer)
    batch, heads, at, ld, max_len, scale, out, lse = _attention_args(pool, q, table, max_len, scale, out, out_f32, lse, return_lse)
    groups = prefix.numel()
    if max_tail is None:
        max_tail = max_len
    if workspace is None:
        workspace = q.new_empty(pool._prefix_bytes(batch, heads, groups, max_len, max_tail), dtype=_th.uint8)
    elif workspace.dtype != _th.uint8 or workspace.device != pool.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be dense uint8 on {pool.device}")
    _check(_lib.qg_prefix_attention(pool._ref, layer, q.data_ptr(), q.stride(0), at, ld, _ints(pool, "lens", lens, batch),
                                    _ints(pool, "starts", starts, groups + 1), _ints(pool, "prefix", prefix), groups, batch, heads,
                                    max_len, max_tail, scale, out.data_ptr(), out.stride(0), out.dtype is _th.float32,
                                    None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                    _stream_now(pool._index)), "qg_prefix_attention")
    return out if lse is None else (out, lse)


def kv_copy_pages(pool, src, dst, stream=None) -> None:
    """Copy pages src[i] to dst[i] (int32 vectors on the device) in every layer of the pool."""
    if stream is not None or _device_now() != pool._index:
        with _on(pool, stream):
            return kv_copy_pages(pool, src, dst)
    count = src.numel()
    _check(_lib.qg_kv_copy_pages(pool._ref, _ints(pool, "src", src), _ints(pool, "dst", dst, count), count,
                                 _stream_now(pool._index)), "qg_kv_copy_pages")


def kv_fork(pool, table, lens, refs, src_rows, dst_rows, new_pages, stream=None) -> None:
    """Table rows dst_rows become second holders of src_rows' tokens: whole pages are shared (refs
    counts them), a partly filled last page is copied to new_pages[i] (a free page, left free where
    there is nothing to copy). table, lens and refs are updated in place; free the destination rows
    first if they hold anything."""
    if stream is not None or _device_now() != pool._index:
        with _on(pool, stream):
            return kv_fork(pool, table, lens, refs, src_rows, dst_rows, new_pages)
    at, ld, rows, pages = _table(pool, table)
    count = src_rows.numel()
    _check(_lib.qg_kv_fork(pool._ref, at, ld, rows, pages, _ints(pool, "lens", lens, rows),
                           _ints(pool, "refs", refs, pool.num_pages), _ints(pool, "src_rows", src_rows),
                           _ints(pool, "dst_rows", dst_rows, count), _ints(pool, "new_pages", new_pages, count), count,
                           _stream_now(pool._index)), "qg_kv_fork")


def kv_free(pool, table, lens, refs, rows, stream=None) -> None:
    """Give up the pages of table rows `rows`: their refs fall by one, the rows become empty."""
    if stream is not None or _device_now() != pool._index:
        with _on(pool, stream):
            return kv_free(pool, table, lens, refs, rows)
    at, ld, table_rows, pages = _table(pool, table)
    _check(_lib.qg_kv_free(pool._ref, at, ld, table_rows, pages, _ints(pool, "lens", lens, table_rows),
                           _ints(pool, "refs", refs, pool.num_pages), _ints(pool, "rows", rows), rows.numel(),
                           _stream_now(pool._index)), "qg_kv_free")


def kv_compact(pool, table, refs, table_out=None, refs_out=None, remap=None, live=None, stream=None):
    """Move the held pages of the pool to its first pages, in every layer. Returns (table_out,
    refs_out, remap, live): the table and the counts for the moved pages (pass table and refs
    themselves to update them in place, else they must not overlap), each page's new index (-1: free),
    and the number of held pages (int32 [1] on the device). What is not given is allocated, the last
    three as views of one buffer when none of them is."""
    if stream is not None or _device_now() != pool._index:
        with _on(pool, stream):
            return kv_compact(pool, table, refs, table_out, refs_out, remap, live)
    at, ld, rows, pages = _table(pool, table)
    need = pool._compact_bytes()

    table_out = table.new_empty((rows, pages)) if table_out is None else table_out
    n = pool.num_pages
    if refs_out is None and remap is None and live is None:      # one allocation for what is counted in pages
        refs_out, remap, live, workspace = refs.new_empty(2 * n + 1 + need // 4).split_with_sizes((n, n, 1, need // 4))
    else:
        refs_out = refs.new_empty(n) if refs_out is None else refs_out
        remap = refs.new_empty(n) if remap is None else remap
        live = refs.new_empty(1) if live is None else live
        workspace = refs.new_empty(need // 4)
    to = _table(pool, table_out)
    if to[2:] != (rows, pages):
        raise ValueError("table_out must have table's shape")
    _check(_lib.qg_kv_compact(pool._ref, at, ld, to[0], to[1], rows, pages, _ints(pool, "refs", refs, pool.num_pages),
                              _ints(pool, "refs_out", refs_out, pool.num_pages),
                              _ints(pool, "remap", remap, pool.num_pages), _ints(pool, "live", live, 1),
                              workspace.data_ptr(), need, _stream_now(pool._index)), "qg_kv_compact")
    return table_out, refs_out, remap, live


def kv_extend(pool, table, lens, refs, add, slots: int, granted=None, starts=None, seqs=None, positions=None, stream=None):
    """Places for a step's new tokens: row r of the table asks for add[r] more (int32 on the device, 0
    or less: none), and gets the free pages that it lacks for them. Returns (granted, seqs, positions):
    the tokens that each row got (add[r], or 0), and the slot map of `slots` places that kv_append
    takes, row after row with the tokens asked for; the places of a row that got none hold -1, as do
    those past the last row's. table, lens and refs are updated in place. A row gets none when the slots,
    its table entries or the free pages (the rows before it come first, those that the free pages did not suffice for among
    them: one request that is too large leaves no page for the rows behind it) do not suffice, or when other rows hold the
    partly filled page that its tokens would go to. starts, int32 [rows + 1], receives each row's first slot
    if given; what else is not given is allocated as views of one buffer when none of it is."""
    if stream is not None or _device_now() != pool._index:
        with _on(pool, stream):
            return kv_extend(pool, table, lens, refs, add, slots, granted, starts, seqs, positions)
    at, ld, rows, pages = _table(pool, table)
    if slots < 0:
        raise ValueError("slots must not be negative")
    need = pool._extend_bytes(rows)
    if granted is None and seqs is None and positions is None:
        granted, seqs, positions, workspace = refs.new_empty(rows + 2 * slots + need // 4).split_with_sizes(
            (rows, slots, slots, need // 4))
    else:
        granted = refs.new_empty(rows) if granted is None else granted
        seqs = refs.new_empty(slots) if seqs is None else seqs
        positions = refs.new_empty(slots) if positions is None else positions
        workspace = refs.new_empty(need // 4)
    _check(_lib.qg_kv_extend(pool._ref, at, ld, rows, pages, _ints(pool, "lens", lens, rows),
                             _ints(pool, "refs", refs, pool.num_pages), _ints(pool, "add", add, rows),
                             _ints(pool, "granted", granted, rows),
                             None if starts is None else _ints(pool, "starts", starts, rows + 1),
                             _ints(pool, "seqs", seqs, slots), _ints(pool, "positions", positions, slots), slots,
                             workspace.data_ptr(), need, _stream_now(pool._index)), "qg_kv_extend")
    return granted, seqs, positions


def kv_trim(pool, table, lens, refs, to, stream=None) -> None:
    """The way back: a row r with 0 <= to[r] < lens[r] keeps its first to[r] tokens (int32 [rows] on
    the device) and gives up the pages past them. table, lens and refs are updated in place."""
    if stream is not None or _device_now() != pool._index:
        with _on(pool, stream):
            return kv_trim(pool, table, lens, refs, to)
    at, ld, rows, pages = _table(pool, table)
    _check(_lib.qg_kv_trim(pool._ref, at, ld, rows, pages, _ints(pool, "lens", lens, rows),
                           _ints(pool, "refs", refs, pool.num_pages), _ints(pool, "to", to, rows),
                           _stream_now(pool._index)), "qg_kv_trim")


ROPE_KINDS = {"plain": 0, "linear": 1, "base": 2, "turns": 3, "parts": 4}


def rope_freqs(rotary_dim: int, base: float = 10000.0, kind: str = "plain", scale: float = 1.0, context: float = 0.0,
               low: float = 1.0, high: float = 32.0) -> np.ndarray:
    """Radians a token of each rotated pair (fp64 [rotary_dim / 2], on the host). kind scales them for
    contexts longer than the trained one: "linear" divides all by scale, "base" raises the base,
    "turns" and "parts" slow the pairs that turn less than `low` times in the trained `context` tokens and
    keep those of over `high` turns (include/qgemv.h has the formulas)."""
    out = np.empty(max(0, rotary_dim // 2), dtype=np.float64)
    _check(_lib.qg_rope_freqs(ROPE_KINDS[kind], rotary_dim, base, scale, context, low, high, _ptr(out)), "qg_rope_freqs")
    return out


class Rotary:
    """What kv_append_rope and qk_rope do to a head of head_dim elements: the norm, if there are
    weights (fp16 [head_dim]), then the rotation of its first 2 * len(freqs) elements by position * freqs
    (fp64, radians a token: an array such as rope_freqs gives, copied to `device`, or a tensor there;
    None: no rotation). interleaved: pairs are neighbours instead of halves apart. factor scales the
    rotated elements. Keeps its tensors alive."""

    def __init__(self, head_dim: int, freqs=None, interleaved: bool = False, q_weight=None, k_weight=None, eps: float = 1e-6,
                 factor: float = 1.0, device="cuda"):
        torch = _torch()
        if freqs is not None and not isinstance(freqs, torch.Tensor):
            freqs = torch.from_numpy(np.ascontiguousarray(freqs, dtype=np.float64)).to(device)
        if freqs is not None and (freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous()):
            raise ValueError("freqs must be a dense fp64 vector")
        held = [t for t in (freqs, q_weight, k_weight) if t is not None]
        for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
            if t is not None and (t.dtype != torch.float16 or t.shape != (head_dim,) or not t.is_contiguous()):
                raise ValueError(f"{name} must be a dense fp16 vector of {head_dim}")
        if len({t.device for t in held}) > 1 or not all(t.is_cuda for t in held):
            raise ValueError("freqs and weights must be on one GPU")
        self.head_dim, self.rotary_dim = head_dim, 0 if freqs is None else 2 * freqs.numel()
        self.freqs, self.q_weight, self.k_weight = freqs, q_weight, k_weight
        self._index = held[0].get_device() if held else None
        address = [None if t is None else t.data_ptr() for t in (freqs, q_weight, k_weight)]
        self._c = _Rotary(*address, eps, factor, self.rotary_dim, bool(interleaved))
        self._ref = ctypes.addressof(self._c)


class _Where:
    """What a pool says of its place, for calls without one."""
    __slots__ = ("device", "_index")

    def __init__(self, t):
        self.device, self._index = t.device, t.get_device()


def _head_rows(index, what: str, t, count: int, head_dim: int):
    """(address, leading dimension, heads) of fp16 rows [count, heads * head_dim], or [count, heads, head_dim]
    with dense heads."""
    shape, ok = t.shape, t.dtype is _th.float16 and t.get_device() == index and t.dim() in (2, 3) and t.shape[0] == count
    if ok and t.dim() == 3:
        ok = shape[2] == head_dim and (t.is_contiguous() or (t.stride(2) == 1 and (shape[1] < 2 or t.stride(1) == head_dim)))
        heads = shape[1]
    elif ok:
        ok = shape[1] % head_dim == 0 and (t.is_contiguous() or t.stride(1) == 1)
        heads = shape[1] // head_dim
    if not ok:
        raise ValueError(f"{what} must be fp16 [{count}, heads * {head_dim}] or [{count}, heads, {head_dim}] with dense rows "
                         f"on cuda:{index}")
    return t.data_ptr(), t.stride(0), heads


def _heads_out(index, what: str, out, t, count: int, heads: int, head_dim: int):
    """(out, address, leading dimension) of an output for t, allocated dense if none is given."""
    if out is None:
        out = t.new_empty(t.shape)
        return out, out.data_ptr(), heads * head_dim
    at, ld, out_heads = _head_rows(index, what, out, count, head_dim)
    if out_heads != heads:
        raise ValueError(f"{what} must have its input's {heads} heads")
    return out, at, ld


def qk_rope(rotary, q, k, positions, q_out=None, k_out=None, stream=None):
    """Norm and rotate queries and keys: fp16 [count, heads * head_dim] (or [count, heads, head_dim]) with any
    row stride, row i at positions[i] (int32 on the device; below 0: the row of the output stays as it
    is). Returns (q_out, k_out), dense where they are allocated here; q and k themselves may be given. k may be
    None (then so is k_out)."""
    if not q.is_cuda:
        raise ValueError("q must be on a GPU")
    where = _Where(q)
    index = where._index
    if stream is not None or _device_now() != index:
        with _on(where, stream):
            return qk_rope(rotary, q, k, positions, q_out, k_out)
    if rotary._index not in (None, index):
        raise ValueError(f"the rotary's tensors are on cuda:{rotary._index}, q on {q.device}")
    count, dim = q.shape[0], rotary.head_dim
    at, ld, heads = _head_rows(index, "q", q, count, dim)
    kat, ldk, kv_heads = (None, 0, 0) if k is None else _head_rows(index, "k", k, count, dim)
    q_out, to, ldo = _heads_out(index, "q_out", q_out, q, count, heads, dim)
    kto, ldko = None, 0
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    if k is not None:
        k_out, kto, ldko = _heads_out(index, "k_out", k_out, k, count, kv_heads, dim)
    _check(_lib.qg_qk_rope(rotary._ref, dim, heads, kv_heads, at, ld, kat, ldk, _ints(where, "positions", positions, count), count,
                           to, ldo, kto, ldko, _stream_now(index)), "qg_qk_rope")
    return q_out, k_out


def kv_append_rope(pool, table, rotary, q, k, v, positions, seqs=None, q_out=None, layer: int = 0, stream=None):
    """qk_rope and kv_append in one pass: the normed and rotated queries are returned (q_out, dense where it
    is allocated here; q itself may be given), the keys and v go into the cache as token positions[i] of table
    row seqs[i] (row i when seqs is None). q: fp16 [count, heads * head_dim] or [count, heads, head_dim],
    or None; k, v: fp16 [count, kv_heads * head_dim]; any row strides. A row with position -1 is
    skipped, its row of q_out stays as it is; one without a page gives its queries only."""
    if stream is not None or _device_now() != pool._index:
        with _on(pool, stream):
            return kv_append_rope(pool, table, rotary, q, k, v, positions, seqs, q_out, layer)
    if rotary._index not in (None, pool._index) or rotary.head_dim != pool.head_dim:
        raise ValueError(f"the rotary must be for heads of {pool.head_dim}, its tensors on {pool.device}")
    count, dim = positions.numel(), pool.head_dim
    at, ld, heads, to, ldo = None, 0, 0, None, 0
    if q is not None:
        at, ld, heads = _head_rows(pool._index, "q", q, count, dim)
        q_out, to, ldo = _heads_out(pool._index, "q_out", q_out, q, count, heads, dim)
    elif q_out is not None:
        raise ValueError("q_out without q")
    _check(_lib.qg_kv_append_rope(pool._ref, layer, *_table(pool, table), rotary._ref, heads, at, ld,
                                  *_rows16(pool, "k", k, count), *_rows16(pool, "v", v, count),
                                  None if seqs is None else _ints(pool, "seqs", seqs, count),
                                  _ints(pool, "positions", positions), count, to, ldo, _stream_now(pool._index)),
           "qg_kv_append_rope")
    return q_out


def dequantize(fmt, w, n: int, k: int, values: bool = True, codes: bool = True, stream=None):
    """Decode the device layout on the device: (W_hat fp32 [n, k] or None, codes uint8 [n, k] or None)."""
    torch = _torch()
    wv = torch.empty((n, k), dtype=torch.float32, device=w.device) if values else None
    cv = torch.empty((n, k), dtype=torch.uint8, device=w.device) if codes else None
    _check(_lib.qg_dequantize(_fmt(fmt), w.data_ptr(), wv.data_ptr() if values else None,
                              cv.data_ptr() if codes else None, n, k, _stream(stream)), "qg_dequantize")
    return wv, cv


def read_probe(buf, nbytes: int, sink, stream=None) -> None:
    """Stream nbytes of a device buffer through non-temporal 128-bit loads (read-ceiling measurement)."""
    _check(_lib.qg_read_probe(buf.data_ptr(), nbytes, sink.data_ptr(), _stream(stream)), "qg_read_probe")

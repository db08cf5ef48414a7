"""Python binding of libkvc.so, the B200 KV-cache codec (C ABI in include/kvc.h).

Argument marshalling only: every step of encoding and decoding runs in the
library's CUDA kernels. PyTorch supplies device memory and streams. There is no
CPU fallback: importing this package fails loudly when libkvc.so is missing.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# KVC_BUILD_VARIANT=<name> loads the in-tree test build libkvc_<name>.so (see
# build.VARIANTS) instead of libkvc.so; a missing library fails the import.
_VARIANT = os.environ.get("KVC_BUILD_VARIANT", "")
if _VARIANT and not _VARIANT.isidentifier():
    raise ImportError(f"bad KVC_BUILD_VARIANT {_VARIANT!r}")
LIB_PATH = os.path.join(_HERE, f"libkvc_{_VARIANT}.so" if _VARIANT else "libkvc.so")

OK, ERR_INVALID, ERR_CAPACITY, ERR_CORRUPT, ERR_TRUNCATED, ERR_PLAN_MISMATCH = 0, 1, 2, 3, 4, 5
ERR_TIMEOUT, ERR_CUDA, ERR_UNSUPPORTED = 6, 7, 8
BF16, FP16, F32 = 1, 2, 3  # value types (f32: lossless only)
DTYPE_F32 = F32
LOSSLESS, TRANSFORM = 0, 1
ABI_VERSION = 2
CACHE_E4M3, CACHE_INT8, CACHE_E2M1 = 1, 2, 3  # formats of the quantised serving cache
RANGES_BLOCK, RANGES_KIVI = 0, 1  # transform value ranges: per block, or KIVI-style per-token values

EXPORTS = [
    "kvc_plan", "kvc_plan_create", "kvc_plan_destroy", "kvc_plan_widths", "kvc_plan_crc",
    "kvc_max_encoded_bytes", "kvc_workspace_bytes",
    "kvc_encode_lossless", "kvc_decode_lossless", "kvc_encode_transform", "kvc_decode_transform",
    "kvc_status_string", "kvc_calibrate_pca", "kvc_allocate_bits",
    "kvc_fixed_basis", "kvc_calibrate_basis",
    "kvc_stage_crc32", "kvc_stage_stream_encode", "kvc_stage_stream_decode",
    "kvc_stage_stream_encode_noalloc",
    "kvc_profile_begin", "kvc_profile_end",
    "kvc_batch_workspace_bytes", "kvc_encode_batch", "kvc_decode_batch",
    "kvc_stream_buffer_bytes", "kvc_stream_encode_host", "kvc_stream_decode_host",
    "kvc_cache_bytes", "kvc_cache_write", "kvc_cache_read",
    "kvc_attend_workspace_bytes", "kvc_attend_workspace_min", "kvc_attend",
]


class KvcError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})" if what else status_string(status))


class PlanDesc(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_uint32), ("dtype", ctypes.c_uint32),
        ("n_layers", ctypes.c_uint32), ("n_heads", ctypes.c_uint32),
        ("n_tokens", ctypes.c_uint32), ("head_dim", ctypes.c_uint32),
        ("values_per_chunk", ctypes.c_uint32),
        ("n_sink", ctypes.c_uint32), ("n_recent", ctypes.c_uint32),
        ("block_tokens", ctypes.c_uint32), ("chunk_tokens", ctypes.c_uint32),
        ("max_bits", ctypes.c_uint32),
        ("rope_theta", ctypes.c_double), ("avg_bits", ctypes.c_double),
        ("bases", ctypes.c_void_p), ("eigvals", ctypes.c_void_p), ("widths", ctypes.c_void_p),
        ("range_mode", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
    ]


class Frame(ctypes.Structure):
    _fields_ = [("first_slice", ctypes.c_uint32), ("n_slices", ctypes.c_uint32),
                ("src", ctypes.c_void_p), ("src_bytes", ctypes.c_size_t),
                ("dst", ctypes.c_void_p), ("dst_cap", ctypes.c_size_t),
                ("res", ctypes.c_void_p)]


class CacheDesc(ctypes.Structure):
    _fields_ = [("format", ctypes.c_uint32), ("n_heads", ctypes.c_uint32), ("head_dim", ctypes.c_uint32),
                ("page_tokens", ctypes.c_uint32), ("n_pages", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("micro", ctypes.c_void_p)]


class AttendDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in ("dtype", "n_rows", "n_q_heads", "n_heads", "head_dim", "n_seqs",
                                               "max_queries", "max_kv")] + [
        ("scale", ctypes.c_float), ("prefix_tokens", ctypes.c_uint32),
        ("q", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
        ("lse", ctypes.c_void_p), ("q_start", ctypes.c_void_p), ("cache", ctypes.POINTER(CacheDesc)),
        ("pages", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("pages_stride", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
        ("prefix_k", ctypes.c_void_p), ("prefix_v", ctypes.c_void_p), ("prefix_head_stride", ctypes.c_int64),
        ("prefix_len", ctypes.c_void_p),
    ]


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 40), ("launches", ctypes.c_uint32),
                ("total_ms", ctypes.c_double)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with transform_codec_b200.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, u32, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32, ctypes.c_int
    i64, cache = ctypes.c_int64, ctypes.POINTER(CacheDesc)
    attend, psz = ctypes.POINTER(AttendDesc), ctypes.POINTER(ctypes.c_size_t)
    sig = {
        "kvc_plan": ([ctypes.POINTER(PlanDesc), ctypes.POINTER(vp)], i32),
        "kvc_plan_create": ([ctypes.POINTER(PlanDesc), ctypes.POINTER(vp)], i32),
        "kvc_plan_destroy": ([vp], None),
        "kvc_plan_widths": ([vp, vp, sz], i32),
        "kvc_plan_crc": ([vp], u32),
        "kvc_max_encoded_bytes": ([vp, i32, u32], sz),
        "kvc_workspace_bytes": ([vp, i32, i32, u32], sz),
        "kvc_encode_lossless": ([vp, u32, u32, vp, vp, sz, vp, sz, vp, vp], i32),
        "kvc_decode_lossless": ([vp, vp, sz, vp, sz, vp, sz, vp, vp], i32),
        "kvc_encode_transform": ([vp, u32, u32, vp, vp, sz, vp, sz, vp, vp], i32),
        "kvc_decode_transform": ([vp, vp, sz, vp, sz, vp, sz, vp, vp], i32),
        "kvc_status_string": ([i32], ctypes.c_char_p),
        "kvc_calibrate_pca": ([ctypes.POINTER(PlanDesc), vp, u32, vp, vp, i32], i32),
        "kvc_allocate_bits": ([vp, ctypes.c_uint64, ctypes.c_double, u32, vp], i32),
        "kvc_fixed_basis": ([i32, u32, vp], i32),
        "kvc_calibrate_basis": ([ctypes.POINTER(PlanDesc), i32, vp, u32, vp, vp, i32], i32),
        "kvc_batch_workspace_bytes": ([vp, i32, i32, u32, u32], sz),
        "kvc_encode_batch": ([vp, i32, ctypes.POINTER(Frame), u32, vp, sz, vp], i32),
        "kvc_decode_batch": ([vp, i32, ctypes.POINTER(Frame), u32, u32, vp, sz, vp], i32),
        "kvc_stream_buffer_bytes": ([vp, i32, u32], sz),
        "kvc_stream_encode_host": ([vp, i32, u32, u32, u32, vp, vp, sz, vp, vp, vp, sz, vp], i32),
        "kvc_stream_decode_host": ([vp, i32, u32, u32, vp, vp, vp, sz, vp, vp, sz, vp], i32),
        "kvc_cache_bytes": ([cache, psz, psz, psz], i32),
        "kvc_cache_write": ([cache, u32, u32, vp, i64, i64, vp, i64, i64, vp, vp, vp], i32),
        "kvc_cache_read": ([cache, u32, u32, vp, u32, vp, vp, vp, u32, vp, vp], i32),
        "kvc_attend_workspace_bytes": ([attend], sz),
        "kvc_attend_workspace_min": ([attend], sz),
        "kvc_attend": ([attend, vp, sz, vp, vp], i32),
        "kvc_profile_begin": ([], i32),
        "kvc_profile_end": ([ctypes.POINTER(KernelTime), i32, ctypes.POINTER(i32)], i32),
        "kvc_stage_crc32": ([vp, sz, vp, vp], i32),
        "kvc_stage_stream_encode": ([vp, u32, vp, vp, vp, vp], i32),
        "kvc_stage_stream_decode": ([vp, u32, u32, vp, vp, vp], i32),
        "kvc_stage_stream_encode_noalloc": ([vp, u32, vp, vp, vp], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def lib():
    return _lib


def status_string(status: int) -> str:
    return _lib.kvc_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != OK:
        raise KvcError(status, what)


def _np_ptr(a):
    return None if a is None else a.ctypes.data


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


@dataclass
class Shape:
    dtype: int
    n_layers: int
    n_heads: int
    n_tokens: int
    head_dim: int
    values_per_chunk: int = 65536
    n_sink: int = 4
    n_recent: int = 128
    block_tokens: int = 64
    chunk_tokens: int = 512
    max_bits: int = 8
    rope_theta: float = 1e4
    avg_bits: float = 2.0
    range_mode: int = 0  # RANGES_BLOCK or RANGES_KIVI

    @property
    def n_slices(self) -> int:
        return self.n_layers * 2 * self.n_heads

    @classmethod
    def from_workload(cls, w) -> "Shape":
        return cls(w.dtype, w.n_layers, w.n_heads, w.n_tokens, w.head_dim, w.values_per_chunk,
                   w.n_sink, w.n_recent, w.block_tokens, w.chunk_tokens, w.max_bits, w.theta,
                   w.avg_bits)

    def desc(self, bases=None, eigvals=None, widths=None) -> PlanDesc:
        return PlanDesc(ABI_VERSION, self.dtype, self.n_layers, self.n_heads, self.n_tokens,
                        self.head_dim, self.values_per_chunk, self.n_sink, self.n_recent,
                        self.block_tokens, self.chunk_tokens, self.max_bits, self.rope_theta,
                        self.avg_bits, _np_ptr(bases), _np_ptr(eigvals), _np_ptr(widths), self.range_mode, 0)


class Plan:
    """A kvc plan on the current CUDA device. Lossless-only when bases is None."""

    def __init__(self, shape: Shape, bases=None, eigvals=None, widths=None):
        self.shape = shape
        b = None if bases is None else np.ascontiguousarray(bases, dtype=np.float32)
        e = None if eigvals is None else np.ascontiguousarray(eigvals, dtype=np.float64)
        w = None if widths is None else np.ascontiguousarray(widths, dtype=np.uint8)
        desc = shape.desc(b, e, w)
        h = ctypes.c_void_p()
        _check(_lib.kvc_plan(ctypes.byref(desc), ctypes.byref(h)), "kvc_plan")
        self._h = h
        # Held by the object: at interpreter exit the module's globals may be
        # cleared before the last plan is collected.
        self._destroy = _lib.kvc_plan_destroy
        self.has_transform = b is not None

    def __del__(self):
        h = getattr(self, "_h", None)
        destroy = getattr(self, "_destroy", None)
        if h is not None and h.value and destroy is not None:
            destroy(h)
            self._h = None

    @property
    def handle(self):
        return self._h

    @property
    def crc(self) -> int:
        return _lib.kvc_plan_crc(self._h)

    def widths(self) -> np.ndarray:
        s = self.shape
        out = np.zeros((s.n_slices, s.head_dim), np.uint8)
        _check(_lib.kvc_plan_widths(self._h, out.ctypes.data, out.size), "kvc_plan_widths")
        return out

    def max_encoded_bytes(self, path: int, n_slices: int) -> int:
        return _lib.kvc_max_encoded_bytes(self._h, path, n_slices)

    def workspace_bytes(self, path: int, decode: bool, n_slices: int) -> int:
        return _lib.kvc_workspace_bytes(self._h, path, int(decode), n_slices)


class Codec:
    """Owns output, workspace and result buffers for repeated calls of one size."""

    def __init__(self, plan: Plan, path: int, n_slices: int, device=None):
        import torch
        self.plan, self.path, self.n_slices = plan, path, n_slices
        dev = torch.device("cuda") if device is None else device
        s = plan.shape
        self.cap = plan.max_encoded_bytes(path, n_slices)
        self.out_elems = n_slices * s.n_tokens * s.head_dim
        vt = torch.int32 if s.dtype == DTYPE_F32 else torch.int16  # one element per value
        self.container = torch.empty(max(self.cap, 16), dtype=torch.uint8, device=dev)
        self.ws_enc = torch.empty(max(plan.workspace_bytes(path, False, n_slices), 256),
                                  dtype=torch.uint8, device=dev)
        self.ws_dec = torch.empty(max(plan.workspace_bytes(path, True, n_slices), 256),
                                  dtype=torch.uint8, device=dev)
        self.res = torch.zeros(4, dtype=torch.int64, device=dev)  # kvc_result (16 bytes) x 2
        self.decoded = torch.empty(max(self.out_elems, 8), dtype=vt, device=dev)

    def encode(self, src, first_slice: int = 0, stream=None, res=None):
        fn = _lib.kvc_encode_lossless if self.path == LOSSLESS else _lib.kvc_encode_transform
        r = self.res[0:2] if res is None else res
        st = fn(self.plan.handle, first_slice, self.n_slices, _dptr(src), _dptr(self.container),
                self.container.numel(), _dptr(self.ws_enc), self.ws_enc.numel(), _dptr(r),
                _stream(stream))
        _check(st, "encode")
        return r

    def decode(self, container, nbytes: int, out=None, stream=None, res=None):
        fn = _lib.kvc_decode_lossless if self.path == LOSSLESS else _lib.kvc_decode_transform
        r = self.res[2:4] if res is None else res
        dst = self.decoded if out is None else out
        cap = dst.numel() * dst.element_size()
        st = fn(self.plan.handle, _dptr(container), nbytes, _dptr(dst), cap, _dptr(self.ws_dec),
                self.ws_dec.numel(), _dptr(r), _stream(stream))
        _check(st, "decode")
        return r


def batch_workspace_bytes(plan: Plan, path: int, decode: bool, n_frames: int,
                          max_slices_per_frame: int) -> int:
    return _lib.kvc_batch_workspace_bytes(plan.handle, path, int(decode), n_frames,
                                          max_slices_per_frame)


def _frames(items):
    arr = (Frame * max(len(items), 1))()
    for i, it in enumerate(items):
        arr[i] = Frame(*it)
    return arr


def encode_batch(plan: Plan, path: int, frames, ws, stream=None):
    """frames: sequence of (first_slice, n_slices, src_tensor, dst_tensor, res_tensor)."""
    items = [(fs, ns, src.data_ptr() if src is not None and src.numel() else None, 0,
              dst.data_ptr(), dst.numel() * dst.element_size(), res.data_ptr())
             for fs, ns, src, dst, res in frames]
    _check(_lib.kvc_encode_batch(plan.handle, path, _frames(items), len(items), _dptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream)),
           "kvc_encode_batch")


def decode_batch(plan: Plan, path: int, frames, ws, max_slices_per_frame: int = 0, stream=None):
    """frames: sequence of (src_tensor, src_bytes, dst_tensor, res_tensor)."""
    items = [(0, 0, src.data_ptr(), nbytes, dst.data_ptr(), dst.numel() * dst.element_size(),
              res.data_ptr()) for src, nbytes, dst, res in frames]
    _check(_lib.kvc_decode_batch(plan.handle, path, _frames(items), len(items),
                                 max_slices_per_frame, _dptr(ws), ws.numel() * ws.element_size(),
                                 _stream(stream)), "kvc_decode_batch")


def stream_buffer_bytes(plan: Plan, path: int, frame_slices: int) -> int:
    return _lib.kvc_stream_buffer_bytes(plan.handle, path, frame_slices)


def _nbytes(t):
    return t.numel() * t.element_size()


def stream_encode_host(plan: Plan, path: int, first_slice: int, n_slices: int, frame_slices: int,
                       h_src, h_dst, h_frame_bytes, h_results, d_buf, stream=None):
    """kvc_stream_encode_host (blocking): h_src / h_dst host tensors (pinned for
    overlap), h_frame_bytes host int64 [n_frames], h_results host int64
    [n_frames, 2] (kvc_result), d_buf device uint8 of stream_buffer_bytes."""
    _check(_lib.kvc_stream_encode_host(plan.handle, path, first_slice, n_slices, frame_slices, _dptr(h_src),
                                       _dptr(h_dst), _nbytes(h_dst), _dptr(h_frame_bytes), _dptr(h_results),
                                       _dptr(d_buf), _nbytes(d_buf), _stream(stream)), "kvc_stream_encode_host")


def stream_decode_host(plan: Plan, path: int, n_slices: int, frame_slices: int, h_src, h_frame_bytes, h_dst,
                       h_results, d_buf, stream=None):
    """kvc_stream_decode_host (blocking); arguments as for stream_encode_host."""
    _check(_lib.kvc_stream_decode_host(plan.handle, path, n_slices, frame_slices, _dptr(h_src),
                                       _dptr(h_frame_bytes), _dptr(h_dst), _nbytes(h_dst), _dptr(h_results),
                                       _dptr(d_buf), _nbytes(d_buf), _stream(stream)), "kvc_stream_decode_host")


def read_result(res) -> tuple[int, int]:
    """(status, bytes) from a device kvc_result (synchronises with its stream)."""
    v = res.cpu().numpy()
    return int(v[0] & 0xFFFFFFFF), int(v[1])


def calibrate_pca(shape: Shape, calib: np.ndarray, n_threads: int = 0):
    """Host PCA per slice: bases [S][D][D] fp32 and eigenvalues [S][D]."""
    c = np.ascontiguousarray(calib, dtype=np.uint16)
    S, n_calib, D = c.shape
    bases = np.zeros((S, D, D), np.float32)
    lam = np.zeros((S, D), np.float64)
    desc = shape.desc()
    _check(_lib.kvc_calibrate_pca(ctypes.byref(desc), c.ctypes.data, n_calib, bases.ctypes.data,
                                  lam.ctypes.data, n_threads), "kvc_calibrate_pca")
    return bases, lam


BASIS_PCA, BASIS_HADAMARD, BASIS_DCT = 0, 1, 2


def fixed_basis(kind: int, D: int) -> np.ndarray:
    """Calibration-free basis [D][D] fp32 (Hadamard or DCT-II)."""
    q = np.zeros((D, D), np.float32)
    _check(_lib.kvc_fixed_basis(kind, D, q.ctypes.data), "kvc_fixed_basis")
    return q


def calibrate_basis(shape: Shape, kind: int, calib: np.ndarray, n_threads: int = 0):
    """Bases [S][D][D] and component variances [S][D] for a basis kind."""
    c = np.ascontiguousarray(calib, dtype=np.uint16)
    S, n_calib, D = c.shape
    bases = np.zeros((S, D, D), np.float32)
    lam = np.zeros((S, D), np.float64)
    desc = shape.desc()
    _check(_lib.kvc_calibrate_basis(ctypes.byref(desc), kind, c.ctypes.data, n_calib, bases.ctypes.data,
                                    lam.ctypes.data, n_threads), "kvc_calibrate_basis")
    return bases, lam


def allocate_bits(eigvals: np.ndarray, avg_bits: float, max_bits: int = 8) -> np.ndarray:
    lam = np.ascontiguousarray(eigvals, dtype=np.float64).ravel()
    w = np.zeros(lam.size, np.uint8)
    _check(_lib.kvc_allocate_bits(lam.ctypes.data, lam.size, avg_bits, max_bits, w.ctypes.data),
           "kvc_allocate_bits")
    return w


def profile_begin():
    _check(_lib.kvc_profile_begin(), "kvc_profile_begin")


def profile_end() -> dict:
    """{kernel name: (launches, total ms)} for the launches since profile_begin()."""
    arr = (KernelTime * 64)()
    n = ctypes.c_int(0)
    _check(_lib.kvc_profile_end(arr, 64, ctypes.byref(n)), "kvc_profile_end")
    return {arr[i].name.decode(): (int(arr[i].launches), float(arr[i].total_ms))
            for i in range(n.value)}


# ---- serving cache
#
# A decoding step makes a handful of these calls, each a few microseconds on the
# GPU when the batch is small, so the checks below stay cheap: plain comparisons,
# the stream as a number, and no objects made that need not be.

_torch = None
_TORCH_DTYPES: dict = {}
_raw_stream = None


def _use_torch():
    """torch, imported by the first call that needs it."""
    global _torch, _raw_stream
    if _torch is None:
        import torch
        _TORCH_DTYPES.update({torch.bfloat16: BF16, torch.float16: FP16, torch.float32: F32})
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _torch = torch
    return _torch


def _value_type(dtype) -> int:
    """BF16, FP16 or F32 of a torch dtype; KvcError (ERR_INVALID) for another."""
    _use_torch()
    dt = _TORCH_DTYPES.get(dtype)
    if dt is None:
        raise KvcError(ERR_INVALID, f"value type {dtype}")
    return dt


def _refuse(what: str):
    raise KvcError(ERR_INVALID, what)


def _require(ok: bool, what: str):
    if not ok:
        _refuse(what)


def _on(t, device, what: str, dtype):
    """t must be a tensor of that device and type."""
    if t.device != device or t.dtype != dtype:
        _refuse(f"{what}: {t.dtype} on {t.device}, not {dtype} on {device}")


def _result(res, device) -> int:
    """The address of a caller's kvc_result: 16 bytes on the tensors' device."""
    if res.device != device or res.numel() * res.element_size() < 16 or not res.is_contiguous():
        _refuse(f"res: {tuple(res.shape)} {res.dtype} on {res.device}")
    return res.data_ptr()


def _launch(device, stream, what: str, fn, *args):
    """fn(*args, stream) with the tensors' device current, on its current stream if none is given."""
    torch = _use_torch()
    if device.type != "cuda":
        _refuse(f"tensors on {device}")
    raw = _raw_stream(device.index) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == device.index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status != OK:
        raise KvcError(status, what)


class QuantCache:
    """A paged, quantised serving cache of one layer (kvc.h, "Serving cache").

    Owns the arrays codes, scales and micro (E2M1 only), or takes given ones:
    codes uint8 [n_pages, 2, n_heads, page_tokens, head_dim or head_dim / 2],
    scales fp32 [n_pages, 2, n_heads, page_tokens], micro uint8 [..., head_dim /
    16]. res is the sticky kvc_result of the calls on this cache that are not
    given one: ERR_INVALID once a slot, page or length was out of range."""

    def __init__(self, fmt: int, n_heads: int, head_dim: int, page_tokens: int, n_pages: int, device=None,
                 codes=None, scales=None, micro=None):
        torch = _use_torch()
        self.format, self.n_heads, self.head_dim = fmt, n_heads, head_dim
        self.page_tokens, self.n_pages = page_tokens, n_pages
        for v in (fmt, n_heads, head_dim, page_tokens, n_pages):
            _require(isinstance(v, int) and 0 < v < 1 << 31, "cache shape")
        self._desc = CacheDesc(fmt, n_heads, head_dim, page_tokens, n_pages, 0, None, None, None)
        _check(_lib.kvc_cache_bytes(ctypes.byref(self._desc), None, None, None), "kvc_cache_bytes")
        rows = (n_pages, 2, n_heads, page_tokens)
        dev = torch.device("cuda") if device is None else torch.device(device)
        if codes is not None:
            dev = codes.device
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        four = fmt == CACHE_E2M1

        def array(t, what, dtype, *last):
            if t is None:
                return torch.zeros(rows + last, dtype=dtype, device=dev)
            _on(t, dev, what, dtype)
            _require(tuple(t.shape) == rows + last and t.is_contiguous(), f"{what} of shape {tuple(t.shape)}")
            return t

        self.codes = array(codes, "codes", torch.uint8, head_dim // 2 if four else head_dim)
        self.scales = array(scales, "scales", torch.float32)
        _require(four or micro is None, "micro-scales of an 8-bit format")
        self.micro = array(micro, "micro", torch.uint8, head_dim // 16) if four else None
        self.res = torch.zeros(2, dtype=torch.int64, device=dev)
        self._desc.codes, self._desc.scales = self.codes.data_ptr(), self.scales.data_ptr()
        self._desc.micro = self.micro.data_ptr() if four else None
        self.ref = ctypes.byref(self._desc)
        self._pointer = ctypes.pointer(self._desc)
        self._res = self.res.data_ptr()


def cache_write(cache: QuantCache, k, v, slots, res=None, stream=None):
    """kvc_cache_write: quantise tokens k, v [n, n_heads, head_dim] (bf16, fp16
    or f32; token and head strides free in 16-byte steps, so [head][token]
    slices go in as slices.transpose(0, 1)) into slots, int64 [n] = page *
    page_tokens + token in page, negative: skipped. Each slot at most once a call."""
    torch = _torch or _use_torch()
    if slots.dim() != 1:
        _refuse(f"slots {tuple(slots.shape)}")
    shape = (slots.shape[0], cache.n_heads, cache.head_dim)
    device, dtype = cache.device, k.dtype
    if k.shape != shape or v.shape != shape:
        _refuse(f"k {tuple(k.shape)}, v {tuple(v.shape)} for {shape}")
    _on(k, device, "k", dtype)
    _on(v, device, "v", dtype)
    _on(slots, device, "slots", torch.int64)
    kt, kh, kc = k.stride()
    vt, vh, vc = v.stride()
    if kc != 1 or vc != 1 or not slots.is_contiguous():
        _refuse("channels and slots are contiguous")
    _launch(device, stream, "kvc_cache_write", _lib.kvc_cache_write, cache.ref, _value_type(dtype), shape[0],
            k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, slots.data_ptr(),
            cache._res if res is None else _result(res, device))


def cache_read(cache: QuantCache, page_table, start, out_start, out, res=None, stream=None):
    """kvc_cache_read: tokens [start[b], start[b] + n_b) of each sequence into
    out [2, n_heads, out_tokens, head_dim] (bf16, fp16 or f32, contiguous: with one
    sequence the slices the codec takes) at out_start[b] .. out_start[b + 1].
    page_table int32 [n_seqs, pages], start int32 [n_seqs], out_start int32
    [n_seqs + 1]; tokens of out outside the ranges are left as they are."""
    torch = _torch or _use_torch()
    device, int32 = cache.device, torch.int32
    _on(page_table, device, "page_table", int32)
    _on(start, device, "start", int32)
    _on(out_start, device, "out_start", int32)
    _on(out, device, "out", out.dtype)
    n = start.numel()
    if page_table.dim() != 2 or page_table.shape[0] != n or out_start.shape != (n + 1,) or start.dim() != 1:
        _refuse("page_table [n], start [n] and out_start [n + 1]")
    if out.dim() != 4 or out.shape[0] != 2 or out.shape[1] != cache.n_heads or out.shape[3] != cache.head_dim:
        _refuse(f"out of shape {tuple(out.shape)}")
    if not (page_table.is_contiguous() and start.is_contiguous() and out_start.is_contiguous()
            and out.is_contiguous()):
        _refuse("contiguous tensors")
    _launch(device, stream, "kvc_cache_read", _lib.kvc_cache_read, cache.ref, _value_type(out.dtype), n,
            page_table.data_ptr(), page_table.shape[1], start.data_ptr(), out_start.data_ptr(), out.data_ptr(),
            out.shape[2], cache._res if res is None else _result(res, device))


class Attention:
    """kvc_attend for batches up to a size: owns the workspace (one call at a
    time) and a sticky kvc_result, res, for calls without one.

    dtype (torch.bfloat16 or torch.float16) is that of q, out and the prefix;
    max_rows query tokens in all, max_seqs sequences, max_queries and max_kv the
    expected most of one sequence (max_kv 0: not known), prefix_tokens the
    longest shared prefix. Runs may be smaller; larger ones are refused with
    ERR_CAPACITY where the workspace does not do. At most 65,535 sequences and
    query heads, and fewer than 2^31 rows times query heads."""

    def __init__(self, dtype, n_q_heads: int, n_heads: int, head_dim: int, max_rows: int, max_seqs: int,
                 max_queries: int = 1, max_kv: int = 0, prefix_tokens: int = 0, device=None):
        torch = _use_torch()
        dev = torch.device("cuda") if device is None else torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device, self.dtype = dev, dtype
        # before they become 32-bit fields; the sizing call answers 0 for what it refuses
        for v, what in ((n_heads, "n_heads"), (n_q_heads, "n_q_heads"), (head_dim, "head_dim"), (max_rows, "max_rows"),
                        (max_seqs, "max_seqs"), (max_queries, "max_queries"), (max_kv, "max_kv"),
                        (prefix_tokens, "prefix_tokens")):
            _require(isinstance(v, int) and 0 <= v < 1 << 31, f"{what} {v}")
        _require(n_q_heads <= 65535 and max_seqs <= 65535 and max_rows * n_q_heads < 1 << 31,
                 f"{n_q_heads} query heads, {max_seqs} sequences, {max_rows} rows")
        d = self._desc = AttendDesc()
        d.dtype, d.n_q_heads, d.n_heads, d.head_dim = _value_type(dtype), n_q_heads, n_heads, head_dim
        d.n_rows, d.n_seqs, d.max_queries, d.max_kv = max_rows, max_seqs, max_queries, max_kv
        d.prefix_tokens, d.scale = prefix_tokens, 1.0
        # any format and page size: the workspace does not depend on them
        shape = CacheDesc(CACHE_E4M3, n_heads, head_dim, 16, 1, 0, None, None, None)
        d.cache = ctypes.pointer(shape)
        self._probe(d)
        self.workspace = torch.empty(max(_lib.kvc_attend_workspace_bytes(ctypes.byref(d)), 16), dtype=torch.uint8,
                                     device=dev)
        self.res = torch.zeros(2, dtype=torch.int64, device=dev)
        self._res = self.res.data_ptr()
        self._ws, self._ws_bytes = self.workspace.data_ptr(), self.workspace.numel()
        self._ref = ctypes.byref(d)

    @staticmethod
    def _probe(d):
        """The status of a bad description: the sizing calls answer 0 for one."""
        _require(d.n_heads > 0 and d.n_q_heads > 0 and d.n_q_heads % d.n_heads == 0, "query heads for each head")
        if d.head_dim not in (64, 128):
            raise KvcError(ERR_UNSUPPORTED, f"head_dim {d.head_dim}")
        _require(d.dtype in (BF16, FP16), "attention value type")

    def run(self, q, out, cache: QuantCache | None = None, page_table=None, kv_len=None, q_start=None, prefix=None,
            prefix_len=None, lse=None, scale: float | None = None, res=None, stream=None):
        """q, out [n, n_q_heads, head_dim] (token and head strides free in 16-byte
        steps); cache with page_table int32 [n_seqs, pages] and kv_len int32
        [n_seqs]; q_start int32 [n_seqs + 1] (None: one query a sequence); prefix
        (k, v), each [n_heads, tokens, head_dim], tokens contiguous, v finite up to
        the longest share and below 2^80 in magnitude (kvc.h); prefix_len
        int32 [n_seqs] (None: all of it); lse fp32 [n, n_q_heads]; scale defaults
        to head_dim ** -0.5."""
        torch = _torch
        d, dev, int32 = self._desc, self.device, torch.int32
        shape = q.shape
        if len(shape) != 3:
            _refuse(f"q {tuple(shape)}")
        n, heads, dim = shape
        _on(q, dev, "q", self.dtype)
        _on(out, dev, "out", self.dtype)
        if heads != d.n_q_heads or dim != d.head_dim or out.shape != shape:
            _refuse(f"q {tuple(shape)}")
        qt, qh, qc = q.stride()
        ot, oh, oc = out.stride()
        if qc != 1 or oc != 1:
            _refuse("channels are contiguous")
        seqs = -1
        if q_start is not None:
            seqs = self._sequences(q_start, "q_start", 1, seqs)
        if kv_len is not None:
            seqs = self._sequences(kv_len, "kv_len", 0, seqs)
        if prefix_len is not None:
            seqs = self._sequences(prefix_len, "prefix_len", 0, seqs)
        if seqs < 0:
            seqs = n
        if q_start is None and n < seqs:
            _refuse("a row for each sequence")
        d.n_rows, d.n_seqs = n, seqs
        d.q, d.q_token_stride, d.q_head_stride = q.data_ptr(), qt, qh
        d.out, d.out_token_stride, d.out_head_stride = out.data_ptr(), ot, oh
        d.q_start = None if q_start is None else q_start.data_ptr()
        d.prefix_len = None if prefix_len is None else prefix_len.data_ptr()
        d.scale = dim ** -0.5 if scale is None else scale
        if lse is None:
            d.lse = None
        else:
            _on(lse, dev, "lse", torch.float32)
            if lse.shape != (n, heads) or not lse.is_contiguous():
                _refuse(f"lse {tuple(lse.shape)}")
            d.lse = lse.data_ptr()
        if cache is None:
            d.cache, d.pages, d.kv_len = None, None, None
        else:
            if cache.device != dev or page_table is None or kv_len is None:
                _refuse("cache")
            _on(page_table, dev, "page_table", int32)
            if page_table.dim() != 2 or page_table.shape[0] != seqs or not page_table.is_contiguous():
                _refuse("page_table")
            d.cache = cache._pointer
            d.pages, d.pages_stride, d.kv_len = page_table.data_ptr(), page_table.shape[1], kv_len.data_ptr()
        if prefix is None:
            d.prefix_tokens = 0
        else:
            pk, pv = prefix
            _on(pk, dev, "prefix keys", self.dtype)
            _on(pv, dev, "prefix values", self.dtype)
            st = pk.stride()
            if (pk.dim() != 3 or pk.shape[0] != d.n_heads or pk.shape[2] != dim or pv.shape != pk.shape
                    or st[1:] != (dim, 1) or pv.stride() != st):
                _refuse(f"prefix {tuple(pk.shape)}")
            d.prefix_tokens, d.prefix_head_stride = pk.shape[1], st[0]
            d.prefix_k, d.prefix_v = pk.data_ptr(), pv.data_ptr()
        _launch(dev, stream, "kvc_attend", _lib.kvc_attend, self._ref, self._ws, self._ws_bytes,
                self._res if res is None else _result(res, dev))

    def _sequences(self, t, what, extra, seqs):
        """The number of sequences that t speaks of, the same as what was said before (-1: nothing yet)."""
        _on(t, self.device, what, _torch.int32)
        m = t.shape[0] - extra if t.dim() == 1 else -1
        if m < 0 or (seqs >= 0 and seqs != m) or not t.is_contiguous():
            _refuse(f"{what} {tuple(t.shape)}")
        return m


def stage_crc32(src, n: int, out, stream=None):
    _check(_lib.kvc_stage_crc32(_dptr(src), n, _dptr(out), _stream(stream)), "kvc_stage_crc32")


def stage_stream_encode(sym, n: int, out, scratch, res, stream=None):
    _check(_lib.kvc_stage_stream_encode(_dptr(sym), n, _dptr(out), _dptr(scratch), _dptr(res),
                                        _stream(stream)), "kvc_stage_stream_encode")


def stage_stream_encode_noalloc(sym, n: int, out, res, stream=None):
    """kvc_stage_stream_encode with the library's own fixed scratch (n <= 65536);
    allocates nothing. Overlapping calls on one device share that scratch."""
    _check(_lib.kvc_stage_stream_encode_noalloc(_dptr(sym), n, _dptr(out), _dptr(res),
                                                _stream(stream)), "kvc_stage_stream_encode_noalloc")


def stage_stream_decode(rec, rec_bytes: int, n: int, sym, res, stream=None):
    _check(_lib.kvc_stage_stream_decode(_dptr(rec), rec_bytes, n, _dptr(sym), _dptr(res),
                                        _stream(stream)), "kvc_stage_stream_decode")

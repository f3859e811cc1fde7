"""Fully-integer attention forward (IntAttention, arXiv 2511.21513) on B200.

Python binding of the C ABI in ``include/intattn.h``: argument marshalling
only.  Every step of the computation runs in the CUDA kernels of
``libintattn.so``; torch supplies device memory and streams.  There is no CPU
fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import os
from typing import Optional, Sequence, Union

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libintattn.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_PARAM_RANGE, ERR_CUDA, ERR_WORKSPACE, ERR_TIMEOUT = range(7)
MAX_HEADS = 128
MAX_CLIPS = 8

# every function declared in include/intattn.h
EXPORTED = ("intattn_derive_params", "intattn_forward", "intattn_forward_variant",
            "intattn_forward_host_workspace_size", "intattn_forward_fp_workspace_size", "intattn_forward_fp",
            "intattn_forward_fp_zp",
            "intattn_calibrate_workspace_size", "intattn_calibrate_clip",
            "intattn_forward_host", "intattn_decode_workspace_size",
            "intattn_decode", "intattn_decode_int4", "intattn_decode_static_scratch", "intattn_quantize",
            "intattn_quantize_zp", "intattn_qk_norm_rope", "intattn_cache_write", "intattn_cache_read",
            "intattn_decode_shared_workspace_size", "intattn_decode_shared",
            "intattn_gelu_derive_params", "intattn_gelu", "intattn_selftest_timeout", "intattn_device_error",
            "intattn_strerror")
DTYPE_FP16, DTYPE_BF16, DTYPE_INT8 = 0, 1, 2
ZERO_LEFT_OUT = 0x100
VARIANT_AUTO, VARIANT_THREE_PASS, VARIANT_SHORT_ROWS = 0, 1, 2
SHORT_ROWS_MAX_KEYS = 256


class _GeluParams(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("s", ctypes.c_int32), ("Mo", ctypes.c_int32), ("so", ctypes.c_int32),
                ("gate", ctypes.c_int32 * 32)]


class IntAttnError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {strerror(code) if _lib is not None else code} (code {code})")


class _Scales(ctypes.Structure):
    # host arrays: float s_q, s_k, s_v, s_o, clip_c; int32 z_k, z_v
    _fields_ = [("per_head", ctypes.c_int32)] + [(n, ctypes.c_void_p) for n in
                                                 ("s_q", "s_k", "s_v", "s_o", "clip_c", "z_k", "z_v")]


class _HeadParams(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("s", ctypes.c_int32), ("D", ctypes.c_int32),
                ("Mo", ctypes.c_int32), ("so", ctypes.c_int32)]


class _Rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p),
                ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64), ("stride_l", ctypes.c_int64)]


class _RopeNorm(ctypes.Structure):
    _fields_ = [("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("table", ctypes.c_void_p), ("n_positions", ctypes.c_int32), ("rot", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("positions", ctypes.c_void_p)]


FloatArg = Union[float, Sequence[float], np.ndarray]


_F32, _I32 = np.dtype(np.float32), np.dtype(np.int32)


def _host_array(x, dtype) -> np.ndarray:
    """x as a contiguous host array of at least one dimension (x itself where it is one)."""
    if type(x) is np.ndarray and x.dtype is dtype and x.ndim == 1 and x.flags.c_contiguous:
        return x
    if type(x) is float or type(x) is int:
        return np.array((x,), dtype)
    return np.array(x, dtype, ndmin=1, order="C")


def _address(a: np.ndarray) -> int:
    """Address of a's data (through the buffer where it is writable, the fastest way)."""
    try:
        return ctypes.addressof(ctypes.c_char.from_buffer(a))
    except (TypeError, ValueError):  # read-only or empty
        return a.ctypes.data


@dataclasses.dataclass
class Scales:
    """Quantisation scales (real = scale * code).  per_head: arrays of H.
    clip: optional per-head clip thresholds (same layout as the scales);
    None: the call's clip_c applies to every head.
    z_k / z_v: optional zero-points (same layout, 0..255): the K / V codes
    are then uint8 tensors and code c stands for c - z."""
    s_q: FloatArg
    s_k: FloatArg
    s_v: FloatArg
    s_o: FloatArg
    per_head: bool = False
    clip: Optional[FloatArg] = None
    z_k: Optional[FloatArg] = None
    z_v: Optional[FloatArg] = None

    def _c(self, names=("s_q", "s_k", "s_v", "s_o", "clip", "z_k", "z_v")):
        """The call's scale struct (only the named arrays that are given, the others null)
        and those arrays by name, to be kept alive for the duration of the call."""
        s, arrs = _Scales(), {}
        s.per_head = bool(self.per_head)
        for n in names:
            x = getattr(self, n)
            if x is not None:
                a = arrs[n] = _host_array(x, _I32 if n in ("z_k", "z_v") else _F32)
                setattr(s, "clip_c" if n == "clip" else n, _address(a))
        return s, arrs

    def _c_heads(self, n_q: int, n_kv: int, names):
        """_c of the named arrays, which hold an entry per head (n_q query
        heads, n_kv K / V heads), or one each."""
        s, arrs = self._c(names)
        for n, a in arrs.items():
            want = (n_q if n in ("s_q", "s_o", "clip") else n_kv) if self.per_head else 1
            if a.size < want:
                raise ValueError(f"scales.{n} holds {a.size} entries; {want} are needed")
        return s, arrs


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m integer_only_quantized_b200.build` (nvcc, sm_100a)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.intattn_derive_params.argtypes = [ctypes.POINTER(_Scales), i32, i32, f32,
                                            ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(_HeadParams)]
        L.intattn_forward.argtypes = [vp, vp, vp, ctypes.POINTER(_Scales), i32, i32, i32, i32, i32,
                                      i32, f32, vp, vp]
        L.intattn_forward_variant.argtypes = [vp, vp, vp, ctypes.POINTER(_Scales), i32, i32, i32, i32, i32,
                                              i32, f32, vp, i32, vp]
        L.intattn_forward_fp_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.intattn_forward_fp_workspace_size.restype = ctypes.c_size_t
        f32p = ctypes.POINTER(ctypes.c_float)
        L.intattn_forward_fp.argtypes = [vp, vp, vp, i32, i32, f32p, f32p, f32, i32, i32, i32, i32, i32, i32,
                                         vp, vp, vp, ctypes.c_size_t, vp]
        L.intattn_forward_fp_zp.argtypes = [vp, vp, vp, i32, i32, f32p, f32p, f32, i32, i32, i32, i32, i32, i32,
                                            vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.intattn_calibrate_workspace_size.argtypes = [i32, i32]
        L.intattn_calibrate_workspace_size.restype = ctypes.c_size_t
        L.intattn_calibrate_clip.argtypes = [vp, vp, ctypes.POINTER(_Scales), i32, i32, i32, i32, i32, i32, i32,
                                             i32, f32, f32, f32p, ctypes.POINTER(ctypes.c_int32), vp,
                                             ctypes.c_size_t, vp]
        L.intattn_forward_host_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.intattn_forward_host_workspace_size.restype = ctypes.c_size_t
        L.intattn_forward_host.argtypes = [vp, vp, vp, ctypes.POINTER(_Scales), i32, i32, i32, i32, i32,
                                           i32, f32, vp, vp, ctypes.c_size_t, vp]
        L.intattn_decode_workspace_size.argtypes = [i32, i32, i32, i32]
        L.intattn_decode_workspace_size.restype = ctypes.c_size_t
        L.intattn_decode.argtypes = [vp, vp, vp, ctypes.POINTER(_Scales), i32, i32, i32, i32, i32,
                                     f32, vp, vp, ctypes.c_size_t, vp]
        L.intattn_decode_int4.argtypes = [vp, vp, vp, ctypes.POINTER(_Scales), i32, i32, i32, i32, i32,
                                          f32, vp, vp, ctypes.c_size_t, vp]
        L.intattn_decode_static_scratch.argtypes = [vp, vp, vp, ctypes.POINTER(_Scales), i32, i32, i32,
                                                    i32, i32, f32, vp, vp]
        L.intattn_quantize.argtypes = [vp, i32, i32, i32, i32, i32, i32, vp, vp, vp]
        L.intattn_quantize_zp.argtypes = [vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp]
        rows, rn, scp = ctypes.POINTER(_Rows), ctypes.POINTER(_RopeNorm), ctypes.POINTER(_Scales)
        L.intattn_qk_norm_rope.argtypes = [rows, rows, rn, i32, i32, i32, i32, i32, i32, rows, rows, vp]
        L.intattn_cache_write.argtypes = [rows, rows, rows, i32, scp, i32, rn, i32, i32, i32, i32, i32, i32, vp, vp,
                                          vp, vp, vp, vp]
        L.intattn_cache_read.argtypes = [vp, vp, scp, i32, i32, i32, i32, i32, i32, vp, vp, i32, vp, vp, vp]
        L.intattn_decode_shared_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.intattn_decode_shared_workspace_size.restype = ctypes.c_size_t
        L.intattn_decode_shared.argtypes = [vp, vp, vp, i32, i32, vp, vp, vp, scp, i32, i32, i32, i32, i32, f32, i32,
                                            vp, vp, ctypes.c_size_t, vp]
        L.intattn_gelu_derive_params.argtypes = [f32, f32, f32, ctypes.POINTER(_GeluParams)]
        L.intattn_gelu.argtypes = [vp, vp, ctypes.c_longlong, f32, f32, f32, vp]
        L.intattn_selftest_timeout.argtypes = [vp]
        L.intattn_device_error.argtypes = [vp]
        L.intattn_strerror.argtypes = [i32]
        L.intattn_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().intattn_strerror(int(code)).decode()


def _check(rc: int, what: str):
    if rc != OK:
        raise IntAttnError(rc, what)


def derive_params(scales: Scales, H: int, d: int, clip_c: float):
    """(lut[32] int32, [H, 5] int32 of M, s, D, Mo, so) as the kernels use them."""
    sc, keep = scales._c()
    lut = np.zeros(32, dtype=np.int32)
    hp = (_HeadParams * H)()
    rc = lib().intattn_derive_params(ctypes.byref(sc), int(H), int(d), float(clip_c),
                                     lut.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), hp)
    _check(rc, "intattn_derive_params")
    del keep
    return lut, np.array([[p.M, p.s, p.D, p.Mo, p.so] for p in hp], dtype=np.int32)


def _stream_handle(stream, device) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check_tensor(t, name: str):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int8 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA int8 tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_codes(t, name: str, zero_point, cuda: bool = True):
    """K or V codes: uint8 when the tensor has a zero-point, else int8."""
    import torch
    want = torch.uint8 if zero_point is not None else torch.int8
    if not isinstance(t, torch.Tensor) or t.dtype != want or t.is_cuda != cuda:
        raise TypeError(f"{name} must be a {'CUDA' if cuda else 'CPU'} {want} tensor"
                        + (" (it has a zero-point)" if zero_point is not None else ""))
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def forward(q, k, v, scales: Scales, causal: bool, clip_c: float, out=None, stream=None, variant: int = 0):
    """out[B,H,Lq,d] int8 = IntAttention forward of int8 q[B,H,Lq,d], k/v[B,H,Lk,d].
    variant: VARIANT_AUTO (intattn_forward), VARIANT_THREE_PASS or
    VARIANT_SHORT_ROWS (intattn_forward_variant); the bytes are the same."""
    import torch
    _check_tensor(q, "q")
    _check_codes(k, "k", scales.z_k)
    _check_codes(v, "v", scales.z_v)
    B, H, Lq, d = q.shape
    Lk = k.shape[2]
    if k.shape != (B, H, Lk, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, H, Lk, d] matching q")
    if out is None:
        out = torch.empty_like(q)
    _check_tensor(out, "out")
    if out.shape != q.shape:
        raise ValueError("out must match q")
    sc, keep = scales._c()
    if variant == VARIANT_AUTO:
        rc = lib().intattn_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(sc), B, H, Lq, Lk,
                                   d, int(bool(causal)), float(clip_c), out.data_ptr(),
                                   _stream_handle(stream, q.device))
    else:
        rc = lib().intattn_forward_variant(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(sc), B, H,
                                           Lq, Lk, d, int(bool(causal)), float(clip_c), out.data_ptr(),
                                           int(variant), _stream_handle(stream, q.device))
    del keep
    _check(rc, "intattn_forward")
    return out


def forward_host_workspace_size(B: int, H: int, Lq: int, Lk: int, d: int) -> int:
    return int(lib().intattn_forward_host_workspace_size(B, H, Lq, Lk, d))


def forward_host(q, k, v, scales: Scales, causal: bool, clip_c: float, out=None, workspace=None, stream=None,
                 device=None):
    """forward on CPU int8 tensors (pinned for asynchronous copies): the
    library copies them in, runs the forward and copies the result out;
    consecutive calls with one workspace overlap.  Returns out (a CPU tensor,
    valid once `stream` has reached the end of the call)."""
    import torch
    if not isinstance(q, torch.Tensor) or q.dtype != torch.int8 or q.is_cuda or not q.is_contiguous():
        raise TypeError("q must be a contiguous CPU int8 tensor")
    _check_codes(k, "k", scales.z_k, cuda=False)
    _check_codes(v, "v", scales.z_v, cuda=False)
    B, H, Lq, d = q.shape
    Lk = k.shape[2]
    if k.shape != (B, H, Lk, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, H, Lk, d]")
    dev = torch.device("cuda") if device is None else torch.device(device)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.int8, pin_memory=True)
    if out.is_cuda or out.dtype != torch.int8 or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous CPU int8 tensor shaped like q")
    need = forward_host_workspace_size(B, H, Lq, Lk, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    sc, keep = scales._c()
    rc = lib().intattn_forward_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(sc), B, H, Lq, Lk, d,
                                    int(bool(causal)), float(clip_c), out.data_ptr(), workspace.data_ptr(),
                                    workspace.numel(), _stream_handle(stream, dev))
    del keep
    _check(rc, "intattn_forward_host")
    return out


def forward_fp_workspace_size(B: int, H: int, Lq: int, Lk: int, d: int) -> int:
    return int(lib().intattn_forward_fp_workspace_size(B, H, Lq, Lk, d))


def forward_fp(q, k, v, per_head: bool, s_o, causal: bool, clip_c: float, clip=None, out=None, scales_out=None,
               workspace=None, stream=None, zero_points=False, zero_points_out=None):
    """intattn_forward_fp: fp16 / bf16 q [B,H,Lq,d], k, v [B,H,Lk,d] (CUDA)
    -> int8 out, quantising on the device.  s_o (and clip, optional): host
    floats, H entries per head or 1.  zero_points=True: intattn_forward_fp_zp
    (K and V quantised with zero-points; zero_points_out, optional CUDA int32
    [2 n], receives z_k then z_v)."""
    import torch
    dt = {torch.float16: DTYPE_FP16, torch.bfloat16: DTYPE_BF16}
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dt or not t.is_contiguous():
            raise TypeError(f"{n} must be a contiguous CUDA fp16 / bf16 tensor")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k and v must have one dtype")
    B, H, Lq, d = q.shape
    Lk = k.shape[2]
    if k.shape != (B, H, Lk, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, H, Lk, d] matching q")
    if out is None:
        out = torch.empty((B, H, Lq, d), dtype=torch.int8, device=q.device)
    _check_tensor(out, "out")
    so = np.ascontiguousarray(np.atleast_1d(np.asarray(s_o, dtype=np.float32)))
    cl = None if clip is None else np.ascontiguousarray(np.atleast_1d(np.asarray(clip, dtype=np.float32)))
    need = forward_fp_workspace_size(B, H, Lq, Lk, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    f32p = ctypes.POINTER(ctypes.c_float)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), dt[q.dtype], int(bool(per_head)), so.ctypes.data_as(f32p),
            None if cl is None else cl.ctypes.data_as(f32p), float(clip_c), B, H, Lq, Lk, d, int(bool(causal)),
            out.data_ptr(), None if scales_out is None else scales_out.data_ptr())
    tail = (workspace.data_ptr(), workspace.numel(), _stream_handle(stream, q.device))
    if zero_points:
        zp = None if zero_points_out is None else zero_points_out.data_ptr()
        rc = lib().intattn_forward_fp_zp(*args, zp, *tail)
        _check(rc, "intattn_forward_fp_zp")
    else:
        rc = lib().intattn_forward_fp(*args, *tail)
        _check(rc, "intattn_forward_fp")
    return out


def calibrate_workspace_size(B: int, H: int) -> int:
    return int(lib().intattn_calibrate_workspace_size(int(B), int(H)))


def calibrate_clip(q, k, scales: Scales, causal: bool, keep: int, stride: int, c_min: float = 0.25,
                   c_max: float = 64.0, workspace=None, stream=None):
    """intattn_calibrate_clip: (thresholds float32 [H or 1], gaps int32 [H or 1])
    for int8 CUDA q [B,H,Lq,d], k [B,H,Lk,d].  Synchronises the stream."""
    import torch
    _check_tensor(q, "q")
    _check_tensor(k, "k")
    B, H, Lq, d = q.shape
    Lk = k.shape[2]
    if k.shape != (B, H, Lk, d):
        raise ValueError("k must be [B, H, Lk, d] matching q")
    n = H if scales.per_head else 1
    clip = np.zeros(n, dtype=np.float32)
    gaps = np.zeros(n, dtype=np.int32)
    if workspace is None:
        workspace = torch.empty(max(int(lib().intattn_calibrate_workspace_size(B, H)), 1), dtype=torch.uint8,
                                device=q.device)
    sc, keep_alive = scales._c()
    rc = lib().intattn_calibrate_clip(q.data_ptr(), k.data_ptr(), ctypes.byref(sc), B, H, Lq, Lk, d,
                                      int(bool(causal)), int(keep), int(stride), float(c_min), float(c_max),
                                      clip.ctypes.data_as(ctypes.POINTER(ctypes.c_float)),
                                      gaps.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), workspace.data_ptr(),
                                      workspace.numel(), _stream_handle(stream, q.device))
    del keep_alive
    _check(rc, "intattn_calibrate_clip")
    return clip, gaps


def decode_workspace_size(B: int, H: int, Lk: int, d: int) -> int:
    return int(lib().intattn_decode_workspace_size(int(B), int(H), int(Lk), int(d)))


def decode(q, k_cache, v_cache, scales: Scales, Lk: int, clip_c: float, out=None, workspace=None,
           stream=None):
    """out[B,H,1,d] int8: one query per (b, h) over the first Lk rows of the caches."""
    import torch
    _check_tensor(q, "q")
    _check_codes(k_cache, "k_cache", scales.z_k)
    _check_codes(v_cache, "v_cache", scales.z_v)
    B, H, one, d = q.shape
    if one != 1:
        raise ValueError("decode takes one query per (b, h): q is [B, H, 1, d]")
    Lmax = k_cache.shape[2]
    if k_cache.shape != (B, H, Lmax, d) or v_cache.shape != k_cache.shape:
        raise ValueError("caches must be [B, H, Lmax, d]")
    if out is None:
        out = torch.empty_like(q)
    _check_tensor(out, "out")
    need = decode_workspace_size(B, H, Lk, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    sc, keep = scales._c()
    rc = lib().intattn_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ctypes.byref(sc), B,
                              H, int(Lk), Lmax, d, float(clip_c), out.data_ptr(), workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(),
                              _stream_handle(stream, q.device))
    del keep
    _check(rc, "intattn_decode")
    return out


def _check_u8_tensor(t, name: str):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA uint8 tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def decode_int4(q, k_cache, v_cache, scales: Scales, Lk: int, clip_c: float, out=None, workspace=None,
                stream=None):
    """out[B,H,1,d] int8 over an int4 KV cache: k_cache/v_cache are uint8
    [B, H, Lmax, d/2], two 4-bit two's-complement channels per byte (channel
    2t in the low nibble of byte t)."""
    import torch
    _check_tensor(q, "q")
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _check_u8_tensor(t, n)
    B, H, one, d = q.shape
    if one != 1:
        raise ValueError("decode takes one query per (b, h): q is [B, H, 1, d]")
    Lmax = k_cache.shape[2]
    if k_cache.shape != (B, H, Lmax, d // 2) or v_cache.shape != k_cache.shape:
        raise ValueError("int4 caches must be [B, H, Lmax, d/2] bytes")
    if out is None:
        out = torch.empty_like(q)
    _check_tensor(out, "out")
    need = decode_workspace_size(B, H, Lk, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    sc, keep = scales._c()
    rc = lib().intattn_decode_int4(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ctypes.byref(sc), B,
                                   H, int(Lk), Lmax, d, float(clip_c), out.data_ptr(), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(),
                                   _stream_handle(stream, q.device))
    del keep
    _check(rc, "intattn_decode_int4")
    return out


def quantize(x, per_head: bool, out=None, scales=None, stream=None):
    """int8 codes and device scales of an fp16 / bf16 CUDA tensor [B, H, L, d]
    (symmetric, dynamic: s = max|x| / 127 per tensor or per head)."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("x must be a CUDA float16 or bfloat16 tensor")
    if not x.is_contiguous() or x.dim() != 4:
        raise ValueError("x must be a contiguous [B, H, L, d] tensor")
    B, H, L, d = x.shape
    if out is None:
        out = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    _check_tensor(out, "out")
    if out.shape != x.shape:
        raise ValueError("out must match x")
    n = H if per_head else 1
    if scales is None:
        scales = torch.empty(n, dtype=torch.float32, device=x.device)
    if scales.dtype != torch.float32 or not scales.is_cuda or scales.numel() < n:
        raise ValueError(f"scales must be a CUDA float32 tensor of at least {n} entries")
    dt = DTYPE_BF16 if x.dtype == torch.bfloat16 else DTYPE_FP16
    _check(lib().intattn_quantize(x.data_ptr(), dt, B, H, L, d, int(bool(per_head)), out.data_ptr(),
                                  scales.data_ptr(), _stream_handle(stream, x.device)), "intattn_quantize")
    return out, scales


def quantize_zp(x, per_head: bool, out=None, scales=None, zero_points=None, stream=None):
    """u8 codes, device scales and device zero-points of an fp16 / bf16 CUDA
    tensor [B, H, L, d] (asymmetric, dynamic, per tensor or per head)."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("x must be a CUDA float16 or bfloat16 tensor")
    if not x.is_contiguous() or x.dim() != 4:
        raise ValueError("x must be a contiguous [B, H, L, d] tensor")
    B, H, L, d = x.shape
    if out is None:
        out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if not isinstance(out, torch.Tensor) or out.dtype != torch.uint8 or not out.is_cuda or not out.is_contiguous():
        raise TypeError("out must be a contiguous CUDA uint8 tensor")
    if out.shape != x.shape:
        raise ValueError("out must match x")
    n = H if per_head else 1
    if scales is None:
        scales = torch.empty(n, dtype=torch.float32, device=x.device)
    if zero_points is None:
        zero_points = torch.empty(n, dtype=torch.int32, device=x.device)
    if scales.dtype != torch.float32 or not scales.is_cuda or scales.numel() < n:
        raise ValueError(f"scales must be a CUDA float32 tensor of at least {n} entries")
    if zero_points.dtype != torch.int32 or not zero_points.is_cuda or zero_points.numel() < n:
        raise ValueError(f"zero_points must be a CUDA int32 tensor of at least {n} entries")
    dt = DTYPE_BF16 if x.dtype == torch.bfloat16 else DTYPE_FP16
    _check(lib().intattn_quantize_zp(x.data_ptr(), dt, B, H, L, d, int(bool(per_head)), out.data_ptr(),
                                     scales.data_ptr(), zero_points.data_ptr(), _stream_handle(stream, x.device)),
           "intattn_quantize_zp")
    return out, scales, zero_points


# ------------------------------------------------ rows, caches and their decode

class _On:
    """Makes `device` and `stream` current for a call, so that what the call
    allocates belongs to the stream it runs on; gives the stream's handle."""

    def __init__(self, device, stream):
        self.device, self.stream = device, stream

    def __enter__(self) -> int:
        import torch
        s = self.stream
        if getattr(s, "device", self.device) != self.device:
            raise ValueError(f"stream is on {s.device}, the tensors are on {self.device}")
        if s is not None and not isinstance(s, torch.cuda.Stream):
            s = torch.cuda.ExternalStream(int(getattr(s, "cuda_stream", s)), device=self.device)
        with contextlib.ExitStack() as guards:  # left again where a step on the way in fails
            guards.enter_context(torch.cuda.device(self.device))
            if s is not None:
                guards.enter_context(torch.cuda.stream(s))
            handle = torch.cuda.current_stream(self.device).cuda_stream
            self.guards = guards.pop_all()
        return handle

    def __exit__(self, *exc):
        self.guards.__exit__(*exc)


class _Here:
    """_On for the current device and its current stream: nothing to switch."""

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self) -> int:
        return self.handle

    def __exit__(self, *exc):
        pass


def _on(device, stream):
    import torch
    if stream is None and device.index == torch.cuda.current_device():
        return _Here(torch._C._cuda_getCurrentRawStream(device.index))
    return _On(device, stream)


def _rows(t, name: str, device, dtype) -> _Rows:
    """A [B, heads, L, d] fp16 / bf16 CUDA tensor whose channels are contiguous."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _row_types():
        raise TypeError(f"{name} must be a CUDA float16 or bfloat16 tensor")
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, heads, L, d]")
    B, h, L, d = t.shape
    sb, sh, sl, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name} must have contiguous channels")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be on {device} in {dtype}")
    # the stride of an extent of one is never used
    return _Rows(t.data_ptr(), sb if B > 1 else 0, sh if h > 1 else 0, sl if L > 1 else 0)


_ROW_TYPES = {}


def _row_types():
    """torch type -> INTATTN_DTYPE_*, of the row operators' floating tensors."""
    if not _ROW_TYPES:
        import torch
        _ROW_TYPES.update({torch.float16: DTYPE_FP16, torch.bfloat16: DTYPE_BF16})
    return _ROW_TYPES


def _index_tensor(t, name: str, shape, device):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device:
        raise TypeError(f"{name} must be an int32 tensor on {device}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)}")
    return t.data_ptr()


@dataclasses.dataclass
class RopeNorm:
    """Norm and rotation of query and key rows (intattn_rope_norm_t).
    table: float32 CUDA [n_positions, rot/2, 2] of (cos, sin) (see rope_table;
    None: no rotation); positions: int32 CUDA [B, L], negative = padding;
    w_q, w_k: float32 CUDA [d] norm weights (None: not normed)."""
    table: Optional[object] = None
    positions: Optional[object] = None
    w_q: Optional[object] = None
    w_k: Optional[object] = None
    eps: float = 1e-6
    interleaved: bool = False

    @staticmethod
    def _weight(w, name: str, d: int, device) -> int:
        import torch
        if not isinstance(w, torch.Tensor) or w.dtype != torch.float32 or w.device != device:
            raise TypeError(f"{name} must be a float32 tensor on {device}")
        if w.shape != (d,) or not w.is_contiguous():
            raise ValueError(f"{name} must be contiguous [{d}]")
        return w.data_ptr()

    def _c(self, B: int, L: int, d: int, device) -> _RopeNorm:
        import torch
        c = _RopeNorm()
        c.eps, c.interleaved = self.eps, bool(self.interleaved)
        if self.w_q is not None:
            c.w_q = self._weight(self.w_q, "w_q", d, device)
        if self.w_k is not None:
            c.w_k = self._weight(self.w_k, "w_k", d, device)
        if self.table is not None:
            t = self.table
            if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.device != device:
                raise TypeError(f"table must be a float32 tensor on {device}")
            if t.dim() != 3 or t.shape[2] != 2 or t.numel() == 0 or not t.is_contiguous():
                raise ValueError("table must be contiguous [n_positions, rot / 2, 2] and not empty")
            c.table, c.n_positions, c.rot = t.data_ptr(), t.shape[0], 2 * t.shape[1]
            c.positions = _index_tensor(self.positions, "positions", (B, L), device)
        elif self.positions is not None:
            raise ValueError("positions without a table")
        return c


def rope_table(n_positions: int, rot: int, base: float = 10000.0, device="cuda"):
    """(cos, sin) of p base^(-2 f / rot) for p < n_positions, f < rot / 2, as
    RopeNorm takes them: float32 [n_positions, rot/2, 2], the angles in double."""
    import torch
    if n_positions < 1 or rot < 2 or rot % 2:
        raise ValueError("rope_table needs n_positions >= 1 and an even rot >= 2")
    f = float(base) ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    a = torch.arange(n_positions, device=device, dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], dim=-1).float().contiguous()


def _rows_out(t, name: str, like, zeroed=False):
    """An output of the shape and type of `like` (None: a new one, cleared
    where `zeroed`) and its _Rows."""
    if t is None:
        B, h, L, d = like.shape
        t = (like.new_zeros if zeroed else like.new_empty)((B, h, L, d))
        return t, _Rows(t.data_ptr(), h * L * d, L * d, d)
    r = _rows(t, name, like.device, like.dtype)
    if t.shape != like.shape:
        raise ValueError(f"{name} must be {list(like.shape)}")
    return t, r


def qk_norm_rope(q, k, norm: RopeNorm, q_out=None, k_out=None, stream=None):
    """(q_out, k_out): norm and position rotation of fp16 / bf16 q [B, H, L, d]
    and k [B, Hkv, L, d] (strided views with contiguous channels; k None:
    queries only) in one pass.  In place: q_out=q, k_out=k.  Rows whose
    position is negative (padding) or past the table are left as they were in outputs that are
    passed, and are 0 in those that are not."""
    import torch
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise TypeError("q must be a CUDA tensor [B, H, L, d]")
    dev, dt = q.device, q.dtype
    qr = _rows(q, "q", dev, dt)
    B, H, L, d = q.shape
    kr = kor = None
    Hkv = 0
    if k is not None:
        kr = _rows(k, "k", dev, dt)
        Hkv = k.shape[1]
        if k.shape != (B, Hkv, L, d):
            raise ValueError("k must be [B, Hkv, L, d] matching q")
    elif k_out is not None:
        raise ValueError("k_out without k")
    c = norm._c(B, L, d, dev)
    kind = _row_types()[dt]
    # rows can be left out: by the kernel where both outputs are new, else in advance
    ragged, mixed = norm.table is not None, k is not None and (q_out is None) != (k_out is None)
    if ragged and q_out is None and not mixed:
        kind |= ZERO_LEFT_OUT
    with _on(dev, stream) as st:
        q_out, qor = _rows_out(q_out, "q_out", q, ragged and mixed)
        if k is not None:
            k_out, kor = _rows_out(k_out, "k_out", k, ragged and mixed)
        _check(lib().intattn_qk_norm_rope(qr, kr, c, kind, B, H, Hkv, L, d, qor, kor, st), "intattn_qk_norm_rope")
    return q_out, k_out


def _check_cache(t, name: str, zero_point, bits: int, shape, device):
    """A cache of `shape` [B, Hkv, Lmax, bytes of a row]."""
    import torch
    want = torch.uint8 if bits == 4 or zero_point is not None else torch.int8
    if not isinstance(t, torch.Tensor) or t.dtype != want or t.device != device:
        raise TypeError(f"{name} must be a {want} tensor on {device}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)}")


def cache_write(k, v, scales: Scales, k_cache, v_cache, start, lengths=None, bits: int = 8, q=None, q_out=None,
                norm: Optional[RopeNorm] = None, stream=None):
    """Quantises fp16 / bf16 rows k, v [B, Hkv, L, d] (strided views) with the
    caches' fixed scales into cache rows start[b] + t, t < lengths[b] (int32
    CUDA [B]; None: L).  k_cache, v_cache: [B, Hkv, Lmax, d] int8 (uint8 with
    zero-points), or, bits = 4, uint8 [B, Hkv, Lmax, d/2].  q [B, H, L, d]:
    also the step's queries, with scales.s_q, into int8 q_out (returned; new
    where none is passed, with 0 in the rows that are not written).
    norm: norm and rotation of q and k first, in the same pass; a token whose
    position is negative or past the table is left out whole, its V row too."""
    import torch
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise TypeError("k must be a CUDA tensor [B, Hkv, L, d]")
    dev, dt = k.device, k.dtype
    kr, vr = _rows(k, "k", dev, dt), _rows(v, "v", dev, dt)
    B, Hkv, L, d = k.shape
    if v.shape != k.shape:
        raise ValueError("v must match k")
    if bits not in (8, 4):
        raise ValueError("bits must be 8 or 4")
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise TypeError("k_cache must be a [B, Hkv, Lmax, d] tensor")
    Lmax = k_cache.shape[2]
    shape = (B, Hkv, Lmax, d * bits // 8)
    _check_cache(k_cache, "k_cache", scales.z_k, bits, shape, dev)
    _check_cache(v_cache, "v_cache", scales.z_v, bits, shape, dev)
    H, qr = 0, None
    if q is not None:
        qr = _rows(q, "q", dev, dt)
        H = q.shape[1]
        if q.shape != (B, H, L, d):
            raise ValueError("q must be [B, H, L, d] matching k")
    elif q_out is not None:
        raise ValueError("q_out without q")
    sp = _index_tensor(start, "start", (B,), dev)
    lp = None if lengths is None else _index_tensor(lengths, "lengths", (B,), dev)
    c = None if norm is None else norm._c(B, L, d, dev)
    sc, keep = scales._c_heads(H, Hkv, ("s_k", "s_v", "z_k", "z_v") if q is None else ("s_k", "s_v", "z_k", "z_v", "s_q"))
    kind = _row_types()[dt] | (ZERO_LEFT_OUT if q is not None and q_out is None else 0)
    with _on(dev, stream) as st:
        if q is not None:
            if q_out is None:
                q_out = q.new_empty((B, H, L, d), dtype=torch.int8)
            _check_tensor(q_out, "q_out")
            if q_out.shape != q.shape or q_out.device != dev:
                raise ValueError("q_out must match q")
        rc = lib().intattn_cache_write(kr, vr, qr, kind, sc, int(bits), c,
                                       B, H, Hkv, L, Lmax, d, sp, lp, k_cache.data_ptr(), v_cache.data_ptr(),
                                       None if q is None else q_out.data_ptr(), st)
    del keep
    _check(rc, "intattn_cache_write")
    return q_out


def cache_read(k_cache, v_cache, scales: Scales, start, L: int, lengths=None, bits: int = 8, dtype=None, k_out=None,
               v_out=None, stream=None):
    """(k_out, v_out): the values of cache rows start[b] + t, t < lengths[b]
    (None: L), as fp16 / bf16 [B, Hkv, L, d] (dtype; default bf16).  Rows past
    lengths[b], and those of cache rows that do not exist, are left as they were in outputs that are
    passed, and are 0 in those that are not.  v_cache None: K only."""
    import torch
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4 or not k_cache.is_cuda:
        raise TypeError("k_cache must be a CUDA tensor [B, Hkv, Lmax, d]")
    if bits not in (8, 4):
        raise ValueError("bits must be 8 or 4")
    dev = k_cache.device
    shape = k_cache.shape
    B, Hkv, Lmax, d = shape
    d = d * 8 // bits
    L = int(L)
    if L < 0:
        raise ValueError("L must not be negative")
    _check_cache(k_cache, "k_cache", scales.z_k, bits, shape, dev)
    if v_cache is not None:
        _check_cache(v_cache, "v_cache", scales.z_v, bits, shape, dev)
    elif v_out is not None:
        raise ValueError("v_out without v_cache")
    dt = dtype or (k_out.dtype if k_out is not None else torch.bfloat16)
    if dt not in _row_types():
        raise TypeError("dtype must be float16 or bfloat16")
    sp = _index_tensor(start, "start", (B,), dev)
    lp = None if lengths is None else _index_tensor(lengths, "lengths", (B,), dev)
    sc, keep = scales._c_heads(0, Hkv, ("s_k", "z_k") if v_cache is None else ("s_k", "s_v", "z_k", "z_v"))
    kind = _row_types()[dt]
    # rows left out become 0 in new outputs: by the kernel where all are new, else in advance
    new = k_cache.new_empty
    if v_cache is not None and (k_out is None) != (v_out is None):
        new = k_cache.new_zeros
    elif k_out is None:
        kind |= ZERO_LEFT_OUT
    with _on(dev, stream) as st:
        if k_out is None:
            k_out = new((B, Hkv, L, d), dtype=dt)
        if v_out is None and v_cache is not None:
            v_out = new((B, Hkv, L, d), dtype=dt)
        for t, n in ((k_out, "k_out"), (v_out, "v_out")):
            if t is None:
                continue
            if not isinstance(t, torch.Tensor) or t.dtype != dt or t.device != dev:
                raise TypeError(f"{n} must be a {dt} tensor on {dev}")
            if t.shape != (B, Hkv, L, d) or not t.is_contiguous():
                raise ValueError(f"{n} must be contiguous {[B, Hkv, L, d]}")
        rc = lib().intattn_cache_read(k_cache.data_ptr(), None if v_cache is None else v_cache.data_ptr(), sc, int(bits),
                                      B, Hkv, L, Lmax, d, sp, lp, kind,
                                      k_out.data_ptr(), None if v_out is None else v_out.data_ptr(), st)
    del keep
    _check(rc, "intattn_cache_read")
    return k_out, v_out


def decode_shared_workspace_size(B: int, H: int, Hkv: int, Lmax: int, d: int) -> int:
    """Bytes of decode_shared's workspace: about 5 B H Lmax + 4 B H d (84 MB for
    64 sequences of 32 heads and caches of 8192 rows, whatever the lengths)."""
    return int(lib().intattn_decode_shared_workspace_size(int(B), int(H), int(Hkv), int(Lmax), int(d)))


def decode_shared(q, k_prefix, v_prefix, k_cache, v_cache, lengths, scales: Scales, clip_c: float, prefix_len=None,
                  dtype=None, out=None, workspace=None, stream=None):
    """out [B, H, 1, d]: one query per (b, h) over the first prefix_len rows
    (None: all) of k_prefix, v_prefix [Hkv, Lp, d], shared by the batch, and
    then the first lengths[b] rows (int32 CUDA [B]; None: all) of k_cache,
    v_cache [B, Hkv, Lmax, d].  H a multiple of Hkv; scales.s_q, s_o, clip: H
    entries per head, s_k, s_v, z_k, z_v: Hkv.  dtype: torch.int8 (default),
    the codes; float16 / bfloat16, the values they stand for.  workspace: a
    uint8 CUDA tensor of decode_shared_workspace_size bytes, one per stream (None: allocated for the
    call).  A length out of
    range leaves its sequence as it was in an `out` that is passed, and 0 in one that is not."""
    import torch
    _check_tensor(q, "q")
    dev = q.device
    if q.dim() != 4 or q.shape[2] != 1:
        raise ValueError("decode_shared takes one query per (b, h): q is [B, H, 1, d]")
    B, H, _, d = q.shape
    for t, n, z in ((k_prefix, "k_prefix", scales.z_k), (v_prefix, "v_prefix", scales.z_v),
                    (k_cache, "k_cache", scales.z_k), (v_cache, "v_cache", scales.z_v)):
        _check_codes(t, n, z)
        if t.device != dev:
            raise ValueError(f"{n} must be on {dev}")
    if k_cache.dim() != 4 or k_prefix.dim() != 3:
        raise ValueError("prefixes are [Hkv, Lp, d], caches [B, Hkv, Lmax, d]")
    Hkv, Lmax = k_cache.shape[1:3]
    if k_cache.shape != (B, Hkv, Lmax, d) or v_cache.shape != k_cache.shape:
        raise ValueError("caches must be [B, Hkv, Lmax, d] matching q")
    Lp_max = k_prefix.shape[1]
    if k_prefix.shape != (Hkv, Lp_max, d) or v_prefix.shape != k_prefix.shape:
        raise ValueError("prefixes must be [Hkv, Lp, d] matching the caches")
    if Hkv < 1 or H % Hkv:
        raise ValueError("the query heads must be a multiple of the K / V heads")
    Lp = Lp_max if prefix_len is None else int(prefix_len)
    lp = None if lengths is None else _index_tensor(lengths, "lengths", (B,), dev)
    dt = dtype or (out.dtype if out is not None else torch.int8)
    kinds = {torch.float16: DTYPE_FP16, torch.bfloat16: DTYPE_BF16, torch.int8: DTYPE_INT8}
    if dt not in kinds:
        raise TypeError("dtype must be int8, float16 or bfloat16")
    sc, keep = scales._c_heads(H, Hkv, ("s_q", "s_k", "s_v", "s_o", "clip", "z_k", "z_v"))
    kind = kinds[dt] | (ZERO_LEFT_OUT if out is None else 0)
    with _on(dev, stream) as st:
        if out is None:
            out = q.new_empty((B, H, 1, d), dtype=dt)
        if not isinstance(out, torch.Tensor) or out.dtype != dt or out.device != dev:
            raise TypeError(f"out must be a {dt} tensor on {dev}")
        if out.shape != q.shape or not out.is_contiguous():
            raise ValueError("out must be contiguous and match q")
        if workspace is None:
            workspace = q.new_empty(decode_shared_workspace_size(B, H, Hkv, Lmax, d), dtype=torch.uint8)
        elif not isinstance(workspace, torch.Tensor) or workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        rc = lib().intattn_decode_shared(q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(), Lp, Lp_max,
                                         k_cache.data_ptr(), v_cache.data_ptr(), lp, sc, B, H, Hkv, Lmax, d,
                                         float(clip_c), kind, out.data_ptr(), workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(), st)
    del keep
    _check(rc, "intattn_decode_shared")
    return out


def gelu_params(s_x: float, s_y: float, c: float):
    """(M, s, gate[32], Mo, so) of the integer GELU, as the kernel uses them."""
    p = _GeluParams()
    _check(lib().intattn_gelu_derive_params(float(s_x), float(s_y), float(c), ctypes.byref(p)),
           "intattn_gelu_derive_params")
    return p.M, p.s, list(p.gate), p.Mo, p.so


def gelu(x, s_x: float, s_y: float, c: float, out=None, stream=None):
    """Integer GELU of a contiguous CUDA int8 tensor (any shape): int8 codes
    of scale s_y for codes x of scale s_x; gate tabulated on [-c, c].
    out may be x itself (in place)."""
    _check_tensor(x, "x")
    if out is None:
        import torch
        out = torch.empty_like(x)
    _check_tensor(out, "out")
    if out.numel() != x.numel():
        raise ValueError("out must have as many elements as x")
    _check(lib().intattn_gelu(x.data_ptr(), out.data_ptr(), x.numel(), float(s_x), float(s_y), float(c),
                              _stream_handle(stream, x.device)), "intattn_gelu")
    return out


def device_error(stream=None) -> int:
    """Synchronise and return/clear the device error word (OK or ERR_TIMEOUT)."""
    import torch
    return int(lib().intattn_device_error(_stream_handle(stream, torch.device("cuda"))))


def selftest_timeout(stream=None) -> int:
    """Run the bounded-wait self-test; returns device_error() afterwards
    (ERR_TIMEOUT when failure detection works)."""
    import torch
    _check(lib().intattn_selftest_timeout(_stream_handle(stream, torch.device("cuda"))),
           "intattn_selftest_timeout")
    return device_error(stream)

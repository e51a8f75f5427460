"""gated_gqa_attention_gb300 -- gated split-KV GQA decode attention for GB300.

A thin ctypes binding over the C ABI in ``include/gda.h`` (``lib/libgda.so``).
Every step of the computation runs in the library's CUDA kernels; this module
only checks tensor metadata, passes device pointers and the current CUDA stream,
and turns status codes into exceptions.  There is no CPU fallback: without the
built library every call raises.

    out = decode(q, gate, k_pool, v_pool, kv_indptr, kv_indices, scale=1/16)

computes, per sequence b and query head h (FreeToken PR #781 "Fuse the BF16
attention output sigmoid gate into the existing Triton decode stage2"):

    O   = softmax(scale * q[b,h] K[rows_b, h // G]^T) V[rows_b, h // G]
    out = bf16( bf16(O) * bf16(sigmoid(gate[b,h])) )     (round-to-nearest-even)

K/V pools of dtype torch.float8_e4m3fn (or uint8 e4m3 codes) select the FP8-cache
kernels; their values are ``k_descale * e4m3(code)`` and ``v_descale * e4m3(code)``.

A 4-bit cache is two uint8 pools of codes [num_slots, Hkv, D / 2] and their scales
``kv_scales`` [num_slots, Hkv, 2, D / 16]: passing ``kv_scales`` to ``decode`` or
``decode_ex`` selects it.  ``kv_write_fp4`` and ``qk_norm_mrope_kv_write`` write it,
``kv_gather_fp4`` reads rows back.  ``kv_write_e4m3`` and ``kv_gather_e4m3`` do the same for an
e4m3 cache.  A prompt of packed sequences goes ``qk_norm_mrope_kv_write`` -> ``prefill_packed``;
new tokens behind cached ones (chunks of prompts, drafted tokens, single tokens, any mix) go into
the cache and then through ``prefill_paged``, over any of the three caches.

Calls run on ``stream`` (default: the current one), and outputs that the decode calls, the
rotary step, ``kv_gather_fp4``, ``kv_gather_e4m3``, ``prefill_packed`` and ``prefill_paged`` allocate belong to it: on another stream
they are used after a wait for it, and kept until that use is over (or given as arguments).
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

__all__ = [
    "load", "decode", "decode_ex", "decode_noalloc", "decode_step_host", "StepHost", "step_layout", "small_path_cluster", "auto_splits", "pack_step", "STEP_MAP_IN", "STEP_MAP_OUT", "prefill", "prefill_read_error", "qk_norm_rope_kv_write", "prefill_packed", "prefill_paged", "prefill_paged_workspace_bytes", "qk_norm_mrope_kv_write", "mrope_pair_axis",
    "kv_write_fp4", "kv_gather_fp4", "kv_write_e4m3", "kv_gather_e4m3", "gate", "workspace_bytes", "workspace_init", "reserve",
    "read_error", "debug_wait_limit", "timing_begin", "timing_end", "status_str", "version", "GdaError", "VARIANT_AUTO", "VARIANT_MMA",
    "VARIANT_SIMT", "VARIANT_TMA", "MAX_SPLITS", "LIB_PATH", "KV_BF16", "KV_E4M3", "KV_E2M1",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libgda.so")

VARIANT_AUTO, VARIANT_MMA, VARIANT_SIMT, VARIANT_TMA = 0, 1, 2, 3
KV_BF16, KV_E4M3, KV_E2M1 = 0, 1, 3
MAX_SPLITS = 256
NOALLOC_SCRATCH_BYTES = 16 << 20
DEVERR_INDEX, DEVERR_TIMEOUT = 0x1, 0x2

_lock = threading.Lock()
_lib = None


class GdaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class _Args(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("k_pool", ctypes.c_void_p),
        ("v_pool", ctypes.c_void_p), ("kv_indptr", ctypes.c_void_p), ("kv_indices", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("num_slots", ctypes.c_int64),
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("scale", ctypes.c_float), ("num_splits", ctypes.c_int), ("fuse_gate", ctypes.c_int),
        ("check_indices", ctypes.c_int), ("variant", ctypes.c_int), ("min_chunk", ctypes.c_int),
        ("window", ctypes.c_int), ("sinks", ctypes.c_void_p), ("kv_dtype", ctypes.c_int),
        ("k_descale", ctypes.c_float), ("v_descale", ctypes.c_float), ("max_len", ctypes.c_int),
        ("total_len", ctypes.c_int64), ("kv_scales", ctypes.c_void_p),
    ]


class _MropeArgs(ctypes.Structure):
    _fields_ = [
        ("qgkv", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("w_q_norm", ctypes.c_void_p),
        ("w_k_norm", ctypes.c_void_p), ("eps", ctypes.c_float), ("n_axes", ctypes.c_int),
        ("positions", ctypes.c_void_p), ("pos_stride", ctypes.c_int64), ("inv_freq", ctypes.c_void_p),
        ("pair_axis", ctypes.c_char_p), ("rope_dim", ctypes.c_int), ("kv_dtype", ctypes.c_int),
        ("q_out", ctypes.c_void_p), ("gate_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
        ("slots", ctypes.c_void_p), ("num_slots", ctypes.c_int64), ("k_pool", ctypes.c_void_p),
        ("v_pool", ctypes.c_void_p), ("kv_scales", ctypes.c_void_p), ("k_descale", ctypes.c_float),
        ("v_descale", ctypes.c_float), ("T", ctypes.c_int64), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
        ("D", ctypes.c_int),
    ]


class _PackedArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("total_q", ctypes.c_int64), ("total_k", ctypes.c_int64),
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("scale", ctypes.c_float), ("causal", ctypes.c_int), ("error_word", ctypes.c_void_p),
    ]


class _PagedArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
        ("gate_stride", ctypes.c_int64), ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
        ("kv_scales", ctypes.c_void_p), ("num_slots", ctypes.c_int64), ("cu_seqlens", ctypes.c_void_p),
        ("kv_indptr", ctypes.c_void_p), ("kv_indices", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("sinks", ctypes.c_void_p), ("total_q", ctypes.c_int64), ("nnz", ctypes.c_int64),
        ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("scale", ctypes.c_float), ("window", ctypes.c_int), ("keep_first", ctypes.c_int),
        ("kv_dtype", ctypes.c_int), ("k_descale", ctypes.c_float), ("v_descale", ctypes.c_float),
        ("error_word", ctypes.c_void_p),
    ]


def load(path: Optional[str] = None):
    """Load the C-ABI library (raises when it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                "libgda.so is not built (%s); run `python -m gated_gqa_attention_gb300.build`" % p)
        lib = ctypes.CDLL(p)
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        lib.gda_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        lib.gda_workspace_bytes.restype = ctypes.c_size_t
        lib.gda_workspace_init.argtypes = [vp, ctypes.c_size_t, vp]
        lib.gda_workspace_init.restype = i32
        lib.gda_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, i32, vp]
        lib.gda_decode.restype = i32
        lib.gda_decode_ex.argtypes = [ctypes.POINTER(_Args), vp, ctypes.c_size_t, vp]
        lib.gda_decode_ex.restype = i32
        lib.gda_decode_e4m3.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, f32, f32, i32, vp]
        lib.gda_decode_e4m3.restype = i32
        lib.gda_decode_fp4.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, f32, f32, i32, vp]
        lib.gda_decode_fp4.restype = i32
        lib.gda_kv_write_fp4.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, vp, f32, f32, i64, i32, i32, vp]
        lib.gda_kv_write_fp4.restype = i32
        lib.gda_kv_gather_fp4.argtypes = [vp, vp, vp, i64, vp, i64, f32, f32, vp, vp, i32, i32, vp]
        lib.gda_kv_gather_fp4.restype = i32
        lib.gda_kv_write_e4m3.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, f32, f32, i64, i32, i32, vp]
        lib.gda_kv_write_e4m3.restype = i32
        lib.gda_kv_gather_e4m3.argtypes = [vp, vp, i64, vp, i64, f32, f32, vp, vp, i32, i32, vp]
        lib.gda_kv_gather_e4m3.restype = i32
        lib.gda_prefill_paged_workspace_bytes.argtypes = [i64, i32, i32, i32, i32]
        lib.gda_prefill_paged_workspace_bytes.restype = ctypes.c_size_t
        lib.gda_prefill_paged.argtypes = [ctypes.POINTER(_PagedArgs), vp, ctypes.c_size_t, vp]
        lib.gda_prefill_paged.restype = i32
        lib.gda_qk_norm_mrope_kv_write.argtypes = [ctypes.POINTER(_MropeArgs), vp]
        lib.gda_qk_norm_mrope_kv_write.restype = i32
        lib.gda_prefill_packed.argtypes = [ctypes.POINTER(_PackedArgs), vp]
        lib.gda_prefill_packed.restype = i32
        lib.gda_prefill.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, vp, vp]
        lib.gda_prefill.restype = i32
        lib.gda_prefill_read_error.argtypes = [vp, i32, ctypes.POINTER(ctypes.c_uint32)]
        lib.gda_prefill_read_error.restype = i32
        lib.gda_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, i32, vp]
        lib.gda_decode_noalloc.restype = i32
        lib.gda_qk_norm_rope_kv_write.argtypes = [vp, i64, vp, vp, f32, vp, vp, i32, vp, i64, vp, vp, vp, vp,
                                                  i32, i32, i32, i32, vp]
        lib.gda_qk_norm_rope_kv_write.restype = i32
        lib.gda_small_path_cluster.argtypes = [i64, i32]
        lib.gda_small_path_cluster.restype = i32
        lib.gda_auto_splits.argtypes = [i32, i32, i32, i32, i32, i64]
        lib.gda_auto_splits.restype = i32
        lib.gda_step_layout.argtypes = [i32, i32, i32, i64, ctypes.POINTER(ctypes.c_size_t)]
        lib.gda_step_layout.restype = ctypes.c_size_t
        lib.gda_decode_step_host.argtypes = [vp, vp, ctypes.c_size_t, vp, vp, i32, f32, f32, vp, vp, i32, i32, i32,
                                             i32, i64, f32, i32, i32, i32, vp]
        lib.gda_decode_step_host.restype = i32
        lib.gda_reserve.argtypes = [i32, i32, i32, i32, i32]
        lib.gda_reserve.restype = i32
        lib.gda_gate.argtypes = [vp, vp, vp, i64, vp]
        lib.gda_gate.restype = i32
        lib.gda_read_error.argtypes = [vp, vp, i32, ctypes.POINTER(ctypes.c_uint32)]
        lib.gda_read_error.restype = i32
        lib.gda_status_str.argtypes = [i32]
        lib.gda_status_str.restype = ctypes.c_char_p
        lib.gda_timing_begin.argtypes = [i32]
        lib.gda_timing_begin.restype = i32
        lib.gda_timing_end.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_double)]
        lib.gda_timing_end.restype = i32
        lib.gda_version.argtypes = []
        lib.gda_version.restype = i32
        lib.gda_debug_wait_limit.argtypes = [i64]
        lib.gda_debug_wait_limit.restype = i32
        _lib = lib
        return lib


def status_str(status: int) -> str:
    return load().gda_status_str(int(status)).decode()


def version() -> int:
    return int(load().gda_version())


def _check(rc: int):
    if rc != 0:
        raise GdaError(rc, status_str(rc))


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_tensor(name, t, dtype, ndim=None, device=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dims" % (name, ndim))


def workspace_bytes(B: int, Hq: int, Hkv: int, D: int, num_splits: int = 0) -> int:
    """Bytes of workspace decode_ex needs (0 for invalid sizes)."""
    return int(load().gda_workspace_bytes(int(B), int(Hq), int(Hkv), int(D), int(num_splits)))


def workspace_init(workspace, stream=None):
    """Zero a caller-owned workspace's header (its device error word)."""
    _launch(load().gda_workspace_init, workspace.get_device(), stream, workspace.data_ptr(),
            workspace.numel() * workspace.element_size())


def reserve(max_B: int, Hq: int = 16, Hkv: int = 2, D: int = 256, max_splits: int = 0):
    """Grow the library's internal workspace on the current device ahead of graph capture."""
    _check(load().gda_reserve(int(max_B), int(Hq), int(Hkv), int(D), int(max_splits)))


def _kv_dtype(k_pool) -> int:
    """KV_E4M3 for float8_e4m3fn / uint8 pools, else KV_BF16."""
    import torch
    return KV_E4M3 if isinstance(k_pool, torch.Tensor) and k_pool.dtype in (torch.float8_e4m3fn, torch.uint8) \
        else KV_BF16


_th = None


def _torch():
    """torch, imported on first use."""
    global _th
    if _th is None:
        import torch
        _th = torch
    return _th


def _need(name, t, dtype, ndim, dev):
    """_check_tensor for device index ``dev``, a quick test before it: these calls take a few
    microseconds, and the checks of ten tensors have to fit in them."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.dim() == ndim and t.is_contiguous():
            return
    except AttributeError:
        pass
    _check_tensor(name, t, dtype, ndim, _torch().device("cuda", dev))


def _need_shape(name, t, dtype, shape, dev, what):
    """As _need, with the sizes ``what`` describes."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return
    except AttributeError:
        pass
    _check_tensor(name, t, dtype, len(shape), _torch().device("cuda", dev))
    if t.shape != shape:
        raise ValueError("%s must %s" % (name, what))


def _first(name, t, dtype, ndim):
    """Checks a call's first tensor; the others have to be on its device, whose index this returns."""
    try:
        i = t.get_device()
        if i >= 0 and t.dtype is dtype and t.dim() == ndim and t.is_contiguous():
            return i
    except AttributeError:
        pass
    _check_tensor(name, t, dtype, ndim)
    return i


def _tokens(name, t, heads=None, dim=None, dev=None):
    """Checks a [T, H, D] bf16 CUDA tensor whose tokens may be any distance apart (the parts of
    a projection's rows) and returns that distance in elements."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not torch.bfloat16:
        raise TypeError("%s must be %s, got %s" % (name, torch.bfloat16, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dev is not None and t.get_device() != dev:
        raise ValueError("%s is on %s, expected cuda:%d" % (name, t.device, dev))
    if t.dim() != 3:
        raise ValueError("%s must have 3 dims" % name)
    T, H, D = t.shape
    if (heads is not None and H != heads) or (dim is not None and D != dim):
        raise ValueError("%s must be [T, %s, %s]" % (name, "H" if heads is None else heads, "D" if dim is None else dim))
    st = t.stride()
    if (D > 1 and st[2] != 1) or (H > 1 and st[1] != D):
        raise ValueError("the heads and dims of a token of %s must be contiguous" % name)
    # one token (or none): its distance to the next is never used
    return st[0] if T > 1 else max(H * D, 8)


def _check_fp4(k_pool, v_pool, kv_scales, D=None, dev=None):
    """Checks a 4-bit cache; returns (num_slots, Hkv)."""
    u8 = _torch().uint8
    if dev is None:
        dev = _first("k_pool", k_pool, u8, 3)
    else:
        _need("k_pool", k_pool, u8, 3, dev)
    n, h, half = shape = k_pool.shape
    _need_shape("v_pool", v_pool, u8, shape, dev, "have k_pool's shape")
    what = "be [num_slots, Hkv, 2, D / 16] for pools [num_slots, Hkv, D / 2]"
    if half % 8 != 0:
        raise ValueError("kv_scales must " + what)
    _need_shape("kv_scales", _scale_bytes(kv_scales), u8, (n, h, 2, half // 8), dev, what)
    if D is not None and 2 * half != D:
        raise ValueError("head dims of q and the pools differ")
    return n, h


def _scale_bytes(kv_scales):
    """kv_scales given as float8_e4m3fn or as its bytes."""
    torch = _torch()
    if isinstance(kv_scales, torch.Tensor) and kv_scales.dtype is torch.float8_e4m3fn:
        return kv_scales.view(torch.uint8)
    return kv_scales


def _alloc(stream, make, *args, **kw):
    """make(*args, **kw), a tensor that a call allocates itself.  Its memory belongs to the stream that the call runs
    on: from the current stream's it could be memory that work queued there still reads, and what the call drops
    could be handed out there while the call still uses it."""
    if stream is None:
        return make(*args, **kw)
    with _torch().cuda.stream(stream):
        return make(*args, **kw)


def _launch(fn, dev, stream, *args):
    """Call a library function on device index ``dev``, where its tensors live, with that device's
    current stream as the default, and raise on an error status (the library launches on the
    current device)."""
    torch = _torch()
    if stream is None:
        if torch._C._cuda_getDevice() == dev:
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
        else:
            with torch.cuda.device(dev):
                rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        if stream.device.index != dev:
            raise ValueError("stream is on %s, the tensors on cuda:%d" % (stream.device, dev))
        with torch.cuda.device(dev):
            rc = fn(*args, stream.cuda_stream)
    if rc != 0:
        _check(rc)


def _decode_checks(q, gate_t, k_pool, v_pool, kv_indptr, kv_indices, out, kv_scales=None):
    """Checks tensor metadata; returns the pools' element type (KV_BF16, KV_E4M3 or KV_E2M1)."""
    torch = _torch()
    bf16, i32 = torch.bfloat16, torch.int32
    dev, shape = _first("q", q, bf16, 3), q.shape
    if gate_t is not None:
        _need_shape("gate", gate_t, bf16, shape, dev, "have q's shape")
    if kv_scales is not None:
        kv = KV_E2M1
        _check_fp4(k_pool, v_pool, kv_scales, shape[2], dev)
    else:
        kv = _kv_dtype(k_pool)
        kdt = k_pool.dtype if kv == KV_E4M3 else bf16
        _need("k_pool", k_pool, kdt, 3, dev)
        _need("v_pool", v_pool, kdt, 3, dev)
        if v_pool.shape != k_pool.shape:
            raise ValueError("k_pool and v_pool must have the same shape")
    _need_shape("kv_indptr", kv_indptr, i32, (shape[0] + 1,), dev, "have B + 1 entries")
    _need("kv_indices", kv_indices, i32, 1, dev)
    if kv != KV_E2M1 and k_pool.shape[2] != shape[2]:
        raise ValueError("head dims of q and the pools differ")
    if out is not None:
        _need_shape("out", out, bf16, shape, dev, "have q's shape")
    return kv


def decode(q, gate_t, k_pool, v_pool, kv_indptr, kv_indices, out=None, scale: Optional[float] = None,
           num_splits: int = 0, stream=None, k_descale: float = 1.0, v_descale: float = 1.0, kv_scales=None):
    """Gated GQA decode attention through ``gda_decode`` (library-owned workspace).

    q, gate_t: [B, Hq, D] bf16; k_pool, v_pool: [num_slots, Hkv, D] bf16, or
    float8_e4m3fn / uint8 e4m3 codes (then ``gda_decode_e4m3`` with the descales), or
    with ``kv_scales`` a 4-bit cache (``gda_decode_fp4``); kv_indptr: [B+1] int32; kv_indices: [nnz] int32 (all CUDA, contiguous).
    ``num_splits <= 0`` lets the kernel plan the splits on the device."""
    import torch
    kv = _decode_checks(q, gate_t, k_pool, v_pool, kv_indptr, kv_indices, out, kv_scales)
    B, Hq, D = q.shape
    Hkv = k_pool.shape[1]
    if out is None:
        out = _alloc(stream, torch.empty_like, q)
    if scale is None:
        scale = 1.0 / (D ** 0.5)
    if kv == KV_E2M1:
        _launch((_lib or load()).gda_decode_fp4, q.get_device(), stream, _ptr(q), _ptr(gate_t), _ptr(k_pool), _ptr(v_pool),
                _ptr(kv_scales), _ptr(kv_indptr), _ptr(kv_indices), _ptr(out), B, Hq, Hkv, D, float(scale),
                float(k_descale), float(v_descale), int(num_splits))
        return out
    if kv == KV_E4M3:
        _check(load().gda_decode_e4m3(_ptr(q), _ptr(gate_t), _ptr(k_pool), _ptr(v_pool), _ptr(kv_indptr),
                                      _ptr(kv_indices), _ptr(out), B, Hq, Hkv, D, float(scale), float(k_descale),
                                      float(v_descale), int(num_splits), _stream(stream)))
        return out
    _check(load().gda_decode(_ptr(q), _ptr(gate_t), _ptr(k_pool), _ptr(v_pool), _ptr(kv_indptr),
                             _ptr(kv_indices), _ptr(out), B, Hq, Hkv, D, float(scale), int(num_splits),
                             _stream(stream)))
    return out


def decode_noalloc(q, gate_t, k_pool, v_pool, kv_indptr, kv_indices, out, scale: Optional[float] = None,
                   num_splits: int = 0, stream=None):
    """``gda_decode_noalloc``: the same result as decode() for callers that must not
    allocate device memory.  ``out`` must be given (this call allocates nothing);
    the library's fixed scratch area (NOALLOC_SCRATCH_BYTES per device) replaces the
    workspace, so calls that may overlap on the GPU must not use it concurrently."""
    if _decode_checks(q, gate_t, k_pool, v_pool, kv_indptr, kv_indices, out) != KV_BF16:
        raise TypeError("decode_noalloc serves bf16 pools only")
    if out is None:
        raise ValueError("decode_noalloc needs a preallocated out tensor")
    B, Hq, D = q.shape
    Hkv = k_pool.shape[1]
    if scale is None:
        scale = 1.0 / (D ** 0.5)
    _check(load().gda_decode_noalloc(_ptr(q), _ptr(gate_t), _ptr(k_pool), _ptr(v_pool), _ptr(kv_indptr),
                                     _ptr(kv_indices), _ptr(out), B, Hq, Hkv, D, float(scale), int(num_splits),
                                     _stream(stream)))
    return out


def auto_splits(B: int, heads: int, grid: int, lmax: int, total: int, min_chunk: int = 0) -> int:
    """``gda_auto_splits``: the automatic split rule for B sequences (longest lmax,
    total ``total`` positions), ``heads`` segments per sequence, ``grid`` stage-1 CTAs:
    the uniform split count, 0 for the stream schedule, -1 for invalid arguments."""
    return int(load().gda_auto_splits(int(B), int(heads), int(grid), int(min_chunk), int(lmax), int(total)))


def small_path_cluster(pairs: int, max_len: int) -> int:
    """``gda_small_path_cluster``: the cluster size (8, 4 or 2) a bf16 decode of
    ``pairs`` = B * Hkv (sequence, KV head) pairs with the length bound ``max_len``
    takes through the one-kernel path on the current device, or 0 (split path)."""
    return int(load().gda_small_path_cluster(int(pairs), int(max_len)))


def step_layout(B: int, Hq: int, D: int, nnz: int):
    """``gda_step_layout``: (offsets of q, gate, kv_indptr, kv_indices; total bytes) of
    one decode step's inputs packed into a single block."""
    off = (ctypes.c_size_t * 4)()
    total = load().gda_step_layout(int(B), int(Hq), int(D), int(nnz), off)
    if total == 0:
        raise ValueError("gda_step_layout: sizes out of range")
    return tuple(int(x) for x in off), int(total)


def pack_step(host_in, q, gate_t, kv_indptr, kv_indices):
    """Write one step's CPU tensors into the packed host block ``host_in`` (a uint8
    CPU tensor, pinned for asynchronous copies) at the offsets of step_layout."""
    import torch
    B, Hq, D = q.shape
    nnz = kv_indices.numel()
    off, total = step_layout(B, Hq, D, nnz)
    if host_in.dtype != torch.uint8 or host_in.device.type != "cpu" or host_in.numel() < total:
        raise ValueError("host_in must be a CPU uint8 tensor of at least %d bytes" % total)
    parts = ((q, torch.bfloat16), (gate_t, torch.bfloat16), (kv_indptr, torch.int32), (kv_indices, torch.int32))
    for (t, dt), o in zip(parts, off):
        if t.dtype != dt:
            raise TypeError("pack_step: expected %s, got %s" % (dt, t.dtype))
        b = t.detach().cpu().contiguous().view(torch.uint8).reshape(-1)
        host_in[o:o + b.numel()].copy_(b)
    return host_in


STEP_MAP_IN, STEP_MAP_OUT = 0x1, 0x2


class StepHost:
    """A decode step bound to fixed buffers: the packed pinned inputs ``host_in``
    (step_layout), the device staging ``dev_in`` / ``dev_out`` (None when mapped) and
    the pinned result ``host_out`` [B, Hq, D] bf16.  Everything is checked and
    marshalled once here; each call is then one ``gda_decode_step_host`` call (copy
    in, decode, copy out, wait).  ``map_in`` / ``map_out``: the kernels read host_in /
    write host_out in place over the host-device link instead of copies."""

    def __init__(self, host_in, dev_in, k_pool, v_pool, dev_out, host_out, B: int, Hq: int, nnz: int,
                 scale: Optional[float] = None, num_splits: int = 0, map_in: bool = False, map_out: bool = False,
                 synchronize: bool = True, stream=None, k_descale: float = 1.0, v_descale: float = 1.0):
        import torch
        kv = _kv_dtype(k_pool)
        dt = torch.bfloat16 if kv == KV_BF16 else k_pool.dtype
        _check_tensor("k_pool", k_pool, dt, 3)
        _check_tensor("v_pool", v_pool, dt, 3, k_pool.device)
        Hkv, D = k_pool.shape[1], k_pool.shape[2]
        _, total = step_layout(B, Hq, D, nnz)
        if host_in.device.type != "cpu" or host_out.device.type != "cpu":
            raise ValueError("host_in and host_out must be CPU tensors")
        if host_in.numel() * host_in.element_size() < total:
            raise ValueError("host_in holds fewer than %d bytes" % total)
        if not map_in and (dev_in is None or not dev_in.is_cuda or dev_in.numel() * dev_in.element_size() < total):
            raise ValueError("dev_in must be a CUDA tensor of at least %d bytes" % total)
        if tuple(host_out.shape) != (B, Hq, D) or host_out.dtype != torch.bfloat16:
            raise ValueError("host_out must be a [B, Hq, D] bf16 tensor")
        if not map_out and (dev_out is None or tuple(dev_out.shape) != (B, Hq, D)):
            raise ValueError("dev_out must be a [B, Hq, D] CUDA tensor")
        if scale is None:
            scale = 1.0 / (D ** 0.5)
        vp = ctypes.c_void_p
        flags = (STEP_MAP_IN if map_in else 0) | (STEP_MAP_OUT if map_out else 0)
        self.host_in, self.dev_in, self.dev_out, self.host_out = host_in, dev_in, dev_out, host_out
        self.k_pool, self.v_pool = k_pool, v_pool   # kept alive with the call's pointers
        self.in_bytes, self.out_bytes = total, host_out.numel() * 2
        self._f = load().gda_decode_step_host
        self._args = (vp(_ptr(host_in)), vp(_ptr(dev_in)), total, vp(_ptr(k_pool)), vp(_ptr(v_pool)),
                      kv, float(k_descale), float(v_descale), vp(_ptr(dev_out)), vp(_ptr(host_out)), int(B), int(Hq),
                      int(Hkv), int(D), int(nnz), float(scale), int(num_splits), flags, 1 if synchronize else 0,
                      _stream(stream))

    def __call__(self):
        rc = self._f(*self._args)
        if rc != 0:
            _check(rc)
        return self.host_out


def decode_step_host(host_in, dev_in, k_pool, v_pool, dev_out, host_out, B: int, Hq: int, nnz: int,
                     scale: Optional[float] = None, num_splits: int = 0, map_in: bool = False,
                     map_out: bool = False, synchronize: bool = True, stream=None, k_descale: float = 1.0,
                     v_descale: float = 1.0):
    """``gda_decode_step_host`` once (see StepHost, which keeps the marshalled call for
    repeated steps)."""
    return StepHost(host_in, dev_in, k_pool, v_pool, dev_out, host_out, B, Hq, nnz, scale=scale,
                    num_splits=num_splits, map_in=map_in, map_out=map_out, synchronize=synchronize,
                    stream=stream, k_descale=k_descale, v_descale=v_descale)()


def decode_ex(q, gate_t, k_pool, v_pool, kv_indptr, kv_indices, out=None, *, workspace=None,
              scale: Optional[float] = None, num_splits: int = 0, fuse_gate: bool = True, lse=None,
              check_indices: bool = False, variant: int = VARIANT_AUTO, min_chunk: int = 0,
              window: int = 0, sinks=None, stream=None, k_descale: float = 1.0, v_descale: float = 1.0,
              max_len: int = 0, total_len: int = 0, kv_scales=None):
    """``gda_decode_ex``: caller workspace (allocated here when None), optional LSE
    output, the unfused first half (``fuse_gate=False``), device index checks, the
    stage-1 variant, a sliding window (last ``window`` positions), per-head
    attention sinks (``sinks``: [Hq] float32 CUDA tensor of logits), for e4m3
    pools the per-tensor descales, ``kv_scales`` for a 4-bit cache (with the descales), and ``max_len``: a host-known bound on every
    sequence's length (0: none), which lets small batches run as one cluster kernel,
    and ``total_len``: the batch's exact number of KV positions (kv_indptr[B], 0: not
    given); with both, the split count is chosen on the host (``auto_splits``)."""
    torch = _torch()
    kv = _decode_checks(q, gate_t if fuse_gate else None, k_pool, v_pool, kv_indptr, kv_indices, out, kv_scales)
    B, Hq, D = q.shape
    Hkv = k_pool.shape[1]
    if out is None:
        out = _alloc(stream, torch.empty_like, q)
    if lse is not None:
        _need("lse", lse, torch.float32, 2, q.get_device())
        if kv == KV_E2M1 and lse.shape != (B, Hq):
            raise ValueError("lse must be [B, Hq]")
    if sinks is not None:
        _check_tensor("sinks", sinks, torch.float32, 1, q.device)
        if sinks.numel() != q.shape[1]:
            raise ValueError("sinks must have Hq entries")
    if scale is None:
        scale = 1.0 / (D ** 0.5)
    if workspace is None:
        nbytes = workspace_bytes(B, Hq, Hkv, D, num_splits)
        workspace = _alloc(stream, torch.empty, max(nbytes, 256), dtype=torch.uint8, device=q.device)
        workspace_init(workspace, stream)
    a = _Args(_ptr(q), _ptr(gate_t) if fuse_gate else None, _ptr(k_pool), _ptr(v_pool), _ptr(kv_indptr),
              _ptr(kv_indices), _ptr(out), _ptr(lse), int(k_pool.shape[0]), B, Hq, Hkv, D, float(scale),
              int(num_splits), 1 if fuse_gate else 0, 1 if check_indices else 0, int(variant), int(min_chunk),
              int(window), _ptr(sinks), kv, float(k_descale), float(v_descale), int(max_len), int(total_len),
              _ptr(kv_scales))
    nbytes = workspace.numel() * workspace.element_size()
    if kv == KV_E2M1:
        if workspace.get_device() != q.get_device():
            raise ValueError("workspace is on %s, expected %s" % (workspace.device, q.device))
        _launch((_lib or load()).gda_decode_ex, q.get_device(), stream, a, workspace.data_ptr(), nbytes)
        return out
    _check(load().gda_decode_ex(a, workspace.data_ptr(), nbytes, _stream(stream)))
    return out


def prefill(q, gate_t, k, v, *, kv_lens=None, out=None, lse=None, scale: Optional[float] = None,
            causal: bool = True, error_word=None, stream=None):
    """Prefill / extend gated SDPA through ``gda_prefill`` (tcgen05 kernel).

    q, gate_t: [B, Sq, Hq, D] bf16 (gate_t None: out = bf16(O)); k, v: [B, Skv, Hkv, D]
    bf16; kv_lens: [B] int32 or None; lse: [B, Hq, Sq] float32 or None; error_word:
    a 1-element int32/uint32 CUDA tensor or None (the library's word)."""
    import torch
    _check_tensor("q", q, torch.bfloat16, 4)
    dev = q.device
    B, Sq, Hq, D = q.shape
    if gate_t is not None:
        _check_tensor("gate", gate_t, torch.bfloat16, 4, dev)
        if gate_t.shape != q.shape:
            raise ValueError("gate must have q's shape")
    _check_tensor("k", k, torch.bfloat16, 4, dev)
    _check_tensor("v", v, torch.bfloat16, 4, dev)
    if v.shape != k.shape or k.shape[0] != B or k.shape[3] != D:
        raise ValueError("k and v must be [B, Skv, Hkv, D] with q's B and D")
    Skv, Hkv = k.shape[1], k.shape[2]
    if kv_lens is not None:
        _check_tensor("kv_lens", kv_lens, torch.int32, 1, dev)
        if kv_lens.numel() != B:
            raise ValueError("kv_lens must have B entries")
    if lse is not None:
        _check_tensor("lse", lse, torch.float32, 3, dev)
        if tuple(lse.shape) != (B, Hq, Sq):
            raise ValueError("lse must be [B, Hq, Sq]")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_tensor("out", out, torch.bfloat16, 4, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if scale is None:
        scale = 1.0 / (D ** 0.5)
    _check(load().gda_prefill(_ptr(q), _ptr(gate_t), _ptr(k), _ptr(v), _ptr(kv_lens), _ptr(out), _ptr(lse),
                              B, Sq, Skv, Hq, Hkv, D, float(scale), 1 if causal else 0, _ptr(error_word),
                              _stream(stream)))
    return out


def prefill_packed(q, gate_t, k, v, cu_seqlens, cu_seqlens_k=None, *, out=None, lse=None,
                   scale: Optional[float] = None, causal: bool = True, error_word=None, stream=None):
    """Gated SDPA over packed sequences through ``gda_prefill_packed``.

    q, gate_t: [Tq, Hq, D] bf16 (gate_t None: out = bf16(O)); k, v: [Tk, Hkv, D] bf16; tokens
    of each may be any multiple of 8 elements apart, so views of a projection's rows
    serve as they are.  cu_seqlens: [B + 1] int32, each sequence's first query row;
    cu_seqlens_k: the same for the keys (None: as the queries), where a sequence has
    more keys than queries when it continues a prefix.  out: [Tq, Hq, D] contiguous (rows
    of no sequence are left as they are: zeros in an ``out`` allocated here); lse:
    [Hq, Tq] float32 or None; error_word as in prefill."""
    torch = _torch()
    sq = _tokens("q", q)
    dev = q.get_device()
    Tq, Hq, D = q.shape
    sg = 0
    if gate_t is not None:
        sg = _tokens("gate", gate_t, Hq, D, dev)
        if gate_t.shape[0] != Tq:
            raise ValueError("gate must have q's shape")
    sk = _tokens("k", k, None, D, dev)
    Tk, Hkv = k.shape[0], k.shape[1]
    sv = _tokens("v", v, Hkv, D, dev)
    if v.shape[0] != Tk:
        raise ValueError("k and v must have the same shape")
    _need("cu_seqlens", cu_seqlens, torch.int32, 1, dev)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must have B + 1 entries")
    if cu_seqlens_k is None:
        if Tk != Tq:
            raise ValueError("k must have q's tokens (or give cu_seqlens_k)")
        cu_seqlens_k = cu_seqlens
    else:
        _need("cu_seqlens_k", cu_seqlens_k, torch.int32, 1, dev)
        if cu_seqlens_k.numel() != cu_seqlens.numel():
            raise ValueError("cu_seqlens_k must have B + 1 entries")
    if lse is not None:
        _need_shape("lse", lse, torch.float32, (Hq, Tq), dev, "be [Hq, Tq]")
    if out is None:
        out = _alloc(stream, torch.zeros, Tq, Hq, D, dtype=torch.bfloat16, device=q.device)
    else:
        _need_shape("out", out, torch.bfloat16, (Tq, Hq, D), dev, "have q's shape")
    if scale is None:
        scale = 1.0 / (D ** 0.5)
    if error_word is not None and (error_word.get_device() != dev or error_word.element_size() != 4
                                   or error_word.numel() < 1):
        raise ValueError("error_word must be a 32-bit word on cuda:%d" % dev)
    a = _PackedArgs(_ptr(q), _ptr(gate_t), _ptr(k), _ptr(v), sq, sg, sk, sv, _ptr(cu_seqlens), _ptr(cu_seqlens_k),
                    _ptr(out), _ptr(lse), Tq, Tk, cu_seqlens.numel() - 1, Hq, Hkv, D, float(scale),
                    1 if causal else 0, _ptr(error_word))
    _launch((_lib or load()).gda_prefill_packed, dev, stream, a)
    return out


def prefill_paged_workspace_bytes(total_q: int, B: int, Hq: int, Hkv: int, D: int) -> int:
    """Bytes of workspace prefill_paged needs (0 for invalid sizes)."""
    return int((_lib or load()).gda_prefill_paged_workspace_bytes(int(total_q), int(B), int(Hq), int(Hkv), int(D)))


def prefill_paged(q, gate_t, k_pool, v_pool, cu_seqlens, kv_indptr, kv_indices, *, out=None, lse=None,
                  scale: Optional[float] = None, window: int = 0, keep_first: int = 0, sinks=None, kv_scales=None,
                  k_descale: float = 1.0, v_descale: float = 1.0, workspace=None, error_word=None, stream=None):
    """Gated causal attention of each sequence's newest tokens over its rows of a paged cache, through
    ``gda_prefill_paged``: chunks of prompts behind a cached prefix, drafted tokens, single tokens.

    q, gate_t: [Tq, Hq, D] bf16 (gate_t None: out = bf16(O)), tokens any multiple of 8 elements apart;
    cu_seqlens: [B + 1] int32, each sequence's first new token (a decode step: 0, 1, .. B);
    k_pool, v_pool, kv_scales, kv_indptr, kv_indices: the cache and each sequence's positions as for
    decode, the new tokens' rows included and last (bf16 pools, e4m3 codes, or a 4-bit cache with
    kv_scales); a slot outside the pools reads as zeros and sets DEVERR_INDEX in the error word.
    A query sees the positions up to its own; with ``window`` the last ``window`` of them and the
    sequence's first ``keep_first``.  sinks: [Hq] float32 sink logits.  out: [Tq, Hq, D] contiguous
    (rows of no sequence are left as they are: zeros in an ``out`` allocated here, which is filled first);
    lse: [Hq, Tq] float32 or None; workspace: at least prefill_paged_workspace_bytes(...) bytes, 42 MB
    (None: allocated here), not shared by calls that may overlap; error_word as in prefill.
    A batch of single tokens alone goes faster through ``decode_ex`` where the cache holds codes."""
    torch = _torch()
    sq = _tokens("q", q)
    dev = q.get_device()
    Tq, Hq, D = q.shape
    sg = 0
    if gate_t is not None:
        sg = _tokens("gate", gate_t, Hq, D, dev)
        if gate_t.shape[0] != Tq:
            raise ValueError("gate must have q's shape")
    if kv_scales is not None:
        kv = KV_E2M1
        num_slots, Hkv = _check_fp4(k_pool, v_pool, kv_scales, D, dev)
    else:
        kv = _kv_dtype(k_pool)
        kdt = k_pool.dtype if kv == KV_E4M3 else torch.bfloat16
        _need("k_pool", k_pool, kdt, 3, dev)
        num_slots, Hkv, d = shape = k_pool.shape
        _need_shape("v_pool", v_pool, kdt, shape, dev, "have k_pool's shape")
        if d != D:
            raise ValueError("head dims of q and the pools differ")
    i32 = torch.int32
    _need("cu_seqlens", cu_seqlens, i32, 1, dev)
    B = cu_seqlens.numel() - 1
    if B < 0:
        raise ValueError("cu_seqlens must have B + 1 entries")
    _need_shape("kv_indptr", kv_indptr, i32, (B + 1,), dev, "have B + 1 entries, as cu_seqlens")
    _need("kv_indices", kv_indices, i32, 1, dev)
    if lse is not None:
        _need_shape("lse", lse, torch.float32, (Hq, Tq), dev, "be [Hq, Tq]")
    if sinks is not None:
        _need_shape("sinks", sinks, torch.float32, (Hq,), dev, "have Hq entries")
    if out is None:
        out = _alloc(stream, torch.zeros, Tq, Hq, D, dtype=torch.bfloat16, device=q.device)
    else:
        _need_shape("out", out, torch.bfloat16, (Tq, Hq, D), dev, "have q's shape")
    if scale is None:
        scale = 1.0 / (D ** 0.5)
    if not (0 <= window < 1 << 31 and 0 <= keep_first < 1 << 31):
        raise ValueError("window and keep_first must be numbers of positions")
    if error_word is not None and (error_word.get_device() != dev or error_word.element_size() != 4
                                   or error_word.numel() < 1):
        raise ValueError("error_word must be a 32-bit word on cuda:%d" % dev)
    if workspace is None:
        n = prefill_paged_workspace_bytes(Tq, B, Hq, Hkv, D)
        workspace = _alloc(stream, torch.empty, max(n, 256), dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on cuda:%d" % dev)
    a = _PagedArgs(_ptr(q), _ptr(gate_t), sq, sg, _ptr(k_pool), _ptr(v_pool), _ptr(kv_scales), num_slots,
                   _ptr(cu_seqlens), _ptr(kv_indptr), _ptr(kv_indices), _ptr(out), _ptr(lse), _ptr(sinks), Tq,
                   kv_indices.numel(), B, Hq, Hkv, D, float(scale), int(window), int(keep_first), kv, float(k_descale),
                   float(v_descale), _ptr(error_word))
    _launch((_lib or load()).gda_prefill_paged, dev, stream, a, workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    return out


def prefill_read_error(clear: bool = True, stream=None) -> int:
    """The library's prefill error word on the current device (synchronises)."""
    w = ctypes.c_uint32(0)
    rc = load().gda_prefill_read_error(_stream(stream), 1 if clear else 0, ctypes.byref(w))
    if rc not in (0, -9):
        _check(rc)
    return int(w.value)


def qk_norm_rope_kv_write(qgkv, slots, k_pool, v_pool, Hq: int, w_q_norm=None, w_k_norm=None, eps: float = 1e-6,
                          cos=None, sin=None, rope_dim: int = 0, q_out=None, gate_out=None, stream=None):
    """The step before attention: q_out = rope(rmsnorm(q)), the token's K row
    rope(rmsnorm(k)) and V row written into the pools at ``slots``, and the gate
    copied out.  qgkv: [B, (2 Hq + 2 Hkv) * D] bf16 rows [q | gate | k | v]."""
    import torch
    _check_tensor("qgkv", qgkv, torch.bfloat16, 2)
    dev = qgkv.device
    _check_tensor("slots", slots, torch.int32, 1, dev)
    _check_tensor("k_pool", k_pool, torch.bfloat16, 3, dev)
    _check_tensor("v_pool", v_pool, torch.bfloat16, 3, dev)
    B = qgkv.shape[0]
    num_slots, Hkv, D = k_pool.shape
    for name, t in (("w_q_norm", w_q_norm), ("w_k_norm", w_k_norm), ("cos", cos), ("sin", sin)):
        if t is not None:
            _check_tensor(name, t, torch.bfloat16, device=dev)
    if q_out is None:
        q_out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=dev)
    if gate_out is None:
        gate_out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=dev)
    _check(load().gda_qk_norm_rope_kv_write(
        _ptr(qgkv), qgkv.shape[1], _ptr(w_q_norm), _ptr(w_k_norm), float(eps), _ptr(cos), _ptr(sin),
        int(rope_dim), _ptr(slots), num_slots, _ptr(q_out), _ptr(gate_out), _ptr(k_pool), _ptr(v_pool),
        B, int(Hq), Hkv, D, _stream(stream)))
    return q_out, gate_out


def mrope_pair_axis(sections, interleaved: bool = False):
    """The axis of each rotated pair for ``sections`` (pairs per axis, e.g. of time, height
    and width): the axes' pairs one after the other, or ``interleaved``: pair i goes to
    axis i mod A while that axis has pairs left, and to axis 0 otherwise."""
    sections = [int(n) for n in sections]
    if not sections or min(sections) < 0:
        raise ValueError("sections must be counts of pairs")
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    A, total = len(sections), sum(sections)
    axis = [0] * total
    for a in range(1, A):
        if sections[a] and a + A * (sections[a] - 1) >= total:
            raise ValueError("axis %d has too many pairs to interleave" % a)
        for i in range(sections[a]):
            axis[a + A * i] = a
    return axis


def _axis_bytes(pair_axis) -> bytes:
    """One byte per pair.  (bytes() of a number is that many zeros, and of an array its memory.)"""
    try:
        return bytes(pair_axis if type(pair_axis) in (list, tuple, bytes) else list(pair_axis))
    except TypeError:
        raise TypeError("pair_axis must be a sequence of axis numbers") from None


def qk_norm_mrope_kv_write(qgkv, positions, inv_freq, pair_axis, Hq: int, Hkv: int, w_q_norm=None, w_k_norm=None,
                           eps: float = 1e-6, q_out=None, k_out=None, gate_out=None, slots=None, k_pool=None,
                           v_pool=None, kv_scales=None, k_descale: float = 1.0, v_descale: float = 1.0, stream=None):
    """The step before attention with rotary positions on several axes, through
    ``gda_qk_norm_mrope_kv_write``: returns (q_out [T, Hq, D], k_out [T, Hkv, D]).

    qgkv: [T, (2 Hq + 2 Hkv) * D] bf16 rows [q | gate | k | v] (rows may be further apart);
    positions: [A, T] int32; inv_freq: [rope_dim / 2] float32; pair_axis: a sequence of
    rope_dim / 2 axis numbers (``mrope_pair_axis``); gate_out: a [T, Hq, D] tensor to copy the
    gate into, or None.  With slots, k_pool and v_pool (bf16, or uint8 codes with kv_scales:
    a 4-bit cache) the K and V rows go into the cache too."""
    torch = _torch()
    bf16 = torch.bfloat16
    _check_rows("qgkv", qgkv)
    dev = qgkv.get_device()
    T, width = qgkv.shape
    Hq, Hkv = int(Hq), int(Hkv)
    if Hq < 1 or Hkv < 1 or width % (2 * Hq + 2 * Hkv) != 0:
        raise ValueError("qgkv's rows must hold (2 Hq + 2 Hkv) * D elements")
    D = width // (2 * Hq + 2 * Hkv)
    axis = _axis_bytes(pair_axis)
    rope_dim = 2 * len(axis)
    if rope_dim:
        _need("positions", positions, torch.int32, 2, dev)
        if positions.shape[1] != T:
            raise ValueError("positions must be [A, T]")
        _need_shape("inv_freq", inv_freq, torch.float32, (len(axis),), dev, "have rope_dim / 2 entries, as pair_axis")
        if max(axis) >= positions.shape[0]:
            raise ValueError("pair_axis names an axis that positions lacks")
    for name, t in (("w_q_norm", w_q_norm), ("w_k_norm", w_k_norm)):
        if t is not None:
            _need_shape(name, t, bf16, (D,), dev, "have D entries")
    outs, device = [], qgkv.device
    for name, t, h in (("q_out", q_out, Hq), ("k_out", k_out, Hkv), ("gate_out", gate_out, Hq)):
        if t is not None:
            _need_shape(name, t, bf16, (T, h, D), dev, "be [T, %d, D]" % h)
        elif name != "gate_out":
            t = _alloc(stream, torch.empty_strided, (T, h, D), (h * D, D, 1), dtype=bf16, device=device)
        outs.append(t)
    q_out, k_out, gate_out = outs
    num_slots, kv = 0, KV_BF16
    if k_pool is not None or v_pool is not None or slots is not None or kv_scales is not None:
        if k_pool is None or v_pool is None or slots is None:
            raise ValueError("a cache write needs slots, k_pool and v_pool")
        _need_shape("slots", slots, torch.int32, (T,), dev, "have T entries")
        if kv_scales is not None:
            kv = KV_E2M1
            num_slots, h = _check_fp4(k_pool, v_pool, kv_scales, D, dev)
        else:
            _need("k_pool", k_pool, torch.bfloat16, 3, dev)
            _need("v_pool", v_pool, torch.bfloat16, 3, dev)
            num_slots, h = k_pool.shape[0], k_pool.shape[1]
            if v_pool.shape != k_pool.shape or k_pool.shape[2] != D:
                raise ValueError("k_pool and v_pool must be [num_slots, Hkv, D]")
        if h != Hkv:
            raise ValueError("the pools must have Hkv heads")
    a = _MropeArgs(_ptr(qgkv), qgkv.stride(0) if T > 1 else width, _ptr(w_q_norm), _ptr(w_k_norm), float(eps),
                   positions.shape[0] if rope_dim else 0, _ptr(positions) if rope_dim else None,
                   T if rope_dim else 0, _ptr(inv_freq) if rope_dim else None,
                   axis, rope_dim, kv, _ptr(q_out), _ptr(gate_out),
                   _ptr(k_out), _ptr(slots), num_slots, _ptr(k_pool), _ptr(v_pool), _ptr(kv_scales), float(k_descale),
                   float(v_descale), T, Hq, Hkv, D)
    _launch((_lib or load()).gda_qk_norm_mrope_kv_write, dev, stream, a)
    return q_out, k_out


def _check_rows(name, t):
    """A 2-D bf16 CUDA tensor with contiguous rows, any distance apart."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not torch.bfloat16:
        raise TypeError("%s must be %s, got %s" % (name, torch.bfloat16, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("%s must have 2 dims and contiguous rows" % name)


def kv_write_fp4(k, v, slots, k_pool, v_pool, kv_scales, k_descale: float = 1.0, v_descale: float = 1.0, stream=None):
    """Quantise the rows of k and v ([T, Hkv, D] bf16, tokens any multiple of 8 elements apart)
    into a 4-bit cache at ``slots`` ([T] int32), through ``gda_kv_write_fp4``."""
    sk = _tokens("k", k)
    (T, Hkv, D), dev = k.shape, k.get_device()
    sv = _tokens("v", v, Hkv, D, dev)
    if v.shape[0] != T:
        raise ValueError("k and v must have the same shape")
    _need_shape("slots", slots, _th.int32, (T,), dev, "have T entries")
    num_slots, h = _check_fp4(k_pool, v_pool, kv_scales, D, dev)
    if h != Hkv:
        raise ValueError("the pools must have Hkv heads")
    _launch((_lib or load()).gda_kv_write_fp4, dev, stream, k.data_ptr(), sk, v.data_ptr(), sv, slots.data_ptr(),
            num_slots, k_pool.data_ptr(), v_pool.data_ptr(), kv_scales.data_ptr(), float(k_descale), float(v_descale),
            T, Hkv, D)


def kv_gather_fp4(k_pool, v_pool, kv_scales, indices, k_descale: float = 1.0, v_descale: float = 1.0, k_out=None,
                  v_out=None, stream=None):
    """The rows of a 4-bit cache that ``indices`` ([N] int32) name, as bf16 [N, Hkv, D] tensors
    (k, v), through ``gda_kv_gather_fp4``; an index outside the pools gives zeros."""
    torch = _torch()
    num_slots, Hkv = _check_fp4(k_pool, v_pool, kv_scales)
    dev, D, bf16 = k_pool.get_device(), 2 * k_pool.shape[2], torch.bfloat16
    _need("indices", indices, torch.int32, 1, dev)
    N = indices.numel()
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None:
            _need_shape(name, t, bf16, (N, Hkv, D), dev, "be [N, Hkv, D]")
    size, strides, device = (N, Hkv, D), (Hkv * D, D, 1), k_pool.device
    if k_out is None:
        k_out = _alloc(stream, torch.empty_strided, size, strides, dtype=bf16, device=device)
    if v_out is None:
        v_out = _alloc(stream, torch.empty_strided, size, strides, dtype=bf16, device=device)
    _launch((_lib or load()).gda_kv_gather_fp4, dev, stream, k_pool.data_ptr(), v_pool.data_ptr(),
            kv_scales.data_ptr(), num_slots, indices.data_ptr(), N, float(k_descale), float(v_descale), k_out.data_ptr(),
            v_out.data_ptr(), Hkv, D)
    return k_out, v_out


def _check_e4m3(k_pool, v_pool, dev=None):
    """Checks an e4m3 cache's pools; returns (num_slots, Hkv, D)."""
    torch = _torch()
    if not isinstance(k_pool, torch.Tensor) or k_pool.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError("k_pool must be a torch.float8_e4m3fn or torch.uint8 tensor")
    if dev is None:
        dev = _first("k_pool", k_pool, k_pool.dtype, 3)
    else:
        _need("k_pool", k_pool, k_pool.dtype, 3, dev)
    _need_shape("v_pool", v_pool, k_pool.dtype, k_pool.shape, dev, "have k_pool's shape")
    return k_pool.shape


def kv_write_e4m3(k, v, slots, k_pool, v_pool, k_descale: float = 1.0, v_descale: float = 1.0, stream=None):
    """Quantise the rows of k and v ([T, Hkv, D] bf16, tokens any multiple of 8 elements apart) into an
    e4m3 cache ([num_slots, Hkv, D] float8_e4m3fn, or uint8 codes) at ``slots`` ([T] int32), through
    ``gda_kv_write_e4m3``."""
    sk = _tokens("k", k)
    (T, Hkv, D), dev = k.shape, k.get_device()
    sv = _tokens("v", v, Hkv, D, dev)
    if v.shape[0] != T:
        raise ValueError("k and v must have the same shape")
    _need_shape("slots", slots, _th.int32, (T,), dev, "have T entries")
    num_slots, h, d = _check_e4m3(k_pool, v_pool, dev)
    if h != Hkv or d != D:
        raise ValueError("the pools must be [num_slots, Hkv, D]")
    _launch((_lib or load()).gda_kv_write_e4m3, dev, stream, k.data_ptr(), sk, v.data_ptr(), sv, slots.data_ptr(),
            num_slots, k_pool.data_ptr(), v_pool.data_ptr(), float(k_descale), float(v_descale), T, Hkv, D)


def kv_gather_e4m3(k_pool, v_pool, indices, k_descale: float = 1.0, v_descale: float = 1.0, k_out=None, v_out=None,
                   stream=None):
    """The rows of an e4m3 cache that ``indices`` ([N] int32) name, as bf16 [N, Hkv, D] tensors (k, v),
    through ``gda_kv_gather_e4m3``; an index outside the pools gives zeros."""
    torch = _torch()
    num_slots, Hkv, D = _check_e4m3(k_pool, v_pool)
    dev, bf16 = k_pool.get_device(), torch.bfloat16
    _need("indices", indices, torch.int32, 1, dev)
    N = indices.numel()
    size, strides, device = (N, Hkv, D), (Hkv * D, D, 1), k_pool.device
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None:
            _need_shape(name, t, bf16, size, dev, "be [N, Hkv, D]")
    if k_out is None:
        k_out = _alloc(stream, torch.empty_strided, size, strides, dtype=bf16, device=device)
    if v_out is None:
        v_out = _alloc(stream, torch.empty_strided, size, strides, dtype=bf16, device=device)
    _launch((_lib or load()).gda_kv_gather_e4m3, dev, stream, k_pool.data_ptr(), v_pool.data_ptr(), num_slots,
            indices.data_ptr(), N, float(k_descale), float(v_descale), k_out.data_ptr(), v_out.data_ptr(), Hkv, D)
    return k_out, v_out


def gate(o, gate_t, out=None, stream=None):
    """Standalone gate: out = bf16(o * bf16(sigmoid(gate))) element by element."""
    import torch
    _check_tensor("o", o, torch.bfloat16)
    _check_tensor("gate", gate_t, torch.bfloat16, device=o.device)
    if gate_t.shape != o.shape:
        raise ValueError("gate must have o's shape")
    if out is None:
        out = torch.empty_like(o)
    _check(load().gda_gate(_ptr(o), _ptr(gate_t), _ptr(out), o.numel(), _stream(stream)))
    return out


def timing_begin(max_calls: int):
    """Time the stage-1 kernel of the next ``max_calls`` decode calls with CUDA events."""
    _check(load().gda_timing_begin(int(max_calls)))


def timing_end():
    """(number of timed stage-1 launches, their total milliseconds); synchronises."""
    n = ctypes.c_int(0)
    ms = ctypes.c_double(0.0)
    _check(load().gda_timing_end(ctypes.byref(n), ctypes.byref(ms)))
    return int(n.value), float(ms.value)


def debug_wait_limit(cycles: int):
    """``gda_debug_wait_limit``: the pipeline wait limit (SM cycles) of later calls;
    a short limit makes the waiting kernels take their timeout path (failure-path
    tests only); ``cycles <= 0`` restores the default."""
    _check(load().gda_debug_wait_limit(int(cycles)))


def read_error(workspace=None, clear: bool = True, stream=None) -> int:
    """The device error word of a workspace (or of the internal one); synchronises."""
    w = ctypes.c_uint32(0)
    ptr = ctypes.c_void_p(workspace.data_ptr()) if workspace is not None else None
    rc = load().gda_read_error(ptr, _stream(stream), 1 if clear else 0, ctypes.byref(w))
    if rc not in (0, -9):
        _check(rc)
    return int(w.value)

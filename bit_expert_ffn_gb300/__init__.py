"""GB300 (sm_103a) routed-expert MoE layer with 2-/3-bit block-quantised experts.

This module is the Python binding of ``libmoe_gb300.so``: every function
named ``moe_*`` here marshals torch tensors into the C call of the same name
declared in ``include/moe_gb300.h`` and raises :class:`MoeError` on a non-OK
status.  All arithmetic runs in the library's CUDA kernels; there is no other
code path, and importing a function of this module without the built library
raises at once.  Tensors are passed by device pointer and work is enqueued on
the current torch CUDA stream.
"""
from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_gb300.so")
SYNTH_PATH = os.path.join(HERE, "libmoe_synth.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "moe_gb300.h")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE = 0, 1, 2, 3
MOE_ERR_CUDA, MOE_ERR_TIMEOUT, MOE_ERR_NONFINITE, MOE_ERR_BOUNDS = 4, 5, 6, 7
MOE_ERR_RANGE = 8
MOE_ID_NOT_LOCAL = -1
MOE_F32, MOE_BF16, MOE_F16 = 0, 1, 2
MOE_PATH_AUTO, MOE_PATH_DECODE, MOE_PATH_PREFILL, MOE_PATH_PREFILL_FP8 = 0, 1, 2, 3
MOE_MX4_PLAIN, MOE_MX4_SWIGLU = 0, 1
MOE_GATE_NONE, MOE_GATE_TOKEN, MOE_GATE_CHANNEL = 0, 1, 2
RMS_EPS = 1e-6  # normalisation in front of each stacked layer

_lock = threading.Lock()
_lib = None
_synth = None


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class moe_expert_arena(ctypes.Structure):
    _fields_ = [
        ("bits", ctypes.c_int32),
        ("H", ctypes.c_int32),
        ("I", ctypes.c_int32),
        ("E", ctypes.c_int32),
        ("gu_codes", ctypes.c_void_p),
        ("gu_scales", ctypes.c_void_p),
        ("d_codes", ctypes.c_void_p),
        ("d_scales", ctypes.c_void_p),
    ]


class moe_layer_weights(ctypes.Structure):
    _fields_ = [
        ("experts", moe_expert_arena),
        ("w_router", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
        ("shared_wg", ctypes.c_void_p),
        ("shared_wu", ctypes.c_void_p),
        ("shared_wd", ctypes.c_void_p),
        ("shared_I", ctypes.c_int32),
    ]


class moe_decode_options(ctypes.Structure):
    _fields_ = [
        ("route_tail_skip", ctypes.c_int32),
        ("hot_experts", ctypes.c_void_p),
    ]


class moe_adamw_tensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("master", ctypes.c_void_p),
        ("m", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("n", ctypes.c_int64),
        ("param_dtype", ctypes.c_int32),
        ("grad_dtype", ctypes.c_int32),
        ("lr_factor", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
    ]


class moe_adamw_options(ctypes.Structure):
    """lr, beta1, beta2, eps, step; and device addresses lr_dev (fp32), step_dev (int64), grad_scale (fp32) or None."""

    _fields_ = [
        ("lr", ctypes.c_double),
        ("beta1", ctypes.c_double),
        ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double),
        ("step", ctypes.c_int64),
        ("lr_dev", ctypes.c_void_p),
        ("step_dev", ctypes.c_void_p),
        ("grad_scale", ctypes.c_void_p),
    ]


_P = ctypes.c_void_p
_I32 = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_PSZ = ctypes.POINTER(ctypes.c_size_t)

# name -> argtypes (restype moe_status = int unless noted)
_SIGS = {
    "moe_check_status": [_P, _I32, _P],
    "moe_packed_size": [_I32, _I64, _I64, _PSZ, _PSZ],
    "moe_pack_experts": [_I32, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P],
    "moe_unpack_experts": [_I32, _I64, _I64, _I64, _P, _P, _P],
    "moe_router_workspace_size": [_I32, _I32, _I32, _I32, _PSZ],
    "moe_router_topk": [_P, _I32, _I32, _P, _P, _I32, _I32, _P, _P, _P, _P, _SZ, _P, _P],
    "moe_topk_from_logits": [_P, _I32, _I32, _I32, _P, _P, _P, _P],
    "moe_permute_workspace_size": [_I32, _I32, _I32, _PSZ],
    "moe_shard_ids": [_P, _I64, _I32, _I32, _P, _P],
    "moe_permute": [_P, _I32, _I32, _I32, _P, _P, _P, _P, _SZ, _P, _P],
    "moe_permute_noalloc": [_P, _I32, _I32, _I32, _P, _P, _P, _P, _P],
    "moe_expert_forward_workspace_size": [ctypes.POINTER(moe_expert_arena), _I32, _I32, _I32, _PSZ],
    "moe_expert_forward": [ctypes.POINTER(moe_expert_arena), _P, _I32, _P, _P, _I32, _P, _P, _P, _P, _I32, _I32,
                           _I32, _P, _SZ, _P, _P],
    "moe_shared_expert_workspace_size": [_I32, _I32, _I32, _PSZ],
    "moe_shared_expert": [_P, _P, _P, _I32, _I32, _P, _I32, _P, _I32, _I32, _P, _SZ, _P, _P],
    "moe_f32_to_bf16": [_P, _P, _I64, _P],
    "moe_decode_workspace_size": [_I32, _I32, _I32, _I32, _I32, _I32, _PSZ],
    "moe_decode_forward": [ctypes.POINTER(moe_layer_weights), _I32, _P, _I32, _I32, ctypes.c_float, _P, _P, _P, _SZ,
                           _P, _P],
    "moe_decode_forward_ex": [ctypes.POINTER(moe_layer_weights), _I32, _P, _I32, _I32, ctypes.c_float,
                              ctypes.POINTER(moe_decode_options), _P, _P, _P, _SZ, _P, _P],
    "moe_rms_norm_bf16": [_P, _P, _I32, _I32, ctypes.c_float, _P],
    "moe_selftest_barrier": [ctypes.c_uint, _I32, _P, _SZ, _P, _P],
    "moe_dispatch": [_P, _I32, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P],
    "moe_dispatch_backward": [_P, _I32, _I32, _I32, _I32, _P, _P, _P],
    "moe_combine": [_P, _I32, _I32, _I32, _I32, _P, _P, _P, _I32, _I32, _P],
    "moe_combine_backward": [_P, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P],
    "moe_mx4_size": [_I64, _I64, _PSZ, _PSZ],
    "moe_mx4_quantise": [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _P],
    "moe_mx4_dequantise": [_P, _P, _I64, _I64, _P, _I32, _P],
    "moe_mx4_matmul": [_P, _P, _I32, _I32, _I32, _P, _P, _I32, _P, _P, _I32, _I32, _P, _P],
    "moe_block_norm": [_P, _I32, _I64, _P, _I32, _I64, _I32, _I32, _P, _P, _P, _I32, ctypes.c_float, ctypes.c_float, _P,
                       _P, _P],
    "moe_block_norm_backward_workspace_size": [_I32, _I32, _I32, _PSZ],
    "moe_block_norm_backward": [_P, _I32, _I64, _P, _I32, _I64, _I32, _I32, _P, _P, _P, _I32, ctypes.c_float,
                                ctypes.c_float, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P],
    "moe_router_loss_workspace_size": [_I32, _I32, _PSZ],
    "moe_router_loss": [_P, _I32, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P, _P],
    "moe_router_loss_backward": [_P, _I32, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _P],
    "moe_cross_entropy_workspace_size": [_I32, _I32, _I32, _PSZ],
    "moe_cross_entropy": [_P, _I32, _I32, _I32, _P, _I32, _P, _P, _P, _P, _SZ, _P, _P],
    "moe_cross_entropy_backward_workspace_size": [_I32, _I32, _I32, _PSZ],
    "moe_cross_entropy_backward": [_P, _I32, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _I32, _I32, _P, _SZ, _P, _P],
    "moe_adamw_step": [ctypes.POINTER(moe_adamw_tensor), _I32, ctypes.POINTER(moe_adamw_options), _P, _P],
    "moe_adamw_states": [ctypes.POINTER(moe_adamw_tensor), _I32, ctypes.POINTER(_P), ctypes.POINTER(_P), _P],
}


def load():
    """Load libmoe_gb300.so (and the input generator library); raise if it is not built."""
    global _lib, _synth
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise MoeError(MOE_ERR_CUDA, f"{LIB_PATH} is not built: run `python -m bit_expert_ffn_gb300.build`")
            L = ctypes.CDLL(LIB_PATH)
            for name, args in _SIGS.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = ctypes.c_int
            L.moe_last_error.restype = ctypes.c_char_p
            L.moe_last_error.argtypes = []
            L.moe_status_name.restype = ctypes.c_char_p
            L.moe_status_name.argtypes = [ctypes.c_int]
            _lib = L
        if _synth is None and os.path.exists(SYNTH_PATH):
            S = ctypes.CDLL(SYNTH_PATH)
            S.moe_synth_codes.argtypes = [ctypes.c_uint64, ctypes.c_uint64, _I64, _I32, _P, _P]
            S.moe_synth_codes.restype = ctypes.c_int
            S.moe_synth_normal.argtypes = [ctypes.c_uint64, ctypes.c_uint64, _I64, ctypes.c_float, ctypes.c_float,
                                           _I32, _P, _P]
            S.moe_synth_normal.restype = ctypes.c_int
            _synth = S
    return _lib


def lib():
    return _lib if _lib is not None else load()


def synth_lib():
    load()
    if _synth is None:
        raise MoeError(MOE_ERR_CUDA, f"{SYNTH_PATH} is not built")
    return _synth


def moe_last_error() -> str:
    return lib().moe_last_error().decode()


def moe_status_name(s: int) -> str:
    return lib().moe_status_name(int(s)).decode()


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoeError(status, f"{what}: {moe_last_error()}")


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr() if t.numel() else None


_INT32, _BYTE = "int32", "uint8"  # element kinds of _packed, beside the moe_dtypes


class _Kinds(dict):
    """Element kind -> the torch types that hold it (the calls also take 16-bit values as bit patterns)."""

    def __missing__(self, kind):
        import torch

        bits = (torch.int16, torch.uint16)
        small = [getattr(torch, n) for n in ("float8_e8m0fnu", "float4_e2m1fn_x2") if hasattr(torch, n)]
        self.update({MOE_F32: (torch.float32,), MOE_BF16: (torch.bfloat16, *bits), MOE_F16: (torch.float16, *bits),
                     _INT32: (torch.int32,), _BYTE: (torch.uint8, torch.int8, *small)})
        return self.get(kind, ())


_KINDS = _Kinds()


class _Host:
    """In an address's place: a tensor that is not on the GPU.  It cannot be passed, and _call reports it, by which time
    the other arguments are known to be of the right types and sizes."""

    def __init__(self, name, t):
        self.what = f"{name} must be on the GPU (got a tensor on {t.device})"


def _packed(t, name, n, kind):
    """The pointer of a packed buffer of at least n elements of a kind (a tensor), or of a raw address."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype in _KINDS[kind] and t.is_contiguous() and t.numel() >= n:
        return (t.data_ptr() if t.is_cuda else _Host(name, t)) if n else None
    want = " or ".join(str(d)[6:] for d in _KINDS[kind]) or f"dtype {kind}"
    raise MoeError(MOE_ERR_INVALID_ARG, f"{name} must be a packed tensor of at least {n} elements of {want} "
                                        f"(got {tuple(t.shape)}, strides {t.stride()}, {t.dtype})")


def _rows(t, name, n, cols, dtype):
    """Pointer and row stride of n rows of `cols` elements: a packed tensor, a 2D one whose rows are packed (stride 0
    repeats one row), or a raw address of packed rows."""
    if t is None or t.__class__ is int:
        return t, cols
    if t.dtype in _KINDS[dtype]:
        if t.is_contiguous():
            if t.numel() >= n * cols:
                return (t.data_ptr() if t.is_cuda else _Host(name, t)) if n else None, cols
        elif t.dim() == 2 and t.shape[0] >= n and t.shape[1] == cols and (t.stride(1) == 1 or cols == 1):
            return (t.data_ptr() if t.is_cuda else _Host(name, t)) if n else None, t.stride(0) if n > 1 else cols
    return _packed(t, name, n * cols, dtype), cols


def _workspace(t, size):
    """The pointer of a workspace said to hold `size` bytes (a tensor of any type), or of a raw address."""
    if t is None or t.__class__ is int:
        return t
    if t.is_contiguous() and t.numel() * t.element_size() >= size:
        return (t.data_ptr() if t.is_cuda else _Host("ws", t)) if size else None
    raise MoeError(MOE_ERR_INVALID_ARG, f"ws must be a packed tensor of at least ws_bytes = {size} bytes "
                                        f"(got {tuple(t.shape)}, strides {t.stride()}, {t.dtype})")


_raw_stream = None  # torch's current stream handle of a device, and the current device, once a GPU is there


def _stream(stream=None):
    """The stream handle: an int, a torch stream, or the current torch stream."""
    global _raw_stream
    if stream is None:
        if _raw_stream is not None:  # (torch.cuda.current_stream() without its Stream object: 0.3 against 3 us)
            return _raw_stream[0](_raw_stream[1]())
        import torch

        if not torch.cuda.is_available():  # host-side argument checks still run
            return 0
        stream = torch.cuda.current_stream()
        fns = [getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice")]
        if None not in fns:
            _raw_stream = fns
    return stream if isinstance(stream, int) else stream.cuda_stream


def _call(fn, *args):
    try:
        status = fn(*args)
    except ctypes.ArgumentError:
        for a in args:
            if a.__class__ is _Host:
                raise MoeError(MOE_ERR_INVALID_ARG, f"{fn.__name__}: {a.what}") from None
        raise
    if status:
        _check(status, fn.__name__)


def _size(fn, *args) -> int:
    out = ctypes.c_size_t(0)
    _check(fn(*args, ctypes.byref(out)), fn.__name__)
    return out.value


# ----------------------------------------------------------------- status

def moe_check_status(dev_status, reset=True, stream=None) -> int:
    """Synchronise and read the device status word; returns the status (no raise)."""
    return lib().moe_check_status(_ptr(dev_status), int(reset), _stream(stream))


# ----------------------------------------------------------------- packing

def moe_packed_size(bits: int, rows: int, cols: int):
    cb, sb = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().moe_packed_size(bits, rows, cols, ctypes.byref(cb), ctypes.byref(sb)), "moe_packed_size")
    return cb.value, sb.value


def moe_pack_experts(bits, n_mats, rows, cols, codes, scales, packed_codes, packed_scales, dev_status=None,
                     stream=None):
    _check(lib().moe_pack_experts(bits, n_mats, rows, cols, _ptr(codes), _ptr(scales), _ptr(packed_codes),
                                  _ptr(packed_scales), _ptr(dev_status), _stream(stream)), "moe_pack_experts")


def moe_unpack_experts(bits, n_mats, rows, cols, packed_codes, codes, stream=None):
    _check(lib().moe_unpack_experts(bits, n_mats, rows, cols, _ptr(packed_codes), _ptr(codes), _stream(stream)),
           "moe_unpack_experts")


# ----------------------------------------------------------------- router

def moe_router_workspace_size(T, H, E, logits_given):
    return _size(lib().moe_router_workspace_size, T, H, E, int(logits_given))


def moe_router_topk(x_bf16, T, H, w_router, bias, E, k, logits_out, topk_ids, topk_w, ws=None, ws_bytes=0,
                    dev_status=None, stream=None):
    _check(lib().moe_router_topk(_ptr(x_bf16), T, H, _ptr(w_router), _ptr(bias), E, k, _ptr(logits_out),
                                 _ptr(topk_ids), _ptr(topk_w), _ptr(ws), ws_bytes, _ptr(dev_status), _stream(stream)),
           "moe_router_topk")


def moe_topk_from_logits(logits, T, E, k, ids, w, dev_status=None, stream=None):
    _check(lib().moe_topk_from_logits(_ptr(logits), T, E, k, _ptr(ids), _ptr(w), _ptr(dev_status), _stream(stream)),
           "moe_topk_from_logits")


# ----------------------------------------------------------------- permute

def moe_permute_workspace_size(T, k, E):
    return _size(lib().moe_permute_workspace_size, T, k, E)


def moe_permute(ids, T, k, E, offsets, perm, inv_perm, ws=None, ws_bytes=0, dev_status=None, stream=None):
    _check(lib().moe_permute(_ptr(ids), T, k, E, _ptr(offsets), _ptr(perm), _ptr(inv_perm), _ptr(ws), ws_bytes,
                             _ptr(dev_status), _stream(stream)), "moe_permute")


def moe_shard_ids(ids, n, e0, e_count, local_ids, stream=None):
    """ids of the shard holding experts [e0, e0 + e_count): local id, or MOE_ID_NOT_LOCAL for other shards."""
    _check(lib().moe_shard_ids(_ptr(ids), n, e0, e_count, _ptr(local_ids), _stream(stream)), "moe_shard_ids")


def moe_permute_noalloc(ids, T, k, E, offsets, perm, inv_perm, dev_status=None, stream=None):
    """moe_permute without a workspace, for callers that cannot allocate (see the header)."""
    _check(lib().moe_permute_noalloc(_ptr(ids), T, k, E, _ptr(offsets), _ptr(perm), _ptr(inv_perm), _ptr(dev_status),
                                     _stream(stream)), "moe_permute_noalloc")


# ----------------------------------------------------------------- experts

def make_arena(bits, H, I, E, gu_codes, gu_scales, d_codes, d_scales) -> moe_expert_arena:
    return moe_expert_arena(bits, H, I, E, _ptr(gu_codes), _ptr(gu_scales), _ptr(d_codes), _ptr(d_scales))


def moe_expert_forward_workspace_size(arena: moe_expert_arena, T, k, path=MOE_PATH_AUTO):
    return _size(lib().moe_expert_forward_workspace_size, ctypes.byref(arena), T, k, path)


def moe_expert_forward(arena: moe_expert_arena, x_bf16, T, ids, w, k, offsets, perm, inv_perm, out, out_dtype=MOE_F32,
                       accumulate=False, path=MOE_PATH_AUTO, ws=None, ws_bytes=0, dev_status=None, stream=None):
    _check(lib().moe_expert_forward(ctypes.byref(arena), _ptr(x_bf16), T, _ptr(ids), _ptr(w), k, _ptr(offsets),
                                    _ptr(perm), _ptr(inv_perm), _ptr(out), out_dtype, int(accumulate), path, _ptr(ws),
                                    ws_bytes, _ptr(dev_status), _stream(stream)), "moe_expert_forward")


def moe_shared_expert_workspace_size(H, I, T):
    return _size(lib().moe_shared_expert_workspace_size, H, I, T)


def moe_shared_expert(wg, wu, wd, H, I, x_bf16, T, out, out_dtype=MOE_F32, accumulate=False, ws=None, ws_bytes=0,
                      dev_status=None, stream=None):
    _check(lib().moe_shared_expert(_ptr(wg), _ptr(wu), _ptr(wd), H, I, _ptr(x_bf16), T, _ptr(out), out_dtype,
                                   int(accumulate), _ptr(ws), ws_bytes, _ptr(dev_status), _stream(stream)),
           "moe_shared_expert")


def moe_f32_to_bf16(in_f32, out_bf16, n, stream=None):
    _check(lib().moe_f32_to_bf16(_ptr(in_f32), _ptr(out_bf16), n, _stream(stream)), "moe_f32_to_bf16")


def moe_decode_workspace_size(T, H, I, E, k, shared_I):
    return _size(lib().moe_decode_workspace_size, T, H, I, E, k, shared_I)


def moe_decode_forward(layers, x, T, k, rms_eps=RMS_EPS, ids_out=None, w_out=None, ws=None, ws_bytes=0,
                       dev_status=None, stream=None):
    """layers: a sequence of moe_layer_weights (host); x: [T][H] fp32 device tensor, updated in place."""
    arr = (moe_layer_weights * len(layers))(*layers)
    _check(lib().moe_decode_forward(arr, len(layers), _ptr(x), T, k, rms_eps, _ptr(ids_out), _ptr(w_out), _ptr(ws),
                                    ws_bytes, _ptr(dev_status), _stream(stream)), "moe_decode_forward")


def moe_decode_forward_ex(layers, x, T, k, rms_eps=RMS_EPS, route_tail_skip=0, hot_experts=None, ids_out=None,
                          w_out=None, ws=None, ws_bytes=0, dev_status=None, stream=None):
    """moe_decode_forward with options: route_tail_skip (rank threshold, 0 = off) and hot_experts (a device
    uint32 tensor [n_layers][(E + 31) // 32] of bit masks, or None)."""
    arr = (moe_layer_weights * len(layers))(*layers)
    opts = moe_decode_options(int(route_tail_skip), _ptr(hot_experts))
    _check(lib().moe_decode_forward_ex(arr, len(layers), _ptr(x), T, k, rms_eps, ctypes.byref(opts), _ptr(ids_out),
                                       _ptr(w_out), _ptr(ws), ws_bytes, _ptr(dev_status), _stream(stream)),
           "moe_decode_forward_ex")


def moe_rms_norm_bf16(x, out, T, H, eps=None, stream=None):
    _check(lib().moe_rms_norm_bf16(_ptr(x), _ptr(out), T, H, RMS_EPS if eps is None else eps, _stream(stream)),
           "moe_rms_norm_bf16")


def moe_selftest_barrier(extra_arrivals, timeout_ms, ws, ws_bytes, dev_status=None, stream=None):
    _check(lib().moe_selftest_barrier(extra_arrivals, timeout_ms, _ptr(ws), ws_bytes, _ptr(dev_status),
                                      _stream(stream)), "moe_selftest_barrier")


# ----------------------------------------------------------------- rows to their experts and back

def moe_dispatch(x, dtype, T, H, k, E, offsets, inv_perm, out, stream=None):
    """out[inv_perm[t, j]] = x[t]; rows of no pair are zero.  x: [T][H], packed rows at any row stride."""
    xp, xs = _rows(x, "x", T, H, dtype)
    _call((_lib or load()).moe_dispatch, xp, dtype, xs, T, H, k, E, _packed(offsets, "offsets", E + 1, _INT32),
          _packed(inv_perm, "inv_perm", T * k, _INT32), _packed(out, "out", T * k * H, dtype), _stream(stream))


def moe_dispatch_backward(drows, dtype, T, H, k, inv_perm, dx, stream=None):
    """dx[t] = sum_j drows[inv_perm[t, j]]."""
    _call((_lib or load()).moe_dispatch_backward, _packed(drows, "drows", T * k * H, dtype), dtype, T, H, k,
          _packed(inv_perm, "inv_perm", T * k, _INT32), _packed(dx, "dx", T * H, dtype), _stream(stream))


def moe_combine(y, dtype, T, H, k, w, inv_perm, out, out_dtype=MOE_F32, accumulate=False, stream=None):
    """out[t] (+)= sum_j w[t, j] * y[inv_perm[t, j]]."""
    _call((_lib or load()).moe_combine, _packed(y, "y", T * k * H, dtype), dtype, T, H, k, _packed(w, "w", T * k, MOE_F32),
          _packed(inv_perm, "inv_perm", T * k, _INT32), _packed(out, "out", T * H, out_dtype), out_dtype, int(accumulate),
          _stream(stream))


def moe_combine_backward(dout, y, dtype, T, H, k, E, offsets, w, inv_perm, dy, dw, stream=None):
    """dy[inv_perm[t, j]] = w[t, j] * dout[t], dw[t, j] = <dout[t], y[inv_perm[t, j]]>."""
    _call((_lib or load()).moe_combine_backward, _packed(dout, "dout", T * H, dtype), _packed(y, "y", T * k * H, dtype),
          dtype, T, H, k, E, _packed(offsets, "offsets", E + 1, _INT32), _packed(w, "w", T * k, MOE_F32),
          _packed(inv_perm, "inv_perm", T * k, _INT32), _packed(dy, "dy", T * k * H, dtype), _packed(dw, "dw", T * k, MOE_F32),
          _stream(stream))


# ----------------------------------------------------------------- 4-bit floating point matrices

def moe_mx4_size(rows: int, cols: int):
    """(bytes of codes, bytes of scales) of a [rows][cols] matrix; cols a multiple of 32."""
    cb, sb = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check((_lib or load()).moe_mx4_size(rows, cols, ctypes.byref(cb), ctypes.byref(sb)), "moe_mx4_size")
    return cb.value, sb.value


def _mx4(codes, codes_name, scales, scales_name, rows, cols):
    return (_packed(codes, codes_name, rows * (cols // 2), _BYTE),
            _packed(scales, scales_name, rows * ((cols + 1023) // 1024) * 32, _BYTE))


def moe_mx4_quantise(x, dtype, rows, cols, codes, scales, dev_status=None, stream=None):
    """x [rows][cols] (rows packed, any row stride) to e2m1 codes and e8m0 scales (uint8 tensors of moe_mx4_size)."""
    xp, xs = _rows(x, "x", rows, cols, dtype)
    cp, sp = _mx4(codes, "codes", scales, "scales", rows, cols)
    _call((_lib or load()).moe_mx4_quantise, xp, dtype, xs, rows, cols, cp, sp, _packed(dev_status, "dev_status", 1, _INT32),
          _stream(stream))


def moe_mx4_dequantise(codes, scales, rows, cols, out, dtype=MOE_BF16, stream=None):
    """The values that codes and scales stand for."""
    cp, sp = _mx4(codes, "codes", scales, "scales", rows, cols)
    _call((_lib or load()).moe_mx4_dequantise, cp, sp, rows, cols, _packed(out, "out", rows * cols, dtype), dtype,
          _stream(stream))


def moe_mx4_matmul(w_codes, w_scales, E, N, K, x_codes, x_scales, rows, offsets, out, out_dtype=MOE_F32,
                   epilogue=MOE_MX4_PLAIN, dev_status=None, stream=None):
    """out[p] = x[p] W_e^T (or silu(gate) * up of it) for the rows p of each group e; offsets None: one group (E = 1)."""
    wc, ws = _mx4(w_codes, "w_codes", w_scales, "w_scales", E * N * (2 if epilogue == MOE_MX4_SWIGLU else 1), K)
    xc, xs = _mx4(x_codes, "x_codes", x_scales, "x_scales", rows, K)
    _call((_lib or load()).moe_mx4_matmul, wc, ws, E, N, K, xc, xs, rows, _packed(offsets, "offsets", E + 1, _INT32),
          _packed(out, "out", rows * N, out_dtype), out_dtype, epilogue, _packed(dev_status, "dev_status", 1, _INT32),
          _stream(stream))


# ----------------------------------------------------------------- norms around a block

def _gate_size(gate_kind, T, H):
    return T if gate_kind == MOE_GATE_TOKEN else H


def moe_block_norm(x, res_dtype, b, dtype, T, H, w_post, w_pre, gate, gate_kind, alpha, eps, y, u, stream=None):
    """y = x + alpha * gate * w_post * rmsnorm(b), u = w_pre * rmsnorm(y).  x and b: packed rows at any row stride."""
    xp, xs = _rows(x, "x", T, H, res_dtype)
    bp, bs = _rows(b, "b", T, H, dtype)
    _call((_lib or load()).moe_block_norm, xp, res_dtype, xs, bp, dtype, bs, T, H, _packed(w_post, "w_post", H, MOE_F32),
          _packed(w_pre, "w_pre", H, MOE_F32), _packed(gate, "gate", _gate_size(gate_kind, T, H), MOE_F32), gate_kind, alpha,
          eps, _packed(y, "y", T * H, res_dtype), _packed(u, "u", T * H, dtype), _stream(stream))


def moe_block_norm_backward_workspace_size(T, H, gate_kind=MOE_GATE_NONE):
    return _size((_lib or load()).moe_block_norm_backward_workspace_size, T, H, gate_kind)


def moe_block_norm_backward(x, res_dtype, b, dtype, T, H, w_post, w_pre, gate, gate_kind, alpha, eps, dy, du, dx, db,
                            dw_post=None, dw_pre=None, dgate=None, ws=None, ws_bytes=0, stream=None):
    """Gradients of moe_block_norm for dy and du (either may be None)."""
    xp, xs = _rows(x, "x", T, H, res_dtype)
    bp, bs = _rows(b, "b", T, H, dtype)
    n = _gate_size(gate_kind, T, H)
    _call((_lib or load()).moe_block_norm_backward, xp, res_dtype, xs, bp, dtype, bs, T, H,
          _packed(w_post, "w_post", H, MOE_F32), _packed(w_pre, "w_pre", H, MOE_F32), _packed(gate, "gate", n, MOE_F32),
          gate_kind, alpha, eps,
          _packed(dy, "dy", T * H, res_dtype), _packed(du, "du", T * H, dtype), _packed(dx, "dx", T * H, res_dtype),
          _packed(db, "db", T * H, dtype), _packed(dw_post, "dw_post", H, MOE_F32), _packed(dw_pre, "dw_pre", H, MOE_F32),
          _packed(dgate, "dgate", n, MOE_F32), _workspace(ws, ws_bytes), ws_bytes, _stream(stream))


# ----------------------------------------------------------------- the router's losses

def moe_router_loss_workspace_size(T, E):
    return _size((_lib or load()).moe_router_loss_workspace_size, T, E)


def moe_router_loss(logits, dtype, T, E, ids, k, keep, loss, counts, mean_prob, lse, ws=None, ws_bytes=0, dev_status=None,
                    stream=None):
    """loss[0] = E sum_e f_e P_e, loss[1] = mean lse^2, counts [E + 1] (the last: tokens that count), mean_prob [E], lse [T].
    keep: bytes or truth values [T], or None."""
    if keep is not None and keep.__class__ is not int and str(keep.dtype) == "torch.bool":
        import torch

        keep = keep.view(torch.uint8)
    _call((_lib or load()).moe_router_loss, _packed(logits, "logits", T * E, dtype), dtype, T, E,
          _packed(ids, "ids", T * k, _INT32), k, _packed(keep, "keep", T, _BYTE), _packed(loss, "loss", 2, MOE_F32),
          _packed(counts, "counts", E + 1, _INT32), _packed(mean_prob, "mean_prob", E, MOE_F32),
          _packed(lse, "lse", T, MOE_F32), _workspace(ws, ws_bytes), ws_bytes, _packed(dev_status, "dev_status", 1, _INT32),
          _stream(stream))


def moe_router_loss_backward(logits, dtype, T, E, ids, k, counts, lse, dloss, w, dw, dlogits, stream=None):
    """dlogits from dloss [2] (or None) and from the routing weights' gradient dw (w and dw, or both None)."""
    _call((_lib or load()).moe_router_loss_backward, _packed(logits, "logits", T * E, dtype), dtype, T, E,
          _packed(ids, "ids", T * k, _INT32), k, _packed(counts, "counts", E + 1, _INT32), _packed(lse, "lse", T, MOE_F32),
          _packed(dloss, "dloss", 2, MOE_F32), _packed(w, "w", T * k, MOE_F32), _packed(dw, "dw", T * k, MOE_F32),
          _packed(dlogits, "dlogits", T * E, dtype), _stream(stream))


# ----------------------------------------------------------------- cross entropy over a vocabulary

def moe_cross_entropy_workspace_size(T, H, V):
    return _size((_lib or load()).moe_cross_entropy_workspace_size, T, H, V)


def moe_cross_entropy(h, dtype, T, H, w, V, labels, loss, lse, ws=None, ws_bytes=0, dev_status=None, stream=None):
    """loss[t] = lse[t] - z[t, labels[t]] of z = h w^T, h [T][H], w [V][H]; labels int32, negative: left out."""
    _call((_lib or load()).moe_cross_entropy, _packed(h, "h", T * H, dtype), dtype, T, H, _packed(w, "w", V * H, dtype), V,
          _packed(labels, "labels", T, _INT32), _packed(loss, "loss", T, MOE_F32), _packed(lse, "lse", T, MOE_F32),
          _workspace(ws, ws_bytes), ws_bytes, _packed(dev_status, "dev_status", 1, _INT32), _stream(stream))


def moe_cross_entropy_backward_workspace_size(T, H, V):
    return _size((_lib or load()).moe_cross_entropy_backward_workspace_size, T, H, V)


def moe_cross_entropy_backward(h, dtype, T, H, w, V, labels, lse, dloss, dlse, dh, dw, dw_dtype=None, accumulate=False, ws=None,
                               ws_bytes=0, dev_status=None, stream=None):
    """dh and dw (either may be None) for dloss [T] and dlse [T] (or None); dw_dtype: dtype (the default) or MOE_F32."""
    wt = dtype if dw_dtype is None else dw_dtype
    _call((_lib or load()).moe_cross_entropy_backward, _packed(h, "h", T * H, dtype), dtype, T, H,
          _packed(w, "w", V * H, dtype), V, _packed(labels, "labels", T, _INT32), _packed(lse, "lse", T, MOE_F32),
          _packed(dloss, "dloss", T, MOE_F32), _packed(dlse, "dlse", T, MOE_F32), _packed(dh, "dh", T * H, dtype),
          _packed(dw, "dw", V * H, wt), wt, int(accumulate), _workspace(ws, ws_bytes), ws_bytes,
          _packed(dev_status, "dev_status", 1, _INT32), _stream(stream))


# ----------------------------------------------------------------- AdamW

class AdamwTensors:
    """The tensors of moe_adamw_step and moe_adamw_states: made once, used every step (make_adamw_tensors)."""

    def __init__(self, array, held):
        self.array, self.held = array, held  # (the torch tensors stay alive with their addresses)
        self.sizes = [a.n for a in array]

    def __len__(self):
        return len(self.array)


def _moe_dtype(t, name):
    for d in (MOE_F32, MOE_BF16, MOE_F16):
        if t.dtype == _KINDS[d][0]:
            return d
    raise MoeError(MOE_ERR_INVALID_ARG, f"{name} must be of float32, bfloat16 or float16 (got {t.dtype})")


def make_adamw_tensors(tensors) -> AdamwTensors:
    """tensors: dicts of torch tensors param, grad, m, v and, where there are, master (fp32) and scales (fp32 [ceil(n / 256)][2]:
    m and v are then uint8), with lr_factor (1) and weight_decay (0)."""
    array, ranges, host = (moe_adamw_tensor * len(tensors))(), [], None
    for i, d in enumerate(tensors):
        unknown = set(d) - {"param", "grad", "master", "m", "v", "scales", "lr_factor", "weight_decay"}
        if unknown or any(d.get(k) is None for k in ("param", "grad", "m", "v")):
            raise MoeError(MOE_ERR_INVALID_ARG, f"tensor {i}: param, grad, m and v are needed, beside them master, scales, "
                                                f"lr_factor and weight_decay (got {sorted(d)})")
        n, a = d["param"].numel(), array[i]
        held = d.get("scales") is not None
        kinds = {"param": _moe_dtype(d["param"], f"tensor {i}: param"), "grad": _moe_dtype(d["grad"], f"tensor {i}: grad"),
                 "master": MOE_F32, "m": _BYTE if held else MOE_F32, "v": _BYTE if held else MOE_F32, "scales": MOE_F32}
        for name, kind in kinds.items():
            t = d.get(name)
            if t is None:
                continue
            want = (n + 255) // 256 * 2 if name == "scales" else n
            if t.dtype in _KINDS[kind] and t.numel() == want and t.is_cuda and t.is_contiguous():
                p = t.data_ptr()
            else:  # (says what is wrong; a step has hundreds of tensors, and the messages' names take their time)
                p = _packed(t, f"tensor {i}: {name}", want, kind)
                if t.numel() != want:
                    raise MoeError(MOE_ERR_INVALID_ARG, f"tensor {i}: {name} must have {want} elements (got {t.numel()})")
                host = host or p
                p = t.data_ptr()
            if want:
                setattr(a, name, p)
                ranges.append((p, p + want * t.element_size(), name != "grad", i, name))
        a.n, a.param_dtype, a.grad_dtype = n, kinds["param"], kinds["grad"]
        a.lr_factor, a.weight_decay = d.get("lr_factor", 1.0), d.get("weight_decay", 0.0)
    end = {True: (0, 0, ""), False: (0, 0, "")}  # how far what is written, and what is read, has come
    for lo, hi, written, i, name in sorted(ranges):
        for other in ((True, False) if written else (True,)):
            if lo < end[other][0]:
                raise MoeError(MOE_ERR_INVALID_ARG, "tensor %d: %s overlaps tensor %d: %s" % (i, name, *end[other][1:]))
        end[written] = max(end[written], (hi, i, name))
    if host:
        raise MoeError(MOE_ERR_INVALID_ARG, host.what)
    return AdamwTensors(array, [dict(d) for d in tensors])


def moe_adamw_step(tensors: AdamwTensors, options: moe_adamw_options, dev_status=None, stream=None):
    """One AdamW step over all tensors, in place."""
    _call((_lib or load()).moe_adamw_step, tensors.array, len(tensors.array), ctypes.byref(options),
          _packed(dev_status, "dev_status", 1, _INT32), _stream(stream))


class AdamwValues:
    """Where moe_adamw_states writes: addresses of fp32 tensors (make_adamw_values)."""

    def __init__(self, m, v, sizes, held):
        self.m, self.v, self.sizes, self.held = m, v, sizes, held


def make_adamw_values(m_values, v_values) -> AdamwValues:
    """m_values and v_values: a packed fp32 tensor for each tensor's state (or None for a tensor, or in place of a list)."""
    arrays, sizes = [], []
    for what, values in (("m_values", m_values), ("v_values", v_values)):
        if values is None:
            arrays.append(None)
            sizes.append(None)
            continue
        arrays.append((_P * len(values))())
        sizes.append([None if t is None else t.numel() for t in values])
        for i, t in enumerate(values):
            p = _packed(t, f"{what}[{i}]", 0 if t is None else t.numel(), MOE_F32)
            if p.__class__ is _Host:
                raise MoeError(MOE_ERR_INVALID_ARG, p.what)
            arrays[-1][i] = p
    return AdamwValues(*arrays, sizes, (m_values, v_values))


def moe_adamw_states(tensors: AdamwTensors, values: AdamwValues, stream=None):
    """The values that the tensors' states stand for, in fp32."""
    for what, sizes in zip(("m_values", "v_values"), values.sizes):
        if sizes is None or sizes == tensors.sizes:  # (lists, compared in one go: a step has hundreds of tensors)
            continue
        if len(sizes) != len(tensors.sizes) or any(s is not None and s != n for s, n in zip(sizes, tensors.sizes)):
            raise MoeError(MOE_ERR_INVALID_ARG, f"{what} must have the tensors' sizes")
    _call((_lib or load()).moe_adamw_states, tensors.array, len(tensors.array), values.m, values.v, _stream(stream))


def header_functions():
    """Names of the functions include/moe_gb300.h declares."""
    import re

    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))

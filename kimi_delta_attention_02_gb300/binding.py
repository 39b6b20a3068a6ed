"""Thin Python binding of libkda (include/kda.h) over ctypes.

Argument marshalling only: every step of prefill and decode runs in the CUDA
kernels of ``libkda.so``. Tensors are torch CUDA tensors (PyTorch provides the
device memory and the stream); the functions check shapes and dtypes, pass raw
pointers, and raise ``KdaError`` on any non-OK status. There is no CPU
fallback: if ``libkda.so`` has not been built, importing the library raises.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")
ROOT = os.path.dirname(_HERE)
HEADERS = [os.path.join(ROOT, "include", "kda.h"), os.path.join(ROOT, "include", "kda_selftest.h")]

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_TIMEOUT, KDA_ERR_RANGE = 0, 1, 2, 3, 4, 5
KDA_F32, KDA_BF16 = 0, 1

_lock = threading.Lock()
_lib = None


KDA_DECAY_CLAMPED, KDA_DECAY_GATED, KDA_DECAY_UNBOUNDED = 0, 1, 2


class PrefillParams(ctypes.Structure):
    """``kda_prefill_params`` of include/kda.h, field for field."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("decay_form", ctypes.c_int32), ("num_seqs", ctypes.c_int32), ("H", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32), ("total_tokens", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("decay", ctypes.c_void_p),
                ("A_log", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p),
                ("init_state", ctypes.c_void_p), ("out_gate", ctypes.c_void_p), ("norm_weight", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("final_state", ctypes.c_void_p), ("decay_bound", ctypes.c_float),
                ("scale", ctypes.c_float), ("norm_eps", ctypes.c_float), ("force_recurrent", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class DecodeParams(ctypes.Structure):
    """``kda_decode_params`` of include/kda.h, field for field."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("decay_form", ctypes.c_int32), ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("decay", ctypes.c_void_p), ("A_log", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("out_gate", ctypes.c_void_p), ("norm_weight", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("conv_weight", ctypes.c_void_p), ("conv_state", ctypes.c_void_p),
                ("decay_bound", ctypes.c_float), ("scale", ctypes.c_float), ("norm_eps", ctypes.c_float),
                ("l2_eps", ctypes.c_float)]


class LinearPrefillParams(ctypes.Structure):
    """``kda_linear_prefill_params`` of include/kda.h, field for field."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("H", ctypes.c_int32), ("H_k", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("decay_per_token", ctypes.c_int32), ("force_recurrent", ctypes.c_int32),
                ("total_tokens", ctypes.c_int64), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("log_decay", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p),
                ("init_state", ctypes.c_void_p), ("out", ctypes.c_void_p), ("final_state", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("scale", ctypes.c_float)]


class LinearDecodeParams(ctypes.Structure):
    """``kda_linear_decode_params`` of include/kda.h, field for field."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("H_k", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("decay_per_token", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("log_decay", ctypes.c_void_p), ("state", ctypes.c_void_p), ("out", ctypes.c_void_p)]


KDA_GATE_NONE, KDA_GATE_CHANNEL, KDA_GATE_ROW = 0, 1, 2


class BlockNormParams(ctypes.Structure):
    """``kda_block_norm_params`` of include/kda.h, field for field."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("x_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("gate_form", ctypes.c_int32), ("post_norm", ctypes.c_int32),
                ("D", ctypes.c_int32), ("scale", ctypes.c_float), ("rows", ctypes.c_int64), ("x", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("post_weight", ctypes.c_void_p),
                ("channel_scale", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p),
                ("residual_out", ctypes.c_void_p), ("out", ctypes.c_void_p), ("post_eps", ctypes.c_float),
                ("pre_eps", ctypes.c_float)]


class DeltaPrefillParams(ctypes.Structure):
    """``kda_delta_prefill_params`` of include/kda.h, field for field."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("H", ctypes.c_int32), ("H_k", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("decay_per_token", ctypes.c_int32), ("force_recurrent", ctypes.c_int32),
                ("total_tokens", ctypes.c_int64), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("log_decay", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("init_state", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("final_state", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("scale", ctypes.c_float)]


class DeltaDecodeParams(ctypes.Structure):
    """``kda_delta_decode_params`` of include/kda.h, field for field."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("H_k", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("decay_per_token", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("log_decay", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("state", ctypes.c_void_p),
                ("out", ctypes.c_void_p)]


KDA_NORM_NONE, KDA_NORM_RMS, KDA_NORM_L2 = 0, 1, 2
_NORMS = {None: KDA_NORM_NONE, "rms": KDA_NORM_RMS, "l2": KDA_NORM_L2}


class NormRotateParams(ctypes.Structure):
    """``kda_norm_rotate_params`` of include/kda.h, field for field."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("norm", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_k", ctypes.c_int32), ("d", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("position_bytes", ctypes.c_int32), ("eps", ctypes.c_float), ("tokens", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
                ("k_out_stride", ctypes.c_int64), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
                ("pair_axis", ctypes.c_uint8 * 128)]


class KdaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what} failed: {status_string(status)}")


def _declare(lib):
    vp, i32, i64, f32, u32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_uint32
    sz = ctypes.c_size_t
    prefill_args = [vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, i32, f32, f32, vp, vp, vp, vp]
    lib.kda_prefill.argtypes = prefill_args[:-1] + [vp, sz, vp]
    lib.kda_prefill.restype = i32
    lib.kda_prefill_workspace_size.argtypes = [i64, i32, i32, i32, i32]
    lib.kda_prefill_workspace_size.restype = sz
    lib.kda_prefill_recurrent.argtypes = prefill_args
    lib.kda_prefill_noalloc.argtypes = prefill_args
    lib.kda_prefill_noalloc.restype = i32
    lib.kda_prefill_recurrent.restype = i32
    lib.kda_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, f32, vp]
    lib.kda_decode.restype = i32
    gated_args = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, i32, f32, f32, vp, vp, vp, vp]
    lib.kda_prefill_gated.argtypes = gated_args
    lib.kda_prefill_gated.restype = i32
    lib.kda_prefill_gated_recurrent.argtypes = gated_args
    lib.kda_prefill_gated_recurrent.restype = i32
    lib.kda_decode_gated.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, f32, vp]
    lib.kda_decode_gated.restype = i32
    lib.kda_prefill_ex.argtypes = [ctypes.POINTER(PrefillParams), vp]
    lib.kda_prefill_ex.restype = i32
    lib.kda_decode_ex.argtypes = [ctypes.POINTER(DecodeParams), vp]
    lib.kda_decode_ex.restype = i32
    lib.kda_prologue.argtypes = [vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, vp, f32, vp, vp, vp, vp, vp]
    lib.kda_prologue.restype = i32
    lib.kda_linear_prefill.argtypes = [ctypes.POINTER(LinearPrefillParams), vp]
    lib.kda_linear_prefill.restype = i32
    lib.kda_linear_decode.argtypes = [ctypes.POINTER(LinearDecodeParams), vp]
    lib.kda_linear_decode.restype = i32
    lib.kda_linear_prefill_workspace_size.argtypes = [i64, i32, i32, i32, i32, i32, i32, i32, i32]
    lib.kda_linear_prefill_workspace_size.restype = sz
    lib.kda_block_norm.argtypes = [ctypes.POINTER(BlockNormParams), vp]
    lib.kda_block_norm.restype = i32
    lib.kda_delta_prefill.argtypes = [ctypes.POINTER(DeltaPrefillParams), vp]
    lib.kda_delta_prefill.restype = i32
    lib.kda_delta_decode.argtypes = [ctypes.POINTER(DeltaDecodeParams), vp]
    lib.kda_delta_decode.restype = i32
    lib.kda_delta_prefill_workspace_size.argtypes = [i64, i32, i32, i32, i32, i32, i32, i32, i32]
    lib.kda_delta_prefill_workspace_size.restype = sz
    lib.kda_norm_rotate.argtypes = [ctypes.POINTER(NormRotateParams), vp]
    lib.kda_norm_rotate.restype = i32
    lib.kda_check_device_error.argtypes = [vp]
    lib.kda_check_device_error.restype = i32
    lib.kda_status_string.argtypes = [i32]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_version.argtypes = []
    lib.kda_version.restype = i32
    lib.kda_selftest_umma.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, u32, u32, u32, u32, vp, vp]
    lib.kda_selftest_umma.restype = i32
    lib.kda_selftest_wait_timeout.argtypes = [vp, vp]
    lib.kda_selftest_wait_timeout.restype = i32


def lib():
    """The loaded libkda (loaded once). Raises if the library was not built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                                   "(the KDA kernels have no fallback)")
            handle = ctypes.CDLL(LIB_PATH)
            _declare(handle)
            _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    if stream is None:
        # torch.cuda.current_stream().cuda_stream without building the Stream object (0.2 against 3 us)
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
    return ctypes.c_void_p(stream.cuda_stream)


def _empty(shape, dtype, device, stream, returned=True):
    """torch.empty for work on ``stream`` (None: the current one). The memory comes from that stream's
    pool: the current stream's may hand out a block that work pending there still uses, which
    another stream's kernel would not wait for. A tensor that is ``returned`` may be used on the
    current stream too, so its memory goes back only when that is done with it."""
    if stream is None or device.index is None or stream.cuda_stream == torch._C._cuda_getCurrentRawStream(device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _io_dtype(dtype) -> int:
    if dtype == torch.bfloat16:
        return KDA_BF16
    if dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"q/k/v and out must be bfloat16 or float32, got {dtype}")


def _check_cuda(*tensors):
    for t in tensors:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("KDA tensors must be contiguous CUDA tensors")


def workspace_size(total_tokens: int, num_seqs: int, H: int, d_k: int = 128, d_v: int = 128) -> int:
    """Bytes of device scratch ``kda_prefill`` can use for these sizes (``kda_prefill_workspace_size``)."""
    return int(lib().kda_prefill_workspace_size(int(total_tokens), int(num_seqs), int(H), int(d_k), int(d_v)))


def _workspace(workspace, T, N, H, d_k, d_v, device, stream):
    """(pointer, bytes) of the scratch handed to the library: ``"auto"`` allocates what
    ``kda_prefill_workspace_size`` asks for (through torch's caching allocator), ``None`` passes
    none (one CTA per chain), a uint8 CUDA tensor is passed as given."""
    if workspace is None:
        return None, 0
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        n = workspace_size(T, N, H, d_k, d_v)
        if n == 0:
            return None, 0
        workspace = _empty(n, torch.uint8, device, stream, returned=False)
    _check_cuda(workspace)
    return ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size()


def prefill(q, k, v, log_alpha, beta, cu_seqlens, init_state=None, *, out=None, final_state=None,
            out_dtype=torch.float32, lower_bound: float = -5.0, scale: float = 1.0, stream=None,
            recurrent: bool = False, want_final: bool = True, workspace="auto"):
    """KDA prefill over packed variable-length sequences (``kda_prefill``).

    q, k [T, H, d_k], v [T, H, d_v] (bf16 or fp32, one dtype); log_alpha [T, H, d_k] fp32;
    beta [T, H] fp32; cu_seqlens [N+1] int32 (device); init_state [N, H, d_k, d_v] fp32 or None.
    Returns (out [T, H, d_v] in ``out_dtype`` (or out's dtype), final_state [N, H, d_k, d_v] or
    None). ``recurrent=True`` forces the fp32 token-recurrent kernel (``kda_prefill_recurrent``).
    ``workspace``: see ``_workspace`` (the default lets the library pick its parallel schedule).
    """
    T, H, d_k = q.shape
    d_v = v.shape[-1]
    N = cu_seqlens.shape[0] - 1
    dt = _io_dtype(q.dtype)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must share one dtype")
    if log_alpha.dtype != torch.float32 or beta.dtype != torch.float32:
        raise TypeError("log_alpha and beta must be float32")
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    if out is None:
        out = _empty((T, H, d_v), out_dtype, q.device, stream)
    odt = _io_dtype(out.dtype)
    if final_state is None and want_final:
        final_state = _empty((N, H, d_k, d_v), torch.float32, q.device, stream)
    _check_cuda(q, k, v, log_alpha, beta, cu_seqlens, init_state, out, final_state)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(cu_seqlens), N, T, H, d_k, d_v, dt,
            odt, float(lower_bound), float(scale), _ptr(init_state), _ptr(out), _ptr(final_state))
    if recurrent:
        st = lib().kda_prefill_recurrent(*args, _stream_handle(stream))
    else:
        ws, ws_bytes = _workspace(workspace, T, N, H, d_k, d_v, q.device, stream)
        st = lib().kda_prefill(*args, ws, ws_bytes, _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_prefill_recurrent" if recurrent else "kda_prefill")
    return out, final_state


def prefill_noalloc(q, k, v, log_alpha, beta, cu_seqlens, init_state=None, *, out, final_state=None,
                    lower_bound: float = -5.0, scale: float = 1.0, stream=None):
    """``kda_prefill_noalloc``: kda_prefill with the library's own scratch instead of a workspace,
    for callers that cannot allocate device memory (the caller still provides ``out`` and, if
    wanted, ``final_state``; nothing is allocated here either)."""
    T, H, d_k = q.shape
    d_v = v.shape[-1]
    N = cu_seqlens.shape[0] - 1
    _check_cuda(q, k, v, log_alpha, beta, cu_seqlens, init_state, out, final_state)
    st = lib().kda_prefill_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(cu_seqlens), N, T,
                                   H, d_k, d_v, _io_dtype(q.dtype), _io_dtype(out.dtype), float(lower_bound),
                                   float(scale), _ptr(init_state), _ptr(out), _ptr(final_state),
                                   _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_prefill_noalloc")
    return out, final_state


def prefill_gated(q, k, v, z, A_log, beta, cu_seqlens, init_state=None, *, out=None, final_state=None,
                  out_dtype=torch.float32, g_min: float = -5.0, scale: float = 1.0, stream=None,
                  recurrent: bool = False, want_final: bool = True):
    """KDA prefill with the gated log-decay g = g_min * Sigmoid(e^{A_h} z) (``kda_prefill_gated``).

    z [T, H, d_k] in the dtype of q/k/v; A_log [H] float32; the rest as in ``prefill``.
    ``recurrent=True`` forces the fp32 token-recurrent kernel (``kda_prefill_gated_recurrent``).
    """
    T, H, d_k = q.shape
    d_v = v.shape[-1]
    N = cu_seqlens.shape[0] - 1
    dt = _io_dtype(q.dtype)
    if k.dtype != q.dtype or v.dtype != q.dtype or z.dtype != q.dtype:
        raise TypeError("q, k, v and z must share one dtype")
    if A_log.dtype != torch.float32 or beta.dtype != torch.float32:
        raise TypeError("A_log and beta must be float32")
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    if out is None:
        out = _empty((T, H, d_v), out_dtype, q.device, stream)
    odt = _io_dtype(out.dtype)
    if final_state is None and want_final:
        final_state = _empty((N, H, d_k, d_v), torch.float32, q.device, stream)
    _check_cuda(q, k, v, z, A_log, beta, cu_seqlens, init_state, out, final_state)
    fn = lib().kda_prefill_gated_recurrent if recurrent else lib().kda_prefill_gated
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(A_log), _ptr(beta), _ptr(cu_seqlens), N, T, H, d_k, d_v, dt,
            odt, float(g_min), float(scale), _ptr(init_state), _ptr(out), _ptr(final_state), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_prefill_gated_recurrent" if recurrent else "kda_prefill_gated")
    return out, final_state


def _decay_fields(q, log_alpha, lower_bound, z, A_log, g_min, unbounded=False):
    """(decay_form, decay tensor, A_log, bound) for exactly one of log_alpha or (z, A_log); with
    ``unbounded`` the logits go through the unbounded map g = -e^{A_h} Softplus(z)."""
    if (log_alpha is None) == (z is None):
        raise ValueError("pass exactly one of log_alpha (clamped form) or z with A_log (gated form)")
    if log_alpha is not None:
        if A_log is not None:
            raise ValueError("A_log belongs to the gated form (z)")
        if log_alpha.dtype != torch.float32:
            raise TypeError("log_alpha must be float32")
        return KDA_DECAY_CLAMPED, log_alpha, None, float(lower_bound)
    if A_log is None or A_log.dtype != torch.float32:
        raise TypeError("the gated form needs A_log [H] float32")
    if z.dtype != q.dtype:
        raise TypeError("z must have the dtype of q")
    return (KDA_DECAY_UNBOUNDED if unbounded else KDA_DECAY_GATED), z, A_log, float(g_min)


def prefill_ex(q, k, v, beta, cu_seqlens, *, log_alpha=None, lower_bound: float = -5.0, z=None, A_log=None,
               g_min: float = -5.0, init_state=None, out_gate=None, norm_weight=None, norm_eps: float = 1e-6,
               out=None, final_state=None, out_dtype=torch.float32, scale: float = 1.0, stream=None,
               recurrent: bool = False, want_final: bool = True, unbounded: bool = False, workspace="auto"):
    """Prefill through the parameter block (``kda_prefill_ex``): the clamped (``log_alpha``) or
    gated (``z``, ``A_log``) log-decay, and optionally the output gate with head-wise RMSNorm,
    ``out = Sigmoid(out_gate) * norm_weight * o / sqrt(mean(o^2) + norm_eps)`` per token and head.
    ``unbounded=True`` (with z, A_log) takes the earlier models' map g = -e^{A_h} Softplus(z)
    (chunked kernel for bf16 with d = 128, else the token-recurrent one).
    out_gate [T, H, d_v] in the dtype of q; norm_weight [d_v] float32 or None (ones).
    Returns (out, final_state or None)."""
    T, H, d_k = q.shape
    d_v = v.shape[-1]
    N = cu_seqlens.shape[0] - 1
    form, decay, A, bound = _decay_fields(q, log_alpha, lower_bound, z, A_log, g_min, unbounded)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must share one dtype")
    if out_gate is not None and out_gate.dtype != q.dtype:
        raise TypeError("out_gate must have the dtype of q")
    if norm_weight is not None and norm_weight.dtype != torch.float32:
        raise TypeError("norm_weight must be float32")
    if beta.dtype != torch.float32 or cu_seqlens.dtype != torch.int32:
        raise TypeError("beta must be float32 and cu_seqlens int32")
    if out is None:
        out = _empty((T, H, d_v), out_dtype, q.device, stream)
    if final_state is None and want_final:
        final_state = _empty((N, H, d_k, d_v), torch.float32, q.device, stream)
    _check_cuda(q, k, v, decay, A, beta, cu_seqlens, init_state, out_gate, norm_weight, out, final_state)
    ws, ws_bytes = _workspace(None if recurrent else workspace, T, N, H, d_k, d_v, q.device, stream)
    p = PrefillParams(struct_size=ctypes.sizeof(PrefillParams), in_dtype=_io_dtype(q.dtype),
                      out_dtype=_io_dtype(out.dtype), decay_form=form, num_seqs=N, H=H, d_k=d_k, d_v=d_v,
                      total_tokens=T, q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), decay=decay.data_ptr(),
                      A_log=None if A is None else A.data_ptr(), beta=beta.data_ptr(),
                      cu_seqlens=cu_seqlens.data_ptr(),
                      init_state=None if init_state is None else init_state.data_ptr(),
                      out_gate=None if out_gate is None else out_gate.data_ptr(),
                      norm_weight=None if norm_weight is None else norm_weight.data_ptr(), out=out.data_ptr(),
                      final_state=None if final_state is None else final_state.data_ptr(), decay_bound=bound,
                      scale=float(scale), norm_eps=float(norm_eps), force_recurrent=int(bool(recurrent)),
                      workspace=ws, workspace_bytes=ws_bytes)
    st = lib().kda_prefill_ex(ctypes.byref(p), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_prefill_ex")
    return out, final_state


def decode_ex(q, k, v, beta, state, *, log_alpha=None, lower_bound: float = -5.0, z=None, A_log=None,
              g_min: float = -5.0, out_gate=None, norm_weight=None, norm_eps: float = 1e-6, conv_weight=None,
              conv_state=None, l2_eps: float = 1e-6, out=None, out_dtype=torch.float32, scale: float = 1.0,
              stream=None, unbounded: bool = False):
    """One decode step through the parameter block (``kda_decode_ex``); ``state`` is updated in
    place. Decay and output-gate options as in ``prefill_ex``. With ``conv_state`` [B, H, 3,
    2 d_k + d_v] (dtype of q; shifted in place) and ``conv_weight`` [H, 2 d_k + d_v, 4] float32,
    q, k, v are the raw projections and pass the prologue of ``prologue`` first.
    Returns out [B, H, d_v]."""
    B, H, d_k = q.shape
    d_v = v.shape[-1]
    form, decay, A, bound = _decay_fields(q, log_alpha, lower_bound, z, A_log, g_min, unbounded)
    if out_gate is not None and out_gate.dtype != q.dtype:
        raise TypeError("out_gate must have the dtype of q")
    if out is None:
        out = _empty((B, H, d_v), out_dtype, q.device, stream)
    _check_cuda(q, k, v, decay, A, beta, state, out_gate, norm_weight, conv_weight, conv_state, out)
    if conv_state is not None and conv_state.dtype != q.dtype:
        raise TypeError("conv_state must have the dtype of q")
    p = DecodeParams(struct_size=ctypes.sizeof(DecodeParams), in_dtype=_io_dtype(q.dtype),
                     out_dtype=_io_dtype(out.dtype), decay_form=form, B=B, H=H, d_k=d_k, d_v=d_v, q=q.data_ptr(),
                     k=k.data_ptr(), v=v.data_ptr(), decay=decay.data_ptr(),
                     A_log=None if A is None else A.data_ptr(), beta=beta.data_ptr(), state=state.data_ptr(),
                     out_gate=None if out_gate is None else out_gate.data_ptr(),
                     norm_weight=None if norm_weight is None else norm_weight.data_ptr(), out=out.data_ptr(),
                     conv_weight=None if conv_weight is None else conv_weight.data_ptr(),
                     conv_state=None if conv_state is None else conv_state.data_ptr(),
                     decay_bound=bound, scale=float(scale), norm_eps=float(norm_eps), l2_eps=float(l2_eps))
    st = lib().kda_decode_ex(ctypes.byref(p), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_ex")
    return out


def prologue(q_raw, k_raw, v_raw, conv_weight, cu_seqlens, conv_init=None, *, l2_eps: float = 1e-6, q=None,
             k=None, v=None, conv_final=None, want_final: bool = True, stream=None):
    """The input prologue (``kda_prologue``): 4-tap causal ShortConv per sequence, Swish, and the
    L2 norm of q and k. q_raw, k_raw [T, H, d_k], v_raw [T, H, d_v] (bf16 or fp32, one dtype);
    conv_weight [H, 2 d_k + d_v, 4] float32; conv_init [N, H, 3, 2 d_k + d_v] or None.
    Returns (q, k, v, conv_final or None), the inputs of ``prefill``."""
    T, H, d_k = q_raw.shape
    d_v = v_raw.shape[-1]
    N = cu_seqlens.shape[0] - 1
    dt = _io_dtype(q_raw.dtype)
    if k_raw.dtype != q_raw.dtype or v_raw.dtype != q_raw.dtype:
        raise TypeError("q, k and v must share one dtype")
    if conv_weight.dtype != torch.float32 or cu_seqlens.dtype != torch.int32:
        raise TypeError("conv_weight must be float32 and cu_seqlens int32")
    if conv_init is not None and conv_init.dtype != q_raw.dtype:
        raise TypeError("conv_init must have the dtype of q")
    q = _empty(q_raw.shape, q_raw.dtype, q_raw.device, stream) if q is None else q
    k = _empty(k_raw.shape, k_raw.dtype, k_raw.device, stream) if k is None else k
    v = _empty(v_raw.shape, v_raw.dtype, v_raw.device, stream) if v is None else v
    if conv_final is None and want_final:
        conv_final = _empty((N, H, 3, 2 * d_k + d_v), q_raw.dtype, q_raw.device, stream)
    _check_cuda(q_raw, k_raw, v_raw, conv_weight, cu_seqlens, conv_init, q, k, v, conv_final)
    st = lib().kda_prologue(_ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(conv_weight), _ptr(cu_seqlens), N, T, H,
                            d_k, d_v, dt, _ptr(conv_init), float(l2_eps), _ptr(q), _ptr(k), _ptr(v),
                            _ptr(conv_final), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_prologue")
    return q, k, v, conv_final


def decode_gated(q, k, v, z, A_log, beta, state, *, out=None, out_dtype=torch.float32, g_min: float = -5.0,
                 scale: float = 1.0, stream=None):
    """One decode step with the gated log-decay (``kda_decode_gated``); ``state`` is updated in place."""
    B, H, d_k = q.shape
    d_v = v.shape[-1]
    dt = _io_dtype(q.dtype)
    if z.dtype != q.dtype or A_log.dtype != torch.float32:
        raise TypeError("z must have the dtype of q, A_log must be float32")
    if out is None:
        out = _empty((B, H, d_v), out_dtype, q.device, stream)
    odt = _io_dtype(out.dtype)
    _check_cuda(q, k, v, z, A_log, beta, state, out)
    st = lib().kda_decode_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(A_log), _ptr(beta), _ptr(state), _ptr(out),
                                B, H, d_k, d_v, dt, odt, float(g_min), float(scale), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_gated")
    return out


def decode(q, k, v, log_alpha, beta, state, *, out=None, out_dtype=torch.float32, lower_bound: float = -5.0,
           scale: float = 1.0, stream=None):
    """One KDA decode step (``kda_decode``); ``state`` [B, H, d_k, d_v] fp32 is updated in place.
    q, k [B, H, d_k], v [B, H, d_v]; log_alpha [B, H, d_k]; beta [B, H]. Returns out [B, H, d_v]."""
    B, H, d_k = q.shape
    d_v = v.shape[-1]
    dt = _io_dtype(q.dtype)
    if out is None:
        out = _empty((B, H, d_v), out_dtype, q.device, stream)
    odt = _io_dtype(out.dtype)
    _check_cuda(q, k, v, log_alpha, beta, state, out)
    st = lib().kda_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(state), _ptr(out), B, H,
                          d_k, d_v, dt, odt, float(lower_bound), float(scale), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode")
    return out


def _one_device(*tensors) -> int:
    """The device index that all given tensors (None: left out) share, each contiguous on it."""
    device = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d < 0 or not t.is_contiguous():
                raise ValueError("KDA tensors must be contiguous CUDA tensors")
            if d != device:
                if device >= 0:
                    raise ValueError("KDA tensors must be on one CUDA device")
                device = d
    return device


def _address(t):
    return None if t is None else t.data_ptr()


def _check_shape(name, t, shape, dtype=None):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")


def _linear_sizes(q, k, v, log_decay, rows_name):
    """Shapes and dtypes shared by linear_prefill and linear_decode: (rows, H_k, H, d_k, d_v)."""
    if q.ndim != 3 or v.ndim != 3 or k.shape != q.shape or v.shape[0] != q.shape[0]:
        raise ValueError(f"q and k must be [{rows_name}, H_k, d_k] and v [{rows_name}, H, d_v]")
    rows, H_k, d_k = q.shape
    _, H, d_v = v.shape
    if H_k < 1 or H % H_k:
        raise ValueError("the value heads must be a multiple of the query / key heads")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must share one dtype")
    if log_decay.dtype != torch.float32:
        raise TypeError("log_decay must be float32")
    if log_decay.shape != (rows, H) and log_decay.shape != (H,):
        raise ValueError(f"log_decay must be [{rows_name}, H] or [H]")
    return rows, H_k, H, d_k, d_v


def linear_workspace_size(total_tokens: int, num_seqs: int, H: int, d_k: int = 128, d_v: int = 128,
                          dtype=torch.bfloat16, out_dtype=torch.float32, recurrent: bool = False, H_k=None) -> int:
    """Bytes of device scratch ``linear_prefill`` can use (``kda_linear_prefill_workspace_size``);
    ``H_k`` query / key heads, H by default."""
    return int(lib().kda_linear_prefill_workspace_size(int(total_tokens), int(num_seqs), int(H),
                                                       int(H if H_k is None else H_k), int(d_k), int(d_v),
                                                       _io_dtype(dtype), _io_dtype(out_dtype), int(bool(recurrent))))


_LINEAR_PREFILL_BYTES = ctypes.sizeof(LinearPrefillParams)
_LINEAR_DECODE_BYTES = ctypes.sizeof(LinearDecodeParams)
_BLOCK_NORM_BYTES = ctypes.sizeof(BlockNormParams)


def linear_prefill(q, k, v, log_decay, cu_seqlens, init_state=None, *, out=None, final_state=None,
                   out_dtype=torch.float32, scale: float = 1.0, stream=None, recurrent: bool = False,
                   want_final: bool = True, workspace="auto"):
    """Linear attention with one decay per head over packed variable-length sequences
    (``kda_linear_prefill``): S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q, k [T, H_k, d_k], v [T, H, d_v] (bf16 or fp32, one dtype; value head h reads query / key head
    h // (H // H_k)); log_decay g [T, H] or, constant, [H] float32; cu_seqlens [N+1] int32 (device);
    init_state [N, H, d_k, d_v] float32 or None. Returns (out [T, H, d_v] in ``out_dtype`` (or
    out's dtype), final_state [N, H, d_k, d_v] or None). ``recurrent=True`` forces the fp32
    token-recurrent kernel. ``workspace``: ``"auto"`` allocates what ``linear_workspace_size``
    asks for, ``None`` passes none, a uint8 CUDA tensor is passed as given."""
    T, H_k, H, d_k, d_v = _linear_sizes(q, k, v, log_decay, "T")
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.ndim != 1 or cu_seqlens.shape[0] < 1:
        raise TypeError("cu_seqlens must be int32 [N + 1]")
    N = cu_seqlens.shape[0] - 1
    given = workspace if isinstance(workspace, torch.Tensor) else None
    device = _one_device(q, k, v, log_decay, cu_seqlens, init_state, out, final_state, given)
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return linear_prefill(q, k, v, log_decay, cu_seqlens, init_state, out=out, final_state=final_state,
                                  out_dtype=out_dtype, scale=scale, stream=stream, recurrent=recurrent,
                                  want_final=want_final, workspace=workspace)
    state_shape = (N, H, d_k, d_v)
    if init_state is not None:
        _check_shape("init_state", init_state, state_shape, torch.float32)
    if out is None:
        out = _empty((T, H, d_v), out_dtype, q.device, stream)
    else:
        _check_shape("out", out, (T, H, d_v))
    if final_state is not None:
        _check_shape("final_state", final_state, state_shape, torch.float32)
    elif want_final:
        final_state = _empty(state_shape, torch.float32, q.device, stream)
    dt, odt, rec = _io_dtype(q.dtype), _io_dtype(out.dtype), 1 if recurrent else 0
    handle = lib()
    if given is None and workspace is not None:
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        n = handle.kda_linear_prefill_workspace_size(T, N, H, H_k, d_k, d_v, dt, odt, rec)
        if n:
            given = _empty(n, torch.uint8, q.device, stream, returned=False)
    p = LinearPrefillParams(_LINEAR_PREFILL_BYTES, dt, odt, N, H, H_k, d_k, d_v, 1 if log_decay.ndim == 2 else 0, rec, T,
                            q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), cu_seqlens.data_ptr(),
                            _address(init_state), out.data_ptr(), _address(final_state), _address(given),
                            0 if given is None else given.numel() * given.element_size(), scale)
    st = handle.kda_linear_prefill(ctypes.byref(p), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_linear_prefill")
    return out, final_state


def linear_decode(q, k, v, log_decay, state, *, out=None, out_dtype=torch.float32, scale: float = 1.0, stream=None):
    """One token of linear attention with one decay per head for B sequences
    (``kda_linear_decode``); ``state`` [B, H, d_k, d_v] float32 is updated in place.
    q, k [B, H_k, d_k], v [B, H, d_v], log_decay [B, H] or [H]. Returns out [B, H, d_v]."""
    B, H_k, H, d_k, d_v = _linear_sizes(q, k, v, log_decay, "B")
    device = _one_device(q, k, v, log_decay, state, out)
    _check_shape("state", state, (B, H, d_k, d_v), torch.float32)
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return linear_decode(q, k, v, log_decay, state, out=out, out_dtype=out_dtype, scale=scale, stream=stream)
    if out is None:
        out = _empty((B, H, d_v), out_dtype, q.device, stream)
    else:
        _check_shape("out", out, (B, H, d_v))
    p = LinearDecodeParams(_LINEAR_DECODE_BYTES, _io_dtype(q.dtype), _io_dtype(out.dtype), B, H, H_k, d_k, d_v,
                           1 if log_decay.ndim == 2 else 0, scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                           log_decay.data_ptr(), state.data_ptr(), out.data_ptr())
    st = lib().kda_linear_decode(ctypes.byref(p), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_linear_decode")
    return out


def block_norm(x, y=None, *, gate=None, post_norm: bool = False, post_weight=None, scale: float = 1.0,
               channel_scale=None, pre_weight=None, eps: float = 1e-6, post_eps=None, residual_out=None, out=None,
               out_dtype=None, want_out: bool = True, want_residual: bool = True, stream=None):
    """The norm after a block, its gate and residual scale, and the norm before the next block
    (``kda_block_norm``), per row of D channels:

        n  = post_weight * y / sqrt(mean(y^2) + post_eps) with ``post_norm``, else y
        x' = x + scale * channel_scale * Sigmoid(gate) * n
        h  = pre_weight * x' / sqrt(mean(x'^2) + eps)

    x [rows, D] and y [rows, D] or None (x' = x), each bf16 or fp32; gate logits in the dtype of y,
    [rows, D] or [rows], or None (factor 1); weights [D] float32 or None (ones); post_eps defaults
    to eps. Returns (x' in x's dtype, h in ``out_dtype`` (x's dtype by default) or out's dtype);
    either is None when not wanted. ``residual_out`` may be x itself. Without y, x' is x and is not
    written unless ``residual_out`` is given."""
    if x.ndim != 2 or (y is not None and y.shape != x.shape):
        raise ValueError("x and y must be [rows, D]")
    rows, D = x.shape
    form = KDA_GATE_NONE
    if y is None:
        if gate is not None or post_norm or post_weight is not None or channel_scale is not None:
            raise ValueError("gate, post_norm, post_weight and channel_scale belong to y")
    elif gate is not None:
        if gate.dtype != y.dtype:
            raise TypeError("gate must have the dtype of y")
        if gate.shape == x.shape:
            form = KDA_GATE_CHANNEL
        elif gate.shape == (rows,):
            form = KDA_GATE_ROW
        else:
            raise ValueError("gate must be [rows, D] or [rows]")
    for w in (post_weight, channel_scale, pre_weight):
        if w is not None:
            _check_shape("a weight", w, (D,), torch.float32)
    device = _one_device(x, y, gate, post_weight, channel_scale, pre_weight, residual_out, out)
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return block_norm(x, y, gate=gate, post_norm=post_norm, post_weight=post_weight, scale=scale,
                              channel_scale=channel_scale, pre_weight=pre_weight, eps=eps, post_eps=post_eps,
                              residual_out=residual_out, out=out, out_dtype=out_dtype, want_out=want_out,
                              want_residual=want_residual, stream=stream)
    if residual_out is not None:
        _check_shape("residual_out", residual_out, (rows, D), x.dtype)
    elif want_residual and y is not None:
        residual_out = _empty(x.shape, x.dtype, x.device, stream)
    if out is not None:
        _check_shape("out", out, (rows, D))
    elif want_out:
        out = _empty(x.shape, out_dtype or x.dtype, x.device, stream)
    p = BlockNormParams(_BLOCK_NORM_BYTES, _io_dtype(x.dtype), KDA_F32 if y is None else _io_dtype(y.dtype),
                        KDA_F32 if out is None else _io_dtype(out.dtype), form, 1 if post_norm else 0, D, scale, rows,
                        x.data_ptr(), _address(y), _address(gate), _address(post_weight), _address(channel_scale),
                        _address(pre_weight), _address(residual_out), _address(out),
                        eps if post_eps is None else post_eps, eps)
    st = lib().kda_block_norm(ctypes.byref(p), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_block_norm")
    return (x if y is None and residual_out is None and want_residual else residual_out), out


def delta_workspace_size(total_tokens: int, num_seqs: int, H: int, d_k: int = 128, d_v: int = 128,
                         dtype=torch.bfloat16, out_dtype=torch.float32, recurrent: bool = False, H_k=None) -> int:
    """Bytes of device scratch ``delta_prefill`` can use (``kda_delta_prefill_workspace_size``);
    ``H_k`` query / key heads, H by default."""
    return int(lib().kda_delta_prefill_workspace_size(int(total_tokens), int(num_seqs), int(H),
                                                      int(H if H_k is None else H_k), int(d_k), int(d_v),
                                                      _io_dtype(dtype), _io_dtype(out_dtype), int(bool(recurrent))))


_DELTA_PREFILL_BYTES = ctypes.sizeof(DeltaPrefillParams)
_DELTA_DECODE_BYTES = ctypes.sizeof(DeltaDecodeParams)
_NORM_ROTATE_BYTES = ctypes.sizeof(NormRotateParams)
_PairAxis = ctypes.c_uint8 * 128
_NO_AXIS = _PairAxis()


def delta_prefill(q, k, v, log_decay, beta, cu_seqlens, init_state=None, *, out=None, final_state=None,
                  out_dtype=torch.float32, scale: float = 1.0, stream=None, recurrent: bool = False,
                  want_final: bool = True, workspace="auto"):
    """The gated delta rule with one decay per head over packed variable-length sequences
    (``kda_delta_prefill``): S_t = (I - beta_t k_t k_t^T) e^{g_t} S_{t-1} + beta_t k_t v_t^T,
    o_t = scale S_t^T q_t.

    beta [T, H] float32; everything else as in ``linear_prefill``: q, k [T, H_k, d_k], v [T, H, d_v]
    (bf16 or fp32, one dtype; value head h reads query / key head h // (H // H_k)); log_decay g
    [T, H] or, constant, [H] float32; cu_seqlens [N+1] int32 (device); init_state [N, H, d_k, d_v]
    float32 or None. Returns (out [T, H, d_v] in ``out_dtype`` (or out's dtype), final_state
    [N, H, d_k, d_v] or None). ``recurrent=True`` forces the fp32 token-recurrent kernel.
    ``workspace``: ``"auto"`` allocates what ``delta_workspace_size`` asks for, ``None`` passes none,
    a uint8 CUDA tensor is passed as given."""
    T, H_k, H, d_k, d_v = _linear_sizes(q, k, v, log_decay, "T")
    _check_shape("beta", beta, (T, H), torch.float32)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.ndim != 1 or cu_seqlens.shape[0] < 1:
        raise TypeError("cu_seqlens must be int32 [N + 1]")
    N = cu_seqlens.shape[0] - 1
    given = workspace if isinstance(workspace, torch.Tensor) else None
    device = _one_device(q, k, v, log_decay, beta, cu_seqlens, init_state, out, final_state, given)
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return delta_prefill(q, k, v, log_decay, beta, cu_seqlens, init_state, out=out, final_state=final_state,
                                 out_dtype=out_dtype, scale=scale, stream=stream, recurrent=recurrent,
                                 want_final=want_final, workspace=workspace)
    state_shape = (N, H, d_k, d_v)
    if init_state is not None:
        _check_shape("init_state", init_state, state_shape, torch.float32)
    if out is None:
        out = _empty((T, H, d_v), out_dtype, q.device, stream)
    else:
        _check_shape("out", out, (T, H, d_v))
    if final_state is not None:
        _check_shape("final_state", final_state, state_shape, torch.float32)
    elif want_final:
        final_state = _empty(state_shape, torch.float32, q.device, stream)
    dt, odt, rec = _io_dtype(q.dtype), _io_dtype(out.dtype), 1 if recurrent else 0
    handle = lib()
    if given is None and workspace is not None:
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        n = handle.kda_delta_prefill_workspace_size(T, N, H, H_k, d_k, d_v, dt, odt, rec)
        if n:
            given = _empty(n, torch.uint8, q.device, stream, returned=False)
    p = DeltaPrefillParams(_DELTA_PREFILL_BYTES, dt, odt, N, H, H_k, d_k, d_v, 1 if log_decay.ndim == 2 else 0, rec, T,
                           q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), beta.data_ptr(),
                           cu_seqlens.data_ptr(), _address(init_state), out.data_ptr(), _address(final_state),
                           _address(given), 0 if given is None else given.numel() * given.element_size(), scale)
    st = handle.kda_delta_prefill(ctypes.byref(p), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_delta_prefill")
    return out, final_state


def delta_decode(q, k, v, log_decay, beta, state, *, out=None, out_dtype=torch.float32, scale: float = 1.0,
                 stream=None):
    """One token of the gated delta rule with one decay per head for B sequences
    (``kda_delta_decode``); ``state`` [B, H, d_k, d_v] float32 is updated in place.
    q, k [B, H_k, d_k], v [B, H, d_v], log_decay [B, H] or [H], beta [B, H]. Returns out [B, H, d_v]."""
    B, H_k, H, d_k, d_v = _linear_sizes(q, k, v, log_decay, "B")
    device = _one_device(q, k, v, log_decay, beta, state, out)
    _check_shape("beta", beta, (B, H), torch.float32)
    _check_shape("state", state, (B, H, d_k, d_v), torch.float32)
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return delta_decode(q, k, v, log_decay, beta, state, out=out, out_dtype=out_dtype, scale=scale,
                                stream=stream)
    if out is None:
        out = _empty((B, H, d_v), out_dtype, q.device, stream)
    else:
        _check_shape("out", out, (B, H, d_v))
    p = DeltaDecodeParams(_DELTA_DECODE_BYTES, _io_dtype(q.dtype), _io_dtype(out.dtype), B, H, H_k, d_k, d_v,
                          1 if log_decay.ndim == 2 else 0, scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                          log_decay.data_ptr(), beta.data_ptr(), state.data_ptr(), out.data_ptr())
    st = lib().kda_delta_decode(ctypes.byref(p), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_delta_decode")
    return out


def _heads_of_rows(name, x):
    """The token stride of [T, heads, d] whose heads and channels are contiguous (a part of a fused
    projection's rows, or a whole tensor)."""
    T, H, d = x.shape
    if x.is_contiguous():
        return H * d
    if (d > 1 and x.stride(2) != 1) or (H > 1 and x.stride(1) != d):
        raise ValueError(f"{name}: a token's heads and channels must be contiguous")
    return x.stride(0) if T > 1 else H * d


def norm_rotate(q, k, positions, inv_freq, *, norm="rms", q_weight=None, k_weight=None, eps: float = 1e-6,
                interleaved: bool = False, pair_axis=None, q_out=None, k_out=None, out_dtype=None, stream=None):
    """The norm of each query and key head, then rotary positions, in one pass (``kda_norm_rotate``):
    n = weight * x / sqrt(mean(x^2) + eps) (``norm="rms"``), x / sqrt(sum(x^2) + eps) (``"l2"``) or x
    (None); then channel pair i of the first 2 * len(inv_freq) channels, (i, i + len(inv_freq)) or,
    ``interleaved``, (2 i, 2 i + 1), turns by position * inv_freq[i].

    q [T, H_q, d], k [T, H_k, d] or None, bf16 or fp32, one dtype; tokens may lie further apart than
    H * d elements (parts of a fused projection's rows). positions int32 or int64, [T] or, for several
    axes, [A, T] with ``pair_axis``, the axis of each pair (a sequence of ints). inv_freq [rot / 2]
    float32, or positions and inv_freq None: no rotation. Weights [d] float32 or None (ones), with
    "rms" only. Returns (q', k' or None) in ``out_dtype`` (the dtype of q by default) or in q_out and
    k_out, which may be q and k themselves."""
    if q.ndim != 3 or (k is not None and (k.ndim != 3 or k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2])):
        raise ValueError("q must be [T, H_q, d] and k [T, H_k, d]")
    T, H_q, d = q.shape
    H_k = 0 if k is None else k.shape[1]
    if k is not None and (H_k < 1 or k.dtype != q.dtype):
        raise TypeError("q and k must share one dtype, k with a head at least")
    if norm not in _NORMS:
        raise ValueError("norm must be 'rms', 'l2' or None")
    for w in (q_weight, k_weight):
        if w is not None:
            _check_shape("a weight", w, (d,), torch.float32)
    if k is None and (k_weight is not None or k_out is not None):
        raise ValueError("k_weight and k_out belong to k")
    half, axes, size = 0, 1, 8
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq belong together")
    if inv_freq is not None:
        if inv_freq.ndim != 1 or inv_freq.dtype != torch.float32:
            raise TypeError("inv_freq must be float32 [rot / 2]")
        half = inv_freq.shape[0]
        if 2 * half > min(d, 256):
            raise ValueError("inv_freq has more pairs than a head has channels for")
        if positions.dtype != torch.int64 and positions.dtype != torch.int32:
            raise TypeError("positions must be int32 or int64")
        size = positions.element_size()
        if positions.ndim == 2 and pair_axis is not None:
            axes = positions.shape[0]
        if positions.shape != ((T,) if pair_axis is None else (axes, T)) or axes < 1:
            raise ValueError("positions must be [T], or [A, T] with pair_axis")
    axis_of = _NO_AXIS
    if pair_axis is not None:
        if len(pair_axis) != half:
            raise ValueError("pair_axis must name an axis for each pair of inv_freq")
        if half and not 0 <= min(pair_axis) <= max(pair_axis) < min(axes, 256):
            raise ValueError("pair_axis names an axis that positions does not have")
        axis_of = _PairAxis.from_buffer_copy(bytes(list(pair_axis)).ljust(128, b"\0"))
    device = _one_device(positions, inv_freq, q_weight, k_weight)
    for t in (q, k, q_out, k_out):
        if t is not None:
            at = t.get_device()
            if at < 0 or (device >= 0 and at != device):
                raise ValueError("KDA tensors must be on one CUDA device")
            device = at
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return norm_rotate(q, k, positions, inv_freq, norm=norm, q_weight=q_weight, k_weight=k_weight, eps=eps,
                               interleaved=interleaved, pair_axis=pair_axis, q_out=q_out, k_out=k_out,
                               out_dtype=out_dtype, stream=stream)
    dtype = out_dtype or q.dtype
    for name, x in (("q_out", q_out), ("k_out", k_out)):
        if x is not None:
            _check_shape(name, x, q.shape if name == "q_out" else k.shape)
            if out_dtype is not None and x.dtype != out_dtype:
                raise TypeError(f"{name} must be {out_dtype}")
            dtype = x.dtype
    # tokens lie q_row (k_row) elements apart in outputs made here
    q_row, k_row = H_q * d, H_k * d
    if q_out is None:
        q_out = _empty(q.shape, dtype, q.device, stream)
    else:
        q_row = _heads_of_rows("q_out", q_out)
    if k is not None:
        if k_out is None:
            k_out = _empty(k.shape, dtype, k.device, stream)
        else:
            k_row = _heads_of_rows("k_out", k_out)
    if k is not None and k_out.dtype != q_out.dtype:
        raise TypeError("q_out and k_out must share one dtype")
    p = NormRotateParams(_NORM_ROTATE_BYTES, _io_dtype(q.dtype), _io_dtype(q_out.dtype), _NORMS[norm], H_q, H_k, d,
                         2 * half, 1 if interleaved else 0, axes, size, eps, T, _heads_of_rows("q", q),
                         0 if k is None else _heads_of_rows("k", k), q_row, k_row, q.data_ptr(), _address(k),
                         _address(q_weight), _address(k_weight), _address(positions), _address(inv_freq),
                         q_out.data_ptr(), _address(k_out), axis_of)
    st = lib().kda_norm_rotate(ctypes.byref(p), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_norm_rotate")
    return q_out, k_out


def check_device_error(stream=None):
    """Synchronise and raise if a kernel recorded a bounded-wait timeout or an input outside
    its range (``KdaError.status`` tells which)."""
    st = lib().kda_check_device_error(_stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_check_device_error")


UMMA_FORMATS = {"f16": 0, "bf16": 1, "tf32": 2}


def selftest_umma(A, B, M, N, K, *, fmt="bf16", sw64=False, a_mn_major=False, b_mn_major=False, negate_a=False,
                  a_lbo=16, a_sbo=1024, b_lbo=16, b_sbo=1024, stream=None):
    """One tcgen05 MMA on the GPU (``kda_selftest_umma``); returns the raw [128, N] accumulator.
    A [M, K] and B [N, K] are rounded on the device to ``fmt`` (f16, bf16 or tf32)."""
    A32 = A.to(torch.float32).contiguous()
    B32 = B.to(torch.float32).contiguous()
    D = torch.full((128, N), float("nan"), dtype=torch.float32, device=A.device)
    status = torch.zeros(1, dtype=torch.int32, device=A.device)
    st = lib().kda_selftest_umma(_ptr(A32), _ptr(B32), _ptr(D), M, N, K, UMMA_FORMATS[fmt], int(sw64), int(a_mn_major),
                                 int(b_mn_major), int(negate_a), a_lbo, a_sbo, b_lbo, b_sbo, _ptr(status),
                                 _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_selftest_umma")
    torch.cuda.synchronize()
    if int(status.item()) != 0:
        raise KdaError(KDA_ERR_TIMEOUT, "kda_selftest_umma")
    return D


def selftest_wait_timeout(stream=None):
    """Runs a bounded wait that is never satisfied (``kda_selftest_wait_timeout``); returns the
    kernel's status word (1 when the wait gave up). The device error word is left set for
    ``check_device_error`` to report."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = lib().kda_selftest_wait_timeout(_ptr(status), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_selftest_wait_timeout")
    torch.cuda.synchronize()
    return int(status.item())


class HostPrefill:
    """End-to-end prefill from pinned HOST buffers, as an application calls it.

    Each ``__call__`` copies the inputs host -> device, runs ``kda_prefill`` and
    copies ``out`` and ``final_state`` back to pinned host memory, all on one
    stream, and waits for the result. Device staging buffers are allocated once.
    """

    def __init__(self, q, k, v, log_alpha, beta, cu_seqlens, init_state=None, device="cuda",
                 out_dtype=torch.float32):
        self.host_in = [t.pin_memory() if not t.is_pinned() else t
                        for t in (q, k, v, log_alpha, beta, cu_seqlens)]
        self.host_init = None if init_state is None else init_state.pin_memory()
        self.dev_in = [torch.empty_like(t, device=device) for t in self.host_in]
        self.dev_init = None if init_state is None else torch.empty_like(self.host_init, device=device)
        T, H, _ = q.shape
        N = cu_seqlens.shape[0] - 1
        self.dev_out = torch.empty((T, H, v.shape[-1]), dtype=out_dtype, device=device)
        self.dev_final = torch.empty((N, H, q.shape[-1], v.shape[-1]), dtype=torch.float32, device=device)
        self.host_out = torch.empty_like(self.dev_out, device="cpu").pin_memory()
        self.host_final = torch.empty_like(self.dev_final, device="cpu").pin_memory()

    @property
    def h2d_bytes(self) -> int:
        n = sum(t.numel() * t.element_size() for t in self.host_in)
        return n + (0 if self.host_init is None else self.host_init.numel() * 4)

    @property
    def d2h_bytes(self) -> int:
        return self.host_out.numel() * self.host_out.element_size() + self.host_final.numel() * 4

    def __call__(self, stream=None, sync: bool = True):
        stream = stream or torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            for d, h in zip(self.dev_in, self.host_in):
                d.copy_(h, non_blocking=True)
            if self.dev_init is not None:
                self.dev_init.copy_(self.host_init, non_blocking=True)
            q, k, v, la, b, cu = self.dev_in
            prefill(q, k, v, la, b, cu, self.dev_init, out=self.dev_out, final_state=self.dev_final,
                    stream=stream)
            self.host_out.copy_(self.dev_out, non_blocking=True)
            self.host_final.copy_(self.dev_final, non_blocking=True)
        if sync:
            stream.synchronize()
        return self.host_out, self.host_final


class HostPrefillStream:
    """Prefill from pinned HOST buffers, streamed: step i's host-to-device copies, its kernel and
    its device-to-host copies run on three CUDA streams, so that step i+1's inputs travel while
    step i computes and step i-1's results come back.

    Every step still moves all its inputs to the device and all its outputs (``out`` and the
    final state) back to pinned host memory; two device staging sets and two host result sets
    alternate between steps. ``run(steps)`` enqueues the steps and waits for the last result.
    """

    def __init__(self, q, k, v, log_alpha, beta, cu_seqlens, init_state=None, device="cuda",
                 out_dtype=torch.float32):
        self.host_in = [t.pin_memory() if not t.is_pinned() else t
                        for t in (q, k, v, log_alpha, beta, cu_seqlens)]
        self.host_init = None if init_state is None else init_state.pin_memory()
        T, H, _ = q.shape
        N = cu_seqlens.shape[0] - 1
        self.dev_in = [[torch.empty_like(t, device=device) for t in self.host_in] for _ in range(2)]
        self.dev_init = [None if init_state is None else torch.empty_like(self.host_init, device=device)
                         for _ in range(2)]
        self.dev_out = [torch.empty((T, H, v.shape[-1]), dtype=out_dtype, device=device) for _ in range(2)]
        self.dev_final = [torch.empty((N, H, q.shape[-1], v.shape[-1]), dtype=torch.float32, device=device)
                          for _ in range(2)]
        self.host_out = [torch.empty_like(self.dev_out[0], device="cpu").pin_memory() for _ in range(2)]
        self.host_final = [torch.empty_like(self.dev_final[0], device="cpu").pin_memory() for _ in range(2)]
        self.s_in, self.s_run, self.s_back = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Stream()
        self.ev_in = [torch.cuda.Event() for _ in range(2)]
        self.ev_run = [torch.cuda.Event() for _ in range(2)]
        self.ev_back = [torch.cuda.Event() for _ in range(2)]
        self.steps_done = 0

    @property
    def h2d_bytes(self) -> int:
        n = sum(t.numel() * t.element_size() for t in self.host_in)
        return n + (0 if self.host_init is None else self.host_init.numel() * 4)

    @property
    def d2h_bytes(self) -> int:
        return self.host_out[0].numel() * self.host_out[0].element_size() + self.host_final[0].numel() * 4

    def _in(self, i):
        b = i & 1
        with torch.cuda.stream(self.s_in):
            if i >= 2:
                self.s_in.wait_event(self.ev_run[b])  # step i-2's kernel has read this staging set
            for d, h in zip(self.dev_in[b], self.host_in):
                d.copy_(h, non_blocking=True)
            if self.dev_init[b] is not None:
                self.dev_init[b].copy_(self.host_init, non_blocking=True)
            self.ev_in[b].record(self.s_in)

    def _run(self, i):
        b = i & 1
        with torch.cuda.stream(self.s_run):
            self.s_run.wait_event(self.ev_in[b])
            if i >= 2:
                self.s_run.wait_event(self.ev_back[b])  # step i-2's results have left this set
            q, k, v, la, bt, cu = self.dev_in[b]
            prefill(q, k, v, la, bt, cu, self.dev_init[b], out=self.dev_out[b], final_state=self.dev_final[b],
                    stream=self.s_run)
            self.ev_run[b].record(self.s_run)

    def _back(self, i, stream):
        b = i & 1
        with torch.cuda.stream(stream):
            stream.wait_event(self.ev_run[b])
            self.host_out[b].copy_(self.dev_out[b], non_blocking=True)
            self.host_final[b].copy_(self.dev_final[b], non_blocking=True)
            self.ev_back[b].record(stream)

    def enqueue(self):
        """Enqueue one step (copies in, kernel, copies back) without waiting."""
        i = self.steps_done
        self._in(i)
        self._run(i)
        self._back(i, self.s_back)
        self.steps_done += 1

    def run(self, steps: int, duplex: bool = True):
        """Run ``steps`` streamed steps and return the last step's (out, final_state) on the host.
        ``duplex``: copies in and copies back on their own streams, so that both directions may
        run at once; otherwise one copy stream carries step i+1's inputs and then step i's
        results, so that the kernel still overlaps the copies but the two directions never do."""
        if duplex:
            for _ in range(steps):
                self.enqueue()
        elif steps > 0:
            i0 = self.steps_done
            self._in(i0)
            for n in range(steps):
                self._run(i0 + n)
                if n + 1 < steps:
                    self._in(i0 + n + 1)
                self._back(i0 + n, self.s_in)
            self.steps_done = i0 + steps
        b = (self.steps_done - 1) & 1
        self.ev_back[b].synchronize()
        return self.host_out[b], self.host_final[b]

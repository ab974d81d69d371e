"""Thin ctypes binding of libqgemm.so (C ABI in include/qgemm.h).

Argument marshalling only: every step of the computation runs in the HIP
library.  Functions take torch tensors on the GPU, pass their device pointers
and torch's current HIP stream, and raise QGemmError on a non-zero status.
There is no fallback: if libqgemm.so is missing, importing this module raises; if
the _calls extension (the compiled marshalling of the calls that stand between two
products) is missing or belongs to another torch, those calls raise.

bf16 data travels as torch.bfloat16 (or int16 / uint16 bit patterns) tensors;
e4m3 codes as torch.uint8 (or torch.float8_e4m3fn) tensors.

Only MoeRouting carries gradients; outputs of everything else are cut off from the
autograd graph of their inputs.
"""
import contextlib
import ctypes
import os

import torch
from torch.autograd.function import once_differentiable

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqgemm.so")

_BUILD = "run `python -m weight_only_quantized_w4a16_amd.build`"

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; {_BUILD} (hipcc, gfx950)")

_lib = ctypes.CDLL(LIB_PATH)


class _NoCalls:
    """In the place of _calls where that cannot be used: every call through it raises."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"{name}: the compiled call marshalling cannot be used ({self._why}); {_BUILD}")

    def __dir__(self):
        return []


try:
    from . import _calls                     # built beside the library
    _built_with = getattr(_calls, "torch_version", "unknown")
    if _built_with != torch.__version__:
        _calls = _NoCalls(f"built with torch {_built_with}, this is {torch.__version__}")
except ImportError as _e:
    _calls = _NoCalls(str(_e))

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t

_SIGS = {
    "qg_status_string": (ctypes.c_char_p, [_I]),
    "qg_version": (ctypes.c_char_p, []),
    "qg_int4_g128_packed_bytes": (_SZ, [_I64, _I64]),
    "qg_int4_g128_scale_bytes": (_SZ, [_I64, _I64]),
    "qg_w4a16_kernel_for": (ctypes.c_char_p, [_I64, _I64, _I64]),
    "qg_w8a8_kernel_for": (ctypes.c_char_p, [_I64, _I64, _I64]),
    "qg_w4a16_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "qg_w8a8_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "pack_int4_g128": (_I, [_P, _I, _I, _P, _P, _P]),
    "pack_int4_g128_mse": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "dequant_int4_g128": (_I, [_P, _P, _I, _I, _P, _P, _P]),
    "qgemm_w4a16": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qgemm_w4a16_noalloc": (_I, [_P, _P, _P, _P, _I, _I, _I, _P]),
    "qg_w4a16_grouped_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64]),
    "qgemm_w4a16_grouped": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "quant_act_per_token": (_I, [_P, _I, _I, _P, _P, _P]),
    "quant_weight_fp8_per_channel": (_I, [_P, _I, _I, _P, _P, _P]),
    "qgemm_w8a8_fp8": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qgemm_w4a8_fp8": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "qgemm_w4a8_fp8_grouped": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "qg_w8a8_int8_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "quant_act_per_token_int8": (_I, [_P, _I, _I, _P, _P, _P]),
    "quant_weight_int8_per_channel": (_I, [_P, _I, _I, _P, _P, _P]),
    "qgemm_w8a8_int8": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qg_w8a8_dynamic_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "qg_w8a8_dynamic_kernel_for": (ctypes.c_char_p, [_I64, _I64, _I64]),
    "qgemm_w8a8_fp8_dynamic": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qgemm_w8a8_int8_dynamic": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qg_w4a8_grouped_dynamic_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64]),
    "qg_w4a8_grouped_dynamic_kernel_for": (ctypes.c_char_p, [_I64, _I64, _I64, _I64]),
    "qgemm_w4a8_fp8_grouped_dynamic": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "rms_norm": (_I, [_P, _P, _P, _F, _I, _I, _P, _P, _P]),
    "rms_norm_quant": (_I, [_P, _P, _P, _F, _I, _I, _P, _P, _P, _P, _P]),
    "rms_norm_quant_int8": (_I, [_P, _P, _P, _F, _I, _I, _P, _P, _P, _P, _P]),
    "swiglu": (_I, [_P, _I, _I, _P, _P]),
    "swiglu_quant": (_I, [_P, _I, _I, _P, _P, _P]),
    "swiglu_quant_int8": (_I, [_P, _I, _I, _P, _P, _P]),
    "qgemm_w4a16_epilogue": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qg_moe_dispatch_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "moe_dispatch": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_gather": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "moe_combine": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "moe_combine_backward": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGS)

# the compiled marshalling calls the functions of the library loaded above
for _name in dir(_calls):
    if _name in _SIGS:
        _calls.bind(_name, ctypes.cast(getattr(_lib, _name), ctypes.c_void_p).value)


class QGemmError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: status {status} ({status_string(status)})")


def status_string(status):
    return _lib.qg_status_string(int(status)).decode()


def version():
    return _lib.qg_version().decode()


def packed_bytes(K, N):
    return _lib.qg_int4_g128_packed_bytes(K, N)


def scale_bytes(K, N):
    return _lib.qg_int4_g128_scale_bytes(K, N)


def w4a16_kernel_for(M, N, K):
    return _lib.qg_w4a16_kernel_for(M, N, K).decode()


def w8a8_kernel_for(M, N, K):
    return _lib.qg_w8a8_kernel_for(M, N, K).decode()


def w8a8_dynamic_kernel_for(M, N, K):
    return _lib.qg_w8a8_dynamic_kernel_for(M, N, K).decode()


def w8a8_dynamic_workspace_bytes(M, N, K):
    return _lib.qg_w8a8_dynamic_workspace_bytes(M, N, K)


def w4a16_workspace_bytes(M, N, K):
    return _lib.qg_w4a16_workspace_bytes(M, N, K)


def w8a8_workspace_bytes(M, N, K):
    return _lib.qg_w8a8_workspace_bytes(M, N, K)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _check(fn, status):
    if status != 0:
        raise QGemmError(fn, status)


# ---- raw entry points (same names and argument order as the C ABI) ----------

def pack_int4_g128(w_bf16, K, N, packed, scales, stream=None):
    _check("pack_int4_g128", _lib.pack_int4_g128(_ptr(w_bf16), K, N, _ptr(packed), _ptr(scales),
                                                 _stream(stream)))


def pack_int4_g128_mse(w_bf16, K, N, n_alpha, packed, scales, stream=None):
    _check("pack_int4_g128_mse", _lib.pack_int4_g128_mse(_ptr(w_bf16), K, N, n_alpha, _ptr(packed),
                                                         _ptr(scales), _stream(stream)))


def dequant_int4_g128(packed, scales, K, N, w_bf16_out, codes_out=None, stream=None):
    _check("dequant_int4_g128", _lib.dequant_int4_g128(_ptr(packed), _ptr(scales), K, N,
                                                       _ptr(w_bf16_out), _ptr(codes_out),
                                                       _stream(stream)))


def qgemm_w4a16(a_bf16, packed, scales, y_bf16, M, N, K, workspace=None, workspace_bytes=0,
                stream=None):
    _check("qgemm_w4a16", _lib.qgemm_w4a16(_ptr(a_bf16), _ptr(packed), _ptr(scales), _ptr(y_bf16),
                                           M, N, K, _ptr(workspace), workspace_bytes,
                                           _stream(stream)))


def qgemm_w4a16_noalloc(a_bf16, packed, scales, y_bf16, M, N, K, stream=None):
    _check("qgemm_w4a16_noalloc", _lib.qgemm_w4a16_noalloc(_ptr(a_bf16), _ptr(packed), _ptr(scales),
                                                           _ptr(y_bf16), M, N, K, _stream(stream)))


NOALLOC_SCRATCH_BYTES = 32 << 20    # QG_NOALLOC_SCRATCH_BYTES of include/qgemm.h


def quant_act_per_token(a_bf16, M, K, a_e4m3, a_scale, stream=None):
    _check("quant_act_per_token", _lib.quant_act_per_token(_ptr(a_bf16), M, K, _ptr(a_e4m3),
                                                           _ptr(a_scale), _stream(stream)))


def quant_weight_fp8_per_channel(w_bf16, K, N, w_e4m3, w_scale, stream=None):
    _check("quant_weight_fp8_per_channel",
           _lib.quant_weight_fp8_per_channel(_ptr(w_bf16), K, N, _ptr(w_e4m3), _ptr(w_scale),
                                             _stream(stream)))


def qgemm_w8a8_fp8(a_e4m3, a_scale, w_e4m3, w_scale, y_bf16, M, N, K, workspace=None,
                   workspace_bytes=0, stream=None):
    _check("qgemm_w8a8_fp8", _lib.qgemm_w8a8_fp8(_ptr(a_e4m3), _ptr(a_scale), _ptr(w_e4m3),
                                                 _ptr(w_scale), _ptr(y_bf16), M, N, K,
                                                 _ptr(workspace), workspace_bytes,
                                                 _stream(stream)))


def qgemm_w4a8_fp8(a_e4m3, a_scale, packed, scales, y_bf16, M, N, K, stream=None):
    _check("qgemm_w4a8_fp8", _lib.qgemm_w4a8_fp8(_ptr(a_e4m3), _ptr(a_scale), _ptr(packed), _ptr(scales),
                                                 _ptr(y_bf16), M, N, K, _stream(stream)))


def qgemm_w4a8_fp8_grouped(a_e4m3, a_scale, offsets_i32, packed, scales, y_bf16, E, T, N, K, workspace,
                           workspace_bytes, stream=None):
    _check("qgemm_w4a8_fp8_grouped",
           _lib.qgemm_w4a8_fp8_grouped(_ptr(a_e4m3), _ptr(a_scale), _ptr(offsets_i32), _ptr(packed),
                                       _ptr(scales), _ptr(y_bf16), E, T, N, K, _ptr(workspace),
                                       workspace_bytes, _stream(stream)))


def w8a8_int8_workspace_bytes(M, N, K):
    return _lib.qg_w8a8_int8_workspace_bytes(M, N, K)


def quant_act_per_token_int8(a_bf16, M, K, a_i8, a_scale, stream=None):
    _check("quant_act_per_token_int8",
           _lib.quant_act_per_token_int8(_ptr(a_bf16), M, K, _ptr(a_i8), _ptr(a_scale), _stream(stream)))


def quant_weight_int8_per_channel(w_bf16, K, N, w_i8, w_scale, stream=None):
    _check("quant_weight_int8_per_channel",
           _lib.quant_weight_int8_per_channel(_ptr(w_bf16), K, N, _ptr(w_i8), _ptr(w_scale),
                                              _stream(stream)))


def qgemm_w8a8_int8(a_i8, a_scale, w_i8, w_scale, y_bf16, M, N, K, workspace=None,
                    workspace_bytes=0, stream=None):
    _check("qgemm_w8a8_int8", _lib.qgemm_w8a8_int8(_ptr(a_i8), _ptr(a_scale), _ptr(w_i8),
                                                   _ptr(w_scale), _ptr(y_bf16), M, N, K,
                                                   _ptr(workspace), workspace_bytes,
                                                   _stream(stream)))


def qgemm_w8a8_fp8_dynamic(a_bf16, w_e4m3, w_scale, y_bf16, M, N, K, workspace=None,
                           workspace_bytes=0, stream=None):
    _check("qgemm_w8a8_fp8_dynamic",
           _lib.qgemm_w8a8_fp8_dynamic(_ptr(a_bf16), _ptr(w_e4m3), _ptr(w_scale), _ptr(y_bf16), M, N, K,
                                       _ptr(workspace), workspace_bytes, _stream(stream)))


def qgemm_w8a8_int8_dynamic(a_bf16, w_i8, w_scale, y_bf16, M, N, K, workspace=None,
                            workspace_bytes=0, stream=None):
    _check("qgemm_w8a8_int8_dynamic",
           _lib.qgemm_w8a8_int8_dynamic(_ptr(a_bf16), _ptr(w_i8), _ptr(w_scale), _ptr(y_bf16), M, N, K,
                                        _ptr(workspace), workspace_bytes, _stream(stream)))


def w4a8_grouped_dynamic_workspace_bytes(E, T, N, K):
    return _lib.qg_w4a8_grouped_dynamic_workspace_bytes(E, T, N, K)


def w4a8_grouped_dynamic_kernel_for(E, T, N, K):
    return _lib.qg_w4a8_grouped_dynamic_kernel_for(E, T, N, K).decode()


def qgemm_w4a8_fp8_grouped_dynamic(a_bf16, offsets_i32, packed, scales, y_bf16, E, T, N, K, workspace,
                                   workspace_bytes, stream=None):
    _check("qgemm_w4a8_fp8_grouped_dynamic",
           _lib.qgemm_w4a8_fp8_grouped_dynamic(_ptr(a_bf16), _ptr(offsets_i32), _ptr(packed), _ptr(scales),
                                               _ptr(y_bf16), E, T, N, K, _ptr(workspace), workspace_bytes,
                                               _stream(stream)))


# ---- the operators between two products: raw entry points ----------------------
# They launch on the device their tensors are on, on that device's current
# stream unless one is given.  The marshalling is compiled (_calls).

def rms_norm(x_bf16, residual_bf16, weight_bf16, eps, M, K, h_bf16, y_bf16, stream=None):
    _check("rms_norm", _calls.rms_norm(x_bf16, residual_bf16, weight_bf16, eps, M, K, h_bf16, y_bf16, stream))


def rms_norm_quant(x_bf16, residual_bf16, weight_bf16, eps, M, K, h_bf16, y_bf16, y_e4m3, y_scale, stream=None):
    _check("rms_norm_quant", _calls.rms_norm_quant(x_bf16, residual_bf16, weight_bf16, eps, M, K, h_bf16, y_bf16, y_e4m3,
                                                   y_scale, stream))


def rms_norm_quant_int8(x_bf16, residual_bf16, weight_bf16, eps, M, K, h_bf16, y_bf16, y_i8, y_scale, stream=None):
    _check("rms_norm_quant_int8", _calls.rms_norm_quant_int8(x_bf16, residual_bf16, weight_bf16, eps, M, K, h_bf16, y_bf16,
                                                             y_i8, y_scale, stream))


def swiglu(gate_up_bf16, M, I, y_bf16, stream=None):
    _check("swiglu", _calls.swiglu(gate_up_bf16, M, I, y_bf16, stream))


def swiglu_quant(gate_up_bf16, M, I, y_e4m3, y_scale, stream=None):
    _check("swiglu_quant", _calls.swiglu_quant(gate_up_bf16, M, I, y_e4m3, y_scale, stream))


def swiglu_quant_int8(gate_up_bf16, M, I, y_i8, y_scale, stream=None):
    _check("swiglu_quant_int8", _calls.swiglu_quant_int8(gate_up_bf16, M, I, y_i8, y_scale, stream))


# qg_activation of include/qgemm.h
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def qgemm_w4a16_epilogue(a_bf16, packed, scales, bias_bf16, activation, residual_bf16, y_bf16, M, N, K, workspace=None,
                         workspace_bytes=0, stream=None):
    """activation: a name of ACTIVATIONS or its qg_activation code."""
    code = ACTIVATIONS.get(activation, activation)
    if not isinstance(code, int):
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    _check("qgemm_w4a16_epilogue", _calls.qgemm_w4a16_epilogue(a_bf16, packed, scales, bias_bf16, code, residual_bf16, y_bf16,
                                                               M, N, K, workspace, workspace_bytes, stream))


def moe_dispatch_workspace_bytes(B, k, E):
    return _lib.qg_moe_dispatch_workspace_bytes(B, k, E)


def moe_dispatch(expert_ids, rows, row_scale, B, k, E, row_bytes, offsets, row_of_slot, rows_out, row_scale_out,
                 workspace=None, workspace_bytes=0, stream=None):
    _check("moe_dispatch", _calls.moe_dispatch(expert_ids, rows, row_scale, B, k, E, row_bytes, offsets, row_of_slot, rows_out,
                                               row_scale_out, workspace, workspace_bytes, stream))


def moe_gather(rows, row_scale, row_of_slot, B, k, row_bytes, rows_out, row_scale_out, stream=None):
    _check("moe_gather", _calls.moe_gather(rows, row_scale, row_of_slot, B, k, row_bytes, rows_out, row_scale_out, stream))


def moe_combine(rows_bf16, row_of_slot, weights, residual_bf16, B, k, K, y_bf16, stream=None):
    _check("moe_combine", _calls.moe_combine(rows_bf16, row_of_slot, weights, residual_bf16, B, k, K, y_bf16, stream))


def moe_combine_backward(dy_bf16, rows_bf16, row_of_slot, weights, B, k, K, drows_bf16, dweights, stream=None):
    _check("moe_combine_backward", _calls.moe_combine_backward(dy_bf16, rows_bf16, row_of_slot, weights, B, k, K, drows_bf16,
                                                               dweights, stream))


# ---- tensor-level helpers (allocate outputs with torch, then call the above) --

_HERE = contextlib.nullcontext()


def _on(stream, t):
    """Context in which `stream` is the current stream (None: no change): what a helper
    allocates, clears or copies then belongs to the stream that launches the work on it,
    and may be freed while that runs."""
    if stream is None:
        return _HERE
    if stream.device_index != t.get_device():
        raise ValueError("the stream belongs to another device than the tensors")
    return torch.cuda.stream(stream)


class _Scratch:
    """A workspace kept from call to call, for calls that do not overlap in time.  A
    call of the largest size before a capture spares the graph one of its own."""

    _ws = None
    _captured = False            # a captured graph uses _ws
    _outgrown = ()               # buffers that captured graphs go on using

    def _scratch(self, need, device, cleared=True):
        """(buffer, need), or (None, 0) if nothing is needed.  A new buffer comes from the
        current stream; a call on another stream follows the one that brought it."""
        if not need:
            return None, 0
        alloc = torch.zeros if cleared else torch.empty
        capturing = torch.cuda.is_current_stream_capturing()
        if self._ws is None or self._ws.numel() * self._ws.element_size() < need:
            if capturing:
                # the graph's own, cleared in every replay: kept, it would not be cleared until the first one
                return alloc(need, dtype=torch.uint8, device=device), need
            if self._captured:
                self._outgrown += (self._ws,)
            elif self._ws is not None:
                # the last calls may have used it on another stream than its own; this call follows them
                self._ws.record_stream(torch.cuda.current_stream(device))
            self._ws, self._captured = alloc(need, dtype=torch.uint8, device=device), False
        self._captured |= capturing
        return self._ws, need


def _bf16(t):
    if t.dtype in (torch.int16, torch.uint16):
        return t
    if t.dtype != torch.bfloat16:
        raise TypeError(f"expected bf16 data, got {t.dtype}")
    return t


class Int4G128Weight:
    """A [K, N] weight in native INT4 g128 form (device buffers owned by torch)."""

    def __init__(self, packed, scales, K, N):
        self.packed, self.scales, self.K, self.N = packed, scales, K, N

    @classmethod
    def from_bf16(cls, w, stream=None, mse_grid=0):
        """Abs-max scales, or with mse_grid > 0 the MSE-optimal clipping
        threshold searched over alpha = i / mse_grid, i = 1 .. mse_grid."""
        K, N = w.shape
        with _on(stream, w):
            packed = torch.empty(max(packed_bytes(K, N) // 4, 1), dtype=torch.int32, device=w.device)
            scales = torch.empty(max(scale_bytes(K, N) // 2, 1), dtype=torch.int16, device=w.device)
            if mse_grid:
                pack_int4_g128_mse(_bf16(w.contiguous()), K, N, mse_grid, packed, scales)
            else:
                pack_int4_g128(_bf16(w.contiguous()), K, N, packed, scales)
        return cls(packed, scales, K, N)

    def dequant(self, with_codes=False, stream=None):
        with _on(stream, self.packed):
            w = torch.empty((self.K, self.N), dtype=torch.bfloat16, device=self.packed.device)
            codes = torch.empty((self.K, self.N), dtype=torch.uint8, device=self.packed.device) \
                if with_codes else None
            dequant_int4_g128(self.packed, self.scales, self.K, self.N, w, codes)
        return (w, codes) if with_codes else w


class W4A16Linear(_Scratch):
    """y = act(a @ w_hat + bias) + residual for a packed INT4 g128 weight; owns a
    reusable workspace.  bias: bf16 [N] or None; activation: a name of ACTIVATIONS."""

    def __init__(self, weight: Int4G128Weight, bias=None, activation="none"):
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
        self.w = weight
        self.bias = None if bias is None else _is(bias, _BF16, (weight.N,), "bias")
        self.activation = activation

    def workspace(self, M):
        # zero-filled once; every call resets the counters it uses
        return self._scratch(w4a16_workspace_bytes(M, self.w.N, self.w.K), self.w.packed.device)

    def __call__(self, a, out=None, stream=None, residual=None):
        """residual: bf16 [M, N] added after the activation; it may be `out` itself."""
        M, K = a.shape
        if K != self.w.K:
            raise ValueError(f"activation K={K} != weight K={self.w.K}")
        with _on(stream, a):
            y = out if out is not None else torch.empty((M, self.w.N), dtype=torch.bfloat16,
                                                        device=a.device)
            ws, nbytes = self.workspace(M)
            if residual is not None or self.bias is not None or self.activation != "none":
                if residual is not None:
                    _is(residual, _BF16, (M, self.w.N), "residual")
                qgemm_w4a16_epilogue(_bf16(a), self.w.packed, self.w.scales, self.bias, self.activation, residual,
                                     _is(y, _BF16, (M, self.w.N), "out"), M, self.w.N, K, ws, nbytes)
            else:
                qgemm_w4a16(_bf16(a), self.w.packed, self.w.scales, y, M, self.w.N, K, ws, nbytes)
        return y


class Fp8Weight:
    """A [K, N] weight as native per-channel e4m3 codes plus fp32 channel scales."""

    def __init__(self, codes, scales, K, N):
        self.codes, self.scales, self.K, self.N = codes, scales, K, N

    @classmethod
    def from_bf16(cls, w, stream=None):
        K, N = w.shape
        with _on(stream, w):
            codes = torch.empty(K * N, dtype=torch.uint8, device=w.device)
            scales = torch.empty(N, dtype=torch.float32, device=w.device)
            quant_weight_fp8_per_channel(_bf16(w.contiguous()), K, N, codes, scales)
        return cls(codes, scales, K, N)


def w4a16_grouped_workspace_bytes(E, T, N, K):
    return _lib.qg_w4a16_grouped_workspace_bytes(E, T, N, K)


def qgemm_w4a16_grouped(a_bf16, offsets_i32, packed, scales, y_bf16, E, T, N, K, workspace,
                        workspace_bytes, stream=None):
    _check("qgemm_w4a16_grouped",
           _lib.qgemm_w4a16_grouped(_ptr(a_bf16), _ptr(offsets_i32), _ptr(packed), _ptr(scales),
                                    _ptr(y_bf16), E, T, N, K, _ptr(workspace), workspace_bytes,
                                    _stream(stream)))


class GroupedInt4Weight(_Scratch):
    """E experts' [K, N] weights packed back to back (device buffers owned by torch)."""

    def __init__(self, packed, scales, E, K, N):
        self.packed, self.scales, self.E, self.K, self.N = packed, scales, E, K, N

    @classmethod
    def from_bf16(cls, w, stream=None):
        """w: [E, K, N] bf16 on the device."""
        E, K, N = w.shape
        words, nsc = packed_bytes(K, N) // 4, scale_bytes(K, N) // 2
        with _on(stream, w):
            packed = torch.empty(E * words, dtype=torch.int32, device=w.device)
            scales = torch.empty(E * nsc, dtype=torch.int16, device=w.device)
            for e in range(E):
                pack_int4_g128(_bf16(w[e].contiguous()), K, N, packed[e * words:(e + 1) * words],
                               scales[e * nsc:(e + 1) * nsc])
        return cls(packed, scales, E, K, N)

    def __call__(self, a, offsets, out=None, stream=None):
        """a: [T, K] bf16 rows grouped by expert; offsets: int32 [E + 1] on the device."""
        T, K = a.shape
        if K != self.K or offsets.numel() != self.E + 1 or offsets.dtype != torch.int32:
            raise ValueError("grouped GEMM: activation K or offsets do not match the weights")
        with _on(stream, a):
            y = out if out is not None else torch.empty((T, self.N), dtype=torch.bfloat16, device=a.device)
            ws, need = self._scratch(w4a16_grouped_workspace_bytes(self.E, T, self.N, K), a.device, cleared=False)
            qgemm_w4a16_grouped(_bf16(a), offsets, self.packed, self.scales, y, self.E, T, self.N, K, ws, need)
        return y

    def w4a8(self, qa, sa, offsets, out=None, stream=None):
        """The W4A8-FP8 product: qa [T, K] e4m3 codes and sa [T] from quant_act_per_token."""
        T, K = qa.shape
        if K != self.K or offsets.numel() != self.E + 1 or offsets.dtype != torch.int32:
            raise ValueError("grouped GEMM: activation K or offsets do not match the weights")
        with _on(stream, qa):
            y = out if out is not None else torch.empty((T, self.N), dtype=torch.bfloat16, device=qa.device)
            ws, need = self._scratch(w4a16_grouped_workspace_bytes(self.E, T, self.N, K), qa.device, cleared=False)
            qgemm_w4a8_fp8_grouped(qa, sa, offsets, self.packed, self.scales, y, self.E, T, self.N, K, ws, need)
        return y

    def w4a8_dynamic(self, a, offsets, out=None, stream=None):
        """The W4A8-FP8 product on bf16 rows, quantized per token inside the call."""
        T, K = a.shape
        if K != self.K or offsets.numel() != self.E + 1 or offsets.dtype != torch.int32:
            raise ValueError("grouped GEMM: activation K or offsets do not match the weights")
        with _on(stream, a):
            y = out if out is not None else torch.empty((T, self.N), dtype=torch.bfloat16, device=a.device)
            ws, need = self._scratch(w4a8_grouped_dynamic_workspace_bytes(self.E, T, self.N, K), a.device, cleared=False)
            qgemm_w4a8_fp8_grouped_dynamic(_bf16(a), offsets, self.packed, self.scales, y, self.E, T, self.N, K, ws, need)
        return y


def quantize_activations(a, stream=None):
    M, K = a.shape
    with _on(stream, a):
        q = torch.empty((M, K), dtype=torch.uint8, device=a.device)
        s = torch.empty(M, dtype=torch.float32, device=a.device)
        quant_act_per_token(_bf16(a), M, K, q, s)
    return q, s


class W8A8Fp8Linear(_Scratch):
    """y = bf16(s_a s_w (qa @ qw)) with per-token quantization of a on every call."""

    def __init__(self, weight: Fp8Weight):
        self.w = weight

    def workspace(self, M, dynamic=False):
        need = (w8a8_dynamic_workspace_bytes if dynamic else w8a8_workspace_bytes)(M, self.w.N, self.w.K)
        # zero-filled once; every call resets the counters it uses
        return self._scratch(need, self.w.codes.device)

    def __call__(self, a, out=None, stream=None, qa=None, sa=None):
        """Without qa / sa the activations are quantized inside the call
        (qgemm_w8a8_fp8_dynamic); with them the GEMM runs on the given codes."""
        M, K = a.shape
        if K != self.w.K:
            raise ValueError(f"activation K={K} != weight K={self.w.K}")
        with _on(stream, a):
            y = out if out is not None else torch.empty((M, self.w.N), dtype=torch.bfloat16,
                                                        device=a.device)
            ws, need = self.workspace(M, dynamic=qa is None)
            if qa is None:
                qgemm_w8a8_fp8_dynamic(_bf16(a), self.w.codes, self.w.scales, y, M, self.w.N, K, ws, need)
            else:
                qgemm_w8a8_fp8(qa, sa, self.w.codes, self.w.scales, y, M, self.w.N, K, ws, need)
        return y


class W4A8Linear:
    """y = bf16(s_a (qa @ w_hat)) for a packed INT4 g128 weight and e4m3 per-token activations."""

    def __init__(self, weight: "Int4G128Weight"):
        self.w = weight

    def __call__(self, a, out=None, stream=None, qa=None, sa=None):
        M, K = a.shape
        if K != self.w.K:
            raise ValueError(f"activation K={K} != weight K={self.w.K}")
        with _on(stream, a):
            if qa is None:
                qa, sa = quantize_activations(a)
            y = out if out is not None else torch.empty((M, self.w.N), dtype=torch.bfloat16, device=a.device)
            qgemm_w4a8_fp8(qa, sa, self.w.packed, self.w.scales, y, M, self.w.N, K)
        return y


class Int8Weight:
    """A [K, N] weight as native per-channel int8 codes plus fp32 channel scales."""

    def __init__(self, codes, scales, K, N):
        self.codes, self.scales, self.K, self.N = codes, scales, K, N

    @classmethod
    def from_bf16(cls, w, stream=None):
        K, N = w.shape
        with _on(stream, w):
            codes = torch.empty(K * N, dtype=torch.int8, device=w.device)
            scales = torch.empty(N, dtype=torch.float32, device=w.device)
            quant_weight_int8_per_channel(_bf16(w.contiguous()), K, N, codes, scales)
        return cls(codes, scales, K, N)


def quantize_activations_int8(a, stream=None):
    M, K = a.shape
    with _on(stream, a):
        q = torch.empty((M, K), dtype=torch.int8, device=a.device)
        s = torch.empty(M, dtype=torch.float32, device=a.device)
        quant_act_per_token_int8(_bf16(a), M, K, q, s)
    return q, s


class W8A8Int8Linear(_Scratch):
    """y = bf16(s_a s_w (qa @ qw)) with int8 codes, per-token quantization of a on every call."""

    def __init__(self, weight: Int8Weight):
        self.w = weight

    def workspace(self, M, dynamic=False):
        need = (w8a8_dynamic_workspace_bytes if dynamic else w8a8_int8_workspace_bytes)(
            M, self.w.N, self.w.K)
        return self._scratch(need, self.w.codes.device)

    def __call__(self, a, out=None, stream=None, qa=None, sa=None):
        """Without qa / sa the activations are quantized inside the call
        (qgemm_w8a8_int8_dynamic); with them the GEMM runs on the given codes."""
        M, K = a.shape
        if K != self.w.K:
            raise ValueError(f"activation K={K} != weight K={self.w.K}")
        with _on(stream, a):
            y = out if out is not None else torch.empty((M, self.w.N), dtype=torch.bfloat16,
                                                        device=a.device)
            ws, need = self.workspace(M, dynamic=qa is None)
            if qa is None:
                qgemm_w8a8_int8_dynamic(_bf16(a), self.w.codes, self.w.scales, y, M, self.w.N, K, ws, need)
            else:
                qgemm_w8a8_int8(qa, sa, self.w.codes, self.w.scales, y, M, self.w.N, K, ws, need)
        return y


# ---- the operators between two products: tensor-level helpers --------------------

def _is(t, dtypes, shape, what):
    """Raises unless t has one of the dtypes and this shape."""
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)

_CODES = {"e4m3": torch.uint8, "int8": torch.int8}


def _codes(M, K, fmt, device):
    if fmt not in _CODES:
        raise ValueError(f"fmt must be 'e4m3' or 'int8', got {fmt!r}")
    return (torch.empty((M, K), dtype=_CODES[fmt], device=device),
            torch.empty(M, dtype=torch.float32, device=device))


class RMSNorm:
    """Residual addition and root-mean-square norm with a bf16 weight [K]."""

    def __init__(self, weight, eps=1e-5):
        self.weight, self.eps = _is(weight, _BF16, (weight.numel(),), "weight"), float(eps)

    def _inputs(self, x, residual):
        M, K = x.shape
        _is(x, _BF16, (M, self.weight.numel()), "x")
        h = None
        if residual is not None:
            _is(residual, _BF16, (M, K), "residual")
            h = torch.empty((M, K), dtype=torch.bfloat16, device=x.device)
        return M, K, h

    def __call__(self, x, residual=None, stream=None):
        """(y, h): the bf16 norm and the new residual stream (x itself without a residual)."""
        with _on(stream, x):
            M, K, h = self._inputs(x, residual)
            y = torch.empty((M, K), dtype=torch.bfloat16, device=x.device)
            rms_norm(x, residual, self.weight, self.eps, M, K, h, y)
        return y, x if h is None else h

    def quantized(self, x, residual=None, fmt="e4m3", with_bf16=False, stream=None):
        """(q, s, h): per-token codes and scales of the norm; with_bf16: (q, s, h, y)."""
        with _on(stream, x):
            M, K, h = self._inputs(x, residual)
            q, s = _codes(M, K, fmt, x.device)
            y = torch.empty((M, K), dtype=torch.bfloat16, device=x.device) if with_bf16 else None
            call = rms_norm_quant if fmt == "e4m3" else rms_norm_quant_int8
            call(x, residual, self.weight, self.eps, M, K, h, y, q, s)
        out = (q, s, x if h is None else h)
        return out + (y,) if with_bf16 else out


def gated_silu(gate_up, stream=None):
    """silu(gate) * up of a fused [M, 2 I] gate_up output, as bf16 [M, I]."""
    M, n = gate_up.shape
    if n % 2:
        raise ValueError("gate_up: the gate and up halves need an even number of columns")
    _is(gate_up, _BF16, (M, n), "gate_up")
    with _on(stream, gate_up):
        y = torch.empty((M, n // 2), dtype=torch.bfloat16, device=gate_up.device)
        swiglu(gate_up, M, n // 2, y)
    return y


def gated_silu_quantized(gate_up, fmt="e4m3", stream=None):
    """The same as per-token codes and scales (q, s)."""
    M, n = gate_up.shape
    if n % 2:
        raise ValueError("gate_up: the gate and up halves need an even number of columns")
    _is(gate_up, _BF16, (M, n), "gate_up")
    with _on(stream, gate_up):
        q, s = _codes(M, n // 2, fmt, gate_up.device)
        (swiglu_quant if fmt == "e4m3" else swiglu_quant_int8)(gate_up, M, n // 2, q, s)
    return q, s


def _differentiable(*tensors):
    """Whether torch records a gradient for one of the tensors (None: no tensor)."""
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


class _Combine(torch.autograd.Function):
    """MoeRouting.combine with the gradients of rows, weights and residual."""

    @staticmethod
    def forward(ctx, rows, weights, residual, routing):
        ctx.routing = routing
        ctx.save_for_backward(rows if ctx.needs_input_grad[1] else None, weights)
        return routing._combine(rows, weights, residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        rows, weights = ctx.saved_tensors
        r, dy = ctx.routing, dy.contiguous()
        of_rows, of_weights, of_residual, _ = ctx.needs_input_grad
        # rows of no slot take part in nothing: their gradient is zero
        drows = torch.zeros((r.B * r.k, dy.shape[1]), dtype=dy.dtype, device=dy.device) if of_rows else None
        dw = torch.empty_like(weights) if of_weights else None
        if of_rows or of_weights:
            moe_combine_backward(dy, rows, r.row_of_slot, weights, r.B, r.k, dy.shape[1], drows, dw)
        return drows, dw, dy if of_residual else None, None


class _Gather(torch.autograd.Function):
    """The rows of MoeRouting.gather; their gradient is combine without weights."""

    @staticmethod
    def forward(ctx, rows, routing):
        ctx.routing = routing
        return routing._gather(rows, None)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, drows):
        return ctx.routing._combine(drows.contiguous(), None, None), None


class MoeRouting:
    """The slots of B tokens with k experts each, sorted by expert: `offsets` int32
    [E + 1] for the grouped products and `row_of_slot` int32 [B, k] (-1: no row).

    dispatch and gather carry gradients of bf16 rows, combine those of rows, weights and
    residual, where torch records them (a router trains over frozen experts).  As with
    torch's own operators, capture a backward pass into a graph only while no eager
    autograd graph of the same leaves is alive."""

    def __init__(self, offsets, row_of_slot):
        self.offsets, self.row_of_slot = offsets, row_of_slot
        self.B, self.k = row_of_slot.shape

    @classmethod
    def dispatch(cls, expert_ids, E, rows=None, row_scale=None, stream=None):
        """(routing, rows [B k, ...], scales [B k] or None) of int32 expert ids [B, k];
        rows: [B, K] bf16 activations, or 8-bit codes with their fp32 row_scale [B].
        Rows from offsets[E] on belong to no expert and are not written."""
        B, k = expert_ids.shape
        _is(expert_ids, (torch.int32,), (B, k), "expert_ids")
        if E < 1:
            raise ValueError(f"E must be positive, got {E}")
        if _differentiable(rows):
            with _on(stream, expert_ids):
                routing = cls.dispatch(expert_ids, E)[0]
                return (routing, *routing.gather(rows, row_scale))
        dev = expert_ids.device
        with _on(stream, expert_ids):
            offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
            row = torch.empty((B, k), dtype=torch.int32, device=dev)
            out, scale_out, width = cls._rows_out(rows, row_scale, B, k)
            need = moe_dispatch_workspace_bytes(B, k, E)
            ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
            moe_dispatch(expert_ids, rows, row_scale, B, k, E, width, offsets, row, out, scale_out, ws, need)
        return cls(offsets, row), out, scale_out

    @staticmethod
    def _rows_out(rows, row_scale, B, k):
        if rows is None:
            if row_scale is not None:
                raise ValueError("row_scale needs rows")
            return None, None, 0
        if rows.dim() != 2 or rows.shape[0] != B:
            raise ValueError(f"rows: expected [{B}, K], got {tuple(rows.shape)}")
        out = torch.empty((B * k, rows.shape[1]), dtype=rows.dtype, device=rows.device)
        scale_out = None
        if row_scale is not None:
            _is(row_scale, (torch.float32,), (B,), "row_scale")
            scale_out = torch.empty(B * k, dtype=torch.float32, device=rows.device)
        return out, scale_out, rows.shape[1] * rows.element_size()

    def _gather(self, rows, row_scale):
        out, scale_out, width = self._rows_out(rows, row_scale, self.B, self.k)
        moe_gather(rows, row_scale, self.row_of_slot, self.B, self.k, width, out, scale_out)
        return out, scale_out

    def gather(self, rows, row_scale=None, stream=None):
        """(rows [B k, K], scales or None): another tensor's rows in the routed order."""
        with _on(stream, rows):
            if not _differentiable(rows):
                return self._gather(rows, row_scale)
            if rows.dtype != torch.bfloat16 or row_scale is not None:
                raise TypeError("gradients of routed rows are those of bf16 rows without scales; detach others")
            return _Gather.apply(rows, self), None

    def _weights(self, weights):
        return None if weights is None else _is(weights, (torch.float32,), (self.B, self.k), "weights")

    def combine(self, rows, weights=None, residual=None, out=None, stream=None):
        """sum_j weights[b, j] rows[row_of_slot[b, j]] + residual[b], bf16 [B, K].
        Without weights and residual: the gradient of dispatch's and gather's rows."""
        K = rows.shape[1]
        _is(rows, _BF16, (self.B * self.k, K), "rows")
        if residual is not None:
            _is(residual, _BF16, (self.B, K), "residual")
        with _on(stream, rows):
            if not _differentiable(rows, weights, residual):
                return self._combine(rows, weights, residual, out)
            if out is not None:
                raise RuntimeError("combine(out=...) carries no gradient; leave out= or detach its inputs")
            return _Combine.apply(rows, weights, residual, self)

    def _combine(self, rows, weights, residual, out=None):
        K = rows.shape[1]
        y = _is(out, _BF16, (self.B, K), "out") if out is not None else \
            torch.empty((self.B, K), dtype=torch.bfloat16, device=rows.device)
        moe_combine(rows, self.row_of_slot, self._weights(weights), residual, self.B, self.k, K, y)
        return y

    def combine_backward(self, dy, rows, weights=None, stream=None):
        """(drows bf16 [B k, K], dweights fp32 [B, k]) of combine; rows of no slot are not written."""
        K = dy.shape[1]
        _is(dy, _BF16, (self.B, K), "dy")
        _is(rows, _BF16, (self.B * self.k, K), "rows")
        with _on(stream, dy):
            drows = torch.empty((self.B * self.k, K), dtype=torch.bfloat16, device=dy.device)
            dw = torch.empty((self.B, self.k), dtype=torch.float32, device=dy.device)
            moe_combine_backward(dy, rows, self.row_of_slot, self._weights(weights), self.B, self.k, K, drows, dw)
        return drows, dw

"""Python binding of librudder (ctypes).

Argument marshalling only: every step of the layer runs in the HIP kernels
behind the C ABI declared in include/.  torch supplies device memory
and the current HIP stream.  If the library is missing this module raises;
there is no CPU fallback.

The calls keep their C names and meanings:
  rudder_quantize_weights  -- offline weight preparation (SteerQuant Fig. 2, §4.2)
  rudder_quant_act         -- fused activation quantization (SteerQuant §4.3, §4.4)
  rudder_linear            -- low-bit GEMM + fused epilogue (SteerQuant §4.4)
  rudder_linear_gelu_quant -- MLP up-projection with GELU (kept in BF16, App. D)
                              and the down layer's quantizer in its epilogue
  rudder_gelu_bf16         -- that GELU alone, elementwise
  rudder_quantize_weights_grouped, rudder_matvec_w4
                           -- few-row products with group-scaled 4-bit weights
  rudder_cache_append, rudder_cache_dequant
                           -- the paged 8-bit cache of keys and values
  rudder_cache_attention, rudder_cross_attention
                           -- attention over that cache, and to bf16 states
  rudder_norm, rudder_norm_quant, rudder_dequant_act
                           -- the RMS norm with the residual's addition, its rows or
                              the next linear's codes, and codes back as values
  rudder_rotary, rudder_rotary_frequencies
                           -- rotary positions on queries and keys
  rudder_prompt_attention  -- causal attention of whole prompts
(SteerQuant = "SteerQuant: Steering Quantization Error with Action-Guided
Scaling in World-Action Models", paperlayer.ai digest.)
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "librudder.so")
BIND_PATH = os.path.join(HERE, "_lib", "rudder_bind.so")

CODES_INT = 0       # int4 split-nibble / int8 codes (int8 matrix cores)
CODES_E2M3 = 1      # codes held as FP6 E2M3 (8-bit codes as two digit planes); f8f6f4 MFMA

RUDDER_OK = 0
RUDDER_ERR_INVALID_ARG = 1
RUDDER_ERR_UNSUPPORTED = 2
RUDDER_ERR_HIP = 3
MAX_STREAMS = 8
CACHE_PAGE = 64     # tokens of a cache page
ROTARY_HALF = 0     # rotary pairs: channels i and i + n of the rotated part
ROTARY_PAIRS = 1    # channels 2 i and 2 i + 1
ROTARY_SCALING = {"plain": 0, "linear": 1, "base": 2, "parts": 3}

EXPORTED = (
    "rudder_packed_weight_bytes", "rudder_packed_act_bytes", "rudder_quant_act_workspace_bytes",
    "rudder_quantize_weights", "rudder_quant_act", "rudder_quant_act_noalloc", "rudder_linear",
    "rudder_linear_gelu_quant", "rudder_gelu_bf16",
    "rudder_dequant_weights", "rudder_stream_sq_error_workspace_bytes", "rudder_stream_sq_error",
    "rudder_status_string", "rudder_last_error",
    "rudder_mfma_ceiling_sink_bytes", "rudder_mfma_ceiling_ops", "rudder_mfma_ceiling",
    "rudder_mfma_ceiling_shape",
    "rudder_grouped_weight_bytes", "rudder_grouped_scale_count",
    "rudder_quantize_weights_grouped", "rudder_matvec_w4",
    "rudder_cache_page_bytes", "rudder_cache_append", "rudder_cache_dequant",
    "rudder_attention_workspace_bytes", "rudder_attention_workspace_bound",
    "rudder_cache_attention", "rudder_cross_attention",
    "rudder_norm", "rudder_norm_quant", "rudder_dequant_act", "rudder_rotary_frequencies",
    "rudder_rotary", "rudder_prompt_attention_workspace_bytes", "rudder_prompt_attention",
)

_lib: Optional[ctypes.CDLL] = None
_bind = None


class RudderError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def load_library() -> ctypes.CDLL:
    """Load the in-tree librudder.so; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RudderError(RUDDER_ERR_HIP,
                          f"{LIB_PATH} not found: build it with __graft_entry__.build() "
                          "or python w4a4_quantized_gemm_rudder_amd/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.rudder_packed_weight_bytes.argtypes = [i, i, i]
    lib.rudder_packed_weight_bytes.restype = sz
    lib.rudder_packed_act_bytes.argtypes = [i, i, i, i]
    lib.rudder_packed_act_bytes.restype = sz
    lib.rudder_quant_act_workspace_bytes.argtypes = [i]
    lib.rudder_quant_act_workspace_bytes.restype = sz
    lib.rudder_quantize_weights.argtypes = [vp, vp, i, i, i, vp, vp, vp, vp]
    lib.rudder_quantize_weights.restype = i
    lib.rudder_quant_act.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, vp, vp]
    lib.rudder_quant_act.restype = i
    lib.rudder_quant_act_noalloc.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp, vp, vp]
    lib.rudder_quant_act_noalloc.restype = i
    lib.rudder_linear.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, vp, vp]
    lib.rudder_linear.restype = i
    lib.rudder_linear_gelu_quant.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                             vp, vp, i, i, vp, vp, vp]
    lib.rudder_linear_gelu_quant.restype = i
    lib.rudder_gelu_bf16.argtypes = [vp, vp, sz, vp]
    lib.rudder_gelu_bf16.restype = i
    lib.rudder_dequant_weights.argtypes = [vp, vp, i, i, i, vp, vp]
    lib.rudder_dequant_weights.restype = i
    lib.rudder_stream_sq_error_workspace_bytes.argtypes = []
    lib.rudder_stream_sq_error_workspace_bytes.restype = sz
    lib.rudder_stream_sq_error.argtypes = [vp, vp, vp, i, i, i, vp, vp, vp]
    lib.rudder_stream_sq_error.restype = i
    lib.rudder_mfma_ceiling_sink_bytes.argtypes = []
    lib.rudder_mfma_ceiling_sink_bytes.restype = sz
    lib.rudder_mfma_ceiling_ops.argtypes = [i, i]
    lib.rudder_mfma_ceiling_ops.restype = ctypes.c_double
    lib.rudder_mfma_ceiling.argtypes = [vp, vp, i, i, i, i, i, i, vp, vp]
    lib.rudder_mfma_ceiling.restype = i
    lib.rudder_mfma_ceiling_shape.argtypes = [vp, vp, i, i, i, i, i, i, i, vp, vp]
    lib.rudder_mfma_ceiling_shape.restype = i
    f = ctypes.c_float
    lib.rudder_grouped_weight_bytes.argtypes = [i, i]
    lib.rudder_grouped_weight_bytes.restype = sz
    lib.rudder_grouped_scale_count.argtypes = [i, i, i]
    lib.rudder_grouped_scale_count.restype = sz
    lib.rudder_quantize_weights_grouped.argtypes = [vp, i, i, i, vp, vp, vp]
    lib.rudder_quantize_weights_grouped.restype = i
    lib.rudder_matvec_w4.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, vp]
    lib.rudder_matvec_w4.restype = i
    lib.rudder_cache_page_bytes.argtypes = [i, i]
    lib.rudder_cache_page_bytes.restype = sz
    lib.rudder_cache_append.argtypes = [vp, vp, vp, vp, vp] + [i] * 9 + [vp, vp, vp]
    lib.rudder_cache_append.restype = i
    lib.rudder_cache_dequant.argtypes = [vp, vp, vp, i, i, i, i, vp, vp, vp]
    lib.rudder_cache_dequant.restype = i
    lib.rudder_attention_workspace_bytes.argtypes = [i] * 7
    lib.rudder_attention_workspace_bytes.restype = sz
    lib.rudder_attention_workspace_bound.argtypes = [i] * 7
    lib.rudder_attention_workspace_bound.restype = sz
    lib.rudder_cache_attention.argtypes = [vp] * 6 + [i] * 11 + [f, i, vp, sz, vp, vp]
    lib.rudder_cache_attention.restype = i
    lib.rudder_cross_attention.argtypes = [vp] * 6 + [i] * 12 + [f, vp, sz, vp, vp]
    lib.rudder_cross_attention.restype = i
    d = ctypes.c_double
    lib.rudder_norm.argtypes = [vp, vp, vp, f] + [i] * 6 + [vp, vp, vp]
    lib.rudder_norm.restype = i
    lib.rudder_norm_quant.argtypes = [vp] * 6 + [f] + [i] * 8 + [vp, vp, vp, vp]
    lib.rudder_norm_quant.restype = i
    lib.rudder_dequant_act.argtypes = [vp, vp, i, i, i, i, vp, vp]
    lib.rudder_dequant_act.restype = i
    lib.rudder_rotary_frequencies.argtypes = [i, d, i, d, d, d, d, vp]
    lib.rudder_rotary_frequencies.restype = i
    lib.rudder_rotary.argtypes = [vp] * 5 + [f] + [i] * 12 + [vp, vp, vp]
    lib.rudder_rotary.restype = i
    lib.rudder_prompt_attention_workspace_bytes.argtypes = [i] * 6
    lib.rudder_prompt_attention_workspace_bytes.restype = sz
    lib.rudder_prompt_attention.argtypes = [vp] * 4 + [i] * 10 + [f, vp, sz, vp, vp]
    lib.rudder_prompt_attention.restype = i
    lib.rudder_status_string.argtypes = [i]
    lib.rudder_status_string.restype = ctypes.c_char_p
    lib.rudder_last_error.argtypes = []
    lib.rudder_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _load_bind():
    """The module that checks and passes on the arguments of the operators between
    the linears, bound to the loaded library; raises if it has not been built."""
    global _bind
    import importlib.util
    import torch  # noqa: F401  (its libraries come first)
    load_library()
    if not os.path.exists(BIND_PATH):
        raise RudderError(RUDDER_ERR_HIP,
                          f"{BIND_PATH} not found: build it with __graft_entry__.build() "
                          "or python -m w4a4_quantized_gemm_rudder_amd.build")
    spec = importlib.util.spec_from_file_location("rudder_bind", BIND_PATH)
    bind = importlib.util.module_from_spec(spec)
    bind.use(LIB_PATH)
    _bind = bind
    return bind


def _check(status: int) -> None:
    if status:
        lib = load_library()
        name = lib.rudder_status_string(status).decode()
        raise RudderError(status, f"{name}: {lib.rudder_last_error().decode()}")


def _ptr(t) -> Optional[int]:
    """Device address of a tensor (None -> NULL).  Plain ints pass through."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to librudder must be contiguous")
    return t.data_ptr()


_raw_stream = _get_device = None


def _current_stream() -> int:
    """Handle of torch's current stream on the current device."""
    if _raw_stream is None:
        _stream_getters()
    return _raw_stream(_get_device())


def _stream_getters() -> None:
    global _raw_stream, _get_device
    import torch
    torch.cuda.init()
    _get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    # the raw handle without a Stream object: a third of the time of current_stream()
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda device: torch.cuda.current_stream(device).cuda_stream)


def _device_and_stream(stream) -> Tuple[int, int]:
    """The current device (-1: none in use yet), where the operators between the linears want all
    of their tensors, and the handle of `stream` (None: the current one)."""
    if stream is None:
        if _raw_stream is None:
            _stream_getters()
        device = _get_device()
        return device, _raw_stream(device)
    import torch
    device = -1
    if torch.cuda.is_initialized():
        if _get_device is None:
            _stream_getters()
        device = _get_device()
    if isinstance(stream, int):
        return device, stream
    of = getattr(stream, "device_index", device)
    if of != device:
        raise ValueError(f"a stream of cuda:{of}, but the current device is cuda:{device}")
    return device, stream.cuda_stream


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---------------------------------------------------------------------------
# Size helpers
# ---------------------------------------------------------------------------

def packed_weight_bytes(K: int, N: int, codes: int = CODES_INT) -> int:
    return int(load_library().rudder_packed_weight_bytes(K, N, codes))


def packed_act_bytes(M: int, K: int, abits: int, codes: int = CODES_INT) -> int:
    return int(load_library().rudder_packed_act_bytes(M, K, abits, codes))


def quant_act_workspace_bytes(S: int) -> int:
    return int(load_library().rudder_quant_act_workspace_bytes(S))


# ---------------------------------------------------------------------------
# The three calls (same names and argument order as the C ABI, sizes passed
# explicitly; tensors are device tensors, bf16 data as torch.bfloat16 or
# int16/uint16 bit patterns)
# ---------------------------------------------------------------------------

def rudder_quantize_weights(W, smooth, K: int, N: int, codes: int, Wq, w_scale, inv_smooth,
                            stream=None) -> None:
    _check(load_library().rudder_quantize_weights(
        _ptr(W), _ptr(smooth), K, N, codes, _ptr(Wq), _ptr(w_scale), _ptr(inv_smooth),
        _stream(stream)))


def rudder_quant_act(X, stream_id, inv_smooth, act_scale, act_scale_out, workspace,
                     M: int, K: int, S: int, abits: int, codes: int, Xq, row_scale,
                     stream=None) -> None:
    _check(load_library().rudder_quant_act(
        _ptr(X), _ptr(stream_id), _ptr(inv_smooth), _ptr(act_scale), _ptr(act_scale_out),
        _ptr(workspace), M, K, S, abits, codes, _ptr(Xq), _ptr(row_scale), _stream(stream)))


def rudder_quant_act_noalloc(X, stream_id, inv_smooth, act_scale_out, M: int, K: int, S: int,
                             abits: int, codes: int, Xq, row_scale, stream=None) -> None:
    _check(load_library().rudder_quant_act_noalloc(
        _ptr(X), _ptr(stream_id), _ptr(inv_smooth), _ptr(act_scale_out), M, K, S, abits, codes,
        _ptr(Xq), _ptr(row_scale), _stream(stream)))


def rudder_linear(Xq, row_scale, stream_id, Wq, w_scale, comp_a, comp_b,
                  M: int, N: int, K: int, S: int, abits: int, codes: int, Y, acc_out=None,
                  stream=None) -> None:
    _check(load_library().rudder_linear(
        _ptr(Xq), _ptr(row_scale), _ptr(stream_id), _ptr(Wq), _ptr(w_scale), _ptr(comp_a),
        _ptr(comp_b), M, N, K, S, abits, codes, _ptr(Y), _ptr(acc_out), _stream(stream)))


def rudder_linear_gelu_quant(Xq, row_scale, stream_id, Wq, w_scale, comp_a, comp_b,
                             M: int, N: int, K: int, S: int, abits: int, codes: int,
                             next_inv_smooth, next_act_scale, next_abits: int, next_codes: int,
                             next_Xq, next_row_scale, stream=None) -> None:
    _check(load_library().rudder_linear_gelu_quant(
        _ptr(Xq), _ptr(row_scale), _ptr(stream_id), _ptr(Wq), _ptr(w_scale), _ptr(comp_a),
        _ptr(comp_b), M, N, K, S, abits, codes, _ptr(next_inv_smooth), _ptr(next_act_scale),
        next_abits, next_codes, _ptr(next_Xq), _ptr(next_row_scale), _stream(stream)))


def rudder_gelu_bf16(x, out, n: int, stream=None) -> None:
    _check(load_library().rudder_gelu_bf16(_ptr(x), _ptr(out), n, _stream(stream)))


def rudder_dequant_weights(Wq, w_scale, K: int, N: int, codes: int, out, stream=None) -> None:
    _check(load_library().rudder_dequant_weights(_ptr(Wq), _ptr(w_scale), K, N, codes, _ptr(out),
                                                 _stream(stream)))


def stream_sq_error_workspace_bytes() -> int:
    return int(load_library().rudder_stream_sq_error_workspace_bytes())


def rudder_stream_sq_error(Y, Yref, stream_id, M: int, N: int, S: int, workspace, sse,
                           stream=None) -> None:
    _check(load_library().rudder_stream_sq_error(_ptr(Y), _ptr(Yref), _ptr(stream_id), M, N, S,
                                                 _ptr(workspace), _ptr(sse), _stream(stream)))


# ---------------------------------------------------------------------------
# Few-row products, cache and attention (include/rudder_attention.h).  Tensors
# are checked for their type, layout and size against the sizes passed and for
# the current device, in csrc/bind.cpp: in Python that took as long as the
# smallest calls.  Device addresses (ints) pass through unchecked.
# ---------------------------------------------------------------------------

def grouped_weight_bytes(K: int, N: int) -> int:
    return int(load_library().rudder_grouped_weight_bytes(K, N))


def grouped_scale_count(K: int, N: int, group: int) -> int:
    return int(load_library().rudder_grouped_scale_count(K, N, group))


def rudder_quantize_weights_grouped(W, K: int, N: int, group: int, Wq, g_scale,
                                    stream=None) -> None:
    bind = _bind or _load_bind()
    device, handle = _device_and_stream(stream)
    _check(bind.quantize_weights_grouped(device, W, K, N, group, Wq, g_scale, handle))


def rudder_matvec_w4(X, stream_id, Wq, g_scale, comp_a, comp_b, M: int, N: int, K: int,
                     group: int, S: int, Y, stream=None) -> None:
    bind = _bind or _load_bind()
    device, handle = _device_and_stream(stream)
    _check(bind.matvec_w4(device, X, stream_id, Wq, g_scale, comp_a, comp_b, M, N, K, group, S, Y,
                          handle))


def cache_page_bytes(Hkv: int, D: int) -> int:
    return int(load_library().rudder_cache_page_bytes(Hkv, D))


def rudder_cache_append(K, V, row_start, pos, page_table, B: int, T: int, max_rows: int,
                        max_pages: int, num_pages: int, Hkv: int, D: int, codes, scales,
                        stream=None, ldk=None, ldv=None) -> None:
    """K, V: [T, Hkv, D] or [T, Hkv * D], rows any distance apart."""
    bind = _bind or _load_bind()
    device, handle = _device_and_stream(stream)
    _check(bind.cache_append(device, K, V, row_start, pos, page_table, B, T, max_rows, max_pages,
                             num_pages, Hkv, D, codes, scales, handle, ldk, ldv))


def rudder_cache_dequant(codes, scales, pages, n: int, num_pages: int, Hkv: int, D: int, K_out,
                         V_out, stream=None) -> None:
    bind = _bind or _load_bind()
    device, handle = _device_and_stream(stream)
    _check(bind.cache_dequant(device, codes, scales, pages, n, num_pages, Hkv, D, K_out, V_out,
                              handle))


def attention_workspace_bytes(B: int, T: int, max_rows: int, max_kv: int, Hq: int, Hkv: int,
                              D: int) -> int:
    return int(load_library().rudder_attention_workspace_bytes(B, T, max_rows, max_kv, Hq, Hkv,
                                                               D))


def attention_workspace_bound(B: int, T: int, max_rows: int, max_kv: int, Hq: int, Hkv: int,
                              D: int) -> int:
    """Bytes that suffice for every call of these heads with B, T, max_rows and max_kv up to
    these; attention_workspace_bytes of a smaller call may be larger than a larger one's."""
    return int(load_library().rudder_attention_workspace_bound(B, T, max_rows, max_kv, Hq, Hkv,
                                                               D))


def rudder_cache_attention(Q, row_start, kv_len, page_table, codes, scales, B: int, T: int,
                           max_rows: int, max_kv: int, max_pages: int, num_pages: int, Hq: int,
                           Hkv: int, D: int, sm: float, causal: bool, workspace, O, stream=None,
                           ldq=None, ldo=None) -> None:
    """Q, O: [T, Hq, D] or [T, Hq * D], rows any distance apart."""
    bind = _bind or _load_bind()
    device, handle = _device_and_stream(stream)
    _check(bind.cache_attention(device, Q, row_start, kv_len, page_table, codes, scales, B, T,
                                max_rows, max_kv, max_pages, num_pages, Hq, Hkv, D, sm, causal,
                                workspace, O, handle, ldq, ldo))


def rudder_cross_attention(Q, K, V, row_start, kv_start, kv_len, B: int, T: int, Tkv: int,
                           max_rows: int, max_kv: int, Hq: int, Hkv: int, D: int, sm: float,
                           workspace, O, stream=None, ldq=None, ldk=None, ldv=None,
                           ldo=None) -> None:
    bind = _bind or _load_bind()
    device, handle = _device_and_stream(stream)
    _check(bind.cross_attention(device, Q, K, V, row_start, kv_start, kv_len, B, T, Tkv, max_rows,
                                max_kv, Hq, Hkv, D, sm, workspace, O, handle, ldq, ldk, ldv, ldo))


# ---------------------------------------------------------------------------
# Norms, rotary positions and prompt attention (include/rudder_block.h), checked
# in the same place
# ---------------------------------------------------------------------------

def rudder_norm(X, R, gamma, eps: float, M: int, K: int, H, Y, stream=None, ldx=None, ldr=None,
                ldh=None, ldy=None) -> None:
    """X, R, H, Y: [M, K], rows any distance apart; R and H both or neither."""
    bind = _bind or _load_bind()
    device, handle = _device_and_stream(stream)
    _check(bind.norm(device, X, R, gamma, eps, M, K, H, Y, handle, ldx, ldr, ldh, ldy))


def rudder_norm_quant(X, R, stream_id, gamma, inv_smooth, act_scale, eps: float, M: int, K: int,
                      S: int, abits: int, codes: int, H, Xq, row_scale, stream=None, ldx=None,
                      ldr=None, ldh=None) -> None:
    """X, R, H: [M, K], rows any distance apart; act_scale None: a step size a row."""
    bind = _bind or _load_bind()
    device, handle = _device_and_stream(stream)
    _check(bind.norm_quant(device, X, R, stream_id, gamma, inv_smooth, act_scale, eps, M, K, S,
                           abits, codes, H, Xq, row_scale, handle, ldx, ldr, ldh))


def rudder_dequant_act(Xq, row_scale, M: int, K: int, abits: int, codes: int, out,
                       stream=None) -> None:
    bind = _bind or _load_bind()
    device, handle = _device_and_stream(stream)
    _check(bind.dequant_act(device, Xq, row_scale, M, K, abits, codes, out, handle))


def rudder_rotary_frequencies(rotary_dim: int, base: float, scaling: int, factor: float,
                              trained: float, low: float, high: float, freq) -> None:
    """freq: a contiguous fp64 tensor of rotary_dim / 2 elements in host memory."""
    import torch
    if (freq.dtype != torch.float64 or freq.device.type != "cpu" or not freq.is_contiguous()
            or freq.numel() < rotary_dim // 2):
        raise ValueError("freq: at least rotary_dim / 2 contiguous fp64 elements in host memory "
                         "expected")
    _check(load_library().rudder_rotary_frequencies(rotary_dim, base, scaling, factor, trained,
                                                    low, high, _ptr(freq)))


def rudder_rotary(Q, K, row_start, pos, freq, magnitude: float, B: int, T: int, max_rows: int,
                  Hq: int, Hkv: int, D: int, rotary_dim: int, layout: int, Qo, Ko, stream=None,
                  ldq=None, ldk=None, ldqo=None, ldko=None) -> None:
    """Q, K, Qo, Ko: [T, H, D] or [T, H * D], rows any distance apart; Qo and Ko may be Q and K."""
    bind = _bind or _load_bind()
    device, handle = _device_and_stream(stream)
    _check(bind.rotary(device, Q, K, row_start, pos, freq, magnitude, B, T, max_rows, Hq, Hkv, D,
                       rotary_dim, layout, Qo, Ko, handle, ldq, ldk, ldqo, ldko))


def prompt_attention_workspace_bytes(B: int, T: int, max_rows: int, Hq: int, Hkv: int,
                                     D: int) -> int:
    return int(load_library().rudder_prompt_attention_workspace_bytes(B, T, max_rows, Hq, Hkv, D))


def rudder_prompt_attention(Q, K, V, row_start, B: int, T: int, max_rows: int, Hq: int, Hkv: int,
                            D: int, sm: float, workspace, O, stream=None, ldq=None, ldk=None,
                            ldv=None, ldo=None) -> None:
    """Q, K, V, O: [T, H, D] or [T, H * D], rows any distance apart."""
    bind = _bind or _load_bind()
    device, handle = _device_and_stream(stream)
    _check(bind.prompt_attention(device, Q, K, V, row_start, B, T, max_rows, Hq, Hkv, D, sm,
                                 workspace, O, handle, ldq, ldk, ldv, ldo))


# ---------------------------------------------------------------------------
# Allocating conveniences (torch allocates; the library computes)
# ---------------------------------------------------------------------------

def quantize_weights(W, smooth, codes: int = CODES_INT, stream=None):
    """W: bf16 [K, N] device tensor, smooth: fp32 [K].
    Returns (Wq uint8, w_scale fp32 [N], inv_smooth fp32 [K])."""
    import torch
    K, N = W.shape
    dev = W.device
    Wq = torch.empty(packed_weight_bytes(K, N, codes), dtype=torch.uint8, device=dev)
    w_scale = torch.empty(N, dtype=torch.float32, device=dev)
    inv_smooth = torch.empty(K, dtype=torch.float32, device=dev)
    rudder_quantize_weights(W, smooth, K, N, codes, Wq, w_scale, inv_smooth, stream)
    return Wq, w_scale, inv_smooth


def quant_act(X, stream_id, inv_smooth, act_scale, S: int, abits: int, codes: int = CODES_INT,
              stream=None, act_scale_out=None, workspace=None):
    """X: bf16 [M, K].  act_scale: fp32 [S] device tensor, or None for dynamic
    (absmax) step sizes.  Returns (Xq uint8, row_scale fp32 [M])."""
    import torch
    M, K = X.shape
    dev = X.device
    Xq = torch.empty(max(packed_act_bytes(M, K, abits, codes), 1), dtype=torch.uint8,
                     device=dev)
    row_scale = torch.empty(max(M, 1), dtype=torch.float32, device=dev)
    if act_scale is None and workspace is None:
        workspace = torch.empty(quant_act_workspace_bytes(S), dtype=torch.uint8, device=dev)
    rudder_quant_act(X, stream_id, inv_smooth, act_scale, act_scale_out, workspace, M, K, S,
                     abits, codes, Xq, row_scale, stream)
    return Xq, row_scale


def linear(Xq, row_scale, stream_id, Wq, w_scale, comp_a, comp_b, M: int, N: int, K: int,
           S: int, abits: int, codes: int = CODES_INT, stream=None, acc_out: bool = False):
    """Returns Y bf16 [M, N] (and int32 accumulators [M, N] if acc_out)."""
    import torch
    dev = Wq.device
    Y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    acc = torch.empty((M, N), dtype=torch.int32, device=dev) if acc_out else None
    rudder_linear(Xq, row_scale, stream_id, Wq, w_scale, comp_a, comp_b, M, N, K, S, abits,
                  codes, Y, acc, stream)
    return (Y, acc) if acc_out else Y


def linear_gelu_quant(Xq, row_scale, stream_id, Wq, w_scale, comp_a, comp_b, M: int, N: int,
                      K: int, S: int, abits: int, next_inv_smooth, next_act_scale,
                      next_abits: int, codes: int = CODES_INT, next_codes: int = CODES_INT,
                      stream=None):
    """Returns (next Xq uint8, next row_scale fp32 [M]): the down layer's
    packed input and row scales, from the up-projection's codes."""
    import torch
    dev = Wq.device
    nxq = torch.empty(max(packed_act_bytes(M, N, next_abits, next_codes), 1), dtype=torch.uint8,
                      device=dev)
    nrs = torch.empty(max(M, 1), dtype=torch.float32, device=dev)
    rudder_linear_gelu_quant(Xq, row_scale, stream_id, Wq, w_scale, comp_a, comp_b, M, N, K, S,
                             abits, codes, next_inv_smooth, next_act_scale, next_abits,
                             next_codes, nxq, nrs, stream)
    return nxq, nrs


def gelu_bf16(x, stream=None):
    """GELU of a bf16 tensor (same table as the fused epilogue)."""
    import torch
    out = torch.empty_like(x)
    rudder_gelu_bf16(x, out, x.numel(), stream)
    return out


def _on(stream, device):
    """Context in which `stream` (None: the current one) and its device are
    current, so that what is allocated and cleared inside belongs to it."""
    import torch
    if stream is None:
        return torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


def quantize_weights_grouped(W, group: int, stream=None):
    """W: bf16 [K, N] device tensor.  Returns (Wq uint8, g_scale bf16) for matvec_w4."""
    import torch
    K, N = W.shape
    with _on(stream, W.device):
        Wq = torch.empty(grouped_weight_bytes(K, N), dtype=torch.uint8, device=W.device)
        g_scale = torch.empty(grouped_scale_count(K, N, group), dtype=torch.bfloat16,
                              device=W.device)
        rudder_quantize_weights_grouped(W, K, N, group, Wq, g_scale)
    return Wq, g_scale


@functools.lru_cache(maxsize=None)
def _grouped_sizes(K: int, N: int, group: int) -> Tuple[int, int]:
    return grouped_weight_bytes(K, N), grouped_scale_count(K, N, group)


def matvec_w4(X, Wq, g_scale, N: int, group: int, stream_id=None, comp_a=None, comp_b=None,
              stream=None):
    """X: bf16 [M, K], weights from quantize_weights_grouped, optionally the
    per-stream compensation (stream_id uint8 [M], comp_a and comp_b fp32
    [S, N]).  Returns Y bf16 [M, N]."""
    import torch
    M, K = X.shape
    if (Wq.numel(), g_scale.numel()) != _grouped_sizes(K, N, group):
        raise ValueError(f"Wq of {Wq.numel()} bytes and {g_scale.numel()} scales are not those of "
                         f"K={K}, N={N}, group={group}")
    S = 1 if comp_a is None else comp_a.shape[0]
    with _on(stream, X.device):
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
        if M:
            rudder_matvec_w4(X, stream_id, Wq, g_scale, comp_a, comp_b, M, N, K, group, S, Y)
    return Y


def new_cache(num_pages: int, Hkv: int, D: int, device="cuda"):
    """An empty cache: (codes int8 [num_pages, Hkv, 2, 64 * D], scales fp32
    [num_pages, Hkv, 2])."""
    import torch
    return (torch.zeros(num_pages, Hkv, 2, CACHE_PAGE * D, dtype=torch.int8, device=device),
            torch.zeros(num_pages, Hkv, 2, dtype=torch.float32, device=device))


def _check_cache(codes, Hkv: int, D: int) -> None:
    page = (Hkv, 2, CACHE_PAGE * D)
    good = (tuple(codes.shape[1:]) == page if codes.dim() == 4 else
            codes.numel() == codes.shape[0] * Hkv * page[1] * page[2])
    if not good:
        raise ValueError(f"codes {tuple(codes.shape)} are not pages of {Hkv} heads of {D} channels")


def cache_append(K, V, row_start, pos, page_table, max_rows: int, codes, scales,
                 stream=None) -> None:
    """Quantizes K, V [T, Hkv, D] into the cache at pos [B] (see
    include/rudder_attention.h)."""
    B, max_pages = page_table.shape
    T, Hkv, D = K.shape
    _check_cache(codes, Hkv, D)
    if T == 0 or B == 0:
        return
    with _on(stream, codes.device):
        rudder_cache_append(K, V, row_start, pos, page_table, B, T, max_rows, max_pages,
                            codes.shape[0], Hkv, D, codes, scales)


def cache_dequant(codes, scales, pages, stream=None):
    """The values of whole pages (int32 [n]): K and V, fp32 [n, Hkv, 64, D]."""
    import torch
    num_pages, Hkv = codes.shape[:2]
    n, D = pages.numel(), codes.shape[3] // CACHE_PAGE
    with _on(stream, codes.device):
        K_out = torch.empty(n, Hkv, CACHE_PAGE, D, dtype=torch.float32, device=codes.device)
        V_out = torch.empty_like(K_out)
        if n:
            rudder_cache_dequant(codes, scales, pages, n, num_pages, Hkv, D, K_out, V_out)
    return K_out, V_out


def _attention_buffers(Q, B, max_rows, max_kv, Hkv):
    import torch
    T, Hq, D = Q.shape
    n = attention_workspace_bytes(B, T, max_rows, max_kv, Hq, Hkv, D)
    ws = torch.empty(n, dtype=torch.uint8, device=Q.device) if n else None
    return ws, torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=Q.device)


def cache_attention(Q, row_start, kv_len, page_table, codes, scales, max_rows: int, max_kv: int,
                    sm: float, causal: bool = True, stream=None):
    """Attention of Q bf16 [T, Hq, D] to the cache.  Returns O bf16 [T, Hq, D]
    (zeros in rows of no sequence)."""
    B, max_pages = page_table.shape
    T, Hq, D = Q.shape
    num_pages, Hkv = codes.shape[:2]
    _check_cache(codes, Hkv, D)
    with _on(stream, Q.device):
        ws, O = _attention_buffers(Q, B, max_rows, max_kv, Hkv)
        if T and B:
            rudder_cache_attention(Q, row_start, kv_len, page_table, codes, scales, B, T,
                                   max_rows, max_kv, max_pages, num_pages, Hq, Hkv, D, sm,
                                   causal, ws, O)
    return O


def cross_attention(Q, K, V, row_start, kv_start, kv_len, max_rows: int, max_kv: int, sm: float,
                    stream=None):
    """Cross attention of Q bf16 [T, Hq, D] to K, V bf16 [Tkv, Hkv, D].
    Returns O bf16 [T, Hq, D] (zeros in rows of no sequence)."""
    B = kv_len.numel()
    T, Hq, D = Q.shape
    Tkv, Hkv = K.shape[:2]
    with _on(stream, Q.device):
        ws, O = _attention_buffers(Q, B, max_rows, max_kv, Hkv)
        if T and B and Tkv:
            rudder_cross_attention(Q, K, V, row_start, kv_start, kv_len, B, T, Tkv, max_rows,
                                   max_kv, Hq, Hkv, D, sm, ws, O)
    return O


def _check_channels(K: int, **vectors) -> None:
    for name, v in vectors.items():
        if v.numel() != K:
            raise ValueError(f"{name} of {v.numel()} elements does not fit K={K} channels")


def norm(X, gamma, eps: float, residual=None, stream=None):
    """RMS norm of X bf16 [M, K], gamma fp32 [K].  Returns Y bf16 [M, K]; with `residual` [M, K]
    (Y, H) of the sum H = bf16(residual + X)."""
    import torch
    M, K = X.shape
    _check_channels(K, gamma=gamma)
    with _on(stream, X.device):
        Y = torch.empty(M, K, dtype=torch.bfloat16, device=X.device)
        H = None if residual is None else torch.empty_like(Y)
        if M:
            rudder_norm(X, residual, gamma, eps, M, K, H, Y)
    return Y if H is None else (Y, H)


def norm_quant(X, gamma, inv_smooth, eps: float, abits: int, codes: int = CODES_INT,
               stream_id=None, act_scale=None, residual=None, stream=None):
    """The same norm as the next linear's packed codes: with stream_id uint8 [M] and act_scale
    fp32 [S] the table's step sizes, without them one a row.  Returns (Xq uint8, row_scale fp32
    [M]), with `residual` (Xq, row_scale, H)."""
    import torch
    M, K = X.shape
    _check_channels(K, gamma=gamma, inv_smooth=inv_smooth)
    S = 1 if act_scale is None else act_scale.numel()
    with _on(stream, X.device):
        Xq = torch.empty(max(packed_act_bytes(M, K, abits, codes), 1), dtype=torch.uint8,
                         device=X.device)
        row_scale = torch.empty(max(M, 1), dtype=torch.float32, device=X.device)
        H = None
        if residual is not None:
            H = torch.empty(M, K, dtype=torch.bfloat16, device=X.device)
        if M:
            rudder_norm_quant(X, residual, stream_id, gamma, inv_smooth, act_scale, eps, M, K, S,
                              abits, codes, H, Xq, row_scale)
    return (Xq, row_scale) if H is None else (Xq, row_scale, H)


def dequant_act(Xq, row_scale, M: int, K: int, abits: int, codes: int = CODES_INT, stream=None):
    """The values of packed activation codes, fp32 [M, K]."""
    import torch
    if Xq.numel() != max(packed_act_bytes(M, K, abits, codes), 1):
        raise ValueError(f"Xq of {Xq.numel()} bytes are not the codes of M={M}, K={K}, "
                         f"abits={abits}, codes={codes}")
    with _on(stream, Xq.device):
        out = torch.empty(M, K, dtype=torch.float32, device=Xq.device)
        if M:
            rudder_dequant_act(Xq, row_scale, M, K, abits, codes, out)
    return out


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "plain",
                       factor: float = 1.0, trained: float = 0.0, low: float = 1.0,
                       high: float = 32.0, device="cuda"):
    """The fp64 frequencies [rotary_dim / 2] that `rotary` takes; scaling "plain", "linear",
    "base" or "parts" (see include/rudder_block.h)."""
    import torch
    freq = torch.empty(max(rotary_dim, 0) // 2, dtype=torch.float64)
    rudder_rotary_frequencies(rotary_dim, base, ROTARY_SCALING[scaling], factor, trained, low,
                              high, freq)
    return freq.to(device)


def rotary(Q, K, row_start, freq, max_rows: int, pos=None, magnitude: float = 1.0,
           layout: int = ROTARY_HALF, in_place: bool = False, stream=None):
    """Rotary positions on Q bf16 [T, Hq, D] and K [T, Hkv, D] (None: Q alone), row i of sequence
    b at pos[b] + i (None: at i).  Returns (Q', K'): Q and K themselves where in_place, else new
    tensors (copies in rows of no sequence)."""
    import torch
    T, Hq, D = Q.shape
    Hkv = 0 if K is None else K.shape[1]
    B = row_start.numel() - 1
    with _on(stream, Q.device):
        Qo = Q if in_place else Q.clone(memory_format=torch.contiguous_format)
        Ko = K if in_place or K is None else K.clone(memory_format=torch.contiguous_format)
        if T and B:
            rudder_rotary(Q, K, row_start, pos, freq, magnitude, B, T, max_rows, Hq, Hkv, D,
                          2 * freq.numel(), layout, Qo, Ko)
    return Qo, Ko


def prompt_attention(Q, K, V, row_start, max_rows: int, sm: float, stream=None):
    """Causal attention of the prompts row_start [B + 1] of Q bf16 [T, Hq, D] to their own K, V
    bf16 [T, Hkv, D].  Returns O bf16 [T, Hq, D] (zeros in rows of no sequence)."""
    import torch
    T, Hq, D = Q.shape
    Hkv, B = K.shape[1], row_start.numel() - 1
    with _on(stream, Q.device):
        O = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=Q.device)
        n = prompt_attention_workspace_bytes(B, T, max_rows, Hq, Hkv, D)
        ws = torch.empty(n, dtype=torch.uint8, device=Q.device) if n else None
        if T and B:
            rudder_prompt_attention(Q, K, V, row_start, B, T, max_rows, Hq, Hkv, D, sm, ws, O)
    return O


# ---------------------------------------------------------------------------
# Measurement (include/rudder_diag.h)
# ---------------------------------------------------------------------------
def mfma_ceiling_sink_bytes() -> int:
    return int(load_library().rudder_mfma_ceiling_sink_bytes())


def mfma_ceiling_ops(iters: int, codes: int) -> float:
    return float(load_library().rudder_mfma_ceiling_ops(iters, codes))


def rudder_mfma_ceiling(Xq, Wq, M: int, N: int, K: int, abits: int, codes: int, iters: int,
                        sink, stream=None) -> None:
    _check(load_library().rudder_mfma_ceiling(_ptr(Xq), _ptr(Wq), M, N, K, abits, codes, iters,
                                              _ptr(sink), _stream(stream)))


CEILING_OWN = 0             # the instruction rudder_linear uses
CEILING_I8_16X16X64 = 1     # v_mfma_i32_16x16x64_i8 (int containers)


def rudder_mfma_ceiling_shape(Xq, Wq, M: int, N: int, K: int, abits: int, codes: int,
                              iters: int, shape: int, sink, stream=None) -> None:
    _check(load_library().rudder_mfma_ceiling_shape(_ptr(Xq), _ptr(Wq), M, N, K, abits, codes,
                                                    iters, shape, _ptr(sink), _stream(stream)))

"""ctypes binding of libmoe (include/moe.h): the same entry points, argument marshalling only.

Tensors are torch CUDA tensors (PyTorch supplies device memory and streams); every step runs in
the library's kernels. There is no CPU path: calling with a CPU tensor, or without the built
library, raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

# MOE_LIBRARY selects another build of the same library (the debug build, libmoe_checks.so)
LIB_PATH = os.environ.get("MOE_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_F32, MOE_BF16 = 0, 1
GROUP_ROWS = 128
MAX_EXPERTS = 256
MAX_TOPK = 16
NORM_MAX_D = 8192
FFN_MAX, FFN_MAX_T = 1 << 20, 1 << 22
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2
ADAMW_F32, ADAMW_F8 = 0, 1
ACT_SILU, ACT_GELU = 0, 1
KEEP_NONE, KEEP_ALL, KEEP_F8 = 0, 1, 2
ADAMW_BLOCK = 256
STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED", -3: "MOE_ERR_CUDA",
          -4: "MOE_ERR_DEVICE_TIMEOUT", -5: "MOE_ERR_BAD_INDEX", -6: "MOE_ERR_CHECK_FAILED"}

_lock = threading.Lock()
_lib = None

_P, _I, _I64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_F, _D = ctypes.c_float, ctypes.c_double


class AdamWTensor(ctypes.Structure):
    """moe_adamw_tensor"""
    _fields_ = [("p", _P), ("master", _P), ("g", _P), ("m", _P), ("v", _P), ("m_scale", _P), ("v_scale", _P),
                ("n", _I64), ("weight_decay", _F), ("dtype", ctypes.c_int32), ("state", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


_SIGS = {
    "moe_route_topk": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "moe_grouped_rows_max": (_I64, [_I, _I, _I]),
    "moe_count_index_workspace_size": (_SZ, [_I, _I, _I]),
    "moe_count_index_hook_offset": (_SZ, [_I]),
    "moe_count_index": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_count_index_static": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "moe_route_count_index": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_permute": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _P, _I64, _P, _P]),
    "moe_grouped_ffn_workspace_size": (_SZ, [_I, _I, _I, _I64, _I, _I]),
    "moe_grouped_ffn_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I64, _I, _P, _P, _P, _P, _SZ, _P]),
    "moe_grouped_ffn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I64, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_grouped_ffn_bwd_recompute": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I64, _I, _P, _P, _P, _P, _P,
                                           _SZ, _P]),
    "moe_grouped_ffn_fwd_gather": (_I, [_P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I64, _I, _P, _P, _P, _P, _SZ, _P]),
    "moe_grouped_ffn_bwd_gather": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I64, _I, _P, _P, _P, _P, _P,
                                        _SZ, _P]),
    "moe_grouped_ffn_bwd_recompute_gather": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I64, _I, _P, _P,
                                                  _P, _P, _P, _SZ, _P]),
    "moe_combine_fwd": (_I, [_P, _P, _P, _I, _I, _I, _I64, _I, _P, _P]),
    "moe_combine_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I64, _I, _P, _P, _P, _P]),
    "moe_router_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "moe_router_fwd": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    "moe_router_bwd": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "moe_norm_fwd": (_I, [_P, _P, _I, _I, _I, _F, _P, _P]),
    "moe_norm_residual_fwd": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _F, _F, _P, _P, _P]),
    "moe_norm_bwd_workspace_size": (_SZ, [_I, _I, _I]),
    "moe_norm_bwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "moe_norm_residual_bwd": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _F, _F, _P, _P, _P, _P, _P, _P, _SZ,
                                   _P]),
    "moe_adamw_plan_size": (_SZ, [_P, _I]),
    "moe_adamw_plan": (_I, [_P, _I, _P, _SZ]),
    "moe_adamw_step": (_I, [_P, _P, _D, _D, _F, _P, _P]),
    "moe_fp4_scale_bytes": (_SZ, [_I64, _I]),
    "moe_fp4_quantize": (_I, [_P, _I, _I64, _I, _P, _P, _P]),
    "moe_fp4_dequantize": (_I, [_P, _P, _I64, _I, _I, _P, _P]),
    "moe_permute_fp4": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _P, _I64, _P, _P, _P]),
    "moe_grouped_ffn_fwd_fp4": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I64, _P, _P, _P, _P, _SZ, _P]),
    "moe_act8_scale_bytes": (_SZ, [_I64, _I]),
    "moe_act8_quantize": (_I, [_P, _I, _I64, _I, _P, _P, _P]),
    "moe_act8_dequantize": (_I, [_P, _P, _I64, _I, _I, _P, _P]),
    "moe_layer_norm_fwd": (_I, [_P, _P, _P, _I, _I, _I, _F, _P, _P, _P, _P, _P, _P]),
    "moe_layer_norm_restore": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "moe_layer_norm_bwd_workspace_size": (_SZ, [_I, _I, _I]),
    "moe_layer_norm_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _F, _P, _P, _P, _P, _SZ, _P]),
    "moe_ffn_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_ffn_fwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_ffn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_read_status": (_I, [_P, _P]),
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_version": (_I, []),
}


class MoeError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} returned {STATUS.get(code, code)}")
        self.code = code


def lib():
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGS.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def exported_symbols():
    return list(_SIGS)


_U8, _I32 = torch.uint8, torch.int32
_CODES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def dtype_code(t: torch.dtype) -> int:
    code = _CODES.get(t)
    if code is None:
        raise TypeError(f"unsupported dtype {t}")
    return code


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libmoe takes CUDA tensors only")
    return t.data_ptr()


# The current stream's handle without building a Stream object (0.1 us instead of 3 us per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _s(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(_device())
    return torch.cuda.current_stream().cuda_stream


def wrong_device(index, dev):
    raise ValueError(f"the buffers are on cuda:{index}, the current device is cuda:{dev}")


def _want(name, t, dtype, shape):
    """A tensor argument that a kernel reads as contiguous memory of this type and shape."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} is needed, got {t.dtype} "
                         f"{tuple(t.shape)} with strides {t.stride()}")


def _ptr(name, t, dtype, shape):
    """The address of a tensor argument that _want accepts."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda:
        return t.data_ptr()
    _want(name, t, dtype, shape)
    return _p(t)


def _scale_bytes(rows, cols):
    return -(-rows // 128) * -(-cols // 128) * 512


def _bytes_at_least(name, t, n):
    """The address of a tensor of at least n bytes."""
    if t.dtype is _U8 and t.numel() >= n and t.is_contiguous() and t.is_cuda:
        return t.data_ptr()
    if t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name}: a contiguous uint8 tensor of at least {n} bytes is needed, got {t.dtype} "
                         f"{tuple(t.shape)}")
    return _p(t)


def _ints(name, t, n):
    """The address of an index tensor: at least n contiguous 32-bit integers. (None is the library's to refuse.)"""
    if t is None:
        return None
    if t.dtype is not _I32 or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 tensor of at least {n} entries is needed, got {t.dtype} "
                         f"{tuple(t.shape)} with strides {t.stride()}")
    return _p(t)


def _ok(fn, rc):
    if rc != 0:
        raise MoeError(fn, rc)


def moe_route_topk(logits, k, topk_idx, topk_w, stream=None):
    T, E = logits.shape
    _ok("moe_route_topk", lib().moe_route_topk(_p(logits), T, E, k, _p(topk_idx), _p(topk_w), _s(stream)))


def moe_grouped_rows_max(T, k, E):
    return int(lib().moe_grouped_rows_max(T, k, E))


def moe_count_index_workspace_size(T, k, E):
    return int(lib().moe_count_index_workspace_size(T, k, E))


def moe_count_index_hook_offset(E):
    return int(lib().moe_count_index_hook_offset(E))


def moe_count_index(topk_idx, E, counts, offsets, tile_offsets, row_of_slot, token_of_row, ws, stream=None):
    T, k = topk_idx.shape
    _ok("moe_count_index", lib().moe_count_index(_p(topk_idx), T, k, E, _p(counts), _p(offsets), _p(tile_offsets),
                                                 _p(row_of_slot), _p(token_of_row), _p(ws), ws.numel() * ws.element_size(),
                                                 _s(stream)))


def moe_route_count_index(logits, k, topk_idx, topk_w, counts, offsets, tile_offsets, row_of_slot, token_of_row, ws,
                          stream=None):
    """moe_route_topk then moe_count_index, in one launch when all its blocks fit on the GPU."""
    T, E = logits.shape
    _ok("moe_route_count_index", lib().moe_route_count_index(
        _p(logits), T, E, k, _p(topk_idx), _p(topk_w), _p(counts), _p(offsets), _p(tile_offsets), _p(row_of_slot),
        _p(token_of_row), _p(ws), ws.numel() * ws.element_size(), _s(stream)))


def moe_count_index_static(topk_idx, E, counts, offsets, tile_offsets, row_of_slot, token_of_row, stream=None):
    """moe_count_index for callers that cannot allocate: the scratch is a fixed array inside libmoe."""
    T, k = topk_idx.shape
    _ok("moe_count_index_static", lib().moe_count_index_static(
        _p(topk_idx), T, k, E, _p(counts), _p(offsets), _p(tile_offsets), _p(row_of_slot), _p(token_of_row),
        _s(stream)))


def moe_permute(x, k, E, row_of_slot, counts, tile_offsets, x_perm, stream=None):
    T, d = x.shape
    _ok("moe_permute", lib().moe_permute(_p(x), dtype_code(x.dtype), T, d, k, E, _p(row_of_slot), _p(counts),
                                         _p(tile_offsets), x_perm.shape[0], _p(x_perm), _s(stream)))


def moe_grouped_ffn_workspace_size(E, d, f, rows_max, dtype, backward):
    return int(lib().moe_grouped_ffn_workspace_size(E, d, f, rows_max, dtype, int(backward)))


def moe_grouped_ffn_fwd(x_perm, w_gate_up, w_down, tile_offsets, offsets, ab, h, y_perm, ws, stream=None):
    E, twof, d = w_gate_up.shape
    _ok("moe_grouped_ffn_fwd", lib().moe_grouped_ffn_fwd(
        _p(x_perm), _p(w_gate_up), _p(w_down), _p(tile_offsets), _p(offsets), E, d, twof // 2, x_perm.shape[0],
        dtype_code(x_perm.dtype), _p(ab), _p(h), _p(y_perm), _p(ws), ws.numel() * ws.element_size(), _s(stream)))


def moe_grouped_ffn_bwd(dy_perm, x_perm, ab, h, w_gate_up, w_down, tile_offsets, offsets, dab, dx_perm, dw_gate_up,
                        dw_down, ws, stream=None):
    E, twof, d = w_gate_up.shape
    _ok("moe_grouped_ffn_bwd", lib().moe_grouped_ffn_bwd(
        _p(dy_perm), _p(x_perm), _p(ab), _p(h), _p(w_gate_up), _p(w_down), _p(tile_offsets), _p(offsets), E, d,
        twof // 2,
        x_perm.shape[0], dtype_code(x_perm.dtype), _p(dab), _p(dx_perm), _p(dw_gate_up), _p(dw_down), _p(ws),
        ws.numel() * ws.element_size(), _s(stream)))


def moe_grouped_ffn_bwd_recompute(dy_perm, x_perm, ab, h, w_gate_up, w_down, tile_offsets, offsets, dab, dx_perm,
                                  dw_gate_up, dw_down, ws, stream=None):
    E, twof, d = w_gate_up.shape
    _ok("moe_grouped_ffn_bwd_recompute", lib().moe_grouped_ffn_bwd_recompute(
        _p(dy_perm), _p(x_perm), _p(ab), _p(h), _p(w_gate_up), _p(w_down), _p(tile_offsets), _p(offsets), E, d,
        twof // 2,
        x_perm.shape[0], dtype_code(x_perm.dtype), _p(dab), _p(dx_perm), _p(dw_gate_up), _p(dw_down), _p(ws),
        ws.numel() * ws.element_size(), _s(stream)))


def moe_grouped_ffn_fwd_gather(x, token_of_row, w_gate_up, w_down, tile_offsets, offsets, ab, h, y_perm, ws,
                               stream=None):
    """moe_grouped_ffn_fwd with GEMM1 gathering its token rows from x [T, d] through token_of_row."""
    E, twof, d = w_gate_up.shape
    _ok("moe_grouped_ffn_fwd_gather", lib().moe_grouped_ffn_fwd_gather(
        _p(x), _p(token_of_row), x.shape[0], _p(w_gate_up), _p(w_down), _p(tile_offsets), _p(offsets), E, d,
        twof // 2, h.shape[0], dtype_code(x.dtype), _p(ab), _p(h), _p(y_perm), _p(ws), ws.numel() * ws.element_size(),
        _s(stream)))


def moe_grouped_ffn_bwd_gather(dy_perm, x, token_of_row, ab, h, w_gate_up, w_down, tile_offsets, offsets, dab, dx_perm,
                               dw_gate_up, dw_down, ws, stream=None):
    """moe_grouped_ffn_bwd with the gate/up weight gradient gathering its token rows from x [T, d]."""
    E, twof, d = w_gate_up.shape
    _ok("moe_grouped_ffn_bwd_gather", lib().moe_grouped_ffn_bwd_gather(
        _p(dy_perm), _p(x), _p(token_of_row), x.shape[0], _p(ab), _p(h), _p(w_gate_up), _p(w_down), _p(tile_offsets),
        _p(offsets), E, d, twof // 2, dy_perm.shape[0], dtype_code(x.dtype), _p(dab), _p(dx_perm), _p(dw_gate_up),
        _p(dw_down), _p(ws), ws.numel() * ws.element_size(), _s(stream)))


def moe_grouped_ffn_bwd_recompute_gather(dy_perm, x, token_of_row, ab, h, w_gate_up, w_down, tile_offsets, offsets,
                                         dab, dx_perm, dw_gate_up, dw_down, ws, stream=None):
    """moe_grouped_ffn_bwd_recompute with GEMM1 and the gate/up weight gradient gathering from x [T, d]."""
    E, twof, d = w_gate_up.shape
    _ok("moe_grouped_ffn_bwd_recompute_gather", lib().moe_grouped_ffn_bwd_recompute_gather(
        _p(dy_perm), _p(x), _p(token_of_row), x.shape[0], _p(ab), _p(h), _p(w_gate_up), _p(w_down), _p(tile_offsets),
        _p(offsets), E, d, twof // 2, dy_perm.shape[0], dtype_code(x.dtype), _p(dab), _p(dx_perm), _p(dw_gate_up),
        _p(dw_down), _p(ws), ws.numel() * ws.element_size(), _s(stream)))


def moe_combine_fwd(y_perm, topk_w, row_of_slot, T, k, out, stream=None):
    d = y_perm.shape[1]
    _ok("moe_combine_fwd", lib().moe_combine_fwd(_p(y_perm), _p(topk_w), _p(row_of_slot), T, d, k, y_perm.shape[0],
                                                 dtype_code(y_perm.dtype), _p(out), _s(stream)))


def moe_combine_bwd(grad_out, y_perm, topk_w, topk_idx, row_of_slot, counts, tile_offsets, E, dy_perm, d_topk_w,
                    d_logits, stream=None):
    T, d = grad_out.shape
    k = topk_idx.shape[1]
    _ok("moe_combine_bwd", lib().moe_combine_bwd(
        _p(grad_out), _p(y_perm), _p(topk_w), _p(topk_idx), _p(row_of_slot), _p(counts), _p(tile_offsets), T, d, k, E,
        y_perm.shape[0], dtype_code(y_perm.dtype), _p(dy_perm), _p(d_topk_w), _p(d_logits), _s(stream)))


def moe_router_workspace_size(T, d, E, dtype):
    return int(lib().moe_router_workspace_size(T, d, E, dtype))


def moe_router_fwd(x, w_router, k, logits, topk_idx, topk_w, ws, stream=None):
    """logits may be None (not written)."""
    T, d = x.shape
    E = w_router.shape[0]
    _ok("moe_router_fwd", lib().moe_router_fwd(
        _p(x), _p(w_router), T, d, E, k, dtype_code(x.dtype), _p(logits), _p(topk_idx), _p(topk_w), _p(ws),
        ws.numel() * ws.element_size(), _s(stream)))


def moe_router_bwd(x, w_router, d_logits, dx, dw_router, ws, accumulate_dx=False, stream=None):
    T, d = x.shape
    E = w_router.shape[0]
    _ok("moe_router_bwd", lib().moe_router_bwd(
        _p(x), _p(w_router), _p(d_logits), T, d, E, dtype_code(x.dtype), int(bool(accumulate_dx)), _p(dx),
        _p(dw_router), _p(ws), ws.numel() * ws.element_size(), _s(stream)))


def _gate_kind(gate, T, d, dtype):
    if gate is None:
        return GATE_NONE
    if gate.dim() == 1:
        _want("gate", gate, dtype, (d,))
        return GATE_CHANNEL
    _want("gate", gate, dtype, (T, d))
    return GATE_TOKEN


def moe_norm_fwd(x, w, n, eps=1e-6, stream=None):
    """n = x rms(x) w, x [T, d]."""
    T, d = x.shape
    dt = x.dtype
    _want("x", x, dt, (T, d))
    _want("w", w, dt, (d,))
    _want("n", n, dt, (T, d))
    _ok("moe_norm_fwd", lib().moe_norm_fwd(_p(x), _p(w), T, d, dtype_code(dt), eps, _p(n), _s(stream)))


def norm_residual_fwd_into(y, x, w_post, gate, kind, w_next, T, d, dt, out, n, res_scale, eps, stream):
    """The call behind moe_norm_residual_fwd and BlockNorms.post: checks its inputs; out and n are the addresses of [T, d]
    outputs of type dt (n None: no next norm)."""
    rows, vec = (T, d), (d,)
    _ok("moe_norm_residual_fwd", lib().moe_norm_residual_fwd(
        _ptr("y", y, dt, rows), _ptr("x", x, dt, rows), _ptr("w_post", w_post, dt, vec),
        _ptr("gate", gate, dt, vec if kind == GATE_CHANNEL else rows) if kind else None, kind,
        None if n is None else _ptr("w_next", w_next, dt, vec), T, d, _CODES[dt], res_scale, eps, out, n, _s(stream)))


def moe_norm_residual_fwd(y, x, w_post, gate, w_next, out, n, res_scale=1.0, eps=1e-6, stream=None):
    """out = res_scale x + gate * (y rms(y) w_post); n = out rms(out) w_next. gate: None, [d] or [T, d];
    w_next and n may be None (no next norm)."""
    T, d = x.shape
    dt = x.dtype
    dtype_code(dt)
    if (w_next is None) != (n is None):
        raise ValueError("w_next and n are given together")
    norm_residual_fwd_into(y, x, w_post, gate, _gate_kind(gate, T, d, dt), w_next, T, d, dt, _ptr("out", out, dt, (T, d)),
                           None if n is None else _ptr("n", n, dt, (T, d)), res_scale, eps, stream)


def moe_norm_bwd_workspace_size(T, d, dtype):
    return int(lib().moe_norm_bwd_workspace_size(T, d, dtype))


def moe_norm_bwd(dn, x, w, dx_in, dx, dw, ws, eps=1e-6, stream=None):
    """Backward of moe_norm_fwd; dx_in (may be None, may be dx) is added to dx."""
    T, d = x.shape
    dt = x.dtype
    for name, t in (("x", x), ("dn", dn), ("dx", dx)) + ((("dx_in", dx_in),) if dx_in is not None else ()):
        _want(name, t, dt, (T, d))
    _want("w", w, dt, (d,))
    _want("dw", dw, dt, (d,))
    _ok("moe_norm_bwd", lib().moe_norm_bwd(_p(dn), _p(x), _p(w), _p(dx_in), T, d, dtype_code(dt), eps, _p(dx), _p(dw),
                                           _p(ws), ws.numel() * ws.element_size(), _s(stream)))


def moe_norm_residual_bwd(dout, dn, out, y, w_post, gate, w_next, dx, dy, dw_post, d_gate, dw_next, ws, res_scale=1.0,
                          eps=1e-6, stream=None):
    """Backward of moe_norm_residual_fwd. dout may be None (zero) when dn is given; dn, out, w_next and dw_next
    belong to the next norm and may be None together; d_gate is None without a gate."""
    T, d = y.shape
    dt = y.dtype
    for name, t in (("y", y), ("dx", dx), ("dy", dy)) + ((("dout", dout),) if dout is not None else ()):
        _want(name, t, dt, (T, d))
    _want("w_post", w_post, dt, (d,))
    _want("dw_post", dw_post, dt, (d,))
    if w_next is not None:
        for name, t in (("dn", dn), ("out", out)):
            _want(name, t, dt, (T, d))
        _want("w_next", w_next, dt, (d,))
        _want("dw_next", dw_next, dt, (d,))
    elif dn is not None or dout is None:
        raise ValueError("dn needs w_next, and without them dout is needed")
    kind = _gate_kind(gate, T, d, dt)
    if kind != GATE_NONE:
        _want("d_gate", d_gate, dt, gate.shape)
    _ok("moe_norm_residual_bwd", lib().moe_norm_residual_bwd(
        _p(dout), _p(dn), _p(out), _p(y), _p(w_post), _p(gate), kind, _p(w_next), T, d, dtype_code(dt), res_scale, eps,
        _p(dx), _p(dy), _p(dw_post), _p(d_gate), _p(dw_next), _p(ws), ws.numel() * ws.element_size(), _s(stream)))


def moe_adamw_plan(tensors):
    """The plan of a list of AdamWTensor: a uint8 host tensor, to be copied to the device as it is."""
    arr = (AdamWTensor * max(1, len(tensors)))(*tensors)
    size = int(lib().moe_adamw_plan_size(arr, len(tensors)))
    plan = torch.empty((size + 7) // 8, dtype=torch.int64).view(torch.uint8)
    _ok("moe_adamw_plan", lib().moe_adamw_plan(arr, len(tensors), ctypes.c_void_p(plan.data_ptr()), plan.numel()))
    return plan


def moe_adamw_step(plan_host, plan_device, beta1, beta2, eps, state, stream=None):
    """state: 24 bytes of device memory laid out as moe_adamw_state."""
    _ok("moe_adamw_step", lib().moe_adamw_step(ctypes.c_void_p(plan_host.data_ptr()), _p(plan_device), beta1, beta2,
                                               eps, _p(state), _s(stream)))


def moe_fp4_scale_bytes(R, K):
    return int(lib().moe_fp4_scale_bytes(R, K))


def _rows(shape):
    """A shape [..., K] as its number of rows and K."""
    K = shape[-1]
    R = 1
    for n in shape[:-1]:
        R *= n
    return R, K


def moe_fp4_quantize(x, codes, scales, stream=None):
    """x [..., K] (rows in order) -> codes [..., K/2] uint8, scales [moe_fp4_scale_bytes(rows, K)] uint8."""
    shape, dt = x.shape, x.dtype
    R, K = _rows(shape)
    _ok("moe_fp4_quantize", lib().moe_fp4_quantize(
        _ptr("x", x, dt, shape), dtype_code(dt), R, K, _ptr("codes", codes, torch.uint8, (*shape[:-1], K // 2)),
        _bytes_at_least("scales", scales, _scale_bytes(R, K)), _s(stream)))


def moe_fp4_dequantize(codes, scales, x, stream=None):
    """The values that codes and scales stand for, into x [..., K]."""
    shape, dt = x.shape, x.dtype
    R, K = _rows(shape)
    _ok("moe_fp4_dequantize", lib().moe_fp4_dequantize(
        _ptr("codes", codes, torch.uint8, (*shape[:-1], K // 2)),
        _bytes_at_least("scales", scales, _scale_bytes(R, K)), R, K, dtype_code(dt), _ptr("x", x, dt, shape), _s(stream)))


def moe_permute_fp4(x, k, E, row_of_slot, counts, tile_offsets, codes, scales, stream=None):
    """moe_permute with MXFP4 output: codes [rows_max, d/2], scales [moe_fp4_scale_bytes(rows_max, d)]."""
    T, d = x.shape
    R = codes.shape[0]
    dt = x.dtype
    _ok("moe_permute_fp4", lib().moe_permute_fp4(
        _ptr("x", x, dt, (T, d)), dtype_code(dt), T, d, k, E, _ints("row_of_slot", row_of_slot, T * k),
        _ints("counts", counts, E), _ints("tile_offsets", tile_offsets, E + 1), R,
        _ptr("codes", codes, torch.uint8, (R, d // 2)), _bytes_at_least("scales", scales, _scale_bytes(R, d)),
        _s(stream)))


def moe_grouped_ffn_fwd_fp4(x_codes, x_scales, wgu_codes, wgu_scales, wd_codes, wd_scales, tile_offsets, offsets,
                            h_codes, h_scales, y_perm, ws, stream=None):
    """wgu_codes [E, 2f, d/2], wd_codes [E, d, f/2]; h_codes [rows_max, f/2] and h_scales are scratch."""
    E, d, f2 = wd_codes.shape
    R, f, u8 = x_codes.shape[0], 2 * f2, _U8
    _ok("moe_grouped_ffn_fwd_fp4", lib().moe_grouped_ffn_fwd_fp4(
        _ptr("x_codes", x_codes, u8, (R, d // 2)), _bytes_at_least("x_scales", x_scales, _scale_bytes(R, d)),
        _ptr("wgu_codes", wgu_codes, u8, (E, 2 * f, d // 2)),
        _bytes_at_least("wgu_scales", wgu_scales, _scale_bytes(E * 2 * f, d)),
        _ptr("wd_codes", wd_codes, u8, (E, d, f2)), _bytes_at_least("wd_scales", wd_scales, _scale_bytes(E * d, f)),
        _ints("tile_offsets", tile_offsets, E + 1), _ints("offsets", offsets, E + 1), E, d, f, R,
        _ptr("h_codes", h_codes, u8, (R, f2)),
        _bytes_at_least("h_scales", h_scales, _scale_bytes(R, f)), _ptr("y_perm", y_perm, torch.bfloat16, (R, d)),
        _p(ws), ws.numel() * ws.element_size(), _s(stream)))


class OwnsBuffers:
    """A class that allocates its buffers once and gives their addresses to every call. Another tensor may be set in the place of
    one of them (a second set of what is kept, say): it has to be of the same type, shape and device, and the calls that follow use
    it. (A captured graph goes on with the one that it was captured with.)"""

    _buffers = ()          # their attributes' names
    _fixed = ()            # attributes that the buffers' sizes follow from, or that say what they are for

    def _take(self):
        """Notes the buffers' addresses: at the end of the construction, and whenever a buffer is set."""
        raise NotImplementedError

    def _built(self):
        self._take()
        self.__dict__["_buffers_taken"] = True

    def __setattr__(self, name, t):
        built = "_buffers_taken" in self.__dict__
        if built and name in self._fixed:
            raise AttributeError(f"{name}: {type(self).__name__} was built for {self.__dict__[name]}")
        taken = built and name in self._buffers
        if taken:
            old = self.__dict__.get(name)
            if old is None or t is None:
                raise ValueError(f"{name}: {type(self).__name__} was built {'without' if old is None else 'with'} this buffer")
            _want(name, t, old.dtype, old.shape)
            if t.device != old.device:
                raise ValueError(f"{name}: the buffers are on {old.device}, got a tensor on {t.device}")
        object.__setattr__(self, name, t)
        if taken:
            self._take()

    def __setstate__(self, state):   # a deep copy has buffers of its own, or was read back onto another GPU
        self.__dict__.update(state)
        self._take()

    def __delattr__(self, name):
        if name in self._buffers:
            raise AttributeError(f"{name}: the calls of {type(self).__name__} use this buffer")
        object.__delattr__(self, name)


_INT_MAX = 0x7fffffff


def _ints_only(*sizes):
    """Sizes that the library takes as 32-bit integers (ctypes would pass on their low bits)."""
    for n in sizes:
        if n > _INT_MAX:
            raise ValueError(f"a size of {n} is past 2^31 - 1")


def moe_act8_scale_bytes(R, K):
    _ints_only(K)
    return int(lib().moe_act8_scale_bytes(R, K))


def _scale_bytes8(rows, cols):
    return rows * -(-cols // 32)


def _at(name, t, dtype, shape, dev):
    """The address of a tensor argument of this type and shape, contiguous, on the current GPU `dev`."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _want(name, t, dtype, shape)
    return _on(name, t, dev)


def _on(name, t, dev):
    """The address of a tensor on the current GPU, on which the launch goes."""
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError("libmoe takes CUDA tensors only")
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")
    return t.data_ptr()


def _rows_on(name, t, dev):
    """The address of a contiguous tensor [..., K] on the current GPU, its number of rows and K."""
    if not t.is_contiguous():
        _want(name, t, t.dtype, t.shape)
    shape = t.shape
    R, K = shape if len(shape) == 2 else _rows(shape)
    if K > _INT_MAX:
        _ints_only(K)
    return (t.data_ptr() if t.get_device() == dev else _on(name, t, dev)), R, K


def _bytes_on(name, t, n, dev):
    """The address of a tensor of at least n bytes on the current GPU."""
    if t.dtype is _U8 and t.numel() >= n and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _bytes_at_least(name, t, n)
    return _on(name, t, dev)


def moe_act8_quantize(x, codes, scales, stream=None):
    """x [..., K] (rows in order) -> codes [..., K] uint8, scales [moe_act8_scale_bytes(rows, K)] uint8."""
    dev = _device()
    p, R, K = _rows_on("x", x, dev)
    _ok("moe_act8_quantize", lib().moe_act8_quantize(
        p, dtype_code(x.dtype), R, K, _at("codes", codes, _U8, x.shape, dev),
        _bytes_on("scales", scales, _scale_bytes8(R, K), dev), _s(stream)))


def moe_act8_dequantize(codes, scales, x, stream=None):
    """The values that codes and scales stand for, into x [..., K]."""
    dev = _device()
    p, R, K = _rows_on("x", x, dev)
    _ok("moe_act8_dequantize", lib().moe_act8_dequantize(
        _at("codes", codes, _U8, x.shape, dev), _bytes_on("scales", scales, _scale_bytes8(R, K), dev), R, K, dtype_code(x.dtype),
        p, _s(stream)))


def layer_norm_fwd_into(dev, x, w, b, T, d, dt, n, mean, rstd, codes, scales, eps, stream):
    """The call behind moe_layer_norm_fwd and LayerNorm.forward: checks its inputs (dev: the current device); n, mean, rstd, codes and
    scales are the addresses of outputs of type dt and fitting size (all but n may be None)."""
    vec = (d,)
    _ok("moe_layer_norm_fwd", lib().moe_layer_norm_fwd(
        _at("x", x, dt, (T, d), dev), _at("w", w, dt, vec, dev), None if b is None else _at("b", b, dt, vec, dev), T, d,
        dtype_code(dt), eps, n, mean, rstd, codes, scales, _s(stream)))


def moe_layer_norm_fwd(x, w, b, n, mean=None, rstd=None, codes=None, scales=None, eps=1e-5, stream=None):
    """n = z w + b, z = (x - mean) rstd, x [T, d]; b may be None (zero). mean, rstd [T] fp32 and z in 8 bits (codes [T, d],
    scales) are written where they are given."""
    T, d = x.shape
    _ints_only(T, d)
    dt, dev, f32 = x.dtype, _device(), torch.float32
    layer_norm_fwd_into(
        dev, x, w, b, T, d, dt, _at("n", n, dt, (T, d), dev), None if mean is None else _at("mean", mean, f32, (T,), dev),
        None if rstd is None else _at("rstd", rstd, f32, (T,), dev), None if codes is None else _at("codes", codes, _U8, (T, d), dev),
        None if scales is None else _bytes_on("scales", scales, _scale_bytes8(T, d), dev), eps, stream)


def layer_norm_restore_into(dev, codes, scales, w, b, T, d, dt, n, stream):
    """The call behind moe_layer_norm_restore and LayerNorm.restore: checks w and b; codes, scales and n are the addresses of buffers
    of type dt and fitting size."""
    vec = (d,)
    _ok("moe_layer_norm_restore", lib().moe_layer_norm_restore(
        codes, scales, _at("w", w, dt, vec, dev), None if b is None else _at("b", b, dt, vec, dev), T, d, dtype_code(dt), n,
        _s(stream)))


def moe_layer_norm_restore(codes, scales, w, b, n, stream=None):
    """n = z w + b with the z that codes and scales stand for; b may be None."""
    T, d = n.shape
    _ints_only(T, d)
    dt, dev = n.dtype, _device()
    layer_norm_restore_into(dev, _at("codes", codes, _U8, (T, d), dev), _bytes_on("scales", scales, _scale_bytes8(T, d), dev), w, b, T, d,
                            dt, _at("n", n, dt, (T, d), dev), stream)


def moe_layer_norm_bwd_workspace_size(T, d, dtype):
    _ints_only(T, d)
    return int(lib().moe_layer_norm_bwd_workspace_size(T, d, dtype))


def layer_norm_bwd_into(dev, dn, x, w, dx_in, T, d, dt, codes, scales, mean, rstd, dx, dw, db, ws, ws_bytes, eps, stream):
    """The call behind moe_layer_norm_bwd and LayerNorm.backward: checks its inputs dn, x, w and dx_in; the others are the addresses of
    buffers of type dt and fitting size."""
    rows = (T, d)
    _ok("moe_layer_norm_bwd", lib().moe_layer_norm_bwd(
        _at("dn", dn, dt, rows, dev), None if x is None else _at("x", x, dt, rows, dev), codes, scales, mean, rstd,
        _at("w", w, dt, (d,), dev), None if dx_in is None else _at("dx_in", dx_in, dt, rows, dev), T, d, dtype_code(dt), eps, dx, dw,
        db, ws, ws_bytes, _s(stream)))


def moe_layer_norm_bwd(dn, x, codes, scales, mean, rstd, w, dx_in, dx, dw, db, ws, eps=1e-5, stream=None):
    """Backward of moe_layer_norm_fwd, from x and mean or from codes and scales (the others None); dx_in (may be None, may be
    dx) is added to dx; db may be None (not wanted)."""
    T, d = dn.shape
    _ints_only(T, d)
    dt, dev, rows, vec, f32 = dn.dtype, _device(), (T, d), (d,), torch.float32

    def opt(name, t, dtype, shape):
        return None if t is None else _at(name, t, dtype, shape, dev)

    layer_norm_bwd_into(
        dev, dn, x, w, dx_in, T, d, dt, opt("codes", codes, _U8, rows),
        None if scales is None else _bytes_on("scales", scales, _scale_bytes8(T, d), dev), opt("mean", mean, f32, (T,)),
        _at("rstd", rstd, f32, (T,), dev), _at("dx", dx, dt, rows, dev), _at("dw", dw, dt, vec, dev), opt("db", db, dt, vec),
        _on("ws", ws, dev), ws.numel() * ws.element_size(), eps, stream)


def moe_ffn_workspace_size(T, d, f, dtype, backward):
    _ints_only(T, d, f)
    return int(lib().moe_ffn_workspace_size(T, d, f, dtype, int(bool(backward))))


def kept(ab, ab_scales, dt, T, f):
    """What `keep` says, and the addresses of ab and ab_scales: nothing, ab in dt, or codes and scales."""
    dev = _device()
    if ab is None:
        if ab_scales is not None:
            raise ValueError("ab_scales belong to an ab in 8 bits")
        return KEEP_NONE, None, None
    if ab_scales is None:
        return KEEP_ALL, _at("ab", ab, dt, (T, 2 * f), dev), None
    return KEEP_F8, _at("ab", ab, _U8, (T, 2 * f), dev), _bytes_on("ab_scales", ab_scales, _scale_bytes8(T, 2 * f), dev)


def ffn_fwd_into(dev, x, w_gate_up, w_down, y_in, T, d, f, dt, act, keep, h, y, ws, ws_bytes, stream):
    """The call behind moe_ffn_fwd and GatedFFN.forward: checks its inputs; keep is what kept() says of fitting buffers; h, y and ws
    are the addresses of buffers of type dt and fitting size."""
    _ok("moe_ffn_fwd", lib().moe_ffn_fwd(
        _at("x", x, dt, (T, d), dev), _at("w_gate_up", w_gate_up, dt, (2 * f, d), dev), _at("w_down", w_down, dt, (d, f), dev),
        None if y_in is None else _at("y_in", y_in, dt, (T, d), dev), T, d, f, dtype_code(dt), act, keep[0], keep[1], keep[2], h, y,
        ws, ws_bytes, _s(stream)))


def moe_ffn_fwd(x, w_gate_up, w_down, y_in, ab, ab_scales, h, y, ws, act=ACT_SILU, stream=None):
    """y = y_in + (act(x Wg^T) * (x Wu^T)) Wd^T, x [T, d], w_gate_up [2f, d], w_down [d, f]. y_in may be None, and may be y.
    ab: None (nothing kept), [T, 2f] in x's type, or [T, 2f] uint8 codes with ab_scales. h [T, f] is written."""
    T, d = x.shape
    f, dt, dev = w_down.shape[1], x.dtype, _device()
    _ints_only(T, d, f)
    ffn_fwd_into(dev, x, w_gate_up, w_down, y_in, T, d, f, dt, act, kept(ab, ab_scales, dt, T, f), _at("h", h, dt, (T, f), dev),
                 _at("y", y, dt, (T, d), dev), _on("ws", ws, dev), ws.numel() * ws.element_size(), stream)


def ffn_bwd_into(dev, dy, x, w_gate_up, w_down, dx_in, T, d, f, dt, act, keep, h, dab, dx, dw_gate_up, dw_down, ws, ws_bytes, stream):
    """The call behind moe_ffn_bwd and GatedFFN.backward: checks its inputs; keep is what kept() says of fitting buffers, h and those
    after it are the addresses of buffers of type dt and fitting size."""
    _ok("moe_ffn_bwd", lib().moe_ffn_bwd(
        _at("dy", dy, dt, (T, d), dev), _at("x", x, dt, (T, d), dev), keep[1], keep[2], h,
        _at("w_gate_up", w_gate_up, dt, (2 * f, d), dev), _at("w_down", w_down, dt, (d, f), dev),
        None if dx_in is None else _at("dx_in", dx_in, dt, (T, d), dev), T, d, f, dtype_code(dt), act, keep[0], dab, dx, dw_gate_up,
        dw_down, ws, ws_bytes, _s(stream)))


def moe_ffn_bwd(dy, x, ab, ab_scales, h, w_gate_up, w_down, dx_in, dab, dx, dw_gate_up, dw_down, ws, act=ACT_SILU,
                stream=None):
    """Backward of moe_ffn_fwd from the ab (and h, or ab_scales) that it kept; dx_in (may be None, may be dx) is added to dx."""
    T, d = dy.shape
    f, dt, dev = w_down.shape[1], dy.dtype, _device()
    _ints_only(T, d, f)
    ffn_bwd_into(dev, dy, x, w_gate_up, w_down, dx_in, T, d, f, dt, act, kept(ab, ab_scales, dt, T, f), _at("h", h, dt, (T, f), dev),
                 _at("dab", dab, dt, (T, 2 * f), dev), _at("dx", dx, dt, (T, d), dev),
                 _at("dw_gate_up", dw_gate_up, dt, (2 * f, d), dev), _at("dw_down", dw_down, dt, (d, f), dev), _on("ws", ws, dev),
                 ws.numel() * ws.element_size(), stream)


def moe_read_status(ws, stream=None):
    return int(lib().moe_read_status(_p(ws), _s(stream)))


def moe_status_string(code):
    return lib().moe_status_string(code).decode()


def moe_version():
    return int(lib().moe_version())

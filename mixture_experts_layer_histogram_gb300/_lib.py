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
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2
ADAMW_F32, ADAMW_F8 = 0, 1
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


def moe_read_status(ws, stream=None):
    return int(lib().moe_read_status(_p(ws), _s(stream)))


def moe_status_string(code):
    return lib().moe_status_string(code).decode()


def moe_version():
    return int(lib().moe_version())

"""ctypes binding of libmoe (include/moe.h): argument marshalling only.

Each function has the name and argument order of the C entry point.  Tensor
arguments may be torch tensors (their ``data_ptr()`` is passed), raw integer
addresses, or None for nullable pointers.  ``stream`` defaults to torch's
current CUDA stream.  A non-zero status raises ``MoEError``.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_MISALIGNED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_UNSUPPORTED = 4
MOE_ERR_CUDA = 5
MOE_ERR_TIMEOUT = 6
MOE_ERR_DEVICE_BOUNDS = 7

MOE_F32 = 0
MOE_BF16 = 1

MOE_OP_ROUTE = 0
MOE_OP_DISPATCH = 1
MOE_OP_EXPERT_FFN = 2
MOE_OP_ROUTE_BWD = 3
MOE_OP_MOD_SELECT = 4
MOE_OP_EXPERT_FFN_BWD = 5
MOE_OP_COMBINE_NORM_BWD = 6
MOE_OP_EXPERT_FFN_W4 = 7
MOE_OP_ORTHOGONALIZE = 8
MOE_OP_MUON_STEP = 9

MOE_GATE_SOFTMAX = 0
MOE_GATE_SIGMOID = 1
MOE_GATE_RENORM = 0x10
MOE_GATE_GROUP_MAX = 0x20

MOE_ROUTE_SOFTMAX_TOPK = 0
MOE_ROUTE_MOD_LINEAR = 1
MOE_ROUTE_LOGIT_GRAD = 2
MOE_ROUTE_DX_WRITE = 0x100
MOE_ROUTE_GATE_RENORM = 0x200

MOE_ROUTE_RENORM = 0x1
MOE_ROUTE_BIAS_SELECT = 0x2

EXPORTS = ("moe_status_str", "moe_version", "moe_kernel_launches", "moe_workspace_bytes", "moe_last_device_error",
           "moe_check_wait_timeout",
           "moe_route", "moe_route_ex", "moe_dispatch", "moe_dispatch_noalloc", "moe_expert_ffn",
           "moe_expert_ffn_ex", "moe_expert_ffn_gather", "moe_expert_ffn_bwd", "moe_combine", "moe_route_bwd",
           "moe_permute_bwd", "mod_select", "moe_ep_plan", "moe_gate", "moe_gate_bwd", "moe_route_group",
           "moe_combine_norm", "moe_combine_norm_bwd", "moe_ckpt_pack", "moe_ckpt_unpack", "moe_ckpt_swiglu",
           "moe_w4_pack", "moe_w4_unpack", "moe_expert_ffn_w4", "moe_orthogonalize", "moe_muon_step")


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int, name: str):
        super().__init__(f"{fn} failed: {name} ({status})")
        self.status = status


_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_Z = ctypes.c_size_t
_F = ctypes.c_float

_SIGS = {
    "moe_status_str": (ctypes.c_char_p, [_I]),
    "moe_version": (_I, []),
    "moe_kernel_launches": (ctypes.c_ulonglong, []),
    "moe_workspace_bytes": (_Z, [_I, _I, _I, _I, _I, _I]),
    "moe_last_device_error": (_I, [_P]),
    "moe_check_wait_timeout": (_I, [ctypes.c_ulonglong, _P]),
    "moe_route": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P]),
    "moe_route_ex": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P]),
    "moe_dispatch": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _Z, _P]),
    "moe_dispatch_noalloc": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "moe_expert_ffn": (_I, [_P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _Z, _P]),
    "moe_expert_ffn_ex": (_I, [_P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P]),
    "moe_expert_ffn_gather": (_I, [_P, _P, _I, _P, _I, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P]),
    "moe_expert_ffn_bwd": (_I, [_P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _Z, _P]),
    "moe_combine": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "moe_route_bwd": (_I, [_I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P]),
    "moe_permute_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "mod_select": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _Z, _P]),
    "moe_gate": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P]),
    "moe_gate_bwd": (_I, [_P, _P, _P, _I, _I, _I, _I, _F, _P, _P]),
    "moe_route_group": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _Z, _P]),
    "moe_combine_norm": (_I, [_P] * 8 + [_F, _I, _I, _I, _I, _P, _P, _P]),
    "moe_combine_norm_bwd": (_I, [_P] * 10 + [_F, _I, _I, _I, _I] + [_P] * 8 + [_Z, _P]),
    "moe_ckpt_pack": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "moe_ckpt_unpack": (_I, [_P, _P, _I, _I, _I, _P, _P]),
    "moe_ckpt_swiglu": (_I, [_P, _P, _I, _I, _I, _P, _P, _P]),
    "moe_w4_pack": (_I, [_P] + [_I] * 6 + [_P, _P, _P]),
    "moe_w4_unpack": (_I, [_P, _P] + [_I] * 6 + [_P, _P]),
    "moe_expert_ffn_w4": (_I, [_P, _P, _I, _P, _I] + [_P] * 6 + [_I] * 5 + [_P, _P, _P, _Z, _P]),
    "moe_orthogonalize": (_I, [_P] + [_I] * 5 + [_F] * 4 + [_P, _P, _Z, _P]),
    "moe_muon_step": (_I, [_P] * 3 + [_I] * 4 + [_F, _I, _F, _F, _F, _I] + [_F] * 4 + [_P] * 4 + [_Z, _P]),
    "moe_ep_plan": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
}


def lib() -> ctypes.CDLL:
    """The loaded libmoe.  Raises if the library has not been built: there is no
    fallback implementation."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmoe.so not built at {LIB_PATH}; run "
                               "`python -m token_dispatch_gb300.build` (needs nvcc)")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = None


def _find_raw_stream():
    """The current stream's address.  torch's own accessor of it where there is one: making a
    Stream object only to read its address took 3.1 of the 10 us of a small call, this 0.2."""
    global _raw_stream
    import torch
    raw, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or dev is None or not torch.cuda.is_initialized():
        torch.cuda.current_stream()  # initialises CUDA, and says so where it cannot
    _raw_stream = (lambda: raw(dev())) if raw and dev else (lambda: torch.cuda.current_stream().cuda_stream)


def _stream(stream):
    if stream is None:
        if _raw_stream is None:
            _find_raw_stream()
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, st: int):
    if st != MOE_OK:
        raise MoEError(fn, st, moe_status_str(st))


def moe_status_str(status: int) -> str:
    return lib().moe_status_str(status).decode()


def moe_version() -> int:
    return lib().moe_version()


def moe_kernel_launches() -> int:
    return lib().moe_kernel_launches()


def moe_workspace_bytes(op: int, T: int, H: int, E: int, K: int, Hp: int) -> int:
    return lib().moe_workspace_bytes(op, T, H, E, K, Hp)


def moe_last_device_error(stream=None) -> int:
    return lib().moe_last_device_error(_stream(stream))


def moe_check_wait_timeout(wait_cycles, stream=None):
    _check("moe_check_wait_timeout", lib().moe_check_wait_timeout(wait_cycles, _stream(stream)))


def moe_route(x, w_router, logit_bias, T, H, E, K, dtype, logits, topk_idx, topk_gate,
              ws=None, ws_bytes=0, stream=None):
    _check("moe_route", lib().moe_route(_ptr(x), _ptr(w_router), _ptr(logit_bias), T, H, E, K, dtype,
                                        _ptr(logits), _ptr(topk_idx), _ptr(topk_gate), _ptr(ws),
                                        ws_bytes, _stream(stream)))


def moe_route_ex(x, w_router, logit_bias, T, H, E, K, dtype, flags, logits, topk_idx, topk_gate,
                 ws=None, ws_bytes=0, stream=None):
    _check("moe_route_ex", lib().moe_route_ex(_ptr(x), _ptr(w_router), _ptr(logit_bias), T, H, E, K, dtype, flags,
                                              _ptr(logits), _ptr(topk_idx), _ptr(topk_gate), _ptr(ws),
                                              ws_bytes, _stream(stream)))


def moe_dispatch(x, topk_idx, T, H, E, K, dtype, cu_seqlens, dst_row, src_tok, xs, ws, ws_bytes,
                 stream=None):
    _check("moe_dispatch", lib().moe_dispatch(_ptr(x), _ptr(topk_idx), T, H, E, K, dtype,
                                              _ptr(cu_seqlens), _ptr(dst_row), _ptr(src_tok), _ptr(xs),
                                              _ptr(ws), ws_bytes, _stream(stream)))


def moe_dispatch_noalloc(x, topk_idx, T, H, E, K, dtype, cu_seqlens, dst_row, src_tok, xs, stream=None):
    """moe_dispatch with the count table in a library-owned static device array
    (for callers that cannot allocate); see include/moe.h for its limits."""
    _check("moe_dispatch_noalloc", lib().moe_dispatch_noalloc(_ptr(x), _ptr(topk_idx), T, H, E, K, dtype,
                                                              _ptr(cu_seqlens), _ptr(dst_row), _ptr(src_tok),
                                                              _ptr(xs), _stream(stream)))


def moe_expert_ffn(xs, cu_seqlens, rows, w_gate, w_up, w_down, E, H, Hp, dtype, act, h,
                   ws=None, ws_bytes=0, stream=None):
    _check("moe_expert_ffn", lib().moe_expert_ffn(_ptr(xs), _ptr(cu_seqlens), rows, _ptr(w_gate),
                                                  _ptr(w_up), _ptr(w_down), E, H, Hp, dtype, _ptr(act),
                                                  _ptr(h), _ptr(ws), ws_bytes, _stream(stream)))


def moe_expert_ffn_ex(xs, cu_seqlens, rows, w_gate, w_up, w_down, E, H, Hp, dtype, act, gu, h,
                      ws=None, ws_bytes=0, stream=None):
    _check("moe_expert_ffn_ex", lib().moe_expert_ffn_ex(_ptr(xs), _ptr(cu_seqlens), rows, _ptr(w_gate), _ptr(w_up),
                                                        _ptr(w_down), E, H, Hp, dtype, _ptr(act), _ptr(gu), _ptr(h),
                                                        _ptr(ws), ws_bytes, _stream(stream)))


def moe_expert_ffn_gather(x, src_tok, T, cu_seqlens, rows, w_gate, w_up, w_down, E, H, Hp, dtype, act, gu, h,
                          ws=None, ws_bytes=0, stream=None):
    _check("moe_expert_ffn_gather", lib().moe_expert_ffn_gather(
        _ptr(x), _ptr(src_tok), T, _ptr(cu_seqlens), rows, _ptr(w_gate), _ptr(w_up), _ptr(w_down), E, H, Hp, dtype,
        _ptr(act), _ptr(gu), _ptr(h), _ptr(ws), ws_bytes, _stream(stream)))


def moe_expert_ffn_bwd(xs, cu_seqlens, rows, w_gate, w_up, w_down, E, H, Hp, dtype, gu, act, dh, dxs,
                       dw_gate, dw_up, dw_down, ws, ws_bytes, stream=None):
    _check("moe_expert_ffn_bwd", lib().moe_expert_ffn_bwd(_ptr(xs), _ptr(cu_seqlens), rows, _ptr(w_gate),
                                                          _ptr(w_up), _ptr(w_down), E, H, Hp, dtype, _ptr(gu),
                                                          _ptr(act), _ptr(dh), _ptr(dxs), _ptr(dw_gate),
                                                          _ptr(dw_up), _ptr(dw_down), _ptr(ws), ws_bytes,
                                                          _stream(stream)))


def moe_combine(h, gate, dst_row, row_scale, residual, out_row, T, H, K, dtype, y, stream=None):
    _check("moe_combine", lib().moe_combine(_ptr(h), _ptr(gate), _ptr(dst_row), _ptr(row_scale),
                                            _ptr(residual), _ptr(out_row), T, H, K, dtype, _ptr(y),
                                            _stream(stream)))


def moe_route_bwd(mode, d_gate, logits, topk_idx, x, w_router, T, H, E, K, dtype, d_logits,
                  dw_router, dx, ws, ws_bytes, stream=None):
    _check("moe_route_bwd", lib().moe_route_bwd(mode, _ptr(d_gate), _ptr(logits), _ptr(topk_idx),
                                                _ptr(x), _ptr(w_router), T, H, E, K, dtype,
                                                _ptr(d_logits), _ptr(dw_router), _ptr(dx), _ptr(ws),
                                                ws_bytes, _stream(stream)))


def moe_permute_bwd(dy, h, gate, dst_row, row_scale, out_row, dxs, T, H, K, dtype, dh, d_gate,
                    d_scale, dx, stream=None):
    _check("moe_permute_bwd", lib().moe_permute_bwd(_ptr(dy), _ptr(h), _ptr(gate), _ptr(dst_row),
                                                    _ptr(row_scale), _ptr(out_row), _ptr(dxs), T, H,
                                                    K, dtype, _ptr(dh), _ptr(d_gate), _ptr(d_scale),
                                                    _ptr(dx), _stream(stream)))


def mod_select(x, w_mod, B, L, H, C, dtype, score, sel, sel_score, mask, x_sel, y_skip,
               ws=None, ws_bytes=0, stream=None):
    _check("mod_select", lib().mod_select(_ptr(x), _ptr(w_mod), B, L, H, C, dtype, _ptr(score),
                                          _ptr(sel), _ptr(sel_score), _ptr(mask), _ptr(x_sel),
                                          _ptr(y_skip), _ptr(ws), ws_bytes, _stream(stream)))


# Tensor arguments of the calls below: names, in the order of the C arguments, and types
# ("x": the call's dtype, "h": bf16, "i": 32-bit words).
_TENSORS = {
    "moe_gate": "logits:f sel_bias:f topk_idx:i topk_gate:f",
    "moe_gate_bwd": "d_gate:f logits:f topk_idx:i d_logits:f",
    "moe_route_group": "x:x w_router:x sel_bias:f logits:f topk_idx:i topk_gate:f ws:b",
    "moe_combine_norm": "h:x gate:f dst_row:i row_scale:f residual:x w_post:f res_scale:f w_next:f y:x xn:x",
    "moe_combine_norm_bwd": "dy:x dxn:x h:x gate:f dst_row:i row_scale:f y:x w_post:f res_scale:f w_next:f d_res:x dh:x "
                            "d_gate:f d_scale:f dw_post:f d_res_scale:f dw_next:f ws:b",
    "moe_ckpt_pack": "x:x q:c scale:b",
    "moe_ckpt_unpack": "q:c scale:b x:x",
    "moe_ckpt_swiglu": "q:c scale:b gu:x act:x",
    "moe_w4_pack": "w:x q:i scale:h",
    "moe_w4_unpack": "q:i scale:h w:x",
    "moe_expert_ffn_w4": "x:x src_tok:i cu_seqlens:i q_gate:i s_gate:h q_up:i s_up:h q_down:i s_down:h act:x h:x ws:b",
    "moe_orthogonalize": "x:x out:h ws:b",
    "moe_muon_step": "w:x dw:f m:f w_out:x w_low:h m_out:f ws:b",
}
_types = {}  # (call, dtype): the types of its tensors
_cuda = None


def _types_of(fn, dtype):
    global _cuda
    import torch
    if dtype not in (MOE_F32, MOE_BF16):
        raise MoEError(fn, MOE_ERR_INVALID_ARG, moe_status_str(MOE_ERR_INVALID_ARG))
    kinds = {"f": torch.float32, "i": torch.int32, "c": torch.int8, "b": torch.uint8, "h": torch.bfloat16,
             "x": torch.bfloat16 if dtype == MOE_BF16 else torch.float32}
    _cuda = torch.cuda
    _types[fn, dtype] = t = tuple(kinds[w.split(":")[1]] for w in _TENSORS[fn].split())
    return t


def _args(fn, dtype, tensors, sizes):
    """Addresses of a call's tensors: each None, a raw address, or a contiguous tensor of its
    type and at least its size, on the current device."""
    types = _types.get((fn, dtype)) or _types_of(fn, dtype)
    dev = None
    out = []
    for t, want, n in zip(tensors, types, sizes):
        if t is None or type(t) is int:
            out.append(t)
            continue
        if dev is None:
            dev = _cuda.current_device() if t.is_cuda else -2
        if t.dtype is not want or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
            name = _TENSORS[fn].split()[len(out)].split(":")[0]
            if t.get_device() != dev:
                raise ValueError(f"{fn}: {name} is not on the current CUDA device")
            raise ValueError(f"{fn}: {name} must be a contiguous {want} tensor of at least {n} elements, "
                             f"not {t.dtype} {tuple(t.shape)} with strides {t.stride()}")
        out.append(t.data_ptr())
    return out


def moe_gate(logits, sel_bias, T, E, K, groups, topk_groups, mode, scale, topk_idx, topk_gate, stream=None):
    l, b, i, g = _args("moe_gate", MOE_F32, (logits, sel_bias, topk_idx, topk_gate), (T * E, E, T * K, T * K))
    _check("moe_gate", lib().moe_gate(l, b, T, E, K, groups, topk_groups, mode, scale, i, g, _stream(stream)))


def moe_gate_bwd(d_gate, logits, topk_idx, T, E, K, mode, scale, d_logits, stream=None):
    dg, l, i, dl = _args("moe_gate_bwd", MOE_F32, (d_gate, logits, topk_idx, d_logits), (T * K, T * E, T * K, T * E))
    _check("moe_gate_bwd", lib().moe_gate_bwd(dg, l, i, T, E, K, mode, scale, dl, _stream(stream)))


def moe_route_group(x, w_router, sel_bias, T, H, E, K, dtype, groups, topk_groups, mode, scale, logits, topk_idx,
                    topk_gate, ws=None, ws_bytes=0, stream=None):
    xp, wp, b, l, i, g, w = _args("moe_route_group", dtype, (x, w_router, sel_bias, logits, topk_idx, topk_gate, ws),
                                  (T * H, H * E, E, T * E, T * K, T * K, ws_bytes))
    _check("moe_route_group", lib().moe_route_group(xp, wp, b, T, H, E, K, dtype, groups, topk_groups, mode, scale, l,
                                                    i, g, w, ws_bytes, _stream(stream)))


def moe_combine_norm(h, gate, dst_row, row_scale, residual, w_post, res_scale, w_next, eps, T, H, K, dtype, y, xn,
                     stream=None):
    n, R = T * H, T * K
    a = _args("moe_combine_norm", dtype, (h, gate, dst_row, row_scale, residual, w_post, res_scale, w_next, y, xn),
              (R * H, R, R, T, n, H, H, H, n, n))
    _check("moe_combine_norm", lib().moe_combine_norm(*a[:8], eps, T, H, K, dtype, a[8], a[9], _stream(stream)))


def moe_combine_norm_bwd(dy, dxn, h, gate, dst_row, row_scale, y, w_post, res_scale, w_next, eps, T, H, K, dtype,
                         d_res, dh, d_gate, d_scale, dw_post, d_res_scale, dw_next, ws=None, ws_bytes=0, stream=None):
    n, R = T * H, T * K
    a = _args("moe_combine_norm_bwd", dtype,
              (dy, dxn, h, gate, dst_row, row_scale, y, w_post, res_scale, w_next, d_res, dh, d_gate, d_scale, dw_post,
               d_res_scale, dw_next, ws),
              (n, n, R * H, R, R, T, n, H, H, H, n, R * H, R, T, H, H, H, ws_bytes))
    _check("moe_combine_norm_bwd", lib().moe_combine_norm_bwd(*a[:10], eps, T, H, K, dtype, *a[10:], ws_bytes,
                                                              _stream(stream)))


def moe_ckpt_pack(x, rows, N, dtype, q, scale, stream=None):
    n, runs = rows * N, rows * ((N + 31) // 32)
    a = _args("moe_ckpt_pack", dtype, (x, q, scale), (n, n, runs))
    _check("moe_ckpt_pack", lib().moe_ckpt_pack(a[0], rows, N, dtype, a[1], a[2], _stream(stream)))


def moe_ckpt_unpack(q, scale, rows, N, dtype, x, stream=None):
    n, runs = rows * N, rows * ((N + 31) // 32)
    a = _args("moe_ckpt_unpack", dtype, (q, scale, x), (n, runs, n))
    _check("moe_ckpt_unpack", lib().moe_ckpt_unpack(a[0], a[1], rows, N, dtype, a[2], _stream(stream)))


def moe_ckpt_swiglu(q, scale, rows, Hp, dtype, gu, act, stream=None):
    n, runs = rows * Hp, rows * ((2 * Hp + 31) // 32)
    a = _args("moe_ckpt_swiglu", dtype, (q, scale, gu, act), (2 * n, runs, 2 * n, n))
    _check("moe_ckpt_swiglu", lib().moe_ckpt_swiglu(a[0], a[1], rows, Hp, dtype, a[2], a[3], _stream(stream)))


def _w4_sizes(E, out, inp, group):
    """Words of codes and scales of a packed tensor with `out` outputs of `inp` inputs."""
    blocks = (inp + 127) // 128
    return E * out * blocks * 16, E * out * blocks * 128 // group if group > 0 else 0


def moe_w4_pack(w, E, rows, cols, axis, group, dtype, q, scale, stream=None):
    out, inp = (cols, rows) if axis == 0 else (rows, cols)
    a = _args("moe_w4_pack", dtype, (w, q, scale), (E * rows * cols, *_w4_sizes(E, out, inp, group)))
    _check("moe_w4_pack", lib().moe_w4_pack(a[0], E, rows, cols, axis, group, dtype, a[1], a[2], _stream(stream)))


def moe_w4_unpack(q, scale, E, rows, cols, axis, group, dtype, w, stream=None):
    out, inp = (cols, rows) if axis == 0 else (rows, cols)
    a = _args("moe_w4_unpack", dtype, (q, scale, w), (*_w4_sizes(E, out, inp, group), E * rows * cols))
    _check("moe_w4_unpack", lib().moe_w4_unpack(a[0], a[1], E, rows, cols, axis, group, dtype, a[2], _stream(stream)))


def moe_expert_ffn_w4(x, src_tok, T, cu_seqlens, rows, q_gate, s_gate, q_up, s_up, q_down, s_down, E, H, Hp, group,
                      dtype, act, h, ws=None, ws_bytes=0, stream=None):
    n_q, n_s = _w4_sizes(E, Hp, H, group)
    d_q, d_s = _w4_sizes(E, H, Hp, group)
    a = _args("moe_expert_ffn_w4", dtype,
              (x, src_tok, cu_seqlens, q_gate, s_gate, q_up, s_up, q_down, s_down, act, h, ws),
              ((rows if src_tok is None else T) * H, rows, E + 1, n_q, n_s, n_q, n_s, d_q, d_s, rows * Hp, rows * H,
               ws_bytes))
    _check("moe_expert_ffn_w4", lib().moe_expert_ffn_w4(a[0], a[1], T, a[2], rows, *a[3:9], E, H, Hp, group, dtype,
                                                        a[9], a[10], a[11], ws_bytes, _stream(stream)))


def moe_orthogonalize(x, E, M, N, dtype, steps, a, b, c, eps, out, ws=None, ws_bytes=0, stream=None):
    n = E * M * N
    t = _args("moe_orthogonalize", dtype, (x, out, ws), (n, n, ws_bytes))
    _check("moe_orthogonalize", lib().moe_orthogonalize(t[0], E, M, N, dtype, steps, a, b, c, eps, t[1], t[2],
                                                        ws_bytes, _stream(stream)))


def moe_muon_step(w, dw, m, E, M, N, dtype, beta, nesterov, lr, weight_decay, scale, steps, a, b, c, eps, w_out, w_low,
                  m_out, ws=None, ws_bytes=0, stream=None):
    n = E * M * N
    t = _args("moe_muon_step", dtype, (w, dw, m, w_out, w_low, m_out, ws), (n, n, n, n, n, n, ws_bytes))
    _check("moe_muon_step", lib().moe_muon_step(*t[:3], E, M, N, dtype, beta, int(nesterov), lr, weight_decay, scale,
                                                steps, a, b, c, eps, *t[3:], ws_bytes, _stream(stream)))


def moe_ep_plan(R, E, S, K, B, counts):
    """Host-side expert-parallel plan from the gathered per-rank expert counts
    (int32 [R, E]).  Returns numpy arrays: piece_count and piece_offset
    [R dst, R src, E], slot_expert [R, B], local_counts [R, E/R + B],
    remote_reads [R]."""
    import numpy as np
    counts = np.ascontiguousarray(counts, dtype=np.int32)
    G = E // R if R > 0 and E % R == 0 else 0
    pc = np.zeros((R, R, E), np.int32)
    po = np.zeros((R, R, E), np.int32)
    se = np.zeros((R, max(B, 0)), np.int32)
    lc = np.zeros((R, G + max(B, 0)), np.int32)
    rr = np.zeros(R, np.int32)

    def a(x):
        return x.ctypes.data_as(ctypes.c_void_p) if x.size else None
    _check("moe_ep_plan", lib().moe_ep_plan(R, E, S, K, B, a(counts), a(pc), a(po), a(se), a(lc), a(rr)))
    return pc, po, se, lc, rr

"""Thin Python binding of libmoe's C ABI (argument marshalling only).

Each function here has the name of the C entry point it calls, takes torch
tensors (device memory) and the current torch stream, and passes their raw
pointers through ctypes.  Every step of the computation runs in libmoe's HIP
kernels; nothing here computes.  If the library is not built the first call
raises, there is no fallback path.

torch is imported before the library is loaded so that libmoe binds to the HIP
runtime already in the process (torch ships one with the same soname).
"""
from __future__ import annotations

import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_F32, MOE_BF16, MOE_MXFP8 = 0, 1, 2
_PREC = {"f32": MOE_F32, "bf16": MOE_BF16, "mxfp8": MOE_MXFP8}

_c_void_p, _i64, _i32, _sz, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int
_f32, _f64 = ctypes.c_float, ctypes.c_double

_SIGS = {
    "moe_abi_version": (_int, []),
    "moe_status_str": (ctypes.c_char_p, [_int]),
    "moe_router_logits": (_int, [_c_void_p, _c_void_p, _int, _i64, _i32, _i32, _c_void_p, _c_void_p]),
    "moe_router_logits_bwd_workspace": (_sz, [_i64, _i32, _i32]),
    "moe_router_logits_bwd": (_int, [_c_void_p, _c_void_p, _int, _c_void_p, _i64, _i32, _i32, _c_void_p, _int,
                                     _c_void_p, _c_void_p, _sz, _c_void_p]),
    "moe_route_topk_workspace": (_sz, [_i64, _i32, _i32]),
    "moe_route_topk": (_int, [_c_void_p, _i64, _i32, _i32] + [_c_void_p] * 8 + [_sz, _c_void_p]),
    "moe_route_topk_noalloc": (_int, [_c_void_p, _i64, _i32, _i32] + [_c_void_p] * 8),
    "moe_route_topk_bwd": (_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i32, _c_void_p, _c_void_p]),
    "moe_dispatch": (_int, [_c_void_p, _int, _i64, _i32, _i32, _c_void_p, _c_void_p, _c_void_p]),
    "moe_dispatch_bwd": (_int, [_c_void_p, _int, _i64, _i32, _i32, _c_void_p, _c_void_p, _c_void_p]),
    "moe_combine": (_int, [_c_void_p, _int, _c_void_p, _c_void_p, _i64, _i32, _i32, _c_void_p, _c_void_p]),
    "moe_combine_bwd": (_int, [_c_void_p, _c_void_p, _int, _c_void_p, _c_void_p, _i64, _i32, _i32, _c_void_p,
                               _c_void_p, _c_void_p]),
    "moe_grouped_ffn_workspace": (_sz, [_i64, _i32, _i32, _i32, _int, _int]),
    "moe_grouped_ffn_fwd": (_int, [_i64, _i32, _i32, _i32, _int] + [_c_void_p] * 11 + [_c_void_p, _sz, _c_void_p]),
    "moe_grouped_ffn_bwd": (_int, [_i64, _i32, _i32, _i32, _int] + [_c_void_p] * 18 + [_c_void_p, _sz, _c_void_p]),
    "moe_mx_act_bytes": (_sz, [_i64, _i32]),
    "moe_mx_tok_rows": (_i64, [_i64, _i32]),
    "moe_mx_tok_bytes": (_sz, [_i64, _i32, _i32]),
    "moe_dispatch_mx_tok": (_int, [_c_void_p, _i64, _i32, _i32, _i32] + [_c_void_p] * 7),
    "moe_combine_bwd_mx_tok": (_int, [_c_void_p] * 7 + [_i64, _i32, _i32, _i32] + [_c_void_p] * 5),
    "moe_dispatch_mx": (_int, [_c_void_p, _i64, _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "moe_combine_bwd_mx": (_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i32, _c_void_p,
                                  _c_void_p, _c_void_p, _c_void_p]),
    "moe_mx_weight_cache_bytes": (_sz, [_i32, _i32, _i32]),
    "moe_route_stats": (_int, [_c_void_p, _i32, _c_void_p, _c_void_p]),
    "moe_mx_weight_cache_build": (_int, [_c_void_p] * 3 + [_i32, _i32, _i32, _c_void_p, _sz, _c_void_p]),
    "mx_quantize": (_int, [_c_void_p, _int, _i64, _i64, _i64, _i32, _c_void_p, _i32, _c_void_p, _c_void_p,
                           _c_void_p]),
    "moe_balance_loss_workspace": (_sz, [_i64, _i32, _i64]),
    "moe_balance_loss": (_int, [_c_void_p, _c_void_p, _i64, _i32, _i32, _c_void_p, _i64, _c_void_p, _f32, _f32]
                         + [_c_void_p] * 6 + [_sz, _c_void_p]),
    "moe_balance_loss_bwd": (_int, [_c_void_p] * 4 + [_i64, _i32, _i32, _c_void_p, _i64, _c_void_p, _f32, _f32]
                             + [_c_void_p] * 6),
    "moe_layernorm": (_int, [_c_void_p] * 4 + [_int, _i64, _i32, _f32] + [_c_void_p] * 5),
    "moe_layernorm_bwd_workspace": (_sz, [_i64, _i32]),
    "moe_layernorm_bwd": (_int, [_c_void_p] * 6 + [_int, _i64, _i32] + [_c_void_p] * 4 + [_sz, _c_void_p]),
    "moe_orthogonalize_workspace": (_sz, [_i32, _i32, _i32, _int]),
    "moe_orthogonalize": (_int, [_c_void_p, _int, _i32, _i32, _i32, _i32, _c_void_p, _f32, _c_void_p, _c_void_p, _sz,
                                 _c_void_p]),
    "moe_muon_step": (_int, [_c_void_p, _int, _i32, _i32, _i32, _c_void_p, _f32, _int, _i32, _c_void_p, _f32,
                             _c_void_p, _f32, _f32, _f32, _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "moe_route_scored_workspace": (_sz, [_i64, _i32, _i32]),
    "moe_route_scored": (_int, [_c_void_p, _c_void_p, _i64, _i32, _i32, _int, _i32, _i32, _i32, _int, _f32]
                         + [_c_void_p] * 8 + [_sz, _c_void_p]),
    "moe_route_scored_bwd": (_int, [_c_void_p] * 3 + [_i64, _i32, _i32, _int, _int, _f32, _int, _c_void_p, _c_void_p]),
    "moe_route_bias_update": (_int, [_c_void_p, _i64, _i32, _f32, _c_void_p, _c_void_p, _c_void_p]),
    "moe_linear_workspace": (_sz, [_int, _i64, _i32, _i32, _int]),
    "moe_linear": (_int, [_c_void_p] * 4 + [_int, _i64, _i32, _i32, _int] + [_c_void_p] * 3 + [_sz, _c_void_p]),
    "moe_linear_bwd": (_int, [_c_void_p] * 4 + [_int, _i64, _i32, _i32, _int, _c_void_p, _int] + [_c_void_p] * 5
                       + [_sz, _c_void_p]),
    "moe_adamw_step": (_int, [_c_void_p, _i32, _int, _int, _i64] + [_c_void_p] * 5 + [_f64] * 4
                       + [_i64, _c_void_p, _c_void_p, ctypes.c_uint32] + [_c_void_p] * 6),
    "moe_adamw_state_values": (_int, [_c_void_p] * 4 + [_i64] + [_c_void_p] * 3),
    "moe_timing_enable": (_int, [_int]),
    "moe_timing_report": (_int, [ctypes.c_char_p, _sz]),
}

_lib = None


class MoeError(RuntimeError):
    pass


def lib():
    """Load libmoe.so (once) and declare its C signatures."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MoeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def exported_symbols():
    return sorted(_SIGS)


def _check(status: int, what: str):
    if status != 0:
        msg = lib().moe_status_str(status).decode()
        raise MoeError(f"{what} failed: {msg} (status {status})")


def _p(t):
    return None if t is None else t.data_ptr()


def _stream():
    # the raw handle of torch.cuda.current_stream(), without building a Stream object per call
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise MoeError(f"unsupported dtype {t.dtype}")


def _ws(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


# --------------------------------------------------------------------------- router

def moe_router_logits(x, w_r, out=None):
    T, d = x.shape
    E = w_r.shape[1]
    out = torch.empty((T, E), dtype=torch.float32, device=x.device) if out is None else out
    _check(lib().moe_router_logits(_p(x), _p(w_r), _dtype_code(x), T, d, E, _p(out), _stream()), "moe_router_logits")
    return out


def moe_router_logits_bwd(x, w_r, dlogits, dx, accumulate_dx=True, dw_r=None, ws=None):
    T, d = x.shape
    E = w_r.shape[1]
    dw_r = torch.empty_like(w_r) if dw_r is None else dw_r
    need = lib().moe_router_logits_bwd_workspace(T, d, E)
    ws = _ws(need, x.device) if ws is None else ws
    _check(lib().moe_router_logits_bwd(_p(x), _p(w_r), _dtype_code(x), _p(dlogits), T, d, E, _p(dx),
                                       int(bool(accumulate_dx)), _p(dw_r), _p(ws), ws.numel(), _stream()),
           "moe_router_logits_bwd")
    return dw_r


def moe_route_topk(logits, k, out=None, ws=None):
    """Returns dict topk_idx, gates, counts, offsets, perm_src, perm_dst, mx_blk_offsets."""
    T, E = logits.shape
    dev = logits.device
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = {
            "topk_idx": torch.empty((T, k), **i32),
            "gates": torch.empty((T, k), dtype=torch.float32, device=dev),
            "counts": torch.empty(E, **i32),
            "offsets": torch.empty(E + 1, **i32),
            "perm_src": torch.empty(T * k, **i32),
            "perm_dst": torch.empty(T * k, **i32),
            "mx_blk_offsets": torch.empty(E + 1, **i32),
        }
    need = lib().moe_route_topk_workspace(T, E, k)
    ws = _ws(need, dev) if ws is None else ws
    _check(lib().moe_route_topk(_p(logits), T, E, k, _p(out["topk_idx"]), _p(out["gates"]), _p(out["counts"]),
                                _p(out["offsets"]), _p(out["perm_src"]), _p(out["perm_dst"]),
                                _p(out.get("mx_blk_offsets")), _p(ws), ws.numel(), _stream()), "moe_route_topk")
    return out


def moe_route_topk_noalloc(logits, k, out):
    """moe_route_topk on the library's static scratch (no workspace); `out` as moe_route_topk returns it."""
    T, E = logits.shape
    _check(lib().moe_route_topk_noalloc(_p(logits), T, E, k, _p(out["topk_idx"]), _p(out["gates"]),
                                        _p(out["counts"]), _p(out["offsets"]), _p(out["perm_src"]),
                                        _p(out["perm_dst"]), _p(out.get("mx_blk_offsets")), _stream()),
           "moe_route_topk_noalloc")
    return out


def moe_route_topk_bwd(gates, dgates, topk_idx, E, out=None):
    T, k = gates.shape
    out = torch.empty((T, E), dtype=torch.float32, device=gates.device) if out is None else out
    _check(lib().moe_route_topk_bwd(_p(gates), _p(dgates), _p(topk_idx), T, E, k, _p(out), _stream()),
           "moe_route_topk_bwd")
    return out


# --------------------------------------------------------------------------- dispatch / combine

def moe_dispatch(x, perm_dst, k, out=None):
    T, d = x.shape
    out = torch.empty((T * k, d), dtype=x.dtype, device=x.device) if out is None else out
    _check(lib().moe_dispatch(_p(x), _dtype_code(x), T, d, k, _p(perm_dst), _p(out), _stream()), "moe_dispatch")
    return out


def moe_mx_act_buffer(rows, cols, device):
    """Caller buffer for moe_dispatch_mx / moe_combine_bwd_mx: E4M3 codes [rows, cols], then grouped scales."""
    n = lib().moe_mx_act_bytes(rows, cols)
    if n == 0:
        raise MoeError(f"moe_mx_act_bytes({rows}, {cols}): unsupported size")
    return _ws(n, device)


def mx_act_split(buf, rows, cols):
    """(codes uint8 [rows, cols], grouped scale bytes uint8 [rows * cols / 32]) views of an MX activation buffer."""
    off = -(-rows * cols // 256) * 256
    return buf[:rows * cols].view(rows, cols), buf[off:off + rows * cols // 32]


def moe_dispatch_mx(x, perm_dst, k, out=None, mx=None):
    """moe_dispatch that also writes the MX rows layout of x_perm (bf16, d % 128 == 0); returns (x_perm, mx)."""
    T, d = x.shape
    out = torch.empty((T * k, d), dtype=x.dtype, device=x.device) if out is None else out
    mx = moe_mx_act_buffer(T * k, d, x.device) if mx is None else mx
    _check(lib().moe_dispatch_mx(_p(x), T, d, k, _p(perm_dst), _p(out), _p(mx), _stream()), "moe_dispatch_mx")
    return out, mx


def moe_mx_tok_buffer(rows, E, cols, device):
    """Caller buffer for the token-axis MX layout: E4M3 codes [cols, moe_mx_tok_rows(rows, E)], then grouped scales."""
    n = lib().moe_mx_tok_bytes(rows, E, cols)
    if n == 0:
        raise MoeError(f"moe_mx_tok_bytes({rows}, {E}, {cols}): unsupported size")
    return _ws(n, device)


def mx_tok_split(buf, rows, E, cols):
    """(codes uint8 [cols, Rp], grouped scale bytes uint8 [Rp / 32 * cols]) views of a token-axis MX buffer."""
    rp = lib().moe_mx_tok_rows(rows, E)
    off = -(-rp * cols // 256) * 256
    return buf[:rp * cols].view(cols, rp), buf[off:off + rp // 32 * cols]


def moe_dispatch_mx_tok(x, route, k, E, out=None, mx=None, mxt=None, write_rows=False):
    """Both MX layouts of the expert rows of x (rows and token-axis), from the routing `route` (perm_src,
    offsets, mx_blk_offsets); the bf16 rows too when write_rows or `out` is given.  Returns (x_perm or None, mx,
    mxt)."""
    T, d = x.shape
    R = T * k
    if out is None and write_rows:
        out = torch.empty((R, d), dtype=x.dtype, device=x.device)
    mx = moe_mx_act_buffer(R, d, x.device) if mx is None else mx
    mxt = moe_mx_tok_buffer(R, E, d, x.device) if mxt is None else mxt
    _check(lib().moe_dispatch_mx_tok(_p(x), T, d, k, E, _p(route["perm_src"]), _p(route["offsets"]),
                                     _p(route["mx_blk_offsets"]), _p(out), _p(mx), _p(mxt), _stream()),
           "moe_dispatch_mx_tok")
    return out, mx, mxt


def moe_dispatch_bwd(dx_perm, perm_dst, k, out=None):
    R, d = dx_perm.shape
    T = R // k
    out = torch.empty((T, d), dtype=dx_perm.dtype, device=dx_perm.device) if out is None else out
    _check(lib().moe_dispatch_bwd(_p(dx_perm), _dtype_code(dx_perm), T, d, k, _p(perm_dst), _p(out), _stream()),
           "moe_dispatch_bwd")
    return out


def moe_combine(y_perm, gates, perm_dst, out=None):
    T, k = gates.shape
    d = y_perm.shape[1]
    out = torch.empty((T, d), dtype=y_perm.dtype, device=y_perm.device) if out is None else out
    _check(lib().moe_combine(_p(y_perm), _dtype_code(y_perm), _p(gates), _p(perm_dst), T, d, k, _p(out), _stream()),
           "moe_combine")
    return out


def moe_combine_bwd(dout, y_perm, gates, perm_dst, dy_perm=None, dgates=None):
    T, k = gates.shape
    d = dout.shape[1]
    dy_perm = torch.empty_like(y_perm) if dy_perm is None else dy_perm
    dgates = torch.empty((T, k), dtype=torch.float32, device=dout.device) if dgates is None else dgates
    _check(lib().moe_combine_bwd(_p(dout), _p(y_perm), _dtype_code(dout), _p(gates), _p(perm_dst), T, d, k,
                                 _p(dy_perm), _p(dgates), _stream()), "moe_combine_bwd")
    return dy_perm, dgates


def moe_combine_bwd_mx(dout, y_perm, gates, perm_dst, dy_perm=None, dgates=None, mx=None):
    """moe_combine_bwd that also writes the MX rows layout of dy_perm; returns (dy_perm, dgates, mx)."""
    T, k = gates.shape
    d = dout.shape[1]
    dy_perm = torch.empty_like(y_perm) if dy_perm is None else dy_perm
    dgates = torch.empty((T, k), dtype=torch.float32, device=dout.device) if dgates is None else dgates
    mx = moe_mx_act_buffer(T * k, d, dout.device) if mx is None else mx
    _check(lib().moe_combine_bwd_mx(_p(dout), _p(y_perm), _p(gates), _p(perm_dst), T, d, k, _p(dy_perm), _p(dgates),
                                    _p(mx), _stream()), "moe_combine_bwd_mx")
    return dy_perm, dgates, mx


def moe_combine_bwd_mx_tok(dout, y_perm, gates, route, E, dy_perm=None, dgates=None, mx=None, mxt=None,
                           write_rows=False):
    """dgates, and dY = gate x dout in both MX layouts (rows and token-axis); the bf16 rows too when write_rows
    or `dy_perm` is given.  Returns (dy_perm or None, dgates, mx, mxt)."""
    T, k = gates.shape
    d = dout.shape[1]
    R = T * k
    if dy_perm is None and write_rows:
        dy_perm = torch.empty_like(y_perm)
    dgates = torch.empty((T, k), dtype=torch.float32, device=dout.device) if dgates is None else dgates
    mx = moe_mx_act_buffer(R, d, dout.device) if mx is None else mx
    mxt = moe_mx_tok_buffer(R, E, d, dout.device) if mxt is None else mxt
    _check(lib().moe_combine_bwd_mx_tok(_p(dout), _p(y_perm), _p(gates), _p(route["perm_dst"]), _p(route["perm_src"]),
                                        _p(route["offsets"]), _p(route["mx_blk_offsets"]), T, d, k, E, _p(dy_perm),
                                        _p(dgates), _p(mx), _p(mxt), _stream()), "moe_combine_bwd_mx_tok")
    return dy_perm, dgates, mx, mxt


def moe_route_stats(counts, out=None):
    """counts [E] int32 (device) -> int32 [4] on the device: max rows, min rows, empty experts, total rows."""
    E = counts.shape[0]
    out = torch.empty(4, dtype=torch.int32, device=counts.device) if out is None else out
    _check(lib().moe_route_stats(_p(counts), E, _p(out), _stream()), "moe_route_stats")
    return out


# --------------------------------------------------------------------------- grouped FFN

def moe_grouped_ffn_workspace(R, E, d, f, prec, is_bwd):
    return lib().moe_grouped_ffn_workspace(R, E, d, f, _PREC[prec], int(is_bwd))


def moe_grouped_ffn_fwd(x_perm, offsets, w_gate, w_up, w_down, prec, out=None, ws=None, mx_wcache=None, x_mx=None,
                        rows=None):
    """x_perm may be None with prec "mxfp8" and x_mx given; then `rows` (R) is required."""
    E, d, f = w_gate.shape
    R = x_perm.shape[0] if x_perm is not None else int(rows)
    dev = w_gate.device
    if out is None:
        out = {name: torch.empty((R, f), dtype=w_gate.dtype, device=dev) for name in ("h_gate", "h_up", "a_act")}
        out["y_perm"] = torch.empty((R, d), dtype=w_gate.dtype, device=dev)
    ws = _ws(moe_grouped_ffn_workspace(R, E, d, f, prec, 0), dev) if ws is None else ws
    _check(lib().moe_grouped_ffn_fwd(R, E, d, f, _PREC[prec], _p(offsets), _p(x_perm), _p(w_gate), _p(w_up),
                                     _p(w_down), _p(mx_wcache), _p(x_mx), _p(out["h_gate"]), _p(out["h_up"]),
                                     _p(out["a_act"]), _p(out["y_perm"]), _p(ws), ws.numel(), _stream()),
           "moe_grouped_ffn_fwd")
    return out


def moe_grouped_ffn_bwd(dy_perm, x_perm, h_gate, h_up, a_act, offsets, mx_blk_offsets, w_gate, w_up, w_down, prec,
                        out=None, ws=None, mx_wcache=None, dy_mx=None, x_mxt=None, dy_mxt=None):
    """With prec "mxfp8", x_perm may be None when x_mxt is given, dy_perm when dy_mx and dy_mxt are."""
    E, d, f = w_gate.shape
    R = h_gate.shape[0]
    dev = h_gate.device
    if out is None:
        out = {"dx_perm": torch.empty((R, d), dtype=h_gate.dtype, device=dev), "dw_gate": torch.empty_like(w_gate),
               "dw_up": torch.empty_like(w_up), "dw_down": torch.empty_like(w_down)}
    ws = _ws(moe_grouped_ffn_workspace(R, E, d, f, prec, 1), dev) if ws is None else ws
    _check(lib().moe_grouped_ffn_bwd(R, E, d, f, _PREC[prec], _p(offsets), _p(mx_blk_offsets), _p(dy_perm),
                                     _p(x_perm), _p(h_gate), _p(h_up), _p(a_act), _p(w_gate), _p(w_up), _p(w_down),
                                     _p(mx_wcache), _p(dy_mx), _p(x_mxt), _p(dy_mxt), _p(out["dx_perm"]),
                                     _p(out["dw_gate"]), _p(out["dw_up"]),
                                     _p(out["dw_down"]), _p(ws), ws.numel(), _stream()), "moe_grouped_ffn_bwd")
    return out


def moe_mx_weight_cache_build(w_gate, w_up, w_down, cache=None):
    """Pre-quantised MXFP8 weights (both orientations); returns the uint8 cache tensor."""
    E, d, f = w_gate.shape
    n = lib().moe_mx_weight_cache_bytes(E, d, f)
    cache = _ws(n, w_gate.device) if cache is None else cache
    _check(lib().moe_mx_weight_cache_build(_p(w_gate), _p(w_up), _p(w_down), E, d, f, _p(cache), cache.numel(),
                                           _stream()), "moe_mx_weight_cache_build")
    return cache


# --------------------------------------------------------------------------- MX quantiser

def mx_quantize(src, axis, seg_offsets=None, nseg=0, q=None, scales=None):
    """src [rows, cols] or [batch, rows, cols]; layouts as documented in include/moe.h."""
    s3 = src if src.dim() == 3 else src.unsqueeze(0)
    B, rows, cols = s3.shape
    dev = src.device
    if q is None:
        if axis == 1:
            q = torch.empty((B, rows, cols), dtype=torch.uint8, device=dev)
            scales = torch.empty((B, rows, cols // 32), dtype=torch.uint8, device=dev)
        elif seg_offsets is None:
            q = torch.empty((B, cols, rows), dtype=torch.uint8, device=dev)
            scales = torch.empty((B, cols, rows // 32), dtype=torch.uint8, device=dev)
        else:
            rp = 32 * (-(-rows // 32) + nseg)
            q = torch.empty((cols, rp), dtype=torch.uint8, device=dev)
            scales = torch.empty((cols, rp // 32), dtype=torch.uint8, device=dev)
    _check(lib().mx_quantize(_p(s3), _dtype_code(src), B, rows, cols, axis, _p(seg_offsets), nseg, _p(q), _p(scales),
                             _stream()), "mx_quantize")
    return q, scales


# --------------------------------------------------------------------------- norm, balance loss, weight update

def _args(what, dev, specs):
    """Device tensors as the C ABI reads them: (name, tensor or None, shape, type) each of this shape and type,
    contiguous, and on the current device, whose current stream the call is enqueued on.  Only what the caller gave
    need be listed: a check costs about as much as allocating a tensor (0.7 us)."""
    for name, t, shape, dtype in specs:
        if t is None or (t.shape == shape and t.dtype is dtype and t.device == dev and t.is_contiguous()):
            continue
        if t.shape != shape or t.dtype is not dtype:
            raise MoeError(f"{what}: {name} is {t.dtype} {list(t.shape)}, expected {dtype} {list(shape)}")
        if not t.is_contiguous():
            raise MoeError(f"{what}: {name} is not contiguous")
        raise MoeError(f"{what}: {name} is on {t.device}, the others on {dev}")
    if dev.type != "cuda" or dev.index != torch.cuda.current_device():
        raise MoeError(f"{what}: the tensors are on {dev}, not on the current GPU")


def _ws_spec(ws):
    return () if ws is None else (("ws", ws, (ws.numel(),), torch.uint8),)


def _storage(what, t, dims):
    """The C code of t's storage type, for a tensor of `dims` dimensions."""
    if t.dim() != dims:
        raise MoeError(f"{what}: a tensor of {dims} dimensions is needed, not {t.dim()}")
    _sizes(what, t)
    return _dtype_code(t)


def _sizes(what, t):
    """The C ABI takes most sizes in 32 bits: a larger one would be cut."""
    if max(t.shape) >> 31:
        raise MoeError(f"{what}: {list(t.shape)} has a size of 2^31 or more")


_F32, _I32 = torch.float32, torch.int32


def moe_layernorm(x, weight=None, bias=None, eps=1e-5, residual=None, out=None):
    """Layer norm of the rows of x [T, d] (of x + residual, also returned as "sum"); {"y", "mean", "rstd"[, "sum"]}."""
    what, dev, dt = "moe_layernorm", x.device, x.dtype
    code = _storage(what, x, 2)
    T, d = x.shape
    rows, cols, per = (T, d), (d,), (T,)
    specs = (("x", x, rows, dt), ("weight", weight, cols, dt), ("bias", bias, cols, dt),
             ("residual", residual, rows, dt))
    if out is None:
        out = {"y": torch.empty_like(x), "mean": torch.empty(T, dtype=_F32, device=dev),
               "rstd": torch.empty(T, dtype=_F32, device=dev)}
        if residual is not None:
            out["sum"] = torch.empty_like(x)
    else:
        specs += (("y", out["y"], rows, dt), ("sum", out.get("sum"), rows, dt), ("mean", out.get("mean"), per, _F32),
                  ("rstd", out.get("rstd"), per, _F32))
    y, total, mean, rstd = out["y"], out.get("sum"), out.get("mean"), out.get("rstd")
    _args(what, dev, specs)
    _check(lib().moe_layernorm(_p(x), _p(residual), _p(weight), _p(bias), code, T, d, eps, _p(y), _p(total), _p(mean),
                               _p(rstd), _stream()), what)
    return out


def moe_layernorm_bwd(dy, x, weight, mean, rstd, dres=None, out=None, ws=None):
    """Gradients of moe_layernorm; x: the rows that were normalised ("sum" with a residual), dres: added to dx.
    {"dx", "dw", "db"}; an out without "dw" or "db" leaves that sum out."""
    what, dev, dt = "moe_layernorm_bwd", x.device, x.dtype
    code = _storage(what, x, 2)
    T, d = x.shape
    rows, cols, per = (T, d), (d,), (T,)
    specs = (("x", x, rows, dt), ("dy", dy, rows, dt), ("weight", weight, cols, dt), ("mean", mean, per, _F32),
             ("rstd", rstd, per, _F32), ("dres", dres, rows, dt)) + _ws_spec(ws)
    if out is None:
        out = {"dx": torch.empty_like(x), "dw": torch.empty(d, dtype=dt, device=dev),
               "db": torch.empty(d, dtype=dt, device=dev)}
    else:
        specs += (("dx", out["dx"], rows, dt), ("dw", out.get("dw"), cols, dt), ("db", out.get("db"), cols, dt))
    dx, dw, db = out["dx"], out.get("dw"), out.get("db")
    _args(what, dev, specs)
    if ws is None:
        ws = _ws(lib().moe_layernorm_bwd_workspace(T, d), dev)
    _check(lib().moe_layernorm_bwd(_p(dy), _p(x), _p(weight), _p(mean), _p(rstd), _p(dres), code, T, d, _p(dx), _p(dw),
                                   _p(db), _p(ws), ws.numel(), _stream()), what)
    return out


def _balance_specs(logits, k, topk_idx, seq_offsets, token_mask):
    if logits.dim() != 2 or (seq_offsets is not None and seq_offsets.dim() != 1):
        raise MoeError("logits of two dimensions and seq_offsets of one are needed")
    _sizes("logits", logits)
    T, E = logits.shape
    S = 1 if seq_offsets is None else seq_offsets.numel() - 1
    mt = torch.bool if token_mask is not None and token_mask.dtype is torch.bool else torch.uint8
    return T, E, S, (("logits", logits, (T, E), _F32), ("topk_idx", topk_idx, (T, k), _I32),
                     ("seq_offsets", seq_offsets, (S + 1,), _I32), ("token_mask", token_mask, (T,), mt))


def moe_balance_loss(logits, topk_idx, alpha, zeta, seq_offsets=None, token_mask=None, out=None, ws=None):
    """Balance and z loss of a routing: {"loss" [2], "counts" [S, E], "probs" [S, E], "lse" [T], "norm" [S + 2]}."""
    what, dev, k = "moe_balance_loss", logits.device, topk_idx.shape[-1] if topk_idx.dim() else 0
    T, E, S, specs = _balance_specs(logits, k, topk_idx, seq_offsets, token_mask)
    specs += _ws_spec(ws)
    if out is None:
        out = {"loss": torch.empty(2, dtype=_F32, device=dev), "counts": torch.empty((S, E), dtype=_I32, device=dev),
               "probs": torch.empty((S, E), dtype=_F32, device=dev), "lse": torch.empty(T, dtype=_F32, device=dev),
               "norm": torch.empty(S + 2, dtype=_F32, device=dev)}
    else:
        specs += (("loss", out["loss"], (2,), _F32), ("counts", out["counts"], (S, E), _I32),
                  ("probs", out["probs"], (S, E), _F32), ("lse", out["lse"], (T,), _F32),
                  ("norm", out["norm"], (S + 2,), _F32))
    loss, counts, probs, lse, norm = out["loss"], out["counts"], out["probs"], out["lse"], out["norm"]
    _args(what, dev, specs)
    if ws is None:
        ws = _ws(lib().moe_balance_loss_workspace(T, E, S), dev)
    _check(lib().moe_balance_loss(_p(logits), _p(topk_idx), T, E, k, _p(seq_offsets), S, _p(token_mask), alpha, zeta,
                                  _p(loss), _p(counts), _p(probs), _p(lse), _p(norm), _p(ws), ws.numel(), _stream()),
           what)
    return out


def moe_balance_loss_bwd(logits, fwd, k, alpha, zeta, dloss=None, seq_offsets=None, token_mask=None, topk_idx=None,
                         gates=None, dgates=None, out=None):
    """dlogits [T, E] of the two losses (fwd: what moe_balance_loss returned for the same arguments), plus the gates'
    gradient when gates, dgates and topk_idx are given."""
    what, dev = "moe_balance_loss_bwd", logits.device
    T, E, S, specs = _balance_specs(logits, k, topk_idx, seq_offsets, token_mask)
    counts, lse, norm = fwd["counts"], fwd["lse"], fwd["norm"]
    _args(what, dev, specs + (("counts", counts, (S, E), _I32), ("lse", lse, (T,), _F32), ("norm", norm, (S + 2,), _F32),
                              ("dloss", dloss, (2,), _F32), ("gates", gates, (T, k), _F32),
                              ("dgates", dgates, (T, k), _F32), ("out", out, (T, E), _F32)))
    if out is None:
        out = torch.empty((T, E), dtype=_F32, device=dev)
    _check(lib().moe_balance_loss_bwd(_p(logits), _p(lse), _p(counts), _p(norm), T, E, k, _p(seq_offsets), S,
                                      _p(token_mask), alpha, zeta, _p(dloss), _p(topk_idx), _p(gates), _p(dgates),
                                      _p(out), _stream()), what)
    return out


def moe_orthogonalize_workspace(E, rows, cols, dtype):
    code = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}.get(dtype)
    if code is None:
        raise MoeError(f"unsupported dtype {dtype}")
    return lib().moe_orthogonalize_workspace(E, rows, cols, code)


def _coef(steps, coef):
    """Per-step (a, b, c): one triple for all steps, a list of `steps` triples, or None."""
    if not 1 <= steps <= 16:
        raise MoeError(f"steps: 1 to 16, not {steps}")
    if coef is None:
        return None
    rows = list(coef) if len(coef) == 0 or hasattr(coef[0], "__len__") else [coef] * steps
    if len(rows) != steps or any(len(r) != 3 for r in rows):
        raise MoeError(f"coef: expected three coefficients, or {steps} triples")
    return (ctypes.c_float * (3 * steps))(*[float(v) for r in rows for v in r])


def moe_orthogonalize(g, steps=5, coef=None, eps=1e-7, out=None, ws=None):
    """Newton-Schulz orthogonalisation of each matrix of g [E, rows, cols]."""
    what, dev, dt = "moe_orthogonalize", g.device, g.dtype
    code = _storage(what, g, 3)
    E, rows, cols = shape = g.shape
    _args(what, dev, (("g", g, shape, dt), ("out", out, shape, dt)) + _ws_spec(ws))
    if out is None:
        out = torch.empty_like(g)
    if ws is None:
        ws = _ws(lib().moe_orthogonalize_workspace(E, rows, cols, code), dev)
    _check(lib().moe_orthogonalize(_p(g), code, E, rows, cols, steps, _coef(steps, coef), eps, _p(out), _p(ws),
                                   ws.numel(), _stream()), what)
    return out


def moe_muon_step(g, mom, w, lr, momentum=0.95, nesterov=True, weight_decay=0.0, scale=1.0, steps=5, coef=None,
                  eps=1e-7, inplace=True, ws=None):
    """One Muon step of the weights w [E, rows, cols] with momentum mom (fp32); returns (w, mom): the tensors given,
    updated, or with inplace=False new ones."""
    what, dev, dt = "moe_muon_step", g.device, g.dtype
    code = _storage(what, g, 3)
    E, rows, cols = shape = g.shape
    _args(what, dev, (("g", g, shape, dt), ("w", w, shape, dt), ("mom", mom, shape, _F32)) + _ws_spec(ws))
    if ws is None:
        ws = _ws(lib().moe_orthogonalize_workspace(E, rows, cols, code), dev)
    w_out, mom_out = (w, mom) if inplace else (torch.empty_like(w), torch.empty_like(mom))
    _check(lib().moe_muon_step(_p(g), code, E, rows, cols, _p(mom), momentum, int(bool(nesterov)), steps,
                               _coef(steps, coef), eps, _p(w), lr, weight_decay, scale, _p(mom_out), _p(w_out),
                               _p(ws), ws.numel(), _stream()), what)
    return w_out, mom_out


# --------------------------------------------------------------------------- routing by scores

_SCORE = {"softmax": 0, "sigmoid": 1}
_ACT = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}


def _named(what, kind, table, name):
    if name not in table:
        raise MoeError(f"{what}: {kind} {name!r}, expected one of {sorted(table)}")
    return table[name]


def _route_sizes(what, logits, k):
    if logits.dim() != 2:
        raise MoeError(f"{what}: logits of two dimensions are needed, not {logits.dim()}")
    _sizes(what, logits)
    T, E = logits.shape
    if not 1 <= k <= E:
        raise MoeError(f"{what}: k = {k} of {E} experts")
    return T, E


def _route_out(T, E, k, dev):
    i32 = dict(dtype=_I32, device=dev)
    return {"topk_idx": torch.empty((T, k), **i32), "gates": torch.empty((T, k), dtype=_F32, device=dev),
            "counts": torch.empty(E, **i32), "offsets": torch.empty(E + 1, **i32), "perm_src": torch.empty(T * k, **i32),
            "perm_dst": torch.empty(T * k, **i32), "mx_blk_offsets": torch.empty(E + 1, **i32)}


def moe_route_scored(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renorm=True, scale=1.0,
                     out=None, ws=None):
    """Routing by softmax or sigmoid scores, a bias and groups of experts; returns what moe_route_topk returns."""
    what, dev = "moe_route_scored", logits.device
    code = _named(what, "score", _SCORE, score)
    T, E = _route_sizes(what, logits, k)
    if (groups | top_groups | group_best) >> 31:  # 32 bits: a larger number would be cut
        raise MoeError(f"{what}: groups, top_groups, group_best = {groups}, {top_groups}, {group_best}")
    specs = (("logits", logits, (T, E), _F32), ("bias", bias, (E,), _F32)) + _ws_spec(ws)
    if out is not None:
        specs += (("topk_idx", out["topk_idx"], (T, k), _I32), ("gates", out["gates"], (T, k), _F32),
                  ("counts", out["counts"], (E,), _I32), ("offsets", out["offsets"], (E + 1,), _I32),
                  ("perm_src", out["perm_src"], (T * k,), _I32), ("perm_dst", out["perm_dst"], (T * k,), _I32),
                  ("mx_blk_offsets", out.get("mx_blk_offsets"), (E + 1,), _I32))
    _args(what, dev, specs)
    if out is None:
        out = _route_out(T, E, k, dev)
    if ws is None:
        ws = _ws(lib().moe_route_scored_workspace(T, E, k), dev)
    _check(lib().moe_route_scored(_p(logits), _p(bias), T, E, k, code, groups, top_groups, group_best, int(bool(renorm)),
                                  scale, _p(out["topk_idx"]), _p(out["gates"]), _p(out["counts"]), _p(out["offsets"]),
                                  _p(out["perm_src"]), _p(out["perm_dst"]), _p(out.get("mx_blk_offsets")), _p(ws),
                                  ws.numel(), _stream()), what)
    return out


def moe_route_scored_bwd(logits, topk_idx, dgates, score="softmax", renorm=True, scale=1.0, out=None, accumulate=False):
    """dlogits [T, E] of moe_route_scored's gates; with accumulate added to `out`."""
    what, dev, k = "moe_route_scored_bwd", logits.device, topk_idx.shape[-1] if topk_idx.dim() else 0
    code = _named(what, "score", _SCORE, score)
    T, E = _route_sizes(what, logits, k)
    if accumulate and out is None:
        raise MoeError(f"{what}: accumulate needs out")
    _args(what, dev, (("logits", logits, (T, E), _F32), ("topk_idx", topk_idx, (T, k), _I32),
                      ("dgates", dgates, (T, k), _F32), ("out", out, (T, E), _F32)))
    if out is None:
        out = torch.empty((T, E), dtype=_F32, device=dev)
    _check(lib().moe_route_scored_bwd(_p(logits), _p(topk_idx), _p(dgates), T, E, k, code, int(bool(renorm)), scale,
                                      int(bool(accumulate)), _p(out), _stream()), what)
    return out


def moe_route_bias_update(counts, bias, rate, inplace=True):
    """bias [E] moved by rate towards the experts below the mean of counts [E] or [S, E]; returns it (or a new one)."""
    what, dev = "moe_route_bias_update", bias.device
    if bias.dim() != 1 or counts.dim() not in (1, 2):
        raise MoeError(f"{what}: bias [E] and counts [E] or [S, E] are needed")
    E, S = bias.shape[0], 1 if counts.dim() == 1 else counts.shape[0]
    _args(what, dev, (("counts", counts, (E,) if counts.dim() == 1 else (S, E), _I32), ("bias", bias, (E,), _F32)))
    out = bias if inplace else torch.empty_like(bias)
    _check(lib().moe_route_bias_update(_p(counts), S, E, rate, _p(bias), _p(out), _stream()), what)
    return out


# --------------------------------------------------------------------------- dense product

def _linear_sizes(what, x, w):
    code = _storage(what, x, 2)
    if w.dim() != 2:
        raise MoeError(f"{what}: w of two dimensions is needed, not {w.dim()}")
    _sizes(what, w)
    return code, x.shape[0], x.shape[1], w.shape[1]


def moe_linear_workspace(x, w, bwd=False):
    """A workspace for moe_linear (or its backward) of these tensors' sizes."""
    code, M, K, N = _linear_sizes("moe_linear_workspace", x, w)
    n = lib().moe_linear_workspace(code, M, K, N, int(bool(bwd)))
    if n == 0:
        raise MoeError(f"moe_linear_workspace: {M} x {K} x {N} is not supported")
    return _ws(n, x.device)


def moe_linear(x, w, bias=None, act="none", residual=None, save=False, out=None, ws=None):
    """{"y"[, "z"]}: y = act(x w + bias) + residual; z (with save, or in out) is what act was applied to."""
    what, dev, dt = "moe_linear", x.device, x.dtype
    acode = _named(what, "act", _ACT, act)
    code, M, K, N = _linear_sizes(what, x, w)
    specs = (("x", x, (M, K), dt), ("w", w, (K, N), dt), ("bias", bias, (N,), dt),
             ("residual", residual, (M, N), dt)) + _ws_spec(ws)
    if out is not None:
        specs += (("y", out["y"], (M, N), dt), ("z", out.get("z"), (M, N), dt))
    _args(what, dev, specs)
    if out is None:
        out = {name: torch.empty((M, N), dtype=dt, device=dev) for name in (("y", "z") if save else ("y",))}
    if ws is None:
        ws = moe_linear_workspace(x, w)
    _check(lib().moe_linear(_p(x), _p(w), _p(bias), _p(residual), code, M, K, N, acode, _p(out["y"]), _p(out.get("z")),
                            _p(ws), ws.numel(), _stream()), what)
    return out


def moe_linear_bwd(dy, x, w, z=None, act="none", in_z=None, in_act="none", dres=None, out=None, ws=None):
    """Gradients {"dx", "dw", "db"} of moe_linear; an out without one of them leaves it out.  With in_act, dx is the
    gradient of in_z, where x = in_act(in_z); dres is added to dx."""
    what, dev, dt = "moe_linear_bwd", x.device, x.dtype
    acode, icode = _named(what, "act", _ACT, act), _named(what, "in_act", _ACT, in_act)
    code, M, K, N = _linear_sizes(what, x, w)
    specs = (("dy", dy, (M, N), dt), ("x", x, (M, K), dt), ("w", w, (K, N), dt), ("z", z, (M, N), dt),
             ("in_z", in_z, (M, K), dt), ("dres", dres, (M, K), dt)) + _ws_spec(ws)
    if out is not None:
        specs += (("dx", out.get("dx"), (M, K), dt), ("dw", out.get("dw"), (K, N), dt), ("db", out.get("db"), (N,), dt))
    _args(what, dev, specs)
    if out is None:
        out = {"dx": torch.empty((M, K), dtype=dt, device=dev), "dw": torch.empty((K, N), dtype=dt, device=dev),
               "db": torch.empty(N, dtype=dt, device=dev)}
    if ws is None:
        ws = moe_linear_workspace(x, w, bwd=True)
    _check(lib().moe_linear_bwd(_p(dy), _p(x), _p(w), _p(z), code, M, K, N, acode, _p(in_z), icode, _p(dres),
                                _p(out.get("dx")), _p(out.get("dw")), _p(out.get("db")), _p(ws), ws.numel(), _stream()),
           what)
    return out


# --------------------------------------------------------------------------- AdamW

class _AdamwTensor(ctypes.Structure):
    _fields_ = [("w", _c_void_p), ("g", _c_void_p), ("w_out", _c_void_p), ("n", _i64), ("offset", _i64),
                ("weight_decay", _f32), ("lr_scale", _f32)]


def _adamw_offsets(params):
    off = [0]
    for t in params:
        off.append(off[-1] + -(-t.numel() // 32) * 32)
    return off


def moe_adamw_state(params, bits=32, master=False):
    """Zero states for a list of tensors, tensor i at [offsets[i], offsets[i] + its size) of each flat buffer:
    {"bits", "offsets", "m", "v"[, "m_scale", "v_scale"][, "master"]}.  bits 8: codes (m, and the root of v) and their
    scales; master: fp32 copies of bf16 weights."""
    if bits not in (32, 8) or not params:
        raise MoeError(f"moe_adamw_state: bits 32 or 8 and a tensor are needed, not {bits} and {len(params)}")
    off, dev = _adamw_offsets(params), params[0].device
    state = {"bits": bits, "offsets": off[:-1]}
    for name in ("m", "v"):
        state[name] = torch.zeros(off[-1], dtype=_F32 if bits == 32 else torch.uint8, device=dev)
        if bits == 8:
            state[name + "_scale"] = torch.zeros(off[-1] // 32, dtype=torch.uint8, device=dev)
    if master:
        state["master"] = torch.zeros(off[-1], dtype=_F32, device=dev)
        for t, o in zip(params, off):
            state["master"][o:o + t.numel()] = t.detach().reshape(-1)
    return state


class AdamwPlan:
    """What moe_adamw_step needs of a list of tensors, checked and laid out once (moe_adamw_plan).  It holds the tensors
    and their addresses; a step refuses tensors that have been given other memory since."""

    def __init__(self, dtype, bits, length, table, params, grads, w_out, state, state_out):
        self.dtype, self.bits, self.length, self.table = dtype, bits, length, table
        self.params, self.grads, self.w_out, self.state, self.state_out = params, grads, w_out, state, state_out
        names = ("m", "v", "m_scale", "v_scale", "master")
        self.device = params[0].device
        self.tensors = ([*params, *grads, *w_out] + [state[n] for n in names if n in state]
                        + [state_out[n] for n in names if n in state_out])
        self.at = [t.data_ptr() for t in self.tensors]
        self.ins, self.outs = [_p(state.get(n)) for n in names], [_p(state_out.get(n)) for n in names]


def moe_adamw_plan(params, grads, state, weight_decay=0.0, lr_scale=1.0, out=None):
    """A plan for steps of params (of one type, fp32 or bf16) from grads (of the same shapes) with state
    (moe_adamw_state).  weight_decay, lr_scale: numbers, or one per tensor.  out: (tensors, state) that take the results;
    None: in place."""
    what = "moe_adamw_plan"
    params, grads = list(params), list(grads)
    if not params or len(grads) != len(params):
        raise MoeError(f"{what}: {len(params)} tensors and {len(grads)} gradients")
    w_out, state_out = (params, state) if out is None else (list(out[0]), out[1])
    if len(w_out) != len(params):
        raise MoeError(f"{what}: {len(params)} tensors and {len(w_out)} outputs")
    n, dev, dt = len(params), params[0].device, params[0].dtype
    code = _dtype_code(params[0])
    per = {"weight_decay": weight_decay, "lr_scale": lr_scale}
    for name, v in per.items():
        per[name] = list(v) if hasattr(v, "__len__") else [v] * n
        if len(per[name]) != n:
            raise MoeError(f"{what}: {len(per[name])} values of {name} for {n} tensors")
    off = _adamw_offsets(params)
    bits = state["bits"]
    kind = _F32 if bits == 32 else torch.uint8
    specs = []
    for i, (w, g, o) in enumerate(zip(params, grads, w_out)):
        specs += [(f"tensor {i}", w, w.shape, dt), (f"gradient {i}", g, w.shape, dt), (f"output {i}", o, w.shape, dt)]
    for st in (state, state_out):
        if st["bits"] != bits or st["offsets"] != off[:-1] or ("master" in st) != ("master" in state):
            raise MoeError(f"{what}: a state of other tensors")
        specs += [(name, st[name], (off[-1],), kind) for name in ("m", "v")]
        if bits == 8:
            specs += [(name, st[name], (off[-1] // 32,), torch.uint8) for name in ("m_scale", "v_scale")]
        specs += [("master", st.get("master"), (off[-1],), _F32)]
    if "master" in state and dt is _F32:
        raise MoeError(f"{what}: a master for fp32 tensors")
    _args(what, dev, specs)
    written = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in w_out if t.numel())
    if any(a[1] > b[0] for a, b in zip(written, written[1:])):
        raise MoeError(f"{what}: outputs overlap (a tensor twice)")
    table = (_AdamwTensor * n)(*[_AdamwTensor(_p(w), _p(g), _p(o), w.numel(), at, wd, ls) for w, g, o, at, wd, ls in
                                 zip(params, grads, w_out, off, per["weight_decay"], per["lr_scale"])])
    return AdamwPlan(code, bits, off[-1], table, params, grads, w_out, state, state_out)


def moe_adamw_step(plan, lr, step=1, betas=(0.9, 0.999), eps=1e-8, seed=0, grad_scale=None, step_dev=None):
    """One AdamW step (step counts from 1; step_dev: an int64 tensor [1] on the device in its place); returns the
    updated (tensors, state)."""
    what = "moe_adamw_step"
    if not -(1 << 63) <= step < 1 << 63:  # 64 bits: a larger number would be cut
        raise MoeError(f"{what}: step = {step}")
    if [t.data_ptr() for t in plan.tensors] != plan.at:
        raise MoeError(f"{what}: a tensor of the plan has other memory now")
    _args(what, plan.device, (("grad_scale", grad_scale, (1,), _F32), ("step_dev", step_dev, (1,), torch.int64)))
    m, v, ms, vs, master = plan.ins
    mo, vo, mso, vso, mastero = plan.outs
    _check(lib().moe_adamw_step(plan.table, len(plan.params), plan.dtype, plan.bits, plan.length, m, v, ms, vs, master,
                                lr, *betas, eps, step, _p(step_dev), _p(grad_scale), seed & 0xFFFFFFFF, mo, vo, mso, vso,
                                mastero, _stream()), what)
    return plan.w_out, plan.state_out


def moe_adamw_state_values(state):
    """The values of an 8-bit state in bf16: {"m", "root"} (the root of v), flat as the state is."""
    what, dev, n = "moe_adamw_state_values", state["m"].device, state["m"].numel()
    if state["bits"] != 8:
        raise MoeError(f"{what}: a state of 8 bits is needed")
    _args(what, dev, tuple((k, state[k], (n,), torch.uint8) for k in ("m", "v"))
          + tuple((k, state[k], (n // 32,), torch.uint8) for k in ("m_scale", "v_scale")))
    out = {"m": torch.empty(n, dtype=torch.bfloat16, device=dev), "root": torch.empty(n, dtype=torch.bfloat16, device=dev)}
    _check(lib().moe_adamw_state_values(_p(state["m"]), _p(state["m_scale"]), _p(state["v"]), _p(state["v_scale"]), n,
                                        _p(out["m"]), _p(out["root"]), _stream()), what)
    return out


# --------------------------------------------------------------------------- diagnostics

def moe_timing_enable(on: bool = True):
    _check(lib().moe_timing_enable(int(bool(on))), "moe_timing_enable")


def moe_timing_report() -> dict:
    """{kernel name: (launches, total ms)} of the launches since the last enable/report."""
    buf = ctypes.create_string_buffer(1 << 16)
    _check(lib().moe_timing_report(buf, len(buf)), "moe_timing_report")
    out = {}
    for line in buf.value.decode().splitlines():
        name, n, ms = line.split()
        out[name] = (int(n), float(ms))
    return out

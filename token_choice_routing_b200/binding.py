"""ctypes binding of libmoe_null.so (include/moe_null.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. Tensors are torch CUDA tensors; their data pointers and the current
CUDA stream are passed through the C ABI. There is no CPU fallback: if the
library is missing this module raises on import.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_null.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_DEVICE_BOUNDS = 0, -1, -2, -3, -4, -5


class MoEError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {code} ({status_string(code)})")
        self.code = code


class Dims(C.Structure):
    _fields_ = [("T", C.c_int32), ("d", C.c_int32), ("N", C.c_int32), ("M", C.c_int32),
                ("K", C.c_int32), ("F", C.c_int32), ("F_shared", C.c_int32), ("flags", C.c_uint32),
                ("C", C.c_int32), ("V", C.c_int32)]


class Weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("w_router", "router_bias", "gate_up", "w_down",
                                           "shared_gate_up", "shared_down", "const_vectors", "router_split")]


OUTPUT_FIELDS = ("logits", "topk_idx", "topk_gate", "n_real", "counts", "offsets", "perm_tok",
                 "slot_row", "xs", "h", "h_shared", "ys", "shared_out", "y", "counts_ext", "P",
                 "losses", "z", "z_shared")


class Outputs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in OUTPUT_FIELDS]


SAVED_FIELDS = ("x", "logits", "topk_idx", "topk_gate", "offsets", "slot_row", "xs", "h", "h_shared", "ys",
                "counts_ext")


class Saved(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in SAVED_FIELDS] + [("t_total", C.c_int64), ("z", C.c_void_p),
                                                          ("z_shared", C.c_void_p)]


GRAD_FIELDS = ("dx", "dw_router", "dbias", "dtok_null_bias", "dw_gate", "dw_up", "dw_down", "dws_gate",
               "dws_up", "dws_down", "dconst")


SAVED8_FIELDS = ("x", "logits", "topk_idx", "topk_gate", "offsets", "slot_row", "counts_ext")
SAVED8_CODES = ("z_codes", "z_scales", "zs_codes", "zs_scales", "ys_codes", "ys_scales")


class Codes8(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in SAVED8_CODES]


class Saved8(C.Structure):
    _fields_ = ([(n, C.c_void_p) for n in SAVED8_FIELDS] + [("t_total", C.c_int64)] +
                [(n, C.c_void_p) for n in SAVED8_CODES])


class Grads(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in GRAD_FIELDS]


def _load() -> C.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"CUDA library not built: {LIB_PATH} is missing "
                          "(run python -m token_choice_routing_b200.build)")
    lib = C.CDLL(LIB_PATH)
    vp, i32, i64, sz = C.c_void_p, C.c_int, C.c_int64, C.c_size_t
    pd = C.POINTER(Dims)
    sig = {
        "moe_abi_version": (i32, []),
        "moe_status_string": (C.c_char_p, [i32]),
        "moe_check_dims": (i32, [pd]),
        "moe_workspace_bytes": (sz, [pd]),
        "moe_packed_gate_up_elems": (sz, [pd, i32]),
        "moe_pack_gate_up": (i32, [pd, vp, vp, vp, vp, vp, vp, vp]),
        "moe_router_split_elems": (sz, [pd]),
        "moe_prepare_router": (i32, [pd, vp, vp, vp]),
        "moe_route": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_route_prepared": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_dispatch": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_ffn": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_gate_up": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_gate_up_gather": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_down": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_combine": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_combine_inplace": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_down_combine": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_gate_up_rows": (i32, [pd, C.c_int64, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_down_rows": (i32, [pd, C.c_int64, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_aux_sums_count": (sz, [pd]),
        "moe_aux_sums": (i32, [pd, vp, vp, vp]),
        "moe_aux_sums_accumulate": (i32, [pd, vp, vp, vp]),
        "moe_aux_finalize": (i32, [pd, vp, vp, vp, vp, vp]),
        "moe_aux": (i32, [pd, vp, vp, vp, vp, vp]),
        "moe_forward": (i32, [pd, C.POINTER(Weights), vp, vp, C.POINTER(Outputs), vp, vp]),
        "moe_get_device_status": (i32, [vp, vp]),
        "moe_clear_device_status": (i32, [vp, vp]),
        "moe_selftest_bounded_wait": (i32, [vp, C.c_uint64, vp]),
        "moe_route_noalloc": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_route_noalloc_device_status": (i32, [vp]),
        "moe_route_noalloc_selftest_bounded_wait": (i32, [C.c_uint64, vp]),
        "moe_backward_workspace_bytes": (sz, [pd]),
        "moe_combine_backward": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_router_backward": (i32, [pd, vp, vp, vp, vp, vp, C.c_int64, C.c_float, C.c_float, vp, vp, vp, vp]),
        "moe_router_weight_grad": (i32, [pd, vp, vp, vp, vp, vp]),
        "moe_expert_ffn_backward": (i32, [pd, C.POINTER(Weights), C.POINTER(Saved), vp, vp, vp, vp,
                                          C.POINTER(Grads), vp, vp]),
        "moe_input_grad": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_swiglu_backward": (i32, [pd, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_swiglu_backward_saved": (i32, [pd, vp, vp, vp, vp, vp]),
        "moe_expert_dgrad_down": (i32, [pd, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_wgrad_down": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_dgrad_gate_up": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_expert_wgrad_gate_up": (i32, [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moe_sort_workspace_bytes": (sz, [i32, i32, i32]),
        "moe_sort_slots": (i32, [i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp]),
        "moe_permute": (i32, [i32, i32, i64, i32, i32, vp, i64, vp, vp, i64, vp, vp]),
        "moe_permute_backward": (i32, [i32, i32, i64, i32, i32, vp, i64, vp, vp, i64, vp, i64, vp, vp]),
        "moe_unpermute": (i32, [i32, i32, i64, i32, i32, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp]),
        "moe_unpermute_backward": (i32, [i32, i32, i64, i32, i32, vp, i64, vp, i64, vp, vp, vp, i64, vp, vp, vp]),
        "moe_unpermute_backward8": (i32, [i32, i32, i64, i32, i32, vp, i64, vp, vp, vp, vp, vp, i64, vp, vp, vp]),
        "moe_checkpoint8_scales": (sz, [i64]),
        "moe_checkpoint8": (i32, [i64, i64, i32, vp, i64, vp, vp, vp, vp, vp]),
        "moe_restore8": (i32, [i64, i64, i32, vp, vp, vp, vp, i64, vp, vp]),
        "moe_swiglu_backward8": (i32, [i64, i64, i32, i32, vp, vp, vp, i64, vp, vp, i64, vp, i64, vp, vp]),
        "moe_forward_checkpoint8": (i32, [pd, C.POINTER(Weights), vp, vp, C.POINTER(Outputs), C.POINTER(Codes8), vp,
                                          vp]),
        "moe_backward_checkpoint8_workspace_bytes": (sz, [pd]),
        "moe_backward_checkpoint8": (i32, [pd, C.POINTER(Weights), C.POINTER(Saved8), vp, C.c_float, C.c_float,
                                           C.POINTER(Grads), vp, vp]),
        "moe_backward": (i32, [pd, C.POINTER(Weights), C.POINTER(Saved), vp, C.c_float, C.c_float,
                               C.POINTER(Grads), vp, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    if lib.moe_abi_version() != 6:
        raise ImportError("libmoe_null ABI version mismatch")
    return lib


LIB = _load()


def status_string(code: int) -> str:
    return LIB.moe_status_string(int(code)).decode()


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _check(fn: str, code: int):
    if code != OK:
        raise MoEError(fn, code)


# moe_dims_t.flags: router product on the fp32 CUDA cores instead of the tensor cores;
# expert GEMMs on CTA pairs instead of single-CTA tiles; the backward's weight gradients on
# CTA pairs
FLAG_ROUTER_FP32_CORES = 1
FLAG_FFN_CTA_PAIR = 2
FLAG_WGRAD_CTA_PAIR = 4


def dims(T, d, N, M, K, F, F_shared, flags=0, C=0, V=0) -> Dims:
    return Dims(int(T), int(d), int(N), int(M), int(K), int(F), int(F_shared), int(flags), int(C), int(V))


def check_dims(dm: Dims) -> int:
    return LIB.moe_check_dims(C.byref(dm))


def workspace_bytes(dm: Dims) -> int:
    return int(LIB.moe_workspace_bytes(C.byref(dm)))


def aux_sums_count(dm: Dims) -> int:
    return int(LIB.moe_aux_sums_count(C.byref(dm)))


def packed_gate_up_elems(dm: Dims, shared: bool) -> int:
    return int(LIB.moe_packed_gate_up_elems(C.byref(dm), 1 if shared else 0))


def pack_gate_up(dm, w_gate, w_up, ws_gate, ws_up, gate_up, shared_gate_up, stream=None):
    _check("moe_pack_gate_up", LIB.moe_pack_gate_up(C.byref(dm), _p(w_gate), _p(w_up), _p(ws_gate),
                                                     _p(ws_up), _p(gate_up), _p(shared_gate_up),
                                                     _stream(stream)))


def router_split_elems(dm: Dims) -> int:
    return int(LIB.moe_router_split_elems(C.byref(dm)))


def prepare_router(dm, w_router, router_split, stream=None):
    _check("moe_prepare_router", LIB.moe_prepare_router(C.byref(dm), _p(w_router), _p(router_split),
                                                         _stream(stream)))


def route(dm, x, w_router, bias, tok_null_bias, logits, topk_idx, topk_gate, n_real, ws, stream=None):
    _check("moe_route", LIB.moe_route(C.byref(dm), _p(x), _p(w_router), _p(bias), _p(tok_null_bias),
                                      _p(logits), _p(topk_idx), _p(topk_gate), _p(n_real), _p(ws),
                                      _stream(stream)))


def route_prepared(dm, x, router_split, bias, tok_null_bias, logits, topk_idx, topk_gate, n_real, ws, stream=None):
    _check("moe_route_prepared",
           LIB.moe_route_prepared(C.byref(dm), _p(x), _p(router_split), _p(bias), _p(tok_null_bias), _p(logits),
                                  _p(topk_idx), _p(topk_gate), _p(n_real), _p(ws), _stream(stream)))


def dispatch(dm, x, topk_idx, ws, counts, offsets, perm_tok, slot_row, xs, stream=None):
    _check("moe_dispatch", LIB.moe_dispatch(C.byref(dm), _p(x), _p(topk_idx), _p(ws), _p(counts),
                                            _p(offsets), _p(perm_tok), _p(slot_row), _p(xs),
                                            _stream(stream)))


def expert_ffn(dm, xs, x, offsets, gate_up, w_down, shared_gate_up, shared_down, h, h_shared, ys,
               shared_out, ws, stream=None):
    _check("moe_expert_ffn", LIB.moe_expert_ffn(C.byref(dm), _p(xs), _p(x), _p(offsets), _p(gate_up),
                                                _p(w_down), _p(shared_gate_up), _p(shared_down), _p(h),
                                                _p(h_shared), _p(ys), _p(shared_out), _p(ws),
                                                _stream(stream)))


def expert_gate_up(dm, xs, x, offsets, gate_up, shared_gate_up, h, h_shared, ws, stream=None):
    _check("moe_expert_gate_up", LIB.moe_expert_gate_up(C.byref(dm), _p(xs), _p(x), _p(offsets), _p(gate_up),
                                                        _p(shared_gate_up), _p(h), _p(h_shared), _p(ws),
                                                        _stream(stream)))


def expert_gate_up_gather(dm, x, perm_tok, offsets, gate_up, shared_gate_up, h, h_shared, ws, stream=None):
    _check("moe_expert_gate_up_gather",
           LIB.moe_expert_gate_up_gather(C.byref(dm), _p(x), _p(perm_tok), _p(offsets), _p(gate_up),
                                         _p(shared_gate_up), _p(h), _p(h_shared), _p(ws), _stream(stream)))


def expert_down(dm, offsets, h, h_shared, w_down, shared_down, ys, shared_out, ws, stream=None):
    _check("moe_expert_down", LIB.moe_expert_down(C.byref(dm), _p(offsets), _p(h), _p(h_shared), _p(w_down),
                                                  _p(shared_down), _p(ys), _p(shared_out), _p(ws),
                                                  _stream(stream)))


def expert_gate_up_rows(dm, rows_cap, xs, x, offsets, gate_up, shared_gate_up, h, h_shared, ws, stream=None):
    """Gate/up grouped GEMM of an expert shard over rows_cap received rows (expert parallelism)."""
    _check("moe_expert_gate_up_rows",
           LIB.moe_expert_gate_up_rows(C.byref(dm), int(rows_cap), _p(xs), _p(x), _p(offsets), _p(gate_up),
                                       _p(shared_gate_up), _p(h), _p(h_shared), _p(ws), _stream(stream)))


def expert_down_rows(dm, rows_cap, offsets, h, h_shared, w_down, shared_down, ys, shared_out, ws, stream=None):
    """Down grouped GEMM of an expert shard over rows_cap received rows (expert parallelism)."""
    _check("moe_expert_down_rows",
           LIB.moe_expert_down_rows(C.byref(dm), int(rows_cap), _p(offsets), _p(h), _p(h_shared), _p(w_down),
                                    _p(shared_down), _p(ys), _p(shared_out), _p(ws), _stream(stream)))


def expert_down_combine(dm, offsets, h, h_shared, w_down, shared_down, ys, topk_gate, slot_row, y, ws,
                        stream=None, topk_idx=None, x=None, const_vectors=None):
    """Down GEMM with the combine in its shared-expert tiles (topk_idx, x and const_vectors
    are needed only with MoE++ copy/constant experts)."""
    _check("moe_expert_down_combine",
           LIB.moe_expert_down_combine(C.byref(dm), _p(offsets), _p(h), _p(h_shared), _p(w_down), _p(shared_down),
                                       _p(ys), _p(topk_gate), _p(slot_row), _p(topk_idx), _p(x),
                                       _p(const_vectors), _p(y), _p(ws), _stream(stream)))


def combine(dm, ys, shared_out, topk_gate, slot_row, y, stream=None, topk_idx=None, x=None,
            const_vectors=None):
    """topk_idx, x and const_vectors are needed only with MoE++ copy/constant experts."""
    _check("moe_combine", LIB.moe_combine(C.byref(dm), _p(ys), _p(shared_out), _p(topk_gate), _p(slot_row),
                                          _p(topk_idx), _p(x), _p(const_vectors), _p(y), _stream(stream)))


def combine_inplace(dm, ys, topk_gate, slot_row, y, ws, stream=None, topk_idx=None, x=None, const_vectors=None):
    """y holds the shared expert's output; adds the routed rows of the tokens the route listed in ws."""
    _check("moe_combine_inplace",
           LIB.moe_combine_inplace(C.byref(dm), _p(ys), _p(topk_gate), _p(slot_row), _p(topk_idx), _p(x),
                                   _p(const_vectors), _p(y), _p(ws), _stream(stream)))


def aux(dm, ws, counts_ext, P, losses, stream=None):
    _check("moe_aux", LIB.moe_aux(C.byref(dm), _p(ws), _p(counts_ext), _p(P), _p(losses), _stream(stream)))


def aux_sums(dm, ws, sums, stream=None):
    _check("moe_aux_sums", LIB.moe_aux_sums(C.byref(dm), _p(ws), _p(sums), _stream(stream)))


def aux_sums_accumulate(dm, ws, sums, stream=None):
    _check("moe_aux_sums_accumulate", LIB.moe_aux_sums_accumulate(C.byref(dm), _p(ws), _p(sums), _stream(stream)))


def aux_finalize(dm, sums, counts_ext, P, losses, stream=None):
    _check("moe_aux_finalize", LIB.moe_aux_finalize(C.byref(dm), _p(sums), _p(counts_ext), _p(P),
                                                    _p(losses), _stream(stream)))


def forward(dm, weights: Weights, x, tok_null_bias, outputs: Outputs, ws, stream=None):
    _check("moe_forward", LIB.moe_forward(C.byref(dm), C.byref(weights), _p(x), _p(tok_null_bias),
                                          C.byref(outputs), _p(ws), _stream(stream)))


def get_device_status(ws, stream=None) -> int:
    return LIB.moe_get_device_status(_p(ws), _stream(stream))


def clear_device_status(ws, stream=None):
    _check("moe_clear_device_status", LIB.moe_clear_device_status(_p(ws), _stream(stream)))


def selftest_bounded_wait(ws, limit_ns: int, stream=None):
    _check("moe_selftest_bounded_wait", LIB.moe_selftest_bounded_wait(_p(ws), int(limit_ns), _stream(stream)))


# ------------------------------------------------------------------------------ backward


def backward_workspace_bytes(dm: Dims) -> int:
    return int(LIB.moe_backward_workspace_bytes(C.byref(dm)))


def combine_backward(dm, dy, ys, topk_gate, slot_row, dys, dg, bws, stream=None, topk_idx=None, x=None,
                     const_vectors=None):
    _check("moe_combine_backward",
           LIB.moe_combine_backward(C.byref(dm), _p(dy), _p(ys), _p(topk_gate), _p(slot_row), _p(topk_idx), _p(x),
                                    _p(const_vectors), _p(dys), _p(dg), _p(bws), _stream(stream)))


def router_backward(dm, logits, topk_idx, topk_gate, dg, counts_ext, t_total, alpha, beta, ds, bws,
                    dtok_null_bias=None, stream=None):
    _check("moe_router_backward",
           LIB.moe_router_backward(C.byref(dm), _p(logits), _p(topk_idx), _p(topk_gate), _p(dg), _p(counts_ext),
                                   int(t_total), float(alpha), float(beta), _p(ds), _p(dtok_null_bias), _p(bws),
                                   _stream(stream)))


def router_weight_grad(dm, x, dw_router, dbias, bws, stream=None):
    _check("moe_router_weight_grad",
           LIB.moe_router_weight_grad(C.byref(dm), _p(x), _p(dw_router), _p(dbias), _p(bws), _stream(stream)))


def expert_ffn_backward(dm, weights: Weights, saved: Saved, dys, dy, dxs, dx_shared, grads: Grads, bws,
                        stream=None):
    _check("moe_expert_ffn_backward",
           LIB.moe_expert_ffn_backward(C.byref(dm), C.byref(weights), C.byref(saved), _p(dys), _p(dy), _p(dxs),
                                       _p(dx_shared), C.byref(grads), _p(bws), _stream(stream)))


def input_grad(dm, dx_shared, dxs, slot_row, topk_idx, topk_gate, dy, dx, bws, stream=None):
    _check("moe_input_grad",
           LIB.moe_input_grad(C.byref(dm), _p(dx_shared), _p(dxs), _p(slot_row), _p(topk_idx), _p(topk_gate),
                              _p(dy), _p(dx), _p(bws), _stream(stream)))


def backward(dm, weights: Weights, saved: Saved, dy, alpha, beta, grads: Grads, bws, stream=None):
    _check("moe_backward", LIB.moe_backward(C.byref(dm), C.byref(weights), C.byref(saved), _p(dy), float(alpha),
                                            float(beta), C.byref(grads), _p(bws), _stream(stream)))


def expert_swiglu_backward(dm, xs, x, offsets, gate_up, shared_gate_up, bws, stream=None):
    _check("moe_expert_swiglu_backward",
           LIB.moe_expert_swiglu_backward(C.byref(dm), _p(xs), _p(x), _p(offsets), _p(gate_up), _p(shared_gate_up),
                                          _p(bws), _stream(stream)))


def expert_dgrad_down(dm, offsets, dys, dy, w_down, shared_down, bws, stream=None):
    _check("moe_expert_dgrad_down", LIB.moe_expert_dgrad_down(C.byref(dm), _p(offsets), _p(dys), _p(dy),
                                                              _p(w_down), _p(shared_down), _p(bws),
                                                              _stream(stream)))


def expert_wgrad_down(dm, offsets, dys, dy, h, h_shared, dw_down, dws_down, bws, stream=None):
    _check("moe_expert_wgrad_down", LIB.moe_expert_wgrad_down(C.byref(dm), _p(offsets), _p(dys), _p(dy), _p(h),
                                                              _p(h_shared), _p(dw_down), _p(dws_down), _p(bws),
                                                              _stream(stream)))


def expert_dgrad_gate_up(dm, offsets, gate_up, shared_gate_up, w_router, dxs, dx_shared, bws, stream=None):
    """w_router (or None): add the router's input gradient ds W_r to dx_shared."""
    _check("moe_expert_dgrad_gate_up",
           LIB.moe_expert_dgrad_gate_up(C.byref(dm), _p(offsets), _p(gate_up), _p(shared_gate_up), _p(w_router),
                                        _p(dxs), _p(dx_shared), _p(bws), _stream(stream)))


def expert_wgrad_gate_up(dm, offsets, xs, x, dw_gate, dw_up, dws_gate, dws_up, bws, stream=None):
    _check("moe_expert_wgrad_gate_up",
           LIB.moe_expert_wgrad_gate_up(C.byref(dm), _p(offsets), _p(xs), _p(x), _p(dw_gate), _p(dw_up),
                                        _p(dws_gate), _p(dws_up), _p(bws), _stream(stream)))


def expert_swiglu_backward_saved(dm, offsets, z, z_shared, bws, stream=None):
    _check("moe_expert_swiglu_backward_saved",
           LIB.moe_expert_swiglu_backward_saved(C.byref(dm), _p(offsets), _p(z), _p(z_shared), _p(bws),
                                                _stream(stream)))


def forward_checkpoint8(dm, weights: Weights, x, tok_null_bias, outputs: Outputs, codes: Codes8, ws, stream=None):
    """moe_forward that keeps an 8-bit checkpoint for ``backward_checkpoint8``."""
    _check("moe_forward_checkpoint8",
           LIB.moe_forward_checkpoint8(C.byref(dm), C.byref(weights), _p(x), _p(tok_null_bias), C.byref(outputs),
                                       C.byref(codes), _p(ws), _stream(stream)))


def backward_checkpoint8_workspace_bytes(dm: Dims) -> int:
    return int(LIB.moe_backward_checkpoint8_workspace_bytes(C.byref(dm)))


def backward_checkpoint8(dm, weights: Weights, saved: Saved8, dy, alpha, beta, grads: Grads, ws, stream=None):
    """moe_backward from the 8-bit checkpoint in ``saved``."""
    _check("moe_backward_checkpoint8",
           LIB.moe_backward_checkpoint8(C.byref(dm), C.byref(weights), C.byref(saved), _p(dy), float(alpha),
                                        float(beta), C.byref(grads), _p(ws), _stream(stream)))


# ------------------------------------------------------ slots from any routing, 8-bit checkpoints
#
# These calls take tensors of several types and row strides, so unlike the calls above they
# check types and shapes here (ValueError) before the library checks sizes (MoEError). Row
# tensors are two-dimensional with adjacent elements in a row; any row stride of at least the
# width will do. Everything else is contiguous.

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _dtype(t: torch.Tensor, name: str) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, not {t.dtype}")
    return code


def _rows(t: torch.Tensor, name: str, rows: Optional[int], cols: Optional[int], dtype: Optional[torch.dtype],
          dev: int):
    """(rows, columns, data pointer, row stride) of a row tensor; None in rows, cols or dtype: any."""
    shape = t.shape
    if (len(shape) == 2 and (rows is None or shape[0] == rows) and (cols is None or shape[1] == cols) and
            (dtype is None or t.dtype is dtype) and t.get_device() == dev):
        ld, inner = t.stride()
        if inner == 1 and ld >= shape[1]:
            return shape[0], shape[1], t.data_ptr(), ld
    _two_d(t, name)
    want = (shape[0] if rows is None else rows, shape[1] if cols is None else cols)
    _placed(t, name, want, t.dtype if dtype is None else dtype, dev)
    if inner != 1 and shape[1] > 1:
        raise ValueError(f"the elements of a row of {name} must be adjacent")
    if ld < shape[1] and shape[0] > 1:
        raise ValueError(f"rows of {name} must not overlap")
    return shape[0], shape[1], t.data_ptr(), max(ld, shape[1])


def _slots(t: torch.Tensor, T: int, dev: int):
    """(K, data pointer) of slot_row [T, K]."""
    shape = t.shape
    if len(shape) == 2 and shape[0] == T and t.dtype is torch.int32 and t.get_device() == dev and t.is_contiguous():
        return shape[1], t.data_ptr()
    _two_d(t, "slot_row")
    return shape[1], _dense(t, "slot_row", (T, shape[1]), torch.int32, dev)


def _dense(t: torch.Tensor, name: str, shape, dtype: torch.dtype, dev: int) -> int:
    """Data pointer of a contiguous tensor."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _placed(t, name, shape, dtype, dev)
    raise ValueError(f"expected a contiguous {name}")


def _placed(t: torch.Tensor, name: str, shape, dtype: torch.dtype, dev: int):
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current device")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")


def _device() -> int:
    return torch.cuda.current_device()


def _raw_stream(stream, dev: int) -> int:
    """The stream's handle, without building a stream object for the current one (3 us a call,
    a third of a decode-sized call's host time)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _status(ws: Optional[torch.Tensor], dev: int):
    """Pointer of the workspace whose status word records device-side errors, or None."""
    if ws is None:
        return None
    if ws.get_device() != dev:
        raise ValueError("ws must be a CUDA tensor on the current device")
    if not ws.is_contiguous() or ws.numel() * ws.element_size() < 4 or ws.data_ptr() % 4:
        raise ValueError("ws must be a workspace: contiguous, at least a status word, 4-byte aligned")
    return ws.data_ptr()


def _two_d(t: torch.Tensor, name: str):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have two dimensions, not {len(shape)}")
    return shape


def sort_workspace_bytes(T: int, K: int, N: int) -> int:
    return int(LIB.moe_sort_workspace_bytes(int(T), int(K), int(N)))


def sort_slots(ids, N, counts, offsets, perm_tok, slot_row, ws, stream=None):
    """Slots sorted by expert: ids [T, K] int32 or int64 (outside [0, N): no expert) ->
    counts [N], offsets [N+1], perm_tok [T*K], slot_row [T, K], all int32. ws: at least
    ``sort_workspace_bytes(T, K, N)`` bytes."""
    T, K = _two_d(ids, "ids")
    dev = _device()
    i32 = torch.int32
    if ids.dtype != i32 and ids.dtype != torch.int64:
        raise ValueError(f"ids must be int32 or int64, not {ids.dtype}")
    need = LIB.moe_sort_workspace_bytes(T, K, N)
    if need and (ws is None or ws.numel() * ws.element_size() < need):
        raise ValueError(f"ws must hold sort_workspace_bytes = {need} bytes")
    _check("moe_sort_slots",
           LIB.moe_sort_slots(T, K, N, _dense(ids, "ids", (T, K), ids.dtype, dev), ids.element_size(),
                              _dense(counts, "counts", (N,), i32, dev), _dense(offsets, "offsets", (N + 1,), i32, dev),
                              _dense(perm_tok, "perm_tok", (T * K,), i32, dev),
                              _dense(slot_row, "slot_row", (T, K), i32, dev), _status(ws, dev),
                              _raw_stream(stream, dev)))


def permute(x, slot_row, xs, ws=None, stream=None):
    """xs[slot_row[t, k]] = x[t] for every slot with a row; the other rows of xs stay as they are."""
    dev, dt = _device(), _dtype(x, "x")
    T, d, px, ldx = _rows(x, "x", None, None, None, dev)
    K, ps = _slots(slot_row, T, dev)
    rows, _, po, ldo = _rows(xs, "xs", None, d, x.dtype, dev)
    _check("moe_permute", LIB.moe_permute(T, K, rows, d, dt, px, ldx, ps, po, ldo, _status(ws, dev),
                                          _raw_stream(stream, dev)))


def permute_backward(dxs, slot_row, dx, base=None, ws=None, stream=None):
    """dx[t] = base[t] + sum_k dxs[slot_row[t, k]]; base None is zero, base may be dx itself."""
    dev, dt = _device(), _dtype(dx, "dx")
    T, d, po, ldo = _rows(dx, "dx", None, None, None, dev)
    K, ps = _slots(slot_row, T, dev)
    rows, _, pi, ldi = _rows(dxs, "dxs", None, d, dx.dtype, dev)
    pb, ldb = (None, 0) if base is None else _rows(base, "base", T, d, dx.dtype, dev)[2:]
    _check("moe_permute_backward",
           LIB.moe_permute_backward(T, K, rows, d, dt, pi, ldi, ps, pb, ldb, po, ldo, _status(ws, dev),
                                    _raw_stream(stream, dev)))


def unpermute(ys, weights, slot_row, y, base=None, ws=None, stream=None):
    """y[t] = base[t] + sum_k weights[t, k] ys[slot_row[t, k]]; base None is zero, base may be y
    itself."""
    dev, dt = _device(), _dtype(y, "y")
    T, d, po, ldo = _rows(y, "y", None, None, None, dev)
    K, ps = _slots(slot_row, T, dev)
    rows, _, pi, ldi = _rows(ys, "ys", None, d, y.dtype, dev)
    pb, ldb = (None, 0) if base is None else _rows(base, "base", T, d, y.dtype, dev)[2:]
    _check("moe_unpermute",
           LIB.moe_unpermute(T, K, rows, d, dt, pi, ldi, _dense(weights, "weights", (T, K), torch.float32, dev), ps,
                             pb, ldb, po, ldo, _status(ws, dev), _raw_stream(stream, dev)))


def unpermute_backward(dy, ys, weights, slot_row, dys, dweights, ws=None, stream=None):
    """dys[slot_row[t, k]] = weights[t, k] dy[t] and dweights[t, k] = <dy[t], ys[slot_row[t, k]]>
    (fp32 [T, K]). dys may be None, or ys and dweights both."""
    if dys is None and ys is None:
        raise ValueError("dys and ys cannot both be None")
    if (ys is None) != (dweights is None):
        raise ValueError("ys and dweights go together")
    dev, dt = _device(), _dtype(dy, "dy")
    f32 = torch.float32
    T, d, pt, ldt = _rows(dy, "dy", None, None, None, dev)
    K, ps = _slots(slot_row, T, dev)
    rows, pi, ldi, po, ldo, pw = None, None, 0, None, 0, None
    if ys is not None:
        rows, _, pi, ldi = _rows(ys, "ys", None, d, dy.dtype, dev)
        pw = _dense(dweights, "dweights", (T, K), f32, dev)
    if dys is not None:
        rows, _, po, ldo = _rows(dys, "dys", rows, d, dy.dtype, dev)
    _check("moe_unpermute_backward",
           LIB.moe_unpermute_backward(T, K, rows, d, dt, pt, ldt, pi, ldi, _dense(weights, "weights", (T, K), f32, dev),
                                      ps, po, ldo, pw, _status(ws, dev), _raw_stream(stream, dev)))


def unpermute_backward8(dy, codes, scales, weights, slot_row, dys, dweights, ws=None, stream=None):
    """``unpermute_backward`` with ys as ``checkpoint8`` stored it. dys may be None."""
    dev, dt = _device(), _dtype(dy, "dy")
    f32 = torch.float32
    T, d, pt, ldt = _rows(dy, "dy", None, None, None, dev)
    K, ps = _slots(slot_row, T, dev)
    rows = _two_d(codes, "codes")[0]
    po, ldo = (None, 0) if dys is None else _rows(dys, "dys", rows, d, dy.dtype, dev)[2:]
    _check("moe_unpermute_backward8",
           LIB.moe_unpermute_backward8(T, K, rows, d, dt, pt, ldt, _dense(codes, "codes", (rows, d), torch.int8, dev),
                                       _dense(scales, "scales", (rows, (d + 31) // 32), torch.uint8, dev),
                                       _dense(weights, "weights", (T, K), f32, dev), ps, po, ldo,
                                       _dense(dweights, "dweights", (T, K), f32, dev), _status(ws, dev),
                                       _raw_stream(stream, dev)))


def checkpoint8_scales(cols: int) -> int:
    return int(LIB.moe_checkpoint8_scales(int(cols)))


def _used(rows_used, dev: int):
    if rows_used is None:
        return None
    if rows_used.numel() != 1:
        raise ValueError("rows_used must be one int32")
    return _dense(rows_used, "rows_used", rows_used.shape, torch.int32, dev)


def checkpoint8(x, codes, scales, rows_used=None, ws=None, stream=None):
    """x [rows, cols] stored in 8 bits: codes [rows, cols] int8, scales [rows, ceil(cols / 32)]
    uint8. rows_used (one int32 on the device, e.g. ``offsets[N:]``): the rows in use."""
    dev, dt = _device(), _dtype(x, "x")
    rows, cols, px, ldx = _rows(x, "x", None, None, None, dev)
    _check("moe_checkpoint8",
           LIB.moe_checkpoint8(rows, cols, dt, px, ldx, _used(rows_used, dev),
                               _dense(codes, "codes", (rows, cols), torch.int8, dev),
                               _dense(scales, "scales", (rows, (cols + 31) // 32), torch.uint8, dev),
                               _status(ws, dev), _raw_stream(stream, dev)))


def restore8(codes, scales, x, rows_used=None, ws=None, stream=None):
    """The activation that ``checkpoint8`` stored, into x [rows, cols]."""
    dev, dt = _device(), _dtype(x, "x")
    rows, cols, px, ldx = _rows(x, "x", None, None, None, dev)
    _check("moe_restore8",
           LIB.moe_restore8(rows, cols, dt, _dense(codes, "codes", (rows, cols), torch.int8, dev),
                            _dense(scales, "scales", (rows, (cols + 31) // 32), torch.uint8, dev),
                            _used(rows_used, dev), px, ldx, _status(ws, dev), _raw_stream(stream, dev)))


def swiglu_backward8(codes, scales, dh, dz, h, packed=True, rows_used=None, ws=None, stream=None):
    """SwiGLU's backward from pre-activations stored by ``checkpoint8`` (codes [rows, 2F]): dz
    [rows, 2F] from dh [rows, F], and the activation h [rows, F] recomputed (None: not written).
    packed: columns in the layer's order (64-column panels of gate, then up), else F gate
    columns, then F up columns."""
    dev, dt = _device(), _dtype(dh, "dh")
    rows, F, pg, ldg = _rows(dh, "dh", None, None, None, dev)
    _, _, pz, ldz = _rows(dz, "dz", rows, 2 * F, dh.dtype, dev)
    ph, ldh = (None, 0) if h is None else _rows(h, "h", rows, F, dh.dtype, dev)[2:]
    _check("moe_swiglu_backward8",
           LIB.moe_swiglu_backward8(rows, F, 1 if packed else 0, dt,
                                    _dense(codes, "codes", (rows, 2 * F), torch.int8, dev),
                                    _dense(scales, "scales", (rows, (2 * F + 31) // 32), torch.uint8, dev),
                                    pg, ldg, _used(rows_used, dev), pz, ldz, ph, ldh, _status(ws, dev),
                                    _raw_stream(stream, dev)))

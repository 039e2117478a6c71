"""ctypes binding of libdsmoe.so with the C ABI's names.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. Torch tensors are passed by data pointer (device tensors for
dsmoe_forward, host tensors for dsmoe_forward_host); streams are torch CUDA
streams or raw cudaStream_t integers. Importing this module raises if the
library has not been built; there is no other code path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
# DSMOE_LIBRARY selects another build of the library, e.g. the profiling build with the
# grouped GEMM's role cycle counters (build.py --role-cycles)
LIB_PATH = os.environ.get("DSMOE_LIBRARY") or os.path.join(_HERE, "libdsmoe.so")

DSMOE_OK, DSMOE_ERR_INVALID_ARG, DSMOE_ERR_UNSUPPORTED, DSMOE_ERR_WORKSPACE, DSMOE_ERR_CUDA, \
    DSMOE_ERR_DEVICE_TIMEOUT = range(6)
DSMOE_SCORE_SOFTMAX, DSMOE_SCORE_SIGMOID, DSMOE_SCORE_SQRT_SOFTPLUS, DSMOE_ROUTE_HASH = range(4)
DSMOE_BIAS_NONE, DSMOE_BIAS_SELECT_ONLY, DSMOE_BIAS_IN_LOGITS = range(3)
DSMOE_GEMM_PAIR, DSMOE_GEMM_SINGLE = range(2)
DSMOE_RANGE_PARTIAL, DSMOE_RANGE_ADD_SHARED = 1, 2

ABI_FUNCTIONS = (
    "dsmoe_abi_version", "dsmoe_status_string", "dsmoe_last_error", "dsmoe_check_config",
    "dsmoe_workspace_bytes", "dsmoe_create", "dsmoe_destroy", "dsmoe_forward", "dsmoe_forward_host",
    "dsmoe_balance_stats", "dsmoe_get_status", "dsmoe_set_wait_limit", "dsmoe_set_timing",
    "dsmoe_stage_times", "dsmoe_stage_name", "dsmoe_launch_count", "dsmoe_workspace_tensor",
    "dsmoe_balance_losses", "dsmoe_sequence_balance", "dsmoe_bias_update",
    "dsmoe_route_noalloc", "dsmoe_set_gemm_kernel", "dsmoe_get_gemm_kernel",
    "dsmoe_set_selection", "dsmoe_get_selection", "dsmoe_set_expert_range", "dsmoe_get_expert_range",
    "dsmoe_round_bf16", "dsmoe_backward_gates", "dsmoe_backward_router", "dsmoe_ep_route", "dsmoe_ep_experts",
    "dsmoe_ep_combine", "dsmoe_forward_host_async", "dsmoe_host_join", "dsmoe_host_sync", "dsmoe_set_training",
    "dsmoe_backward_experts", "dsmoe_backward_weights", "dsmoe_gemm_role_cycles",
    "dsmoe_q8_scale_cols", "dsmoe_q8_quantize", "dsmoe_q8_quantize_weights", "dsmoe_norm_q8", "dsmoe_norm_backward",
    "dsmoe_q8_matmul", "dsmoe_q8_gated_matmul", "dsmoe_q8_tiling", "dsmoe_forward_q8",
)
ROLE_CTAS, ROLE_SLOTS = 160, 9
ROLE_KINDS = ("gemm_down", "gemm_gate_up", "shared_down", "shared_gate_up", "weight_grad")
ROLE_SLOT_NAMES = ("cycles", "nanoseconds", "producer_wait_stage", "mma_wait_stage", "mma_wait_acc", "mma_loop",
                   "epi_wait_acc", "epi_loop", "tiles")


class DsmoeCfg(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("n_routed", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("d_ff", ctypes.c_int32), ("n_shared", ctypes.c_int32), ("d_ff_shared", ctypes.c_int32),
                ("score", ctypes.c_int32), ("bias_mode", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("hash_mult", ctypes.c_uint32), ("hash_mod", ctypes.c_uint32)]


DSMOE_Q8_BF16, DSMOE_Q8_GATED, DSMOE_Q8_FP32 = range(3)
Q8_WEIGHTS = ("W_gate", "W_up", "W_down", "Ws_gate", "Ws_up", "Ws_down")


class DsmoeQ8Weights(ctypes.Structure):
    _fields_ = [(n + s, ctypes.c_void_p) for n in Q8_WEIGHTS for s in ("", "_scales")]


class DsmoeQ8Tiles(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tokens", "splits", "chains", "grid")]


class DsmoeError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: {status_string(status)} ({status}): {message}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python mixture_experts_layer_score_b200/build.py` (there is no fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u64, f32p, i32p = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64,
                                     ctypes.c_void_p, ctypes.c_void_p)
    cfgp = ctypes.POINTER(DsmoeCfg)
    sig = {
        "dsmoe_abi_version": (i32, []),
        "dsmoe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "dsmoe_last_error": (ctypes.c_char_p, []),
        "dsmoe_check_config": (ctypes.c_int, [cfgp]),
        "dsmoe_workspace_bytes": (ctypes.c_int, [cfgp, ctypes.POINTER(ctypes.c_size_t)]),
        "dsmoe_create": (ctypes.c_int, [cfgp, i32, ctypes.POINTER(vp)]),
        "dsmoe_destroy": (None, [vp]),
        "dsmoe_forward": (ctypes.c_int, [vp, i32] + [vp] * 18 + [vp]),
        "dsmoe_forward_host": (ctypes.c_int, [vp, i32] + [vp] * 16 + [vp]),
        "dsmoe_forward_host_async": (ctypes.c_int, [vp, i32] + [vp] * 16 + [vp]),
        "dsmoe_host_join": (ctypes.c_int, [vp, vp]),
        "dsmoe_host_sync": (ctypes.c_int, [vp]),
        "dsmoe_set_training": (ctypes.c_int, [vp, i32]),
        "dsmoe_backward_experts": (ctypes.c_int, [vp, i32] + [vp] * 10 + [vp]),
        "dsmoe_backward_weights": (ctypes.c_int, [vp, i32] + [vp] * 9 + [vp]),
        "dsmoe_balance_stats": (ctypes.c_int, [vp, i64, vp, vp, vp, vp, vp]),
        "dsmoe_get_status": (ctypes.c_int, [vp]),
        "dsmoe_set_wait_limit": (ctypes.c_int, [vp, u64]),
        "dsmoe_set_timing": (ctypes.c_int, [vp, i32]),
        "dsmoe_set_gemm_kernel": (ctypes.c_int, [vp, i32]),
        "dsmoe_get_gemm_kernel": (i32, [vp]),
        "dsmoe_set_selection": (ctypes.c_int, [vp, i32, i32]),
        "dsmoe_get_selection": (ctypes.c_int, [vp, ctypes.POINTER(i32), ctypes.POINTER(i32)]),
        "dsmoe_stage_times": (ctypes.c_int, [vp, ctypes.POINTER(ctypes.c_float), i32, ctypes.POINTER(i32)]),
        "dsmoe_stage_name": (ctypes.c_char_p, [i32]),
        "dsmoe_launch_count": (ctypes.c_int, [vp, ctypes.POINTER(i64)]),
        "dsmoe_gemm_role_cycles": (ctypes.c_int, [vp, i32]),
        "dsmoe_balance_losses": (ctypes.c_int, [vp, vp, vp, i32, vp, ctypes.c_float, ctypes.c_float, vp, vp, vp,
                                                vp]),
        "dsmoe_sequence_balance": (ctypes.c_int, [vp, i32, i32, vp, vp, ctypes.c_float, vp, vp, vp, vp]),
        "dsmoe_bias_update": (ctypes.c_int, [vp, i64, vp, ctypes.c_float, vp, vp]),
        "dsmoe_workspace_tensor": (ctypes.c_int, [vp, ctypes.c_char_p, ctypes.POINTER(vp),
                                                  ctypes.POINTER(i64), ctypes.POINTER(i64)]),
        "dsmoe_route_noalloc": (ctypes.c_int, [cfgp, i32] + [vp] * 8 + [vp]),
        "dsmoe_set_expert_range": (ctypes.c_int, [vp, i32, i32, i32]),
        "dsmoe_get_expert_range": (ctypes.c_int, [vp, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                                  ctypes.POINTER(i32)]),
        "dsmoe_round_bf16": (ctypes.c_int, [vp, i64, vp, vp, vp]),
        "dsmoe_backward_gates": (ctypes.c_int, [vp, i32, vp, vp, vp, vp, vp]),
        "dsmoe_ep_route": (ctypes.c_int, [vp, i32] + [vp] * 11 + [i32, vp, vp]),
        "dsmoe_ep_experts": (ctypes.c_int, [vp, i32, i32, i32, vp, i64, vp, vp, vp, vp, vp, vp]),
        "dsmoe_ep_combine": (ctypes.c_int, [vp, i32] + [vp] * 7 + [vp]),
        "dsmoe_backward_router": (ctypes.c_int, [vp, i32, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp,
                                                 vp]),
        "dsmoe_q8_scale_cols": (i32, [i32]),
        "dsmoe_forward_q8": (ctypes.c_int, [vp, i32] + [vp] * 7 + [ctypes.POINTER(DsmoeQ8Weights)] + [vp] * 8 + [vp]),
        "dsmoe_q8_quantize": (ctypes.c_int, [vp, i64, i32] + [vp] * 3 + [vp]),
        "dsmoe_q8_quantize_weights": (ctypes.c_int, [vp, i32, i32, i32] + [vp] * 3 + [vp]),
        "dsmoe_norm_q8": (ctypes.c_int, [vp, i32, vp, vp, vp, ctypes.c_float] + [vp] * 4 + [vp]),
        "dsmoe_norm_backward": (ctypes.c_int, [vp, i32, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp]),
        "dsmoe_q8_tiling": (ctypes.c_int, [i32, i32, i64, i32, i32, i32, i32, ctypes.POINTER(DsmoeQ8Tiles)]),
        "dsmoe_q8_matmul": (ctypes.c_int, [vp, i32, i64, i32, i32] + [vp] * 6 + [vp]),
        "dsmoe_q8_gated_matmul": (ctypes.c_int, [vp, i32, i64, i32, i32] + [vp] * 9 + [vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def status_string(status: int) -> str:
    return _lib.dsmoe_status_string(int(status)).decode()


def dsmoe_status_string(status: int) -> str:
    return status_string(status)


def dsmoe_last_error() -> str:
    return _lib.dsmoe_last_error().decode()


def _check(status: int, where: str):
    if status != DSMOE_OK:
        raise DsmoeError(status, where, dsmoe_last_error())


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_cfg(d_model: int, n_routed: int, top_k: int, d_ff: int, n_shared: int = 0, d_ff_shared: int = 0,
             score: int = DSMOE_SCORE_SOFTMAX, bias_mode: int = DSMOE_BIAS_NONE, renormalize: bool = False,
             max_tokens: int = 1, hash_mult: int = 2654435761, hash_mod: int = 0) -> DsmoeCfg:
    return DsmoeCfg(d_model, n_routed, top_k, d_ff, n_shared, d_ff_shared, score, bias_mode, int(renormalize),
                    max_tokens, hash_mult, hash_mod)


def cfg_from(obj, max_tokens: int) -> DsmoeCfg:
    """dsmoe_cfg from any object with the layer's field names (d_model, n_routed, top_k, ...)."""
    return make_cfg(obj.d_model, obj.n_routed, obj.top_k, obj.d_ff, obj.n_shared, obj.d_ff_shared, obj.score,
                    obj.bias_mode, obj.renormalize, max_tokens, getattr(obj, "hash_mult", 2654435761), 0)


def dsmoe_abi_version() -> int:
    return _lib.dsmoe_abi_version()


def dsmoe_check_config(cfg: DsmoeCfg) -> int:
    return _lib.dsmoe_check_config(ctypes.byref(cfg))


def dsmoe_workspace_bytes(cfg: DsmoeCfg) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.dsmoe_workspace_bytes(ctypes.byref(cfg), ctypes.byref(n)), "dsmoe_workspace_bytes")
    return n.value


class _Live:
    """What a handle was made and set up with: the checks of tensors against it need no call."""
    __slots__ = ("device", "cfg", "experts", "k", "flags")

    def __init__(self, device: int, cfg: DsmoeCfg):
        self.device, self.cfg = device, DsmoeCfg.from_buffer_copy(cfg)
        self.experts, self.k, self.flags = cfg.n_routed, cfg.top_k, DSMOE_RANGE_ADD_SHARED


_handles: Dict[int, _Live] = {}


def dsmoe_create(cfg: DsmoeCfg, device: int = 0) -> int:
    h = ctypes.c_void_p()
    _check(_lib.dsmoe_create(ctypes.byref(cfg), int(device), ctypes.byref(h)), "dsmoe_create")
    _handles[h.value] = _Live(int(device), cfg)
    return h.value


def dsmoe_destroy(handle: int) -> None:
    _handles.pop(handle, None)
    _lib.dsmoe_destroy(handle)


def dsmoe_forward(handle, T, x, token_ids, W_router, b, W_gate, W_up, W_down, Ws_gate, Ws_up, Ws_down,
                  h, topk_idx, gates, counts, f, P, P_sum=None, scores_dbg=None, stream=None) -> None:
    st = _lib.dsmoe_forward(handle, int(T), *[_ptr(t) for t in (
        x, token_ids, W_router, b, W_gate, W_up, W_down, Ws_gate, Ws_up, Ws_down, h, topk_idx, gates, counts, f,
        P, P_sum, scores_dbg)], _stream(stream))
    _check(st, "dsmoe_forward")


def dsmoe_forward_host(handle, T, x_host, token_ids_host, W_router, b, W_gate, W_up, W_down, Ws_gate, Ws_up,
                       Ws_down, h_host, topk_idx_host, gates_host, counts_host, f_host, P_host,
                       stream=None) -> None:
    st = _lib.dsmoe_forward_host(handle, int(T), *[_ptr(t) for t in (
        x_host, token_ids_host, W_router, b, W_gate, W_up, W_down, Ws_gate, Ws_up, Ws_down, h_host,
        topk_idx_host, gates_host, counts_host, f_host, P_host)], _stream(stream))
    _check(st, "dsmoe_forward_host")


def dsmoe_forward_host_async(handle, T, x_host, token_ids_host, W_router, b, W_gate, W_up, W_down, Ws_gate, Ws_up,
                             Ws_down, h_host, topk_idx_host, gates_host, counts_host, f_host, P_host,
                             stream=None) -> None:
    st = _lib.dsmoe_forward_host_async(handle, int(T), *[_ptr(t) for t in (
        x_host, token_ids_host, W_router, b, W_gate, W_up, W_down, Ws_gate, Ws_up, Ws_down, h_host,
        topk_idx_host, gates_host, counts_host, f_host, P_host)], _stream(stream))
    _check(st, "dsmoe_forward_host_async")


def dsmoe_host_join(handle, stream=None) -> None:
    _check(_lib.dsmoe_host_join(handle, _stream(stream)), "dsmoe_host_join")


def dsmoe_host_sync(handle) -> None:
    _check(_lib.dsmoe_host_sync(handle), "dsmoe_host_sync")


def dsmoe_balance_stats(handle, T_total, counts, P_sum, f, P, stream=None) -> None:
    _check(_lib.dsmoe_balance_stats(handle, int(T_total), _ptr(counts), _ptr(P_sum), _ptr(f), _ptr(P),
                                    _stream(stream)), "dsmoe_balance_stats")


def dsmoe_get_status(handle) -> int:
    return _lib.dsmoe_get_status(handle)


def dsmoe_set_wait_limit(handle, ns: int) -> None:
    _check(_lib.dsmoe_set_wait_limit(handle, int(ns)), "dsmoe_set_wait_limit")


def dsmoe_set_gemm_kernel(handle, kind: int) -> None:
    _check(_lib.dsmoe_set_gemm_kernel(handle, int(kind)), "dsmoe_set_gemm_kernel")


def dsmoe_get_gemm_kernel(handle) -> int:
    return int(_lib.dsmoe_get_gemm_kernel(handle))


def dsmoe_set_selection(handle, mask_top: int, k_active: int) -> None:
    _check(_lib.dsmoe_set_selection(handle, int(mask_top), int(k_active)), "dsmoe_set_selection")
    if handle in _handles:
        _handles[handle].k = int(k_active)


def dsmoe_get_selection(handle):
    m, k = ctypes.c_int32(), ctypes.c_int32()
    _check(_lib.dsmoe_get_selection(handle, ctypes.byref(m), ctypes.byref(k)), "dsmoe_get_selection")
    return m.value, k.value


def dsmoe_set_expert_range(handle, e_begin: int, e_end: int, flags: int) -> None:
    _check(_lib.dsmoe_set_expert_range(handle, int(e_begin), int(e_end), int(flags)), "dsmoe_set_expert_range")
    if handle in _handles:
        _handles[handle].experts, _handles[handle].flags = int(e_end) - int(e_begin), int(flags)


def dsmoe_get_expert_range(handle):
    b, e, f = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(_lib.dsmoe_get_expert_range(handle, ctypes.byref(b), ctypes.byref(e), ctypes.byref(f)),
           "dsmoe_get_expert_range")
    return b.value, e.value, f.value


def dsmoe_round_bf16(handle, n: int, src, dst, stream=None) -> None:
    _check(_lib.dsmoe_round_bf16(handle, int(n), _ptr(src), _ptr(dst), _stream(stream)), "dsmoe_round_bf16")


def dsmoe_ep_route(handle, T, x, token_ids, W_router, b, topk_idx, gates, counts, f, P, P_sum, scores_dbg, world,
                   send_rows, stream=None) -> None:
    _check(_lib.dsmoe_ep_route(handle, int(T), *[_ptr(t) for t in (
        x, token_ids, W_router, b, topk_idx, gates, counts, f, P, P_sum, scores_dbg)], int(world), _ptr(send_rows),
        _stream(stream)), "dsmoe_ep_route")


def dsmoe_ep_experts(handle, n_src, e_begin, e_end, recv_counts, n_rows, rows, W_gate, W_up, W_down, Y,
                     stream=None) -> None:
    _check(_lib.dsmoe_ep_experts(handle, int(n_src), int(e_begin), int(e_end), _ptr(recv_counts), int(n_rows),
                                 *[_ptr(t) for t in (rows, W_gate, W_up, W_down, Y)], _stream(stream)),
           "dsmoe_ep_experts")


def dsmoe_ep_combine(handle, T, x, Ws_gate, Ws_up, Ws_down, gates, Y, h, stream=None) -> None:
    _check(_lib.dsmoe_ep_combine(handle, int(T), *[_ptr(t) for t in (x, Ws_gate, Ws_up, Ws_down, gates, Y, h)],
                                 _stream(stream)), "dsmoe_ep_combine")


def dsmoe_set_training(handle, enable: bool) -> None:
    _check(_lib.dsmoe_set_training(handle, int(bool(enable))), "dsmoe_set_training")


def dsmoe_backward_experts(handle, T, dh, dY, W_gate, W_up, W_down, Ws_gate, Ws_up, Ws_down, dx_add, dx,
                           stream=None) -> None:
    _check(_lib.dsmoe_backward_experts(handle, int(T), *[_ptr(t) for t in (
        dh, dY, W_gate, W_up, W_down, Ws_gate, Ws_up, Ws_down, dx_add, dx)], _stream(stream)),
        "dsmoe_backward_experts")


def dsmoe_backward_weights(handle, T, dh, dY, x, dW_gate, dW_up, dW_down, dWs_gate, dWs_up, dWs_down,
                           stream=None) -> None:
    _check(_lib.dsmoe_backward_weights(handle, int(T), *[_ptr(t) for t in (
        dh, dY, x, dW_gate, dW_up, dW_down, dWs_gate, dWs_up, dWs_down)], _stream(stream)),
        "dsmoe_backward_weights")


def dsmoe_backward_gates(handle, T, dh, gates, dg, dY, stream=None) -> None:
    _check(_lib.dsmoe_backward_gates(handle, int(T), _ptr(dh), _ptr(gates), _ptr(dg), _ptr(dY), _stream(stream)),
           "dsmoe_backward_gates")


def dsmoe_backward_router(handle, T, x, W_router, topk_idx, gates, scores, dg, f, alpha, dlogits, dx, dW_router,
                          stream=None) -> None:
    _check(_lib.dsmoe_backward_router(handle, int(T), *[_ptr(t) for t in (
        x, W_router, topk_idx, gates, scores, dg, f)], float(alpha), _ptr(dlogits), _ptr(dx), _ptr(dW_router),
        _stream(stream)), "dsmoe_backward_router")


def dsmoe_set_timing(handle, enable: bool) -> None:
    _check(_lib.dsmoe_set_timing(handle, int(bool(enable))), "dsmoe_set_timing")


def dsmoe_stage_name(i: int) -> Optional[str]:
    r = _lib.dsmoe_stage_name(int(i))
    return None if r is None else r.decode()


def stage_names() -> Sequence[str]:
    out, i = [], 0
    while (n := dsmoe_stage_name(i)) is not None:
        out.append(n)
        i += 1
    return out


def dsmoe_stage_times(handle) -> Dict[str, float]:
    names = stage_names()
    buf = (ctypes.c_float * len(names))()
    n = ctypes.c_int32(0)
    _check(_lib.dsmoe_stage_times(handle, buf, len(names), ctypes.byref(n)), "dsmoe_stage_times")
    return {names[i]: float(buf[i]) for i in range(n.value)}


def dsmoe_gemm_role_cycles():
    """The one-CTA grouped GEMM's role counters since the last call, as a uint64 array
    [launch kind, CTA, slot] (kinds ROLE_KINDS, slots ROLE_SLOT_NAMES); a profiling build
    of the library is required (DsmoeError with DSMOE_ERR_UNSUPPORTED otherwise)."""
    import numpy as np
    buf = np.zeros((len(ROLE_KINDS), ROLE_CTAS, ROLE_SLOTS), dtype=np.uint64)
    _check(_lib.dsmoe_gemm_role_cycles(buf.ctypes.data, buf.size), "dsmoe_gemm_role_cycles")
    return buf


def dsmoe_launch_count(handle) -> int:
    n = ctypes.c_int64(0)
    _check(_lib.dsmoe_launch_count(handle, ctypes.byref(n)), "dsmoe_launch_count")
    return n.value


def dsmoe_route_noalloc(cfg: DsmoeCfg, T, x, W_router, b, topk_idx, gates, counts, f, P, stream=None) -> None:
    """The routing stage without a handle or any allocation (scratch is a fixed array in
    the library); for callers that cannot allocate device memory when they route."""
    st = _lib.dsmoe_route_noalloc(ctypes.byref(cfg), int(T), *[_ptr(t) for t in (
        x, W_router, b, topk_idx, gates, counts, f, P)], _stream(stream))
    _check(st, "dsmoe_route_noalloc")


def dsmoe_balance_losses(handle, f, P, n_groups, group_of, alpha1, alpha2, f_dev, P_dev, losses, stream=None):
    _check(_lib.dsmoe_balance_losses(handle, _ptr(f), _ptr(P), int(n_groups), _ptr(group_of), float(alpha1),
                                     float(alpha2), _ptr(f_dev), _ptr(P_dev), _ptr(losses), _stream(stream)),
           "dsmoe_balance_losses")


def dsmoe_sequence_balance(handle, T, seq_len, topk_idx, scores, beta, f_seq, p_seq, loss, stream=None):
    _check(_lib.dsmoe_sequence_balance(handle, int(T), int(seq_len), _ptr(topk_idx), _ptr(scores), float(beta),
                                       _ptr(f_seq), _ptr(p_seq), _ptr(loss), _stream(stream)),
           "dsmoe_sequence_balance")


def dsmoe_bias_update(handle, T, counts, alpha, b, stream=None):
    _check(_lib.dsmoe_bias_update(handle, int(T), _ptr(counts), float(alpha), _ptr(b), _stream(stream)),
           "dsmoe_bias_update")


# ---- the 8-bit path. Byte tensors (e4m3 values, e8m0 scales) may be of any one-byte dtype, e.g.
# torch.float8_e4m3fn and torch.float8_e8m0fnu.
_DTYPES: Dict[str, tuple] = {}
_raw_stream = None


def _setup():
    import torch
    global _raw_stream
    _raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream() without the Stream object
    _DTYPES.update(bf16=(torch.bfloat16,), f32=(torch.float32,), i32=(torch.int32,),
                   q8=(torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.uint8, torch.int8))


def _take(where: str, handle, stream, *tensors):
    """Check the torch tensors of a call ((name, tensor, kind, elements); raw addresses pass) and
    return their addresses in order, and the stream: the caller's, or the current stream of
    the handle's device."""
    if not _DTYPES:
        _setup()
    device = _handles[handle].device if handle in _handles else None
    ptrs = []
    for name, t, kind, n in tensors:
        if t is not None and t.__class__ is not int:
            if t.dtype not in _DTYPES[kind] or t.numel() != n or not t.is_contiguous() or \
                    (t.get_device() != device if device is not None else not t.is_cuda):
                _refuse(where, name, t, kind, n)
            t = t.data_ptr()
        ptrs.append(t)
    if stream is None and device is not None:
        return ptrs, _raw_stream(device)
    return ptrs, _stream(stream)


def _take_outputs(where: str, live, *tensors):
    """As _take, for outputs, which may be longer than the call needs."""
    ptrs = []
    for name, t, kind, n in tensors:
        if t is not None and t.__class__ is not int:
            if live is not None and (t.dtype not in _DTYPES[kind] or t.numel() < n or not t.is_contiguous() or
                                     t.get_device() != live.device):
                _refuse(where, name, t, kind, n, least=True)
            t = t.data_ptr()
        ptrs.append(t)
    return ptrs


def _refuse(where: str, name: str, t, kind: str, n: int, least: bool = False):
    if t.dtype not in _DTYPES[kind]:
        why = f"is {t.dtype}, not {' or '.join(map(str, _DTYPES[kind]))}"
    elif t.numel() < n or (t.numel() != n and not least):
        why = f"has {t.numel()} elements, not {n}"
    elif not t.is_contiguous():
        why = "is not contiguous"
    else:
        why = f"is on {t.device}, not on the handle's GPU"
    raise DsmoeError(DSMOE_ERR_INVALID_ARG, where, f"{name} {why}")


def _norm_width(where, handle, w) -> int:
    """d of the handle's rows, which w has to match."""
    known = _handles.get(handle)
    if known is None:
        return w.numel() if hasattr(w, "numel") else 0
    d = known.cfg.d_model
    if w is not None and w.__class__ is not int and w.numel() != d:
        raise DsmoeError(DSMOE_ERR_INVALID_ARG, where, f"w has {w.numel()} elements, not d_model = {d}")
    return d


def dsmoe_q8_scale_cols(C: int) -> int:
    """Scale bytes of a row of C values: 4 ceil(C / 512)."""
    return int(_lib.dsmoe_q8_scale_cols(int(C)))


def _scale_cols(C: int) -> int:
    return 4 * ((C + 511) // 512)


def dsmoe_q8_quantize(handle, R, C, x, q, scales, stream=None) -> None:
    where, R, C = "dsmoe_q8_quantize", int(R), int(C)
    p, s = _take(where, handle, stream, ("x", x, "bf16", R * C), ("q", q, "q8", R * C),
                 ("scales", scales, "q8", R * _scale_cols(C)))
    _check(_lib.dsmoe_q8_quantize(handle, R, C, *p, s), where)


def dsmoe_q8_quantize_weights(handle, E, N, K, W, q, scales, stream=None) -> None:
    where, E, N, K = "dsmoe_q8_quantize_weights", int(E), int(N), int(K)
    p, s = _take(where, handle, stream, ("W", W, "bf16", E * N * K), ("q", q, "q8", E * N * K),
                 ("scales", scales, "q8", E * -(-N // 128) * _scale_cols(K)))
    _check(_lib.dsmoe_q8_quantize_weights(handle, E, N, K, *p, s), where)


def dsmoe_norm_q8(handle, T, x, residual, w, eps, r, u, q, scales, stream=None) -> None:
    where, T = "dsmoe_norm_q8", int(T)
    d = _norm_width(where, handle, w)
    n = T * d
    (x, residual, w, r, u, q, scales), s = _take(
        where, handle, stream, ("x", x, "bf16", n), ("residual", residual, "bf16", n), ("w", w, "bf16", d),
        ("r", r, "bf16", n), ("u", u, "bf16", n), ("q", q, "q8", n),
        ("scales", scales, "q8", T * _scale_cols(d)))
    _check(_lib.dsmoe_norm_q8(handle, T, x, residual, w, float(eps), r, u, q, scales, s), where)


def dsmoe_norm_backward(handle, T, dy, dres, r, w, eps, dx, dw, stream=None) -> None:
    where, T = "dsmoe_norm_backward", int(T)
    d = _norm_width(where, handle, w)
    n = T * d
    (dy, dres, r, w, dx, dw), s = _take(
        where, handle, stream, ("dy", dy, "f32", n), ("dres", dres, "bf16", n), ("r", r, "bf16", n),
        ("w", w, "bf16", d), ("dx", dx, "bf16", n), ("dw", dw, "f32", d))
    _check(_lib.dsmoe_norm_backward(handle, T, dy, dres, r, w, float(eps), dx, dw, s), where)


def dsmoe_q8_matmul(handle, E, R, N, K, offsets, a, a_scales, W, W_scales, out, stream=None) -> None:
    where, E, R, N, K = "dsmoe_q8_matmul", int(E), int(R), int(N), int(K)
    S = _scale_cols(K)
    p, s = _take(
        where, handle, stream, ("offsets", offsets, "i32", E + 1), ("a", a, "q8", R * K),
        ("a_scales", a_scales, "q8", R * S), ("W", W, "q8", E * N * K),
        ("W_scales", W_scales, "q8", E * -(-N // 128) * S), ("out", out, "bf16", R * N))
    _check(_lib.dsmoe_q8_matmul(handle, E, R, N, K, *p, s), where)


def dsmoe_q8_gated_matmul(handle, E, R, N, K, offsets, a, a_scales, W_gate, gate_scales, W_up, up_scales, q, scales,
                          stream=None) -> None:
    where, E, R, N, K = "dsmoe_q8_gated_matmul", int(E), int(R), int(N), int(K)
    S = _scale_cols(K)
    nw, ns = E * N * K, E * -(-N // 128) * S
    p, s = _take(
        where, handle, stream, ("offsets", offsets, "i32", E + 1), ("a", a, "q8", R * K),
        ("a_scales", a_scales, "q8", R * S), ("W_gate", W_gate, "q8", nw), ("gate_scales", gate_scales, "q8", ns),
        ("W_up", W_up, "q8", nw), ("up_scales", up_scales, "q8", ns), ("q", q, "q8", R * N),
        ("scales", scales, "q8", R * _scale_cols(N)))
    _check(_lib.dsmoe_q8_gated_matmul(handle, E, R, N, K, *p, s), where)


def dsmoe_q8_tiling(E, R, N, K, output: int, E_all=None, num_sms: int = 148) -> Dict[str, int]:
    """How a product is cut up: tokens of a tile, CTAs per tile (splits), chains of K, CTAs (grid)."""
    t = DsmoeQ8Tiles()
    _check(_lib.dsmoe_q8_tiling(int(E), int(E if E_all is None else E_all), int(R), int(N), int(K), int(output),
                                int(num_sms), ctypes.byref(t)), "dsmoe_q8_tiling")
    return {n: getattr(t, n) for n, _ in t._fields_}


def _q8_weight_shapes(cfg: DsmoeCfg):
    """(experts, N, K) of each expert tensor by name; experts None: as many as the handle applies."""
    d, F, Fs, Ks = cfg.d_model, cfg.d_ff, cfg.d_ff_shared, cfg.n_shared
    return {"W_gate": (None, F, d), "W_up": (None, F, d), "W_down": (None, d, F),
            "Ws_gate": (Ks, Fs, d), "Ws_up": (Ks, Fs, d), "Ws_down": (Ks, d, Fs)}


def _take_q8_weights(where: str, handle, weights: Dict, experts: Optional[int]) -> DsmoeQ8Weights:
    """The struct of 8-bit weights given as (values, scales) pairs by name, each checked against
    the handle's configuration and the number of routed experts (raw addresses pass)."""
    ptrs = []
    for name, (E, N, K) in _q8_weight_shapes(_handles[handle].cfg).items():
        values, scales = (E != 0 and weights.get(name)) or (None, None)  # (0: no shared experts)
        E = (experts or 0) if E is None else E
        for what, t, rows, cols in (("values", values, N, K), ("scales", scales, -(-N // 128), _scale_cols(K))):
            if getattr(t, "ndim", 0) == 3 and tuple(t.shape) != (E, rows, cols):
                raise DsmoeError(DSMOE_ERR_INVALID_ARG, where,
                                 f"{name} {what} are {tuple(t.shape)}, not {(E, rows, cols)}")
            ptrs += _take(where, handle, 0, (f"{name} {what}", t, "q8", E * rows * cols))[0]
    return DsmoeQ8Weights(*ptrs)


def dsmoe_forward_q8(handle, T, x, x_q, x_scales, residual, token_ids, W_router, b, weights, h, topk_idx, gates,
                     counts, f, P, P_sum=None, scores_dbg=None, stream=None) -> None:
    """weights: a dict of (values, scales) tensor pairs by name (Q8_WEIGHTS), or a DsmoeQ8Weights, whose
    addresses are taken as they are. Outputs may be longer than T tokens need."""
    where, T = "dsmoe_forward_q8", int(T)
    live = _handles.get(handle)
    if not isinstance(weights, DsmoeQ8Weights):
        weights = DsmoeQ8Weights() if live is None else _take_q8_weights(where, handle, weights, live.experts)
    d, N, k = (live.cfg.d_model, live.cfg.n_routed, live.k) if live is not None else (0, 0, 0)
    n = T * d
    (x, x_q, x_scales, residual, token_ids, W_router, b), s = _take(
        where, handle, stream, ("x", x, "bf16", n), ("x_q", x_q, "q8", n),
        ("x_scales", x_scales, "q8", T * _scale_cols(d)), ("residual", residual, "bf16", n),
        ("token_ids", token_ids, "i32", T), ("W_router", W_router, "bf16", N * d), ("b", b, "f32", N))
    outs = _take_outputs(
        where, live, ("h", h, "f32" if live is not None and live.flags & DSMOE_RANGE_PARTIAL else "bf16", n),
        ("topk_idx", topk_idx, "i32", T * k), ("gates", gates, "f32", T * k), ("counts", counts, "i32", N),
        ("f", f, "f32", N), ("P", P, "f32", N), ("P_sum", P_sum, "f32", N), ("scores_dbg", scores_dbg, "f32", T * N))
    _check(_lib.dsmoe_forward_q8(handle, T, x, x_q, x_scales, residual, token_ids, W_router, b, ctypes.byref(weights),
                                 *outs, s), where)


_WS_DTYPES = {"logits": "float32", "offsets": "int32", "slot_of": "int32", "Xp": "bfloat16",
              "A1": "bfloat16", "A1s": "bfloat16", "Y": "bfloat16", "Hs": "float32", "AB": "bfloat16",
              "ABs": "bfloat16", "dAB": "bfloat16", "dABs": "bfloat16", "dXp": "bfloat16", "dXs": "float32"}


def dsmoe_workspace_tensor(handle, name: str):
    """(device address, rows, cols) of an intermediate workspace buffer."""
    p, r, c = ctypes.c_void_p(), ctypes.c_int64(), ctypes.c_int64()
    _check(_lib.dsmoe_workspace_tensor(handle, name.encode(), ctypes.byref(p), ctypes.byref(r), ctypes.byref(c)),
           "dsmoe_workspace_tensor")
    return p.value, r.value, c.value


def workspace_view(handle, name: str, device: int = 0):
    """A torch tensor aliasing a workspace buffer (copy it before the next forward)."""
    import torch
    ptr, rows, cols = dsmoe_workspace_tensor(handle, name)
    dt = getattr(torch, _WS_DTYPES[name])
    n = rows * cols
    esz = torch.empty((), dtype=dt).element_size()

    class _Buf:  # minimal __cuda_array_interface__ exporter over the raw device pointer
        pass

    b = _Buf()
    typestr = {"float32": "<f4", "int32": "<i4", "bfloat16": "<i2"}[_WS_DTYPES[name]]
    b.__cuda_array_interface__ = dict(shape=(n,), typestr=typestr, data=(ptr, False), version=3)
    with torch.cuda.device(device):
        t = torch.as_tensor(b, device=f"cuda:{device}")
    if _WS_DTYPES[name] == "bfloat16":
        t = t.view(torch.bfloat16)
    assert t.element_size() == esz
    return t.view(rows, cols)


def _empty(stream, device: int, shapes):
    """Tensors for work on `stream` (None: the current one), as [(shape, dtype), ...]. torch reuses freed
    memory in the order of the stream it was allocated on, so they are allocated on `stream`: a
    block whose last use there or elsewhere is still to come is not taken. The current stream is
    recorded as their user, so that what it still reads of them is not overwritten once they are freed."""
    import torch
    dev = torch.device("cuda", device)
    if not _DTYPES:
        _setup()
    raw, here = None if stream is None else _stream(stream), _raw_stream(device)
    if raw is None or raw == here:
        return [torch.empty(shape, dtype=dtype, device=dev) for shape, dtype in shapes]
    on = torch.cuda.ExternalStream(raw, device=dev) if raw else torch.cuda.default_stream(dev)
    current = torch.cuda.current_stream(dev)
    with torch.cuda.stream(on):
        out = [torch.empty(shape, dtype=dtype, device=dev) for shape, dtype in shapes]
    for t in out:
        t.record_stream(current)
    return out


class DSMoE:
    """A handle plus the weight tensors of one layer; forward() allocates the outputs with
    torch (device memory only) and calls dsmoe_forward."""

    def __init__(self, cfg: DsmoeCfg, weights: Dict, device: int = 0):
        self.cfg = cfg
        self.device = device
        self.w = weights
        self.handle = dsmoe_create(cfg, device)
        self.mask_top, self.k_active = 0, cfg.top_k
        self.range_flags = DSMOE_RANGE_ADD_SHARED

    def set_selection(self, mask_top: int = 0, k_active: Optional[int] = None):
        """Selection variant for later forwards (see dsmoe_set_selection)."""
        k = self.cfg.top_k if k_active is None else int(k_active)
        dsmoe_set_selection(self.handle, mask_top, k)
        self.mask_top, self.k_active = int(mask_top), k

    def set_expert_range(self, e_begin: int, e_end: int, partial: bool = True, add_shared: bool = False):
        """Apply only routed experts [e_begin, e_end) in later forwards (see
        dsmoe_set_expert_range); the weights given at construction must then hold those
        experts only. With partial, forward() returns h as fp32 partial sums."""
        flags = (DSMOE_RANGE_PARTIAL if partial else 0) | (DSMOE_RANGE_ADD_SHARED if add_shared else 0)
        dsmoe_set_expert_range(self.handle, e_begin, e_end, flags)
        self.range_flags = flags

    def close(self):
        if self.handle:
            dsmoe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def alloc_outputs(self, T: int, with_scores: bool = False, stream=None):
        """forward()'s outputs for T tokens, for use on `stream` (None: the current one)."""
        import torch
        c, f32, i32 = self.cfg, torch.float32, torch.int32
        N, K = (c.n_routed,), (T, self.k_active)
        shapes = dict(h=((T, c.d_model), f32 if self.range_flags & DSMOE_RANGE_PARTIAL else torch.bfloat16),
                      topk_idx=(K, i32), gates=(K, f32), counts=(N, i32), f=(N, f32), P=(N, f32), P_sum=(N, f32))
        if with_scores and c.score != DSMOE_ROUTE_HASH:
            shapes["scores"] = ((T, c.n_routed), f32)
        out = dict(zip(shapes, _empty(stream, self.device, shapes.values())))
        out.setdefault("scores", None)
        return out

    def forward(self, x, token_ids=None, out=None, with_scores: bool = False, stream=None):
        T = x.shape[0]
        o = self.alloc_outputs(T, with_scores, stream) if out is None else out
        w = self.w
        dsmoe_forward(self.handle, T, x, token_ids, w.get("W_router"), w.get("b"), w["W_gate"], w["W_up"],
                      w["W_down"], w.get("Ws_gate"), w.get("Ws_up"), w.get("Ws_down"), o["h"], o["topk_idx"],
                      o["gates"], o["counts"], o["f"], o["P"], o["P_sum"], o["scores"], stream)
        return o


class DSMoEQ8(DSMoE):
    """The layer with its expert weights in 8 bits. weights: DSMoE's dict; the six expert tensors
    may be bf16 (quantised here, once, and waited for; the bf16 tensors are not kept) or (values, scales)
    pairs that already are in 8 bits, with scales of dsmoe_q8_scale_cols bytes a row; they are checked
    here against cfg, and their number of experts against the expert range in force at a forward. sharded.expert_sharded_forward takes it as it takes a
    DSMoE; the token-dispatch form and the backward pass need the bf16 weights."""

    def __init__(self, cfg: DsmoeCfg, weights: Dict, device: int = 0):
        import torch
        super().__init__(cfg, {k: v for k, v in weights.items() if k not in Q8_WEIGHTS}, device)
        where, shapes = "DSMoEQ8", _q8_weight_shapes(cfg)
        self.q, self.experts = {}, None
        for name in Q8_WEIGHTS:
            W, (E, N, K) = weights.get(name), shapes[name]
            if W is None or E == 0:  # (a configuration without shared experts reads none)
                continue
            pair = isinstance(W, (tuple, list))
            values = W[0] if pair else W
            if hasattr(values, "numel"):  # (raw addresses are taken as they are)
                if E is None:
                    E = values.numel() // (N * K) if self.experts is None else self.experts
                    self.experts = E
                if not pair and tuple(W.shape) != (E, N, K):
                    raise DsmoeError(DSMOE_ERR_INVALID_ARG, where, f"{name} is {tuple(W.shape)}, not {(E, N, K)}")
            if not pair:
                values = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=W.device)
                scales = torch.empty((E, -(-N // 128), dsmoe_q8_scale_cols(K)), dtype=torch.float8_e8m0fnu,
                                     device=W.device)
                dsmoe_q8_quantize_weights(self.handle, E, N, K, W, values, scales)
                W = (values, scales)
            self.q[name] = tuple(W)
        if any(n in weights and not isinstance(weights[n], (tuple, list)) for n in Q8_WEIGHTS):
            torch.cuda.current_stream(device).synchronize()  # the weights are ready for forwards on any stream
        self._weights = _take_q8_weights(where, self.handle, self.q, self.experts)

    def _check_experts(self, experts: int):
        if self.experts is not None and self.experts != experts:
            raise DsmoeError(DSMOE_ERR_INVALID_ARG, "DSMoEQ8", f"the weights hold {self.experts} routed experts, not "
                             f"the {experts} of the expert range")

    def set_expert_range(self, e_begin: int, e_end: int, partial: bool = True, add_shared: bool = False):
        self._check_experts(int(e_end) - int(e_begin))
        super().set_expert_range(e_begin, e_end, partial, add_shared)

    def alloc_rows(self, T: int, stream=None):
        """Buffers of T 8-bit rows, values [T, d] and scales [T, S(d)], for use on `stream`."""
        import torch
        d = self.cfg.d_model
        return tuple(_empty(stream, self.device, [((T, d), torch.float8_e4m3fn),
                                                  ((T, dsmoe_q8_scale_cols(d)), torch.float8_e8m0fnu)]))

    def forward(self, x, token_ids=None, out=None, with_scores: bool = False, stream=None, residual=None, x_q=None):
        """The layer on x; x_q: its 8-bit rows (values, scales) where the caller has them, else they are
        made here and returned as "x_q", which lives as long as the outputs; an `out` that holds it
        from an earlier call with as many tokens has it overwritten like the other outputs.
        residual: what the layer's output is added to in place of x."""
        T = x.shape[0]
        if self.handle in _handles:
            self._check_experts(_handles[self.handle].experts)
        o = self.alloc_outputs(T, with_scores, stream) if out is None else out
        if x_q is None:
            x_q = o.get("x_q")
            if x_q is None or x_q[0].shape[0] != T:
                x_q = o["x_q"] = self.alloc_rows(T, stream)
            dsmoe_q8_quantize(self.handle, T, self.cfg.d_model, x, *x_q, stream)
        w = self.w
        dsmoe_forward_q8(self.handle, T, x, *x_q, residual, token_ids, w.get("W_router"), w.get("b"), self._weights,
                         o["h"], o["topk_idx"], o["gates"], o["counts"], o["f"], o["P"], o["P_sum"], o["scores"],
                         stream)
        return o

    def forward_norm(self, x, residual, w, eps: float, token_ids=None, with_scores: bool = False, stream=None):
        """A block: r = x + residual, u = RMSNorm(r) w, h = r + the layer's experts on u. Returns the
        layer's outputs and "r", "u", "x_q" (the 8-bit rows of u)."""
        import torch
        T = x.shape[0]
        r, u = _empty(stream, self.device, [(x.shape, torch.bfloat16)] * 2)
        x_q = self.alloc_rows(T, stream)
        dsmoe_norm_q8(self.handle, T, x, residual, w, eps, r, u, *x_q, stream)
        o = self.forward(u, token_ids, None, with_scores, stream, r, x_q)
        o["r"], o["u"], o["x_q"] = r, u, x_q
        return o

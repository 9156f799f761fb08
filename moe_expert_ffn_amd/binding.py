"""Thin ctypes binding of libmoe_ffn.so (C ABI in include/moe_ffn.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  torch provides device memory and the current HIP stream.  The
library must have been built (``python moe_expert_ffn_amd/build.py`` or
``__graft_entry__.build()``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import itertools
import os
from bisect import bisect_left

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_ffn.so")

ABI_VERSION = 5                 # MOE_ABI_VERSION of the header these signatures follow
MOE_OK, MOE_ERR_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 0, -1, -2, -3, -4
MOE_F32, MOE_BF16, MOE_FP8_E4M3, MOE_INT8 = 0, 1, 2, 3
PLAN_FWD, PLAN_BWD, PLAN_QUOTA = 0, 1, 2
DEV_BAD_EXPERT, DEV_BAD_PLAN, DEV_BAD_OWNER, DEV_WAIT_TIMEOUT = 1, 2, 4, 8
DEV_BAD_LOGIT, DEV_BAD_GRAD = 16, 32
SCORES = {"softmax": 0, "sigmoid": 1}         # moe_score
GROUP_SCORES = {"max": 0, "top2": 1}          # moe_group_score
GATE_NONE, GATE_TOKEN, GATE_FEATURE = 0, 1, 2  # moe_gate_kind
ADAMW_BLOCK = 128                             # MOE_ADAMW_BLOCK
EXEC_TWO_PHASE = 1              # MOE_EXEC_TWO_PHASE
EXEC_SPLIT_SHIFT = 8            # MOE_EXEC_SPLIT(n1) = n1 << 8
EXEC_FP8_ACT = 2                # MOE_EXEC_FP8_ACT


def exec_flags(two_phase=False, split=0, fp8_act=False):
    """exec_flags of moe_forward / moe_backward: the two-phase launch and its
    producer workgroups per worker (0: every workgroup runs both phases)."""
    split = int(split)
    if split and not two_phase:
        raise MoeError("a producer/consumer split needs the two-phase launch")
    if not 0 <= split <= 0xFF:
        raise MoeError(f"split={split} outside 0..255")
    return ((EXEC_TWO_PHASE if two_phase else 0) | (split << EXEC_SPLIT_SHIFT) |
            (EXEC_FP8_ACT if fp8_act else 0))
TIMELINE_MAX_WG, TL_PHASES = 1024, 5          # MOE_TIMELINE_MAX_WG, MOE_TL_PHASES
TL_FC1, TL_FC2, TL_DA, TL_DX, TL_DW = range(5)

EXPORTS = ["moe_abi_version", "moe_status_str", "moe_max_slots", "moe_max_blocks",
           "moe_workspace_size", "moe_route_stats", "moe_route_stats_noalloc", "moe_plan",
           "moe_plan_gate",
           "moe_predict_cost", "moe_predict_split", "moe_quantize_token_blocks",
           "moe_quantize_act_rows", "moe_quantize_int8_rows", "moe_forward",
           "moe_backward", "moe_backward_gates", "moe_gate_grad",
           "moe_router_workspace_size", "moe_router_forward", "moe_router_backward",
           "moe_router_forward_choice", "moe_router_bias_update",
           "moe_norm_workspace_size", "moe_norm_in", "moe_norm_in_backward", "moe_norm_out",
           "moe_norm_out_backward",
           "moe_adamw_workspace_size", "moe_adamw_prepare", "moe_adamw",
           "moe_grad_workspace_size", "moe_grad_prepare", "moe_grad_norm", "moe_grad_scale",
           "moe_event_create", "moe_event_destroy", "moe_event_record", "moe_event_elapsed_ms",
           "moe_device_info"]


class MoeError(RuntimeError):
    pass


class Layer(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int), ("d", ctypes.c_int), ("d_ff", ctypes.c_int),
                ("act_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
                ("w1", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("w1_scale", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p)]


class Router(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int), ("k", ctypes.c_int), ("dtype", ctypes.c_int),
                ("score", ctypes.c_int), ("renorm", ctypes.c_int), ("scale", ctypes.c_float)]


class Choice(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("groups", ctypes.c_int), ("top_groups", ctypes.c_int),
                ("group_score", ctypes.c_int)]
    tensor = None                             # the bias, which the choice keeps alive


class Norm(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("d", ctypes.c_int), ("dtype", ctypes.c_int),
                ("w_dtype", ctypes.c_int), ("gate_kind", ctypes.c_int), ("alpha", ctypes.c_float),
                ("eps", ctypes.c_float), ("w", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("token_mask", ctypes.c_void_p)]


class AdamwTensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("master", ctypes.c_void_p), ("g", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("p_dtype", ctypes.c_int),
                ("g_dtype", ctypes.c_int)]


class AdamwList(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("tensors", ctypes.c_int),
                ("state_bits", ctypes.c_int), ("items", ctypes.c_uint32), ("item", ctypes.c_int)]


class AdamwHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("step", ctypes.c_int), ("seed", ctypes.c_uint32), ("step_dev", ctypes.c_void_p),
                ("lr_dev", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p)]


class GradTensor(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int)]


class GradList(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("tensors", ctypes.c_int), ("items", ctypes.c_uint32),
                ("apart", ctypes.c_int)]


class Clip(ctypes.Structure):
    _fields_ = [("max_norm", ctypes.c_double), ("mult", ctypes.c_double), ("mult_dev", ctypes.c_void_p)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t


def load():
    """Load the built library (raises MoeError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise MoeError(f"{LIB_PATH} is missing: build it with moe_expert_ffn_amd/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    lib.moe_abi_version.restype = _I
    lib.moe_status_str.restype = ctypes.c_char_p
    lib.moe_status_str.argtypes = [_I]
    lib.moe_max_slots.restype = _SZ
    lib.moe_max_slots.argtypes = [_I, _I, _I, _I]
    lib.moe_max_blocks.restype = _SZ
    lib.moe_max_blocks.argtypes = [_I, _I, _I, _I]
    lib.moe_workspace_size.restype = _SZ
    lib.moe_workspace_size.argtypes = [ctypes.POINTER(Layer), _I, _I, _I, _I, _I, _I]
    lib.moe_route_stats.restype = _I
    lib.moe_route_stats.argtypes = [_P, _I, _I, _I, _I] + [_P] * 8 + [_P, _SZ, _P]
    lib.moe_route_stats_noalloc.restype = _I
    lib.moe_route_stats_noalloc.argtypes = [_P, _I, _I, _I, _I] + [_P] * 8 + [_P]
    lib.moe_plan.restype = _I
    lib.moe_plan.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I] + [_P] * 3 + [_I] + [_P] * 2 + [_P, _SZ, _P]
    lib.moe_quantize_token_blocks.restype = _I
    lib.moe_quantize_token_blocks.argtypes = [_P, _I, _I, _P, _I, _I, _P, _I, _I, _I, _P, _P, _P]
    lib.moe_predict_cost.restype = _I
    lib.moe_predict_cost.argtypes = [_P] * 5 + [_I] * 6 + [_P, _P, _P]
    lib.moe_quantize_act_rows.restype = _I
    lib.moe_quantize_act_rows.argtypes = [_P, _I, _I, _P, _P, _P]
    lib.moe_quantize_int8_rows.restype = _I
    lib.moe_quantize_int8_rows.argtypes = [_P, _I, _I, _I, _I, _P, _P, _P]
    lib.moe_predict_split.restype = _I
    lib.moe_predict_split.argtypes = [_P] * 3 + [_I] * 7 + [_P, _P, _P, _P]
    lib.moe_plan_gate.restype = _I
    lib.moe_plan_gate.argtypes = [_P, _P, _P, _I, _I, _I] + [_P] * 3 + [_I] + [_P] * 2 + [_P]
    lib.moe_forward.restype = _I
    lib.moe_forward.argtypes = ([ctypes.POINTER(Layer), _P, _P, _P, _I, _I, _I, _I]
                                + [_P] * 8 + [_P, _SZ, _I, _P, _P, _P])
    lib.moe_backward.restype = _I
    lib.moe_backward.argtypes = ([ctypes.POINTER(Layer), _P, _P, _P, _P, _P, _I, _I, _I, _I, _I]
                                 + [_P] * 10 + [_P, _SZ, _I, _P, _P, _P])
    lib.moe_backward_gates.restype = _I
    lib.moe_backward_gates.argtypes = ([ctypes.POINTER(Layer)] + [_P] * 5 + [_I] * 5
                                       + [_P] * 11 + [_P, _SZ, _I, _P, _P, _P])
    lib.moe_gate_grad.restype = _I
    lib.moe_gate_grad.argtypes = [_P, _P, _I, _P, _I, _I, _I, _P, _P]
    R, N = ctypes.POINTER(Router), ctypes.POINTER(Norm)
    lib.moe_router_workspace_size.restype = _SZ
    lib.moe_router_workspace_size.argtypes = [R, _I]
    lib.moe_router_forward.restype = _I
    lib.moe_router_forward.argtypes = [R, _P, _I, _P, _I] + [_P] * 7 + [_P, _SZ, _P]
    lib.moe_router_backward.restype = _I
    lib.moe_router_backward.argtypes = [R, _P, _I, _P, _I] + [_P] * 6 + [_I, _P]
    lib.moe_router_forward_choice.restype = _I
    lib.moe_router_forward_choice.argtypes = [R, ctypes.POINTER(Choice), _P, _I, _P, _I] + [_P] * 7 + [_P, _SZ, _P]
    lib.moe_router_bias_update.restype = _I
    lib.moe_router_bias_update.argtypes = [_P, _I, ctypes.c_float, _P, _P]
    lib.moe_norm_workspace_size.restype = _SZ
    lib.moe_norm_workspace_size.argtypes = [_I, _I]
    lib.moe_norm_in.restype = _I
    lib.moe_norm_in.argtypes = [N] + [_P, _I] * 4 + [_P, _P]
    lib.moe_norm_in_backward.restype = _I
    lib.moe_norm_in_backward.argtypes = [N] + [_P, _I] * 4 + [_P] + [_P, _I] * 2 + [_P, _P, _P, _SZ, _P]
    lib.moe_norm_out.restype = _I
    lib.moe_norm_out.argtypes = [N] + [_P, _I] * 3 + [_P, _P]
    lib.moe_norm_out_backward.restype = _I
    lib.moe_norm_out_backward.argtypes = [N] + [_P, _I] * 2 + [_P] + [_P, _I] + [_P, _P, _P, _SZ, _P]
    lib.moe_adamw_workspace_size.restype = _SZ
    lib.moe_adamw_workspace_size.argtypes = [_I]
    lib.moe_adamw_prepare.restype = _I
    lib.moe_adamw_prepare.argtypes = [ctypes.POINTER(AdamwTensor), _I, _I, ctypes.POINTER(AdamwList),
                                      _P, _SZ, _P]
    lib.moe_adamw.restype = _I
    lib.moe_adamw.argtypes = [ctypes.POINTER(AdamwList), ctypes.POINTER(AdamwHyper), _P]
    lib.moe_grad_workspace_size.restype = _SZ
    lib.moe_grad_workspace_size.argtypes = [_I]
    lib.moe_grad_prepare.restype = _I
    lib.moe_grad_prepare.argtypes = [ctypes.POINTER(GradTensor), _I, ctypes.POINTER(GradList), _P, _SZ, _P]
    lib.moe_grad_norm.restype = _I
    lib.moe_grad_norm.argtypes = [ctypes.POINTER(GradList), ctypes.POINTER(Clip), _P, _P, _P, _P]
    lib.moe_grad_scale.restype = _I
    lib.moe_grad_scale.argtypes = [ctypes.POINTER(GradList), _P, _P]
    lib.moe_event_create.argtypes = [ctypes.POINTER(_P)]
    lib.moe_event_destroy.argtypes = [_P]
    lib.moe_event_record.argtypes = [_P, _P]
    lib.moe_event_elapsed_ms.argtypes = [_P, _P, ctypes.POINTER(ctypes.c_float)]
    lib.moe_device_info.argtypes = [ctypes.POINTER(_I)] * 3
    if lib.moe_abi_version() != ABI_VERSION:
        raise MoeError(f"{LIB_PATH} has ABI {lib.moe_abi_version()}, the binding expects "
                       f"{ABI_VERSION}: rebuild it")
    _lib = lib
    return lib


def _check(rc):
    if rc != MOE_OK:
        raise MoeError(f"libmoe_ffn: {load().moe_status_str(rc).decode()} ({rc})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _require_device(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise MoeError("all buffers must be contiguous device tensors")


def _expect(t, dtype, min_numel, name):
    """Element type and minimum size of a buffer the library writes or reads."""
    if t.dtype != dtype:
        raise MoeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() < min_numel:
        raise MoeError(f"{name}: needs at least {min_numel} elements, has {t.numel()}")


def act_code(dtype) -> int:
    return MOE_F32 if dtype == torch.float32 else MOE_BF16


def _act_dtype(layer) -> torch.dtype:
    return torch.float32 if layer.act_dtype == MOE_F32 else torch.bfloat16


def _ids_shape(topk_ids):
    if topk_ids.dim() != 2:
        raise MoeError(f"topk_ids: expected [T][k], got {tuple(topk_ids.shape)}")
    _expect(topk_ids, torch.int32, 0, "topk_ids")
    return topk_ids.shape


def _expect_route(rs, T, k, E, beta):
    """The routing statistics the executors read (from route_stats)."""
    _expect(rs["counts"], torch.int32, E, "counts")
    _expect(rs["block_offsets"], torch.int32, E + 1, "block_offsets")
    _expect(rs["row_to_slot"], torch.int32, T * k, "row_to_slot")
    _expect(rs["slot_to_row"], torch.int32, max_slots(T, k, E, beta), "slot_to_row")


def _expect_plan_out(out, E, P):
    _expect(out["q"], torch.int32, E * P, "q")
    _expect(out["load"], torch.int32, P, "load")
    # block_worker [>= sum b]: its size goes to the library, which writes nothing
    # (and flags the plan) when the blocks do not fit
    _expect(out["block_worker"], torch.int32, 1, "block_worker")
    _expect(out["plan_info"], torch.int32, 4, "plan_info")


def make_layer(w1, w2, w1_scale=None, w2_scale=None, act_dtype=torch.bfloat16) -> Layer:
    _require_device(w1, w2, w1_scale, w2_scale)
    if w1.dim() != 3 or w2.dim() != 3:
        raise MoeError("w1 and w2 are [E][2 d_ff][d] and [E][d][d_ff]")
    E, two_dff, d = w1.shape
    if tuple(w2.shape) != (E, d, two_dff // 2) or two_dff % 2:
        raise MoeError(f"w2: expected {(E, d, two_dff // 2)}, got {tuple(w2.shape)}")
    if w2.dtype != w1.dtype:
        raise MoeError(f"w2: expected {w1.dtype}, got {w2.dtype}")
    if w1.dtype == torch.uint8:
        wcode = MOE_FP8_E4M3
        if w1_scale is None or w2_scale is None:
            raise MoeError("e4m3 weights need w1_scale and w2_scale")
        _expect(w1_scale, torch.float32, E * -(-two_dff // 128) * -(-d // 128), "w1_scale")
        _expect(w2_scale, torch.float32, E * -(-d // 128) * -(-(two_dff // 2) // 128), "w2_scale")
    elif w1.dtype == torch.int8:
        wcode = MOE_INT8
        if w1_scale is None or w2_scale is None:
            raise MoeError("int8 weights need w1_scale and w2_scale")
        if act_dtype != torch.bfloat16:
            raise MoeError(f"int8 weights take bfloat16 activations, not {act_dtype}")
        _expect(w1_scale, torch.float32, E * two_dff, "w1_scale")
        _expect(w2_scale, torch.float32, E * d, "w2_scale")
    elif w1.dtype == torch.float32:
        wcode = MOE_F32
    elif w1.dtype == torch.bfloat16:
        wcode = MOE_BF16
    else:
        raise MoeError(f"w1: unsupported element type {w1.dtype}")
    return Layer(E, d, two_dff // 2, act_code(act_dtype), wcode, w1.data_ptr(), w2.data_ptr(),
                 w1_scale.data_ptr() if w1_scale is not None else None,
                 w2_scale.data_ptr() if w2_scale is not None else None)


def max_slots(T, k, E, beta) -> int:
    return int(load().moe_max_slots(T, k, E, beta))


def max_blocks(T, k, E, beta) -> int:
    return int(load().moe_max_blocks(T, k, E, beta))


def workspace(layer: Layer, T, k, beta, P, s, with_backward, device) -> torch.Tensor:
    n = int(load().moe_workspace_size(ctypes.byref(layer), T, k, beta, P, s, int(with_backward)))
    if n == 0:
        raise MoeError("moe_workspace_size rejected the sizes")
    return torch.empty(n + 256, dtype=torch.uint8, device=device)


def _aligned(ws: torch.Tensor):
    p = ws.data_ptr()
    off = (-p) % 256
    return ctypes.c_void_p(p + off), ws.numel() - off


def alloc_route(T, k, E, beta, device):
    i32 = dict(dtype=torch.int32, device=device)
    return {
        "counts": torch.empty(E, **i32), "offsets": torch.empty(E + 1, **i32),
        "block_counts": torch.empty(E, **i32), "block_offsets": torch.empty(E + 1, **i32),
        "row_to_slot": torch.empty(max(T * k, 1), **i32),
        "slot_to_row": torch.empty(max(max_slots(T, k, E, beta), 1), **i32),
        "kappa": torch.empty(1, dtype=torch.float64, device=device),
    }


def route_stats(topk_ids: torch.Tensor, E: int, beta: int, out: dict, ws: torch.Tensor,
                status: torch.Tensor):
    _require_device(topk_ids, ws, status, *out.values())
    T, k = _ids_shape(topk_ids)
    _expect(out["counts"], torch.int32, E, "counts")
    _expect(out["offsets"], torch.int32, E + 1, "offsets")
    _expect(out["block_counts"], torch.int32, E, "block_counts")
    _expect(out["block_offsets"], torch.int32, E + 1, "block_offsets")
    _expect(out["row_to_slot"], torch.int32, T * k, "row_to_slot")
    _expect(out["slot_to_row"], torch.int32, max_slots(T, k, E, beta), "slot_to_row")
    _expect(out["kappa"], torch.float64, 1, "kappa")
    _expect(status, torch.int32, 1, "status")
    wsp, wsn = _aligned(ws)
    _check(load().moe_route_stats(_ptr(topk_ids), T, k, E, beta, _ptr(out["counts"]),
                                  _ptr(out["offsets"]), _ptr(out["block_counts"]),
                                  _ptr(out["block_offsets"]), _ptr(out["row_to_slot"]),
                                  _ptr(out["slot_to_row"]), _ptr(out["kappa"]), _ptr(status),
                                  wsp, wsn, _stream()))
    return out


def route_stats_noalloc(topk_ids: torch.Tensor, E: int, beta: int, out: dict,
                        status: torch.Tensor):
    """route_stats without a workspace (moe_route_stats_noalloc): the library's
    own scratch array holds the per-chunk counts."""
    _require_device(topk_ids, status, *out.values())
    T, k = _ids_shape(topk_ids)
    _expect(out["counts"], torch.int32, E, "counts")
    _expect(out["offsets"], torch.int32, E + 1, "offsets")
    _expect(out["block_counts"], torch.int32, E, "block_counts")
    _expect(out["block_offsets"], torch.int32, E + 1, "block_offsets")
    _expect(out["row_to_slot"], torch.int32, T * k, "row_to_slot")
    _expect(out["slot_to_row"], torch.int32, max_slots(T, k, E, beta), "slot_to_row")
    _expect(out["kappa"], torch.float64, 1, "kappa")
    _expect(status, torch.int32, 1, "status")
    _check(load().moe_route_stats_noalloc(_ptr(topk_ids), T, k, E, beta, _ptr(out["counts"]),
                                          _ptr(out["offsets"]), _ptr(out["block_counts"]),
                                          _ptr(out["block_offsets"]), _ptr(out["row_to_slot"]),
                                          _ptr(out["slot_to_row"]), _ptr(out["kappa"]),
                                          _ptr(status), _stream()))
    return out


def alloc_plan(E, P, nblocks_cap, device):
    i32 = dict(dtype=torch.int32, device=device)
    return {"q": torch.empty((E, P), **i32), "load": torch.empty(P, **i32),
            "block_worker": torch.full((max(nblocks_cap, 1),), -1, **i32),
            "plan_info": torch.empty(4, **i32)}


def predict_cost(counts, block_offsets, bw_fwd, bw_bwd, owner, beta, P, d, d_ff, cost, status,
                 num_workgroups=0):
    """Wave-quantized predicted cost (int64, thousandths of a K step) into cost[0]."""
    _require_device(counts, block_offsets, bw_fwd, bw_bwd, owner, cost, status)
    _check(load().moe_predict_cost(_ptr(counts), _ptr(block_offsets), _ptr(bw_fwd), _ptr(bw_bwd),
                                   _ptr(owner), counts.numel(), beta, P, d, d_ff, num_workgroups,
                                   _ptr(cost), _ptr(status), _stream()))
    return cost


def predict_split(counts, block_offsets, block_worker, beta, P, d, d_ff, backward, costs, choice,
                  status, num_workgroups=0):
    """Predicted time (int64, thousandths of a K step) of every two-phase mode
    into costs[m + 1] (m = -1 two launches, 0 one launch, n1 > 0 producer /
    consumer split) and the chosen mode into choice[0]."""
    _require_device(counts, block_offsets, block_worker, costs, choice, status)
    _expect(costs, torch.int64, costs.numel(), "costs")
    _expect(choice, torch.int32, 1, "choice")
    G = num_workgroups if num_workgroups > 0 else device_info()["num_cus"]
    if P > 0 and G % P == 0 and costs.numel() < G // P + 1:
        raise MoeError(f"costs holds {costs.numel()} entries, the model writes {G // P + 1}")
    _check(load().moe_predict_split(_ptr(counts), _ptr(block_offsets), _ptr(block_worker),
                                    counts.numel(), beta, P, d, d_ff, num_workgroups,
                                    1 if backward else 0, _ptr(costs), _ptr(choice), _ptr(status),
                                    _stream()))
    return costs, choice


def quantize_act_rows(src, codes, exps):
    """e4m3 codes [rows][cols] and power-of-two exponents [cols/128][rows]
    (int32) of the bf16 rows src [rows][cols], blocks of 128 features."""
    _require_device(src, codes, exps)
    if src.dim() != 2:
        raise MoeError("src must be [rows][cols]")
    rows, cols = src.shape
    _expect(src, torch.bfloat16, rows * cols, "src")
    _expect(codes, torch.uint8, rows * cols, "codes")
    _expect(exps, torch.int32, rows * (cols // 128), "exps")
    _check(load().moe_quantize_act_rows(_ptr(src), rows, cols, _ptr(codes), _ptr(exps), _stream()))
    return codes, exps


def quantize_token_blocks(src, rows, cols, block_rows, codes, scales, row_map=None, gather=False,
                          row_div=1, row_scale=None, ld=None, src_rows=None):
    """Token-axis e4m3 codes [rows][cols] and scales [ceil(rows/block_rows)][cols].

    src holds src_rows rows of ld elements (default: rows, the rows read in
    place); gathered map values past src_rows * row_div read as zero rows, and
    row_scale must hold src_rows * row_div entries."""
    _require_device(src, codes, scales, *[t for t in (row_map, row_scale) if t is not None])
    ld = cols if ld is None else ld
    if src_rows is None:
        if gather:
            raise MoeError("gathered rows need src_rows (the rows of src)")
        src_rows = rows
    if rows > 0 and block_rows > 0:
        nblk = (rows + block_rows - 1) // block_rows
        _expect(codes, torch.uint8, rows * cols, "codes")
        _expect(scales, torch.float32, nblk * cols, "scales")
        _expect(src, torch.bfloat16, (src_rows - 1) * ld + cols if src_rows > 0 else 0, "src")
        if row_map is not None:
            _expect(row_map, torch.int32, rows, "row_map")
        if row_scale is not None:
            _expect(row_scale, torch.float32, src_rows * row_div, "row_scale")
    _check(load().moe_quantize_token_blocks(
        _ptr(src), ld, src_rows, _ptr(row_map) if row_map is not None else None,
        1 if gather else 0, row_div, _ptr(row_scale) if row_scale is not None else None, rows, cols,
        block_rows, _ptr(codes), _ptr(scales), _stream()))
    return codes, scales


def plan_gate(block_counts, block_offsets, owner, P, rho_milli, out, status):
    _require_device(block_counts, block_offsets, owner, status, *out.values())
    E = block_counts.numel()
    _expect(block_counts, torch.int32, E, "block_counts")
    _expect(block_offsets, torch.int32, E + 1, "block_offsets")
    _expect(owner, torch.int32, E, "owner")
    _expect_plan_out(out, E, P)
    _expect(status, torch.int32, 1, "status")
    _check(load().moe_plan_gate(_ptr(block_counts), _ptr(block_offsets), _ptr(owner), E, P,
                                rho_milli, _ptr(out["q"]), _ptr(out["load"]),
                                _ptr(out["block_worker"]), out["block_worker"].numel(),
                                _ptr(out["plan_info"]), _ptr(status), _stream()))
    return out


def plan(block_counts, block_offsets, owner, P, s, mode, lam, out, ws, status):
    _require_device(block_counts, block_offsets, owner, ws, status, *out.values())
    E = block_counts.numel()
    _expect(block_counts, torch.int32, E, "block_counts")
    _expect(block_offsets, torch.int32, E + 1, "block_offsets")
    _expect(owner, torch.int32, E, "owner")
    _expect_plan_out(out, E, P)
    _expect(status, torch.int32, 1, "status")
    wsp, wsn = _aligned(ws)
    _check(load().moe_plan(_ptr(block_counts), _ptr(block_offsets), _ptr(owner), E, P, s, mode,
                           lam, _ptr(out["q"]), _ptr(out["load"]), _ptr(out["block_worker"]),
                           out["block_worker"].numel(), _ptr(out["plan_info"]), _ptr(status),
                           wsp, wsn, _stream()))
    return out


def alloc_timeline(device):
    """Timeline buffer [TL_PHASES][TIMELINE_MAX_WG][2] of the GPU's 100 MHz counter."""
    return torch.zeros((TL_PHASES, TIMELINE_MAX_WG, 2), dtype=torch.int64, device=device)


def _expect_timeline(timeline):
    if timeline is not None:
        _expect(timeline, torch.int64, TL_PHASES * TIMELINE_MAX_WG * 2, "timeline")


def forward(layer: Layer, x, gates, topk_ids, beta, P, rs, block_worker, y, z_save, ws, status,
            events=None, timeline=None, two_phase=False, split=0, fp8_act=False):
    _require_device(x, gates, topk_ids, y, z_save, ws, status, block_worker, timeline)
    _expect_timeline(timeline)
    T, k = _ids_shape(topk_ids)
    act, E, d, dff = _act_dtype(layer), layer.E, layer.d, layer.d_ff
    _expect(x, act, T * d, "x")
    _expect(gates, torch.float32, T * k, "gates")
    _expect(y, act, T * d, "y")
    if z_save is not None:
        _expect(z_save, act, max_slots(T, k, E, beta) * 2 * dff, "z_save")
    _expect_route(rs, T, k, E, beta)
    _expect(block_worker, torch.int32, max_blocks(T, k, E, beta), "block_worker")
    _expect(status, torch.int32, 1, "status")
    wsp, wsn = _aligned(ws)
    ev = None if events is None else (ctypes.c_void_p * len(events))(*events)
    _check(load().moe_forward(ctypes.byref(layer), _ptr(x), _ptr(gates), _ptr(topk_ids), T, k,
                              beta, P, _ptr(rs["counts"]), _ptr(rs["block_offsets"]),
                              _ptr(rs["row_to_slot"]), _ptr(rs["slot_to_row"]),
                              _ptr(block_worker), _ptr(y), _ptr(z_save), _ptr(status), wsp, wsn,
                              exec_flags(two_phase, split, fp8_act), ev, _ptr(timeline),
                              _stream()))


def backward(layer: Layer, x, gates, dy, z_save, topk_ids, beta, P, s, rs, owner, block_worker,
             dx, dw1, dw2, ws, status, events=None, timeline=None, two_phase=False, split=0,
             fp8_act=False, dlogp=None):
    """moe_backward; with dlogp [T][k] fp32, moe_backward_gates (the gate gradients too)."""
    _require_device(x, gates, dy, z_save, topk_ids, owner, block_worker, dx, dw1, dw2, ws, status,
                    timeline)
    _expect_timeline(timeline)
    T, k = _ids_shape(topk_ids)
    act, E, d, dff = _act_dtype(layer), layer.E, layer.d, layer.d_ff
    _expect(x, act, T * d, "x")
    _expect(gates, torch.float32, T * k, "gates")
    _expect(dy, act, T * d, "dy")
    _expect(z_save, act, max_slots(T, k, E, beta) * 2 * dff, "z_save")
    _expect_route(rs, T, k, E, beta)
    _expect(owner, torch.int32, E, "owner")
    _expect(block_worker, torch.int32, max_blocks(T, k, E, beta), "block_worker")
    _expect(dx, act, T * d, "dx")
    _expect(dw1, torch.float32, E * 2 * dff * d, "dw1")
    _expect(dw2, torch.float32, E * d * dff, "dw2")
    _expect(status, torch.int32, 1, "status")
    wsp, wsn = _aligned(ws)
    ev = None if events is None else (ctypes.c_void_p * len(events))(*events)
    args = [ctypes.byref(layer), _ptr(x), _ptr(gates), _ptr(dy), _ptr(z_save), _ptr(topk_ids), T, k,
            beta, P, s, _ptr(rs["counts"]), _ptr(rs["block_offsets"]), _ptr(rs["row_to_slot"]),
            _ptr(rs["slot_to_row"]), _ptr(owner), _ptr(block_worker), _ptr(dx), _ptr(dw1),
            _ptr(dw2)]
    rest = [_ptr(status), wsp, wsn, exec_flags(two_phase, split, fp8_act), ev, _ptr(timeline),
            _stream()]
    if dlogp is None:
        _check(load().moe_backward(*args, *rest))
    else:
        _require_device(dlogp)
        _expect(dlogp, torch.float32, T * k, "dlogp")
        _check(load().moe_backward_gates(*args, _ptr(dlogp), *rest))


# ---- around the layer: router, gate gradients, norms, optimizer ---------------

# These calls take a few microseconds on the GPU, so their checks are kept cheap: device and
# stream come from torch's own raw queries, and pointers travel as plain numbers.

def _here(first, *rest):
    """Every tensor given is on the current device; that device's current stream."""
    dev = first.get_device()                    # -1: not on a GPU
    for t in rest:
        if t is not None and t.get_device() != dev:
            dev = -1
    if dev < 0 or dev != torch.cuda.current_device():
        raise MoeError("all buffers must be tensors on the current device")
    return torch._C._cuda_getCurrentRawStream(dev)


def _at(t):
    return None if t is None else t.data_ptr()


def _ws_at(ws):
    if ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise MoeError("ws: expected contiguous uint8")
    p = ws.data_ptr()
    off = -p % 256
    return p + off, max(ws.numel() - off, 0)


_INT_MAX = 2 ** 31 - 1


def _int(n, name):
    """n, refused where a C int does not hold it: ctypes would cut it down without a word."""
    if not -_INT_MAX <= n <= _INT_MAX:
        raise MoeError(f"{name}: {n} is beyond a 32-bit int")
    return n


def _rows(t, T, cols, dtype, name):
    """Row stride of a [T][cols] matrix whose rows' elements lie side by side."""
    if t.dtype == dtype and t.shape == (T, cols) and T <= _INT_MAX:
        stride = t.stride()
        if stride[1] == 1 and cols <= stride[0] <= _INT_MAX:
            return stride[0]
    if t.dtype != dtype:
        raise MoeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] != T or t.shape[1] != cols:
        raise MoeError(f"{name}: expected {(T, cols)}, got {tuple(t.shape)}")
    _int(T, f"rows of {name}")
    _int(cols, f"columns of {name}")
    if T == 0 or (T == 1 and (cols <= 1 or t.stride(1) == 1)):
        return cols
    ld = t.stride(0)
    if (cols > 1 and t.stride(1) != 1) or ld < cols:
        raise MoeError(f"{name}: strides {tuple(t.stride())} are not those of rows of {cols}")
    return _int(ld, f"row stride of {name}")


def _vector(t, n, dtype, name):
    if t.dtype != dtype or t.numel() < n or not t.is_contiguous():
        raise MoeError(f"{name}: expected {n} contiguous elements of {dtype}, got "
                       f"{tuple(t.shape)} of {t.dtype}")


def _mask_at(mask, T):
    if mask is None:
        return None
    if mask.dtype not in (torch.uint8, torch.bool):
        raise MoeError(f"mask: expected uint8 or bool, got {mask.dtype}")
    _vector(mask, T, mask.dtype, "mask")
    return mask.data_ptr()


_CODES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def _dtype_code(dtype, name):
    code = _CODES.get(dtype)
    if code is None:
        raise MoeError(f"{name}: unsupported element type {dtype}")
    return code


def make_router(E, k, dtype=torch.float32, score="softmax", renorm=True, scale=1.0) -> Router:
    """A top-k router of logits [T][E] of this dtype (moe_router)."""
    if score not in SCORES:
        raise MoeError(f"score {score!r}: one of {sorted(SCORES)}")
    r = Router(_int(E, "E"), _int(k, "k"), _dtype_code(dtype, "logits"), SCORES[score], int(bool(renorm)), scale)
    if load().moe_router_workspace_size(ctypes.byref(r), 0) == 0:
        raise MoeError(f"router of E={E}, k={k}, scale={scale} is not supported")
    return r


def alloc_router(router: Router, T, device):
    f32, i32 = dict(dtype=torch.float32, device=device), dict(dtype=torch.int32, device=device)
    return {"topk_ids": torch.empty((T, router.k), **i32), "gates": torch.empty((T, router.k), **f32),
            "counts": torch.empty(router.E, **i32), "prob_sum": torch.empty(router.E, **f32),
            "live": torch.empty(1, **i32), "losses": torch.empty(2, **f32)}


def router_workspace(router: Router, T, device) -> torch.Tensor:
    n = int(load().moe_router_workspace_size(ctypes.byref(router), _int(T, "T")))
    if n == 0:
        raise MoeError("moe_router_workspace_size rejected the sizes")
    return torch.empty(n + 256, dtype=torch.uint8, device=device)


def make_choice(router: Router, bias=None, groups=1, top_groups=None, group_score="top2") -> Choice:
    """A choice by values, score + bias [E] (float32, read when a forward pass runs; None: 0), in the
    top_groups (None: all) best of so many groups of consecutive experts, by their best ("max") or the
    sum of their two best ("top2")."""
    if group_score not in GROUP_SCORES:
        raise MoeError(f"group_score {group_score!r}: one of {sorted(GROUP_SCORES)}")
    top_groups = groups if top_groups is None else top_groups
    if not (1 <= top_groups <= groups <= 64 and router.E % groups == 0 and
            router.k <= top_groups * (router.E // groups)):
        raise MoeError(f"{top_groups} of {groups} groups are not supported for E={router.E}, k={router.k}")
    if bias is not None:
        _vector(bias, router.E, torch.float32, "bias")
    c = Choice(_at(bias), groups, top_groups, GROUP_SCORES[group_score])
    c.tensor = bias
    return c


def router_bias_update(bias, counts, rate):
    """The balancing step of a choice's bias, in place: bias += rate * sign(mean(counts) - counts)."""
    st = _here(bias, counts)
    E = _int(bias.numel(), "bias")
    _vector(bias, E, torch.float32, "bias")
    _vector(counts, E, torch.int32, "counts")
    _check(load().moe_router_bias_update(_at(counts), E, rate, _at(bias), st))
    return bias


def _router_args(router, logits, mask):
    if logits.dim() != 2:
        raise MoeError(f"logits: expected [T][E], got {tuple(logits.shape)}")
    T = logits.shape[0]
    dt = torch.float32 if router.dtype == MOE_F32 else torch.bfloat16
    ld = _rows(logits, T, router.E, dt, "logits")
    _mask_at(mask, T)
    return T, ld, dt


def router_forward(router: Router, logits, out: dict, ws, status, mask=None, choice=None):
    """Routes logits [T][E] into out (alloc_router): ids, gates, counts, prob_sum, live, losses.  choice
    (make_choice, for a router of as many experts): by values instead of logits."""
    if choice is not None and choice.tensor is not None:
        _vector(choice.tensor, router.E, torch.float32, "bias")
        _here(choice.tensor)
    st = _here(logits, mask, ws, status, *out.values())
    T, ld, _ = _router_args(router, logits, mask)
    _vector(out["topk_ids"], T * router.k, torch.int32, "topk_ids")
    _vector(out["gates"], T * router.k, torch.float32, "gates")
    _vector(out["counts"], router.E, torch.int32, "counts")
    _vector(out["prob_sum"], router.E, torch.float32, "prob_sum")
    _vector(out["live"], 1, torch.int32, "live")
    _vector(out["losses"], 2, torch.float32, "losses")
    _vector(status, 1, torch.int32, "status")
    wsp, wsn = _ws_at(ws)
    args = (_at(logits), ld, _at(mask), T, _at(out["topk_ids"]), _at(out["gates"]), _at(out["counts"]),
            _at(out["prob_sum"]), _at(out["live"]), _at(out["losses"]), _at(status), wsp, wsn, st)
    if choice is None:
        _check(load().moe_router_forward(ctypes.byref(router), *args))
    else:
        _check(load().moe_router_forward_choice(ctypes.byref(router), ctypes.byref(choice), *args))
    return out


def router_backward(router: Router, logits, out: dict, dlogp, dlosses, dlogits, mask=None):
    """dlogits [T][E] from dlogp [T][k] (log-form gate gradients) and dlosses [2], each nullable;
    out: router_forward's on the same logits and mask."""
    st = _here(logits, mask, dlogp, dlosses, dlogits, out["topk_ids"], out["counts"], out["live"])
    T, ld, dt = _router_args(router, logits, mask)
    ld_out = _rows(dlogits, T, router.E, dt, "dlogits")
    _vector(out["topk_ids"], T * router.k, torch.int32, "topk_ids")
    _vector(out["counts"], router.E, torch.int32, "counts")
    _vector(out["live"], 1, torch.int32, "live")
    if dlogp is not None:
        _vector(dlogp, T * router.k, torch.float32, "dlogp")
    if dlosses is not None:
        _vector(dlosses, 2, torch.float32, "dlosses")
    _check(load().moe_router_backward(
        ctypes.byref(router), _at(logits), ld, _at(mask), T, _at(out["topk_ids"]), _at(dlogp),
        _at(out["counts"]), _at(out["live"]), _at(dlosses), _at(dlogits), ld_out, st))
    return dlogits


def gate_grad(z, dz, row_to_slot, dlogp):
    """Log-form gate gradients <dU, U> of routed rows from rows [G, U] and [dG, dU] [slots][2 d_ff]."""
    st = _here(z, dz, row_to_slot, dlogp)
    if z.dim() != 2 or z.shape[1] % 2:
        raise MoeError(f"z: expected [slots][2 d_ff], got {tuple(z.shape)}")
    slots, two = z.shape
    code = _dtype_code(z.dtype, "z")
    _vector(z, z.numel(), z.dtype, "z")
    _vector(dz, z.numel(), z.dtype, "dz")
    rows = _int(row_to_slot.numel(), "rows")
    _int(slots, "slots")
    _int(two, "columns of z")
    _vector(row_to_slot, rows, torch.int32, "row_to_slot")
    _vector(dlogp, rows, torch.float32, "dlogp")
    _check(load().moe_gate_grad(_at(z), _at(dz), code, _at(row_to_slot), rows, slots, two // 2,
                                _at(dlogp), st))
    return dlogp


def quantize_int8_rows(src, codes, scales):
    """Rows of src [rows][cols] (float32 or bfloat16) as int8 codes [rows][cols] with a scale each: a weight's
    channels, or activations' tokens."""
    st = _here(src, codes, scales)
    if src.dim() != 2:
        raise MoeError(f"src: expected [rows][cols], got {tuple(src.shape)}")
    rows, cols = src.shape
    ld = _rows(src, rows, cols, src.dtype, "src")
    _vector(codes, rows * cols, torch.int8, "codes")
    _vector(scales, rows, torch.float32, "scales")
    _check(load().moe_quantize_int8_rows(_at(src), ld, _dtype_code(src.dtype, "src"), rows, cols, _at(codes), _at(scales), st))
    return codes


def norm_workspace(T, d, device) -> torch.Tensor:
    n = int(load().moe_norm_workspace_size(_int(T, "T"), _int(d, "d")))
    if n == 0:
        raise MoeError("moe_norm_workspace_size rejected the sizes")
    return torch.empty(n + 256, dtype=torch.uint8, device=device)


def _norm_desc(rows, w, gate, alpha, eps, mask, name):
    """The moe_norm of rows [T][d] of the tensor `rows`, and their row stride."""
    if rows.dim() != 2:
        raise MoeError(f"{name}: expected [T][d], got {tuple(rows.shape)}")
    T, d = rows.shape
    code = _dtype_code(rows.dtype, name)
    w_code = _dtype_code(w.dtype, "w")
    if w_code != code and w_code != MOE_F32:
        raise MoeError(f"w: expected float32 or {rows.dtype}, got {w.dtype}")
    if w.shape != (d,) or not w.is_contiguous():
        raise MoeError(f"w: expected {d} contiguous elements, got {tuple(w.shape)}")
    kind = GATE_NONE
    if gate is not None:
        if gate.shape == (T, 1):
            kind = GATE_TOKEN
        elif gate.shape == (d,):
            kind = GATE_FEATURE
        else:
            raise MoeError(f"gate: expected {(T, 1)} or {(d,)}, got {tuple(gate.shape)}")
        _vector(gate, 0, torch.float32, "gate")
    N = Norm(T, d, code, w_code, kind, alpha, eps, w.data_ptr(),
             None if gate is None else gate.data_ptr(), _mask_at(mask, T))
    return N, T, d, _rows(rows, T, d, rows.dtype, name)


def _opt_rows(t, T, d, dtype, name):
    if t is None:
        return None, 0
    return t.data_ptr(), _rows(t, T, d, dtype, name)


def norm_in(x, w, eps, n, rstd, u=None, gate=None, alpha=1.0, r=None, mask=None):
    """Before the block: r = x + alpha gate u, n = w r / rms(r); rstd [T] for the backward pass.
    mask [T]: 0 where a row is padding (r = x, n = 0); the gradients take the same."""
    st = _here(x, w, n, rstd, u, gate, r, mask)
    N, T, d, ldx = _norm_desc(x, w, gate, alpha, eps, mask, "x")
    _vector(rstd, T, torch.float32, "rstd")
    _check(load().moe_norm_in(ctypes.byref(N), _at(x), ldx, *_opt_rows(u, T, d, x.dtype, "u"),
                              *_opt_rows(r, T, d, x.dtype, "r"), _at(n),
                              _rows(n, T, d, x.dtype, "n"), _at(rstd), st))
    return n


def _norm_grads(T, d, gate, dw, dgate, ws):
    _vector(dw, d, torch.float32, "dw")
    if gate is not None and dgate is not None:
        _vector(dgate, gate.numel(), torch.float32, "dgate")
    return _ws_at(ws)


def norm_in_backward(dn, r, w, rstd, dx, dw, ws, dr=None, u=None, gate=None, alpha=1.0, du=None,
                     dgate=None, mask=None):
    """Gradients of norm_in: dx (r's and x's), dw, and with u also du and dgate (shaped like gate)."""
    st = _here(dn, r, w, rstd, dx, dw, ws, dr, u, gate, du, dgate, mask)
    N, T, d, ldr = _norm_desc(r, w, gate, alpha, 1.0, mask, "r")
    dt = r.dtype
    _vector(rstd, T, torch.float32, "rstd")
    wsp, wsn = _norm_grads(T, d, gate, dw, dgate, ws)
    _check(load().moe_norm_in_backward(
        ctypes.byref(N), _at(dn), _rows(dn, T, d, dt, "dn"), *_opt_rows(dr, T, d, dt, "dr"),
        _at(r), ldr, *_opt_rows(u, T, d, dt, "u"), _at(rstd), _at(dx),
        _rows(dx, T, d, dt, "dx"), *_opt_rows(du, T, d, dt, "du"), _at(dw), _at(dgate), wsp, wsn,
        st))
    return dx


def norm_out(y, x, w, eps, out, rstd, gate=None, alpha=1.0, mask=None):
    """After the block: out = x + alpha gate w y / rms(y); rstd [T] for the backward pass.
    mask [T]: 0 where a row is padding (out = x); the gradients take the same."""
    st = _here(y, x, w, out, rstd, gate, mask)
    N, T, d, ldy = _norm_desc(y, w, gate, alpha, eps, mask, "y")
    _vector(rstd, T, torch.float32, "rstd")
    _check(load().moe_norm_out(ctypes.byref(N), _at(y), ldy, _at(x),
                               _rows(x, T, d, y.dtype, "x"), _at(out),
                               _rows(out, T, d, y.dtype, "out"), _at(rstd), st))
    return out


def norm_out_backward(dout, y, w, rstd, dy, dw, ws, gate=None, alpha=1.0, dgate=None, mask=None):
    """Gradients of norm_out: dy, dw and dgate (shaped like gate); x's is dout."""
    st = _here(dout, y, w, rstd, dy, dw, ws, gate, dgate, mask)
    N, T, d, ldy = _norm_desc(y, w, gate, alpha, 1.0, mask, "y")
    _vector(rstd, T, torch.float32, "rstd")
    wsp, wsn = _norm_grads(T, d, gate, dw, dgate, ws)
    _check(load().moe_norm_out_backward(
        ctypes.byref(N), _at(dout), _rows(dout, T, d, y.dtype, "dout"), _at(y), ldy, _at(rstd),
        _at(dy), _rows(dy, T, d, y.dtype, "dy"), _at(dw), _at(dgate), wsp, wsn, st))
    return dy


class PreparedAdamw:
    """A prepared list of tensors (moe_adamw_prepare), its workspace, and the tensors, which it keeps
    alive."""

    def __init__(self, c_list, ws, keep):
        self.list, self.ws, self.keep = c_list, ws, keep


def make_adamw(p, g, m, v, m_scale=None, v_scale=None, master=None) -> PreparedAdamw:
    """Prepares AdamW over lists of contiguous tensors: parameters p, gradients g, states m and v
    (float32, or uint8 e4m3 codes with m_scale and v_scale, one float32 per 128 elements), and
    optionally master (a float32 copy, or None, for each bfloat16 parameter)."""
    count = len(p)
    lists = {"g": g, "m": m, "v": v, "m_scale": m_scale, "v_scale": v_scale, "master": master}
    for name, ts in lists.items():
        if ts is not None and len(ts) != count:
            raise MoeError(f"{name}: expected {count} tensors, got {len(ts)}")
    bits = 8 if m_scale is not None else 32
    if (m_scale is None) != (v_scale is None):
        raise MoeError("m_scale and v_scale go together")
    state = torch.uint8 if bits == 8 else torch.float32
    arr = (AdamwTensor * max(count, 1))()
    keep = []
    for i in range(count):
        n = p[i].numel()
        ts = [p[i], g[i], m[i], v[i]]
        _vector(p[i], n, p[i].dtype, f"p[{i}]")
        _vector(g[i], n, g[i].dtype, f"g[{i}]")
        _vector(m[i], n, state, f"m[{i}]")
        _vector(v[i], n, state, f"v[{i}]")
        a = arr[i]
        if bits == 8:
            blocks = -(-n // ADAMW_BLOCK)
            _vector(m_scale[i], blocks, torch.float32, f"m_scale[{i}]")
            _vector(v_scale[i], blocks, torch.float32, f"v_scale[{i}]")
            ts += [m_scale[i], v_scale[i]]
            a.m_scale, a.v_scale = m_scale[i].data_ptr(), v_scale[i].data_ptr()
        if master is not None and master[i] is not None:
            _vector(master[i], n, torch.float32, f"master[{i}]")
            ts.append(master[i])
            a.master = master[i].data_ptr()
        _here(*ts)
        keep += ts
        a.p, a.g, a.m, a.v, a.n = (p[i].data_ptr(), g[i].data_ptr(), m[i].data_ptr(),
                                   v[i].data_ptr(), n)
        a.p_dtype, a.g_dtype = _dtype_code(p[i].dtype, f"p[{i}]"), _dtype_code(g[i].dtype, f"g[{i}]")
    size = int(load().moe_adamw_workspace_size(count))
    if size == 0 and count:
        raise MoeError("moe_adamw_workspace_size rejected the list")
    ws = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
    wsp, wsn = _aligned(ws)
    out = AdamwList()
    _check(load().moe_adamw_prepare(arr, count, bits, ctypes.byref(out), wsp, wsn, _stream()))
    return PreparedAdamw(out, ws, keep)


def adamw(prepared: PreparedAdamw, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1,
          seed=0, grad_scale=None):
    """One AdamW step on every tensor of the list.  step (from 1 on) is a number or an int32 tensor,
    lr a number or a float32 tensor, grad_scale nothing or a float32 tensor: tensors are read when
    the step runs, also in a captured graph."""
    h = AdamwHyper(0.0, beta1, beta2, eps, weight_decay, 0, seed & 0xFFFFFFFF)
    if isinstance(step, torch.Tensor):
        _here(step)
        _vector(step, 1, torch.int32, "step")
        h.step_dev = step.data_ptr()
    else:
        h.step = _int(step, "step")
    if isinstance(lr, torch.Tensor):
        _here(lr)
        _vector(lr, 1, torch.float32, "lr")
        h.lr_dev = lr.data_ptr()
    else:
        h.lr = lr
    if grad_scale is not None:
        _here(grad_scale)
        _vector(grad_scale, 1, torch.float32, "grad_scale")
        h.grad_scale = grad_scale.data_ptr()
    _check(load().moe_adamw(ctypes.byref(prepared.list), ctypes.byref(h), _here(prepared.ws)))


class PreparedGrads:
    """A prepared list of gradients (moe_grad_prepare), its workspace, and the gradients, which it keeps
    alive."""

    def __init__(self, c_list, ws, keep):
        self.list, self.ws, self.keep = c_list, ws, keep
        sizes = [(t.data_ptr(), t.nbytes) for t in (*keep, ws)]
        spans = sorted((at, at + n) for at, n in sizes if n)
        self.begins = [b for b, _ in spans]
        self.ends = list(itertools.accumulate((e for _, e in spans), max))    # the furthest of those up to each

    def holds(self, at):
        """Whether the 4 bytes at an address lie in a gradient or the workspace, or a part of them."""
        i = bisect_left(self.begins, at + 4)
        return i > 0 and self.ends[i - 1] > at


def make_grads(grads) -> PreparedGrads:
    """Prepares a list of contiguous gradients (float32 or bfloat16) for grad_norm and grad_scale.  A list
    of its own: it may hold the gradients of several optimizers."""
    grads = list(grads)
    count = len(grads)
    arr = (GradTensor * max(count, 1))()
    for i, g in enumerate(grads):
        _vector(g, g.numel(), g.dtype, f"grads[{i}]")
        _here(g)
        arr[i].g, arr[i].n, arr[i].dtype = g.data_ptr(), g.numel(), _dtype_code(g.dtype, f"grads[{i}]")
    size = int(load().moe_grad_workspace_size(count))
    if size == 0:
        raise MoeError("moe_grad_workspace_size rejected the list")
    ws = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
    wsp, wsn = _aligned(ws)
    out = GradList()
    _check(load().moe_grad_prepare(arr, count, ctypes.byref(out), wsp, wsn, _stream()))
    return PreparedGrads(out, ws, grads)


def grad_norm(prepared: PreparedGrads, max_norm, norm, scale, status, mult=1.0):
    """The list's norm (times |mult|) into norm [1], and into scale [1] what brings mult times the gradients
    to a norm of max_norm at most: adamw's grad_scale, or grad_scale's.  mult is a number or a float32
    tensor, read when the call runs."""
    st = _here(prepared.ws, norm, scale, status)
    c = Clip(max_norm, 1.0, None)
    if isinstance(mult, torch.Tensor):
        _here(mult)
        _vector(mult, 1, torch.float32, "mult")
        c.mult_dev = mult.data_ptr()
    else:
        c.mult = mult
    _vector(norm, 1, torch.float32, "norm")
    _vector(scale, 1, torch.float32, "scale")
    _vector(status, 1, torch.int32, "status")
    _check(load().moe_grad_norm(ctypes.byref(prepared.list), ctypes.byref(c), _at(norm), _at(scale), _at(status), st))
    return norm


def grad_scale(prepared: PreparedGrads, scale):
    """Every gradient of the list times scale [1], which lies in none of them, in place."""
    at = scale.data_ptr()
    if prepared.holds(at):
        raise MoeError("scale: lies in the list's memory")
    st = _here(prepared.ws, scale)
    _vector(scale, 1, torch.float32, "scale")
    _check(load().moe_grad_scale(ctypes.byref(prepared.list), at, st))


class Events:
    """n hipEvent_t created through the library, for stage timing on the
    stream the kernels run on."""

    def __init__(self, n):
        lib = load()
        self.ev = []
        for _ in range(n):
            p = ctypes.c_void_p()
            _check(lib.moe_event_create(ctypes.byref(p)))
            self.ev.append(p.value)

    def elapsed_ms(self, i, j) -> float:
        ms = ctypes.c_float()
        _check(load().moe_event_elapsed_ms(ctypes.c_void_p(self.ev[i]), ctypes.c_void_p(self.ev[j]),
                                          ctypes.byref(ms)))
        return float(ms.value)

    def record(self, i):
        _check(load().moe_event_record(ctypes.c_void_p(self.ev[i]), _stream()))

    def __del__(self):
        try:
            lib = load()
            for e in self.ev:
                lib.moe_event_destroy(ctypes.c_void_p(e))
        except Exception:
            pass


def device_info():
    a, b, c = _I(), _I(), _I()
    _check(load().moe_device_info(ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
    return {"num_cus": a.value, "num_xcds": b.value, "gemm_wg_per_cu": c.value}

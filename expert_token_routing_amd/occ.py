"""Thin ctypes binding of libocc.so (the C ABI in include/occ.h).

Argument marshalling only: every function checks the tensors it is handed
(device, dtype, shape, contiguity), passes their device addresses and the
current HIP stream to the C entry point of the same name, and raises
``OccError`` on a non-OK status.  All computation happens in the library's
kernels; when the library is missing this module raises instead of falling
back to anything else.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

from .workloads import Workload

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libocc.so")

OCC_OK, OCC_ERR_INVALID_ARG, OCC_ERR_UNSUPPORTED, OCC_ERR_WORKSPACE, OCC_ERR_HIP = range(5)
OCC_F32, OCC_BF16 = 0, 1
OCC_PRUNE_OFF, OCC_PRUNE_TRAVERSE, OCC_PRUNE_GROUPSUM, OCC_PRUNE_SIMILARITY = 0, 1, 2, 3
OCC_FLAG_TRAIN = 1
OCC_FLAG_DETERMINISTIC = 2
OCC_NOALLOC_SCRATCH_BYTES = 128 << 20
OCC_GATE_NONE, OCC_GATE_CHANNEL, OCC_GATE_TOKEN = 0, 1, 2
OCC_ADAMW_32BIT, OCC_ADAMW_8BIT = 0, 1
OCC_SCORE_SOFTMAX, OCC_SCORE_SIGMOID = 0, 1
OCC_ADAMW_BLOCK = 256
BSTAGES = ["dispatch", "dgrad_down", "dgrad_up", "shared", "combine", "wgrad_down", "wgrad_up",
           "route"]
OCC_BSTAGE_COUNT = len(BSTAGES)
STAGES = ["route", "brim", "dispatch", "shared_up", "shared_down", "gemm_up", "gemm_down_first",
          "gemm_down_rest", "combine"]
OCC_STAGE_COUNT = len(STAGES)

EXPORTED = ["occ_status_string", "occ_workspace_size", "occ_route",
            "occ_similarity_accumulate", "occ_similarity_rank", "occ_route_similarity",
            "occ_build_brim", "occ_moe_forward", "occ_moe_forward_routed", "occ_gate",
            "occ_moe_forward_gated", "occ_moe_backward", "occ_forward_views",
            "occ_coactivation_stats", "occ_place_experts", "occ_events_create",
            "occ_events_destroy", "occ_event_elapsed_ms", "occ_moe_forward_noalloc",
            "occ_block_workspace_size", "occ_block_norm", "occ_block_norm_backward",
            "occ_balance_loss", "occ_balance_backward", "occ_gate_backward", "occ_adamw_step",
            "occ_route_scored", "occ_route_scored_backward", "occ_route_bias_step",
            "occ_quantize_int8", "occ_int8_workspace_size", "occ_moe_forward_int8"]


class OccError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


class LayerDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "d", "Ne", "k", "Nd", "F", "n_shared", "F_shared", "prune_rule",
                 "prune_groups", "dtype", "flags")]


class Brim(ctypes.Structure):
    _fields_ = [("brim0", ctypes.c_void_p), ("sfd_off", ctypes.c_void_p),
                ("epd_off", ctypes.c_void_p), ("epd_src", ctypes.c_void_p),
                ("epd_w", ctypes.c_void_p), ("tok_epd", ctypes.c_void_p),
                ("brim1", ctypes.c_void_p), ("down_rows", ctypes.c_void_p),
                ("first_cnt", ctypes.c_void_p), ("tile_off", ctypes.c_void_p)]


class ForwardView(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("brim", Brim),
                ("x_sfd", ctypes.c_void_p), ("epd", ctypes.c_void_p),
                ("sfd_out", ctypes.c_void_p), ("h_shared", ctypes.c_void_p),
                ("y_shared", ctypes.c_void_p)]


class NormDesc(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("scale", ctypes.c_float), ("gate", ctypes.c_int32)]


class BalanceDesc(ctypes.Structure):
    _fields_ = [("balance", ctypes.c_float), ("group", ctypes.c_float), ("z", ctypes.c_float)]


class AdamwDesc(ctypes.Structure):
    _fields_ = ([("state", ctypes.c_int32), ("grad_dtype", ctypes.c_int32)] +
                [(n, ctypes.c_double) for n in
                 ("lr", "beta1", "beta2", "eps", "weight_decay", "grad_scale")] +
                [("step", ctypes.c_int64)])


class ScoreDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("score", "top_groups", "group_best",
                                               "renormalise")] + [("scale", ctypes.c_float)])


class Int8Pointers(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("gate", "up", "down", "gate_scale", "up_scale",
                                               "down_scale")]


class AdamwTensor(ctypes.Structure):
    _fields_ = ([("n", ctypes.c_int64)] +
                [(n, ctypes.c_void_p) for n in
                 ("p", "g", "m", "v", "m_scale", "v_scale", "p_out", "m_out", "v_out",
                  "m_scale_out", "v_scale_out", "p_bf16")])


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OccError(OCC_ERR_HIP, f"{LIB_PATH} is missing; run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        dp = ctypes.POINTER(LayerDesc)
        sigs = {
            "occ_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "occ_workspace_size": ([dp, ctypes.POINTER(sz)], ctypes.c_int),
            "occ_route": ([dp, vp, vp, vp, vp, vp], ctypes.c_int),
            "occ_similarity_accumulate": ([i32, i32, vp, vp, vp], ctypes.c_int),
            "occ_similarity_rank": ([i32, vp, vp, vp, vp], ctypes.c_int),
            "occ_route_similarity": ([dp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
            "occ_build_brim": ([dp, vp, vp, vp, ctypes.c_int, vp, sz, ctypes.POINTER(Brim), vp],
                               ctypes.c_int),
            "occ_moe_forward": ([dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp],
                                ctypes.c_int),
            "occ_moe_forward_noalloc": ([dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp],
                                        ctypes.c_int),
            "occ_moe_forward_routed": ([dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                        vp, vp], ctypes.c_int),
            "occ_gate": ([dp, vp, vp, vp, vp], ctypes.c_int),
            "occ_moe_backward": ([dp] + [vp] * 20 + [sz, vp, vp], ctypes.c_int),
            "occ_moe_forward_gated": ([dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp],
                                      ctypes.c_int),
            "occ_forward_views": ([dp, vp, ctypes.POINTER(ForwardView)], ctypes.c_int),
            "occ_coactivation_stats": ([dp, vp, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
            "occ_place_experts": ([vp, i32, i32, vp], ctypes.c_int),
            "occ_block_workspace_size": ([dp, ctypes.POINTER(sz)], ctypes.c_int),
            "occ_block_norm": ([dp, ctypes.POINTER(NormDesc)] + [vp] * 8, ctypes.c_int),
            "occ_block_norm_backward": ([dp, ctypes.POINTER(NormDesc)] + [vp] * 13 + [sz, vp],
                                        ctypes.c_int),
            "occ_balance_loss": ([dp, ctypes.POINTER(BalanceDesc)] + [vp] * 8 + [sz, vp],
                                 ctypes.c_int),
            "occ_balance_backward": ([dp, ctypes.POINTER(BalanceDesc)] + [vp] * 4 +
                                     [ctypes.c_float, vp, vp, vp], ctypes.c_int),
            "occ_gate_backward": ([dp] + [vp] * 7 + [sz, vp], ctypes.c_int),
            "occ_adamw_step": ([ctypes.POINTER(AdamwDesc), vp, i32, vp, vp], ctypes.c_int),
            "occ_route_scored": ([dp, ctypes.POINTER(ScoreDesc)] + [vp] * 6, ctypes.c_int),
            "occ_route_scored_backward": ([dp, ctypes.POINTER(ScoreDesc)] + [vp] * 6,
                                          ctypes.c_int),
            "occ_route_bias_step": ([dp, ctypes.c_float] + [vp] * 6 + [sz, vp], ctypes.c_int),
            "occ_quantize_int8": ([ctypes.c_int64, i32, i32] + [vp] * 4, ctypes.c_int),
            "occ_int8_workspace_size": ([dp, ctypes.POINTER(sz)], ctypes.c_int),
            "occ_moe_forward_int8": ([dp] + [vp] * 4 + [ctypes.POINTER(Int8Pointers)] * 2 +
                                     [vp, vp, sz, vp], ctypes.c_int),
            "occ_events_create": ([i32, vp], ctypes.c_int),
            "occ_events_destroy": ([i32, vp], ctypes.c_int),
            "occ_event_elapsed_ms": ([vp, vp, ctypes.POINTER(ctypes.c_float)], ctypes.c_int),
        }
        for name, (args, res) in sigs.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().occ_status_string(status).decode()
    except OccError:
        return f"status {status}"


def _check(status: int, what: str):
    if status != OCC_OK:
        raise OccError(status, what)


def desc_of(w: Workload, **over) -> LayerDesc:
    f = dict(T=w.T, d=w.d, Ne=w.Ne, k=w.k, Nd=w.Nd, F=w.F, n_shared=w.n_shared,
             F_shared=w.F_shared, prune_rule=w.prune_rule, prune_groups=w.prune_groups,
             dtype=w.dtype, flags=0)
    f.update(over)
    return LayerDesc(**f)


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t: torch.Tensor | None, name: str, dtype=None, shape=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


def _host_i32(a, name: str, shape=None) -> np.ndarray:
    a = np.ascontiguousarray(a, dtype=np.int32)
    if shape is not None and a.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {a.shape}")
    return a


def _hp(a: np.ndarray) -> ctypes.c_void_p:
    return ctypes.c_void_p(a.ctypes.data)


def occ_workspace_size(desc: LayerDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().occ_workspace_size(ctypes.byref(desc), ctypes.byref(n)), "occ_workspace_size")
    return n.value


def alloc_workspace(desc: LayerDesc, device="cuda") -> torch.Tensor:
    """A device byte tensor of occ_workspace_size bytes (torch allocations are 256-aligned)."""
    return torch.empty(occ_workspace_size(desc), dtype=torch.uint8, device=device)


def occ_route(desc: LayerDesc, logits, placement, ids, w, stream=None):
    T, Ne, k = desc.T, desc.Ne, desc.k
    L = _host_i32(placement, "placement", (desc.Nd, Ne // desc.Nd))
    _check(lib().occ_route(ctypes.byref(desc), _dev(logits, "logits", torch.float32, (T, Ne)),
                           _hp(L), _dev(ids, "ids", torch.int32, (T, k)),
                           _dev(w, "w", torch.float32, (T, k)), _stream(stream)), "occ_route")


def occ_similarity_accumulate(logits, gram, stream=None):
    """gram (Ne x Ne fp64) += logits^T logits, one batch (appendix A.3)."""
    T, Ne = logits.shape
    _check(lib().occ_similarity_accumulate(
        T, Ne, _dev(logits, "logits", torch.float32, (T, Ne)),
        _dev(gram, "gram", torch.float64, (Ne, Ne)), _stream(stream)), "occ_similarity_accumulate")


def occ_similarity_rank(gram, rank, t2=None, stream=None):
    """Squared cosine table (optional t2) and per-row ranking from a Gram matrix."""
    Ne = gram.shape[0]
    _check(lib().occ_similarity_rank(
        Ne, _dev(gram, "gram", torch.float64, (Ne, Ne)),
        _dev(t2, "t2", torch.float64, (Ne, Ne)), _dev(rank, "rank", torch.int32, (Ne, Ne)),
        _stream(stream)), "occ_similarity_rank")


def occ_route_similarity(desc: LayerDesc, logits, placement, sim_rank, ids, w, stream=None):
    T, Ne, k = desc.T, desc.Ne, desc.k
    L = _host_i32(placement, "placement", (desc.Nd, Ne // desc.Nd))
    _check(lib().occ_route_similarity(
        ctypes.byref(desc), _dev(logits, "logits", torch.float32, (T, Ne)), _hp(L),
        _dev(sim_rank, "sim_rank", torch.int32, (Ne, Ne)), _dev(ids, "ids", torch.int32, (T, k)),
        _dev(w, "w", torch.float32, (T, k)), _stream(stream)), "occ_route_similarity")


def occ_build_brim(desc: LayerDesc, ids, w, placement, workspace, dense_brim1=True,
                   stream=None) -> Brim:
    T, k = desc.T, desc.k
    L = _host_i32(placement, "placement", (desc.Nd, desc.Ne // desc.Nd))
    out = Brim()
    _check(lib().occ_build_brim(ctypes.byref(desc), _dev(ids, "ids", torch.int32, (T, k)),
                                _dev(w, "w", torch.float32, (T, k)), _hp(L), int(dense_brim1),
                                _dev(workspace, "workspace", torch.uint8),
                                workspace.numel(), ctypes.byref(out), _stream(stream)),
           "occ_build_brim")
    return out


def occ_moe_forward(desc: LayerDesc, x, logits, placement, w_gate, w_up, w_down, ws_gate, ws_up,
                    ws_down, y, workspace, stage_events=None, stream=None):
    T, d, Ne, F = desc.T, desc.d, desc.Ne, desc.F
    dt = torch.bfloat16 if desc.dtype == OCC_BF16 else torch.float32
    L = _host_i32(placement, "placement", (desc.Nd, Ne // desc.Nd))
    nsh, Fsh = desc.n_shared, desc.F_shared
    sh = [None, None, None]
    if nsh > 0:
        sh = [_dev(ws_gate, "ws_gate", dt, (nsh, Fsh, d)), _dev(ws_up, "ws_up", dt, (nsh, Fsh, d)),
              _dev(ws_down, "ws_down", dt, (nsh, d, Fsh))]
    ev = None
    if stage_events is not None:
        ev = (ctypes.c_void_p * (OCC_STAGE_COUNT + 1))(*stage_events)
    _check(lib().occ_moe_forward(
        ctypes.byref(desc), _dev(x, "x", dt, (T, d)),
        _dev(logits, "logits", torch.float32, (T, Ne)), _hp(L),
        _dev(w_gate, "w_gate", dt, (Ne, F, d)), _dev(w_up, "w_up", dt, (Ne, F, d)),
        _dev(w_down, "w_down", dt, (Ne, d, F)), *sh, _dev(y, "y", dt, (T, d)),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(),
        ctypes.cast(ev, ctypes.c_void_p) if ev is not None else None, _stream(stream)),
        "occ_moe_forward")


def occ_moe_forward_noalloc(desc: LayerDesc, x, logits, placement, w_gate, w_up, w_down, ws_gate,
                            ws_up, ws_down, y, stage_events=None, stream=None):
    """occ_moe_forward with the library's static per-GPU scratch array as the
    workspace (nothing allocated; shapes up to OCC_NOALLOC_SCRATCH_BYTES of
    workspace; calls on one GPU must not overlap)."""
    T, d, Ne, F = desc.T, desc.d, desc.Ne, desc.F
    dt = torch.bfloat16 if desc.dtype == OCC_BF16 else torch.float32
    L = _host_i32(placement, "placement", (desc.Nd, Ne // desc.Nd))
    nsh, Fsh = desc.n_shared, desc.F_shared
    sh = [None, None, None]
    if nsh > 0:
        sh = [_dev(ws_gate, "ws_gate", dt, (nsh, Fsh, d)), _dev(ws_up, "ws_up", dt, (nsh, Fsh, d)),
              _dev(ws_down, "ws_down", dt, (nsh, d, Fsh))]
    ev = None
    if stage_events is not None:
        ev = (ctypes.c_void_p * (OCC_STAGE_COUNT + 1))(*stage_events)
    _check(lib().occ_moe_forward_noalloc(
        ctypes.byref(desc), _dev(x, "x", dt, (T, d)),
        _dev(logits, "logits", torch.float32, (T, Ne)), _hp(L),
        _dev(w_gate, "w_gate", dt, (Ne, F, d)), _dev(w_up, "w_up", dt, (Ne, F, d)),
        _dev(w_down, "w_down", dt, (Ne, d, F)), *sh, _dev(y, "y", dt, (T, d)),
        ctypes.cast(ev, ctypes.c_void_p) if ev is not None else None, _stream(stream)),
        "occ_moe_forward_noalloc")


def occ_moe_forward_routed(desc: LayerDesc, x, ids, w, placement, w_gate, w_up, w_down, ws_gate,
                           ws_up, ws_down, y, workspace, stage_events=None, stream=None):
    T, d, Ne, F, k = desc.T, desc.d, desc.Ne, desc.F, desc.k
    dt = torch.bfloat16 if desc.dtype == OCC_BF16 else torch.float32
    L = _host_i32(placement, "placement", (desc.Nd, Ne // desc.Nd))
    nsh, Fsh = desc.n_shared, desc.F_shared
    sh = [None, None, None]
    if nsh > 0:
        sh = [_dev(ws_gate, "ws_gate", dt, (nsh, Fsh, d)), _dev(ws_up, "ws_up", dt, (nsh, Fsh, d)),
              _dev(ws_down, "ws_down", dt, (nsh, d, Fsh))]
    ev = None
    if stage_events is not None:
        ev = (ctypes.c_void_p * (OCC_STAGE_COUNT + 1))(*stage_events)
    _check(lib().occ_moe_forward_routed(
        ctypes.byref(desc), _dev(x, "x", dt, (T, d)), _dev(ids, "ids", torch.int32, (T, k)),
        _dev(w, "w", torch.float32, (T, k)), _hp(L),
        _dev(w_gate, "w_gate", dt, (Ne, F, d)), _dev(w_up, "w_up", dt, (Ne, F, d)),
        _dev(w_down, "w_down", dt, (Ne, d, F)), *sh, _dev(y, "y", dt, (T, d)),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(),
        ctypes.cast(ev, ctypes.c_void_p) if ev is not None else None, _stream(stream)),
        "occ_moe_forward_routed")


def occ_gate(desc: LayerDesc, x, w_router, logits, stream=None):
    T, d, Ne = desc.T, desc.d, desc.Ne
    dt = torch.bfloat16 if desc.dtype == OCC_BF16 else torch.float32
    _check(lib().occ_gate(ctypes.byref(desc), _dev(x, "x", dt, (T, d)),
                          _dev(w_router, "w_router", dt, (Ne, d)),
                          _dev(logits, "logits", torch.float32, (T, Ne)), _stream(stream)),
           "occ_gate")


def occ_moe_forward_gated(desc: LayerDesc, x, w_router, placement, w_gate, w_up, w_down, ws_gate,
                          ws_up, ws_down, y, workspace, stage_events=None, stream=None):
    T, d, Ne, F = desc.T, desc.d, desc.Ne, desc.F
    dt = torch.bfloat16 if desc.dtype == OCC_BF16 else torch.float32
    L = _host_i32(placement, "placement", (desc.Nd, Ne // desc.Nd))
    nsh, Fsh = desc.n_shared, desc.F_shared
    sh = [None, None, None]
    if nsh > 0:
        sh = [_dev(ws_gate, "ws_gate", dt, (nsh, Fsh, d)), _dev(ws_up, "ws_up", dt, (nsh, Fsh, d)),
              _dev(ws_down, "ws_down", dt, (nsh, d, Fsh))]
    ev = None
    if stage_events is not None:
        ev = (ctypes.c_void_p * (OCC_STAGE_COUNT + 1))(*stage_events)
    _check(lib().occ_moe_forward_gated(
        ctypes.byref(desc), _dev(x, "x", dt, (T, d)), _dev(w_router, "w_router", dt, (Ne, d)),
        _hp(L), _dev(w_gate, "w_gate", dt, (Ne, F, d)), _dev(w_up, "w_up", dt, (Ne, F, d)),
        _dev(w_down, "w_down", dt, (Ne, d, F)), *sh, _dev(y, "y", dt, (T, d)),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(),
        ctypes.cast(ev, ctypes.c_void_p) if ev is not None else None, _stream(stream)),
        "occ_moe_forward_gated")


def occ_moe_backward(desc: LayerDesc, dy, x, logits, placement, w_gate, w_up, w_down, ws_gate,
                     ws_up, ws_down, dx, dw_gate, dw_up, dw_down, dws_gate, dws_up, dws_down,
                     dw, dlogits, workspace, stage_events=None, stream=None):
    """Backward pass; the workspace must hold a training forward's state."""
    T, d, Ne, F, k = desc.T, desc.d, desc.Ne, desc.F, desc.k
    dt = torch.bfloat16 if desc.dtype == OCC_BF16 else torch.float32
    f32 = torch.float32
    L = _host_i32(placement, "placement", (desc.Nd, Ne // desc.Nd))
    nsh, Fsh = desc.n_shared, desc.F_shared
    sh = [None] * 6
    if nsh > 0:
        sh = [_dev(ws_gate, "ws_gate", dt, (nsh, Fsh, d)), _dev(ws_up, "ws_up", dt, (nsh, Fsh, d)),
              _dev(ws_down, "ws_down", dt, (nsh, d, Fsh)),
              _dev(dws_gate, "dws_gate", f32, (nsh, Fsh, d)),
              _dev(dws_up, "dws_up", f32, (nsh, Fsh, d)),
              _dev(dws_down, "dws_down", f32, (nsh, d, Fsh))]
    ev = None
    if stage_events is not None:
        ev = (ctypes.c_void_p * (OCC_BSTAGE_COUNT + 1))(*stage_events)
    _check(lib().occ_moe_backward(
        ctypes.byref(desc), _dev(dy, "dy", dt, (T, d)), _dev(x, "x", dt, (T, d)),
        _dev(logits, "logits", f32, (T, Ne)), _hp(L),
        _dev(w_gate, "w_gate", dt, (Ne, F, d)), _dev(w_up, "w_up", dt, (Ne, F, d)),
        _dev(w_down, "w_down", dt, (Ne, d, F)), *sh[:3], _dev(dx, "dx", dt, (T, d)),
        _dev(dw_gate, "dw_gate", f32, (Ne, F, d)), _dev(dw_up, "dw_up", f32, (Ne, F, d)),
        _dev(dw_down, "dw_down", f32, (Ne, d, F)), *sh[3:], _dev(dw, "dw", f32, (T, k)),
        _dev(dlogits, "dlogits", f32, (T, Ne)), _dev(workspace, "workspace", torch.uint8),
        workspace.numel(), ctypes.cast(ev, ctypes.c_void_p) if ev is not None else None,
        _stream(stream)), "occ_moe_backward")


# ---- around the layer in a training step ----

_TORCH = {OCC_F32: torch.float32, OCC_BF16: torch.bfloat16}


def _addr(t: torch.Tensor | None, name: str, dtype, shape: tuple, index: int):
    """The address of a contiguous device tensor of this type and shape on the call's device."""
    if t is None:
        return None
    if (index < 0 or t.get_device() != index or t.dtype is not dtype or t.shape != shape
            or not t.is_contiguous()):
        _dev(t, name, dtype, shape)  # says which check fails
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{index}")
    return t.data_ptr()


def _device(t: torch.Tensor | None) -> int:
    """The device of a call's tensors, taken from one that it cannot do without (-1: the tensor
    is missing, which the library refuses, or is a host tensor, which _addr refuses)."""
    return -1 if t is None else t.get_device()


def _current(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the current stream's handle without an object around it (0.1 us instead of 1.1, where a small
# call takes 7)
_current = getattr(torch._C, "_cuda_getCurrentRawStream", _current)


def _queue(what: str, fn, index: int, stream, *args):
    """fn(*args, stream) with device `index` as the current one."""
    if index < 0:
        raise OccError(OCC_ERR_INVALID_ARG, what)
    if stream is None:
        stream = _current(index)
    elif stream.device.index != index:
        raise ValueError(f"{what}: tensors on cuda:{index}, stream on {stream.device}")
    else:
        stream = stream.cuda_stream
    if torch.cuda.current_device() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != OCC_OK:
        raise OccError(status, what)


def occ_block_workspace_size(desc: LayerDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().occ_block_workspace_size(ctypes.byref(desc), ctypes.byref(n)),
           "occ_block_workspace_size")
    return n.value


def alloc_block_workspace(desc: LayerDesc, device="cuda") -> torch.Tensor:
    """A device byte tensor of occ_block_workspace_size bytes."""
    return torch.empty(occ_block_workspace_size(desc), dtype=torch.uint8, device=device)


def _ws(workspace, index: int):
    if workspace is None:
        return None, 0
    return (_addr(workspace, "workspace", torch.uint8, (workspace.numel(),), index),
            workspace.numel())


def _norm_gate(desc: LayerDesc, opt: NormDesc):
    """The type and shape of a gate (its gradient has that shape in fp32)."""
    if opt.gate == OCC_GATE_TOKEN:
        return torch.float32, (desc.T,)
    return _TORCH.get(desc.dtype), (desc.d,)


def occ_block_norm(desc: LayerDesc, opt: NormDesc, x, y, w_post, gate, w_pre, r, h, stream=None):
    """r = x + scale gate w_post n(y), h = w_pre n(r); y, w_post, gate and w_pre with h may be
    None (see occ.h)."""
    dt, d, i = _TORCH.get(desc.dtype), (desc.d,), _device(x)
    rows = (desc.T, desc.d)
    _queue("occ_block_norm", lib().occ_block_norm, i, stream, desc, opt,
           _addr(x, "x", dt, rows, i), _addr(y, "y", dt, rows, i),
           _addr(w_post, "w_post", dt, d, i), _addr(gate, "gate", *_norm_gate(desc, opt), i),
           _addr(w_pre, "w_pre", dt, d, i), _addr(r, "r", dt, rows, i), _addr(h, "h", dt, rows, i))


def occ_block_norm_backward(desc: LayerDesc, opt: NormDesc, dr, dh, r, y, w_post, gate, w_pre, dx,
                            dy, dw_post, dgate, dw_pre, workspace, stream=None):
    """Gradients of occ_block_norm from dr and dh (r: its r, or its x without y)."""
    dt, d, i, f32 = _TORCH.get(desc.dtype), (desc.d,), _device(dx), torch.float32
    rows, (gate_dt, gate_shape) = (desc.T, desc.d), _norm_gate(desc, opt)
    _queue("occ_block_norm_backward", lib().occ_block_norm_backward, i, stream, desc, opt,
           _addr(dr, "dr", dt, rows, i), _addr(dh, "dh", dt, rows, i), _addr(r, "r", dt, rows, i),
           _addr(y, "y", dt, rows, i), _addr(w_post, "w_post", dt, d, i),
           _addr(gate, "gate", gate_dt, gate_shape, i), _addr(w_pre, "w_pre", dt, d, i),
           _addr(dx, "dx", dt, rows, i), _addr(dy, "dy", dt, rows, i),
           _addr(dw_post, "dw_post", f32, d, i), _addr(dgate, "dgate", f32, gate_shape, i),
           _addr(dw_pre, "dw_pre", f32, d, i), *_ws(workspace, i))


def _mask(valid, T: int, index: int):
    if valid is not None and valid.dtype is not torch.bool and valid.dtype is not torch.uint8:
        raise ValueError(f"valid must be torch.bool or torch.uint8, got {valid.dtype}")
    return None if valid is None else _addr(valid, "valid", valid.dtype, (T,), index)


def _place(desc: LayerDesc, placement):
    """The placement as host int32 in bytes (the library reads it within the call; an array's
    address costs 1 us more), or None."""
    if placement is None:
        return None
    return _host_i32(placement, "placement", (desc.Nd, desc.Ne // max(desc.Nd, 1))).tobytes()


def occ_balance_loss(desc: LayerDesc, opt: BalanceDesc, logits, ids, valid, placement, counts,
                     probs, loss, workspace, stream=None):
    """Router losses [sum, balance, group, z], mean probabilities, and the counts (Ne, then the
    valid tokens)."""
    T, Ne, f32, i32, i = desc.T, desc.Ne, torch.float32, torch.int32, _device(logits)
    place = _place(desc, placement)
    _queue("occ_balance_loss", lib().occ_balance_loss, i, stream, desc, opt,
           _addr(logits, "logits", f32, (T, Ne), i), _addr(ids, "ids", i32, (T, desc.k), i),
           _mask(valid, T, i), place, _addr(counts, "counts", i32, (Ne + 1,), i),
           _addr(probs, "probs", f32, (Ne,), i), _addr(loss, "loss", f32, (4,), i),
           *_ws(workspace, i))


def occ_balance_backward(desc: LayerDesc, opt: BalanceDesc, logits, valid, placement, counts,
                         dloss: float, dlogits_in, dlogits, stream=None):
    """dlogits = dlogits_in + dloss times the losses' gradient in the logits."""
    T, Ne, f32, i = desc.T, desc.Ne, torch.float32, _device(logits)
    place = _place(desc, placement)
    _queue("occ_balance_backward", lib().occ_balance_backward, i, stream, desc, opt,
           _addr(logits, "logits", f32, (T, Ne), i), _mask(valid, T, i), place,
           _addr(counts, "counts", torch.int32, (Ne + 1,), i), dloss,
           _addr(dlogits_in, "dlogits_in", f32, (T, Ne), i),
           _addr(dlogits, "dlogits", f32, (T, Ne), i))


def occ_gate_backward(desc: LayerDesc, dlogits, x, w_router, dx_in, dx, dw_router, workspace,
                      stream=None):
    """dx = dx_in + dlogits w_router, dw_router = dlogits^T x; dx or dw_router may be None."""
    T, d, Ne, dt, f32 = desc.T, desc.d, desc.Ne, _TORCH.get(desc.dtype), torch.float32
    i = _device(dlogits)
    _queue("occ_gate_backward", lib().occ_gate_backward, i, stream, desc,
           _addr(dlogits, "dlogits", f32, (T, Ne), i), _addr(x, "x", dt, (T, d), i),
           _addr(w_router, "w_router", dt, (Ne, d), i), _addr(dx_in, "dx_in", dt, (T, d), i),
           _addr(dx, "dx", dt, (T, d), i), _addr(dw_router, "dw_router", f32, (Ne, d), i),
           *_ws(workspace, i))


class AdamwTensors:
    """The tensors of an optimizer, laid out once for occ_adamw_step (which holds no state of
    its own): a list of dicts of device tensors

      p (fp32), g (opt.grad_dtype), m, v (fp32, or torch.float8_e4m3fn with 8-bit states and
      then m_scale, v_scale: one fp32 per OCC_ADAMW_BLOCK elements), and optionally p_bf16, the
      bf16 copy to write, and p_out, m_out, v_out, m_scale_out, v_scale_out (in place otherwise).

    The table keeps the tensors alive."""

    def __init__(self, opt: AdamwDesc, tensors: list[dict]):
        self.state, self.grad_dtype = opt.state, opt.grad_dtype
        self.tensors = [dict(t) for t in tensors]
        self.table = (AdamwTensor * max(len(self.tensors), 1))()
        self.index = None  # the tensors' device
        eight, f32 = opt.state == OCC_ADAMW_8BIT, torch.float32
        state = torch.float8_e4m3fn if eight else f32
        names = {n for n, _ in AdamwTensor._fields_[1:]}
        for k, (t, row) in enumerate(zip(self.tensors, self.table)):
            if set(t) - names:
                raise ValueError(f"tensor {k}: unknown entries {sorted(set(t) - names)}")

            def address(name, dtype, shape):
                return _addr(t.get(name), f"tensor {k}: {name}", dtype, shape, self.index)

            if t.get("p") is None:
                raise ValueError(f"tensor {k}: p must be given")
            if self.index is None:
                self.index = _device(t["p"])
            shape = tuple(t["p"].shape)
            row.n = t["p"].numel()
            units = (-(-row.n // OCC_ADAMW_BLOCK),)
            for name, dtype in (("p", f32), ("g", _TORCH.get(opt.grad_dtype)), ("m", state),
                                ("v", state), ("m_scale", f32), ("v_scale", f32)):
                scale = name.endswith("_scale")
                given = t.get(name) is not None
                if given == (scale and not eight):
                    raise ValueError(f"tensor {k}: {name} must be {'None' if given else 'given'}")
                want = units if scale else shape
                setattr(row, name, address(name, dtype, want))
                if name == "g":
                    continue
                out = name + "_out"
                if t.get(out) is None:
                    setattr(row, out, getattr(row, name))
                elif given:
                    setattr(row, out, address(out, dtype, want))
                else:
                    raise ValueError(f"tensor {k}: {out} must be None")
            row.p_bf16 = address("p_bf16", torch.bfloat16, shape)


def occ_adamw_step(opt: AdamwDesc, tensors: AdamwTensors, dynamic=None, stream=None):
    """One AdamW step over the tensors; dynamic: None or a device fp32 tensor
    [lr, step, grad_scale] that replaces the descriptor's."""
    if opt.state != tensors.state or opt.grad_dtype != tensors.grad_dtype:
        raise ValueError("the descriptor's state and grad_dtype differ from the table's")
    if not tensors.tensors:
        return
    _queue("occ_adamw_step", lib().occ_adamw_step, tensors.index, stream, opt, tensors.table,
           len(tensors.tensors), _addr(dynamic, "dynamic", torch.float32, (3,), tensors.index))


# ---- routing by scores ----

def occ_route_scored(desc: LayerDesc, opt: ScoreDesc, logits, bias, placement, ids, w,
                     stream=None):
    """The k experts of the best scores (softmax or sigmoid, plus a bias for the choice) in the
    best groups, and their weights; bias may be None, placement too when all groups are used."""
    T, Ne, f32, i = desc.T, desc.Ne, torch.float32, _device(logits)
    place = _place(desc, placement)
    _queue("occ_route_scored", lib().occ_route_scored, i, stream, desc, opt,
           _addr(logits, "logits", f32, (T, Ne), i), _addr(bias, "bias", f32, (Ne,), i), place,
           _addr(ids, "ids", torch.int32, (T, desc.k), i), _addr(w, "w", f32, (T, desc.k), i))


def occ_route_scored_backward(desc: LayerDesc, opt: ScoreDesc, logits, ids, dw, dlogits_in,
                              dlogits, stream=None):
    """dlogits = dlogits_in + the gradient of occ_route_scored's weights in the logits."""
    T, Ne, f32, i = desc.T, desc.Ne, torch.float32, _device(logits)
    _queue("occ_route_scored_backward", lib().occ_route_scored_backward, i, stream, desc, opt,
           _addr(logits, "logits", f32, (T, Ne), i),
           _addr(ids, "ids", torch.int32, (T, desc.k), i), _addr(dw, "dw", f32, (T, desc.k), i),
           _addr(dlogits_in, "dlogits_in", f32, (T, Ne), i),
           _addr(dlogits, "dlogits", f32, (T, Ne), i))


def occ_route_bias_step(desc: LayerDesc, rate: float, ids, valid, bias_in, counts, bias,
                        workspace, stream=None):
    """bias = bias_in + rate sign(mean load - load), with the counts (Ne, then the valid
    tokens); bias may be bias_in."""
    Ne, f32, i32, i = desc.Ne, torch.float32, torch.int32, _device(ids)
    _queue("occ_route_bias_step", lib().occ_route_bias_step, i, stream, desc, rate,
           _addr(ids, "ids", i32, (desc.T, desc.k), i), _mask(valid, desc.T, i),
           _addr(bias_in, "bias_in", f32, (Ne,), i), _addr(counts, "counts", i32, (Ne + 1,), i),
           _addr(bias, "bias", f32, (Ne,), i), *_ws(workspace, i))


# ---- experts in 8-bit integers ----

_OCC = {torch.float32: OCC_F32, torch.bfloat16: OCC_BF16}


def occ_quantize_int8(x, q, scale, stream=None):
    """Rows of x (its last dimension; bf16 or fp32) as int8 codes q and a scale each."""
    i = _device(x)
    if x.dim() < 1 or x.dtype not in _OCC:
        raise ValueError("x must be rows of torch.float32 or torch.bfloat16")
    cols = x.shape[-1]
    _queue("occ_quantize_int8", lib().occ_quantize_int8, i, stream,
           x.numel() // cols if cols else 0, cols, _OCC[x.dtype],
           _addr(x, "x", x.dtype, x.shape, i), _addr(q, "q", torch.int8, x.shape, i),
           _addr(scale, "scale", torch.float32, x.shape[:-1], i))


class Int8Experts:
    """The weights of experts in 8 bits, laid out once: device tensors gate and up (N x F x d
    int8), down (N x d x F int8), gate_scale and up_scale (N x F fp32), down_scale (N x d fp32),
    as occ_quantize_int8 makes them of bf16 weights.  Keeps the tensors alive."""

    def __init__(self, gate, up, down, gate_scale, up_scale, down_scale):
        self.index, self.shape = _device(gate), tuple(gate.shape)
        if len(self.shape) != 3:
            raise ValueError(f"gate must be N x F x d, got {self.shape}")
        N, F, d = self.shape
        self.tensors = (gate, up, down, gate_scale, up_scale, down_scale)
        i8, f32 = torch.int8, torch.float32
        wants = (("gate", i8, (N, F, d)), ("up", i8, (N, F, d)), ("down", i8, (N, d, F)),
                 ("gate_scale", f32, (N, F)), ("up_scale", f32, (N, F)),
                 ("down_scale", f32, (N, d)))
        for t, (name, _, _) in zip(self.tensors, wants):
            if t is None:
                raise ValueError(f"{name} must be given")
        self.table = Int8Pointers(*[_addr(t, name, dtype, shape, self.index)
                                    for t, (name, dtype, shape) in zip(self.tensors, wants)])


def _int8_table(group, name: str, shape: tuple, index: int):
    if group is None:
        return None
    if group.shape != shape or group.index != index:
        raise ValueError(f"{name} are {group.shape} on cuda:{group.index}, expected {shape} on "
                         f"cuda:{index}")
    return group.table


def occ_int8_workspace_size(desc: LayerDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().occ_int8_workspace_size(ctypes.byref(desc), ctypes.byref(n)),
           "occ_int8_workspace_size")
    return n.value


def alloc_int8_workspace(desc: LayerDesc, device="cuda") -> torch.Tensor:
    """A device byte tensor of occ_int8_workspace_size bytes."""
    return torch.empty(occ_int8_workspace_size(desc), dtype=torch.uint8, device=device)


def occ_moe_forward_int8(desc: LayerDesc, x, ids, w, placement, experts: Int8Experts,
                         shared: Int8Experts | None, y, workspace, stream=None):
    """The layer on a given routing with experts in 8 bits (x and y bf16)."""
    T, d, k, i = desc.T, desc.d, desc.k, _device(x)
    bf16, place = torch.bfloat16, _place(desc, placement)
    _queue("occ_moe_forward_int8", lib().occ_moe_forward_int8, i, stream, desc,
           _addr(x, "x", bf16, (T, d), i), _addr(ids, "ids", torch.int32, (T, k), i),
           _addr(w, "w", torch.float32, (T, k), i), place,
           _int8_table(experts, "experts", (desc.Ne, desc.F, d), i),
           _int8_table(shared, "shared experts", (desc.n_shared, desc.F_shared, d), i),
           _addr(y, "y", bf16, (T, d), i), *_ws(workspace, i))


def occ_forward_views(desc: LayerDesc, workspace) -> ForwardView:
    out = ForwardView()
    _check(lib().occ_forward_views(ctypes.byref(desc), _dev(workspace, "workspace", torch.uint8),
                                   ctypes.byref(out)), "occ_forward_views")
    return out


def occ_coactivation_stats(desc: LayerDesc, ids, placement, C, P, n_sfd, ct, intra, stream=None):
    T, k, Ne = desc.T, desc.k, desc.Ne
    L = _host_i32(placement, "placement", (desc.Nd, Ne // desc.Nd))
    _check(lib().occ_coactivation_stats(
        ctypes.byref(desc), _dev(ids, "ids", torch.int32, (T, k)), _hp(L),
        _dev(C, "C", torch.int32, (Ne, Ne)), _dev(P, "P", torch.float32, (Ne, Ne)),
        _dev(n_sfd, "n_sfd", torch.int64, (1,)), _dev(ct, "ct", torch.float64, (1,)),
        _dev(intra, "intra", torch.float64, (1,)), _stream(stream)), "occ_coactivation_stats")


def occ_place_experts(C, Nd: int) -> np.ndarray:
    """Algorithm 1 on host counts C (Ne x Ne); returns the (Nd, Ne/Nd) placement."""
    Cc = np.ascontiguousarray(C, dtype=np.int32)
    Ne = Cc.shape[0]
    if Cc.shape != (Ne, Ne):
        raise ValueError("C must be square")
    L = np.empty((Nd, Ne // max(Nd, 1)), np.int32)
    _check(lib().occ_place_experts(_hp(Cc), Ne, Nd, _hp(L)), "occ_place_experts")
    return L


class StageEvents:
    """stages+1 HIP events for a call's stage timing (occ_moe_forward's by
    default; OCC_BSTAGE_COUNT for occ_moe_backward)."""

    def __init__(self, stages: int = OCC_STAGE_COUNT):
        self.n = stages + 1
        self.arr = (ctypes.c_void_p * self.n)()
        _check(lib().occ_events_create(self.n, self.arr), "occ_events_create")

    @property
    def handles(self):
        return list(self.arr)

    def elapsed_ms(self) -> list[float]:
        out = []
        for i in range(self.n - 1):
            ms = ctypes.c_float(0)
            _check(lib().occ_event_elapsed_ms(self.arr[i], self.arr[i + 1], ctypes.byref(ms)),
                   "occ_event_elapsed_ms")
            out.append(ms.value)
        return out

    def close(self):
        if self.arr is not None:
            lib().occ_events_destroy(self.n, self.arr)
            self.arr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def ws_view(workspace: torch.Tensor, ptr: int, shape, dtype: torch.dtype) -> torch.Tensor:
    """A torch view of a buffer the library placed inside `workspace` (a device
    address returned by occ_build_brim / occ_forward_views)."""
    off = int(ptr) - workspace.data_ptr()
    numel = int(np.prod(shape)) if len(shape) else 1
    nbytes = numel * torch.empty(0, dtype=dtype).element_size()
    if off < 0 or off + nbytes > workspace.numel():
        raise ValueError("address outside the workspace")
    return workspace[off:off + nbytes].view(dtype).view(*shape)

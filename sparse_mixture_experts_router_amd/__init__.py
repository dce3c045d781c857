"""Sparse mixture-of-experts layer (forward and backward) on AMD MI355X (gfx950).

A thin ctypes binding of ``libmoe.so``: every function below only marshals
PyTorch tensors (device memory) and the current HIP stream into the C ABI
declared in ``include/moe.h``; every step of the layer runs in the library's
HIP kernels.  There is no CPU fallback: if the library is not built, calls
raise.
"""

from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional, Sequence

import torch

__all__ = [
    "LIB_PATH", "MOE_OK", "MOE_ERR_INVALID_ARG", "MOE_ERR_UNSUPPORTED", "MOE_ERR_WORKSPACE",
    "MOE_ERR_HIP", "MOE_F32", "MOE_BF16", "MOE_WEIGHTS_DTYPE", "MOE_WEIGHTS_FP8_E4M3", "STAGES", "BACKWARD_STAGES",
    "MoEError", "MoEConfig", "MoEWeights",
    "MoERouting", "lib", "make_config", "moe_workspace_size", "moe_status_string",
    "alloc_workspace", "moe_route", "moe_layer_forward", "moe_balance_stats", "MoELayer",
    "MoEGrads", "moe_backward_workspace_size", "alloc_backward_workspace", "moe_layer_backward",
    "moe_update_select_bias", "MoEPlanInfo", "moe_forward_plan", "moe_layer_forward_noalloc",
    "NOALLOC_SCRATCH_BYTES",
    "ACTIVATIONS", "CHECKPOINT_BLOCK", "MoELinearConfig", "MoELinearArgs", "MoELinearGradArgs",
    "make_linear_config", "moe_linear_workspace_size", "alloc_linear_workspace",
    "moe_grouped_linear", "moe_linear_backward_workspace_size", "alloc_linear_backward_workspace",
    "moe_grouped_linear_backward", "moe_checkpoint_pack", "moe_checkpoint_unpack",
    "moe_group_workspace_size", "alloc_group_workspace", "moe_group_rows", "moe_combine",
    "moe_combine_backward",
]

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
MOE_F32, MOE_BF16 = 0, 1
MOE_WEIGHTS_DTYPE, MOE_WEIGHTS_FP8_E4M3 = 0, 1
NOALLOC_SCRATCH_BYTES = 64 << 20   # MOE_NOALLOC_SCRATCH_BYTES of include/moe.h
_SCALES = ("w_gate_scale", "w_up_scale", "w_down_scale", "ws_gate_scale", "ws_up_scale",
           "ws_down_scale")
ACTIVATIONS = ("none", "relu", "gelu", "silu", "swiglu")   # moe_activation, in its order
CHECKPOINT_BLOCK = 64   # columns of a row that share one scale of an 8-bit checkpoint
STAGES = ("route", "permute", "expert_up", "expert_down", "combine")
BACKWARD_STAGES = ("route", "transpose_w", "recompute", "grad_h", "grad_x", "segments", "grad_w",
                   "grad_wr")


class MoEError(RuntimeError):
    def __init__(self, status: int, detail: str = ""):
        self.status = status
        msg = moe_status_string(status)
        super().__init__(f"{msg} ({detail})" if detail else msg)


class MoEConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("d_ff", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("weight_format", ctypes.c_int32)]


class MoEWeights(ctypes.Structure):
    _fields_ = [("w_router", ctypes.c_void_p), ("w_gate", ctypes.c_void_p),
                ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("ws_gate", ctypes.c_void_p), ("ws_up", ctypes.c_void_p),
                ("ws_down", ctypes.c_void_p), ("logit_bias", ctypes.c_void_p),
                ("select_bias", ctypes.c_void_p)] + [(n, ctypes.c_void_p) for n in _SCALES]


class MoERouting(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("topk_idx", ctypes.c_void_p),
                ("topk_gate", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("prob_sum", ctypes.c_void_p), ("f", ctypes.c_void_p), ("P", ctypes.c_void_p),
                ("aux", ctypes.c_void_p), ("balance_alpha", ctypes.c_float)]


class MoEPlanInfo(ctypes.Structure):
    _fields_ = [("up_kernel", ctypes.c_int32), ("up_tile_rows", ctypes.c_int32),
                ("down_kernel", ctypes.c_int32), ("down_tile_rows", ctypes.c_int32),
                ("route_split", ctypes.c_int32), ("route_kernel", ctypes.c_int32),
                ("down_split", ctypes.c_int32),
                ("tail_split_cols", ctypes.c_int32), ("up_narrow_tails", ctypes.c_int32),
                ("down_narrow_tails", ctypes.c_int32), ("compute_units", ctypes.c_int32),
                ("all_token_pass", ctypes.c_int32),
                ("split_plan_offset", ctypes.c_uint64), ("workspace_bytes", ctypes.c_uint64)]


class MoEGrads(ctypes.Structure):
    _fields_ = [("dx", ctypes.c_void_p), ("dw_router", ctypes.c_void_p),
                ("dlogit_bias", ctypes.c_void_p), ("dw_gate", ctypes.c_void_p),
                ("dw_up", ctypes.c_void_p), ("dw_down", ctypes.c_void_p),
                ("dws_gate", ctypes.c_void_p), ("dws_up", ctypes.c_void_p),
                ("dws_down", ctypes.c_void_p)]


class MoELinearConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("rows", "x_rows", "groups", "in_dim", "out_dim", "dtype", "weight_format",
                 "activation")]


class MoELinearArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("x", "row_index", "offsets", "w", "w_scale", "bias", "residual", "y", "z_codes",
                 "z_scale")]


class MoELinearGradArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("x", "row_index", "offsets", "w", "dy", "z_codes", "z_scale", "dx", "dw",
                 "dbias")]


_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run "
                               "`python -m sparse_mixture_experts_router_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
        cfgp, wp, rp = (ctypes.POINTER(MoEConfig), ctypes.POINTER(MoEWeights),
                        ctypes.POINTER(MoERouting))
        L.moe_workspace_size.argtypes = [cfgp]
        L.moe_workspace_size.restype = sz
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_route.argtypes = [cfgp, vp, wp, rp, vp, sz, vp]
        L.moe_route.restype = ctypes.c_int
        L.moe_layer_forward.argtypes = [cfgp, vp, wp, vp, rp, vp, sz, vp]
        L.moe_layer_forward.restype = ctypes.c_int
        L.moe_layer_forward_timed.argtypes = [cfgp, vp, wp, vp, rp, vp, sz, vp,
                                              ctypes.POINTER(vp)]
        L.moe_layer_forward_timed.restype = ctypes.c_int
        L.moe_balance_stats.argtypes = [i32, i32, i32, vp, vp, ctypes.c_float, vp, vp, vp, vp]
        L.moe_balance_stats.restype = ctypes.c_int
        L.moe_backward_workspace_size.argtypes = [cfgp]
        L.moe_backward_workspace_size.restype = sz
        L.moe_layer_backward.argtypes = [cfgp, vp, wp, vp, ctypes.c_float, ctypes.c_float,
                                         ctypes.POINTER(MoEGrads), vp, sz, vp]
        L.moe_layer_backward.restype = ctypes.c_int
        L.moe_layer_backward_timed.argtypes = L.moe_layer_backward.argtypes + [ctypes.POINTER(vp)]
        L.moe_layer_backward_timed.restype = ctypes.c_int
        L.moe_update_select_bias.argtypes = [i32, vp, ctypes.c_float, vp, vp]
        L.moe_update_select_bias.restype = ctypes.c_int
        L.moe_forward_plan.argtypes = [cfgp, ctypes.POINTER(MoEPlanInfo)]
        L.moe_forward_plan.restype = ctypes.c_int
        L.moe_layer_forward_noalloc.argtypes = [cfgp, vp, wp, vp, rp, vp]
        L.moe_layer_forward_noalloc.restype = ctypes.c_int
        lcfg = ctypes.POINTER(MoELinearConfig)
        i64 = ctypes.c_int64
        L.moe_group_workspace_size.argtypes = [i32, i32, i32]
        L.moe_group_workspace_size.restype = sz
        L.moe_group_rows.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_linear_workspace_size.argtypes = [lcfg]
        L.moe_linear_workspace_size.restype = sz
        L.moe_grouped_linear.argtypes = [lcfg, ctypes.POINTER(MoELinearArgs), vp, sz, vp]
        L.moe_linear_backward_workspace_size.argtypes = [lcfg]
        L.moe_linear_backward_workspace_size.restype = sz
        L.moe_grouped_linear_backward.argtypes = [lcfg, ctypes.POINTER(MoELinearGradArgs), vp, sz,
                                                  vp]
        L.moe_checkpoint_pack.argtypes = [i64, i32, i32, vp, vp, vp, vp]
        L.moe_checkpoint_unpack.argtypes = [i64, i32, i32, vp, vp, vp, vp]
        L.moe_combine.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, vp, vp]
        L.moe_combine_backward.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
        for fn in (L.moe_group_rows, L.moe_grouped_linear, L.moe_grouped_linear_backward,
                   L.moe_checkpoint_pack, L.moe_checkpoint_unpack, L.moe_combine,
                   L.moe_combine_backward):
            fn.restype = ctypes.c_int
        _LIB = L
    return _LIB


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def _check(status: int):
    if status != MOE_OK:
        raise MoEError(status, lib().moe_last_error().decode())


_TORCH_DTYPE = {MOE_BF16: torch.bfloat16, MOE_F32: torch.float32}


def make_config(T: int, d_model: int, n_experts: int, top_k: int, d_ff: int,
                n_shared: int = 0, dtype=torch.bfloat16, capacity: int = 0,
                weight_format: int = MOE_WEIGHTS_DTYPE) -> MoEConfig:
    """``capacity``: 0 = dropless, else the most (token, slot) assignments a
    routed expert takes per call (the rest are dropped).  ``weight_format``:
    MOE_WEIGHTS_FP8_E4M3 for expert weights given as uint8 E4M3 codes plus
    fp32 per-output-channel scales (``*_scale`` entries of the weights)."""
    code = MOE_BF16 if dtype in (torch.bfloat16, "bf16", MOE_BF16) else MOE_F32
    return MoEConfig(int(T), int(d_model), int(n_experts), int(top_k), int(d_ff),
                     int(n_shared), code, int(capacity), int(weight_format))


def moe_workspace_size(cfg: MoEConfig) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(cfg)))


def alloc_workspace(cfg: MoEConfig, device="cuda") -> torch.Tensor:
    n = moe_workspace_size(cfg)
    if n == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "configuration rejected")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_forward_plan(cfg: MoEConfig) -> Dict[str, int]:
    """How moe_layer_forward runs ``cfg`` on the current device (kernel
    choices, tile rows, reduction splits, and the workspace offset of the
    device-side split plan); see ``moe_forward_plan`` in include/moe.h."""
    info = MoEPlanInfo()
    _check(lib().moe_forward_plan(ctypes.byref(cfg), ctypes.byref(info)))
    return {name: int(getattr(info, name)) for name, _ in MoEPlanInfo._fields_}


def _ptr(t: Optional[torch.Tensor], dtype=None, name="tensor",
         numel: Optional[int] = None) -> Optional[int]:
    """Device address of ``t`` after checking placement, layout, dtype and,
    when ``numel`` is given, its element count: the C ABI sees only pointers,
    so a tensor of the wrong size would be read or written out of bounds."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, the configuration needs {numel}")
    return t.data_ptr()


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _weight_numels(cfg: MoEConfig) -> Dict[str, int]:
    """Element count of every weight, bias and scale that ``cfg`` implies."""
    N, d, F, S = cfg.n_experts, cfg.d_model, cfg.d_ff, cfg.n_shared
    return {"w_router": N * d, "w_gate": N * F * d, "w_up": N * F * d, "w_down": N * d * F,
            "ws_gate": S * F * d, "ws_up": S * F * d, "ws_down": S * d * F,
            "logit_bias": N, "select_bias": N,
            "w_gate_scale": N * F, "w_up_scale": N * F, "w_down_scale": N * d,
            "ws_gate_scale": S * F, "ws_up_scale": S * F, "ws_down_scale": S * d}


def _weights(cfg: MoEConfig, w: Dict[str, Optional[torch.Tensor]], experts=True) -> MoEWeights:
    dt = _TORCH_DTYPE[cfg.dtype]
    fp8 = cfg.weight_format == MOE_WEIGHTS_FP8_E4M3
    n = _weight_numels(cfg)
    args = {"w_router": _ptr(w.get("w_router"), dt, "w_router", n["w_router"])}
    if experts:
        for name in ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down"):
            args[name] = _ptr(w.get(name), torch.uint8 if fp8 else dt, name, n[name])
        if fp8:
            for name in _SCALES:
                args[name] = _ptr(w.get(name), torch.float32, name, n[name])
    args["logit_bias"] = _ptr(w.get("logit_bias"), torch.float32, "logit_bias", n["logit_bias"])
    args["select_bias"] = _ptr(w.get("select_bias"), torch.float32, "select_bias",
                               n["select_bias"])
    return MoEWeights(**args)


def _routing(cfg: MoEConfig, logits=None, topk_idx=None, topk_gate=None, counts=None,
             prob_sum=None, f=None, P=None, aux=None, alpha=0.01):
    T, N, k = cfg.T, cfg.n_experts, cfg.top_k
    return MoERouting(_ptr(logits, torch.float32, "logits", T * N),
                      _ptr(topk_idx, torch.int32, "topk_idx", T * k),
                      _ptr(topk_gate, torch.float32, "topk_gate", T * k),
                      _ptr(counts, torch.int32, "counts", N),
                      _ptr(prob_sum, torch.float32, "prob_sum", N),
                      _ptr(f, torch.float32, "f", N), _ptr(P, torch.float32, "P", N),
                      _ptr(aux, torch.float32, "aux", 2), float(alpha))


def moe_route(cfg: MoEConfig, x: torch.Tensor, weights: Dict[str, Optional[torch.Tensor]], *,
              topk_idx: torch.Tensor, topk_gate: torch.Tensor, workspace: torch.Tensor,
              logits=None, counts=None, prob_sum=None, f=None, P=None, aux=None, alpha=0.01,
              stream=None) -> None:
    """Routing only; see ``moe_route`` in include/moe.h."""
    w = _weights(cfg, weights, experts=False)
    r = _routing(cfg, logits, topk_idx, topk_gate, counts, prob_sum, f, P, aux, alpha)
    _check(lib().moe_route(ctypes.byref(cfg),
                           _ptr(x, _TORCH_DTYPE[cfg.dtype], "x", cfg.T * cfg.d_model),
                           ctypes.byref(w), ctypes.byref(r), _ptr(workspace, None, "workspace"),
                           workspace.numel(), _stream(stream)))


def moe_layer_forward(cfg: MoEConfig, x: torch.Tensor, weights: Dict[str, Optional[torch.Tensor]],
                      y: torch.Tensor, *, workspace: torch.Tensor, logits=None, topk_idx=None,
                      topk_gate=None, counts=None, prob_sum=None, f=None, P=None, aux=None,
                      alpha=0.01, stream=None,
                      stage_events: Optional[Sequence[torch.cuda.Event]] = None) -> None:
    """Whole layer forward into ``y``; see ``moe_layer_forward`` in include/moe.h.

    ``f``, ``P``, ``aux``: optional balance statistics written by the same
    call (``aux`` = [N sum f P, alpha N sum f P]).
    ``stage_events``: optional list of len(STAGES) + 1 ``torch.cuda.Event``
    (enable_timing=True) or None, recorded before each stage and after the
    last; None entries are skipped.
    """
    dt = _TORCH_DTYPE[cfg.dtype]
    w = _weights(cfg, weights)
    r = _routing(cfg, logits, topk_idx, topk_gate, counts, prob_sum, f, P, aux, alpha)
    td = cfg.T * cfg.d_model
    args = (ctypes.byref(cfg), _ptr(x, dt, "x", td), ctypes.byref(w), _ptr(y, dt, "y", td),
            ctypes.byref(r), _ptr(workspace, None, "workspace"), workspace.numel(),
            _stream(stream))
    if stage_events is None:
        _check(lib().moe_layer_forward(*args))
        return
    if len(stage_events) != len(STAGES) + 1:
        raise ValueError("need one event per stage plus one")
    s = torch.cuda.current_stream() if stream is None else stream
    for ev in stage_events:      # torch creates the HIP event on first record
        if ev is not None and not ev.cuda_event:
            ev.record(s)
    arr = (ctypes.c_void_p * len(stage_events))(
        *[None if ev is None else ev.cuda_event for ev in stage_events])
    _check(lib().moe_layer_forward_timed(*args, arr))


def moe_layer_forward_noalloc(cfg: MoEConfig, x: torch.Tensor,
                              weights: Dict[str, Optional[torch.Tensor]], y: torch.Tensor, *,
                              logits=None, topk_idx=None, topk_gate=None, counts=None,
                              prob_sum=None, f=None, P=None, aux=None, alpha=0.01,
                              stream=None) -> None:
    """moe_layer_forward without a workspace argument: the library's own
    per-GPU device array of NOALLOC_SCRATCH_BYTES serves as the workspace, so
    the call allocates nothing; see ``moe_layer_forward_noalloc`` in
    include/moe.h (larger configurations raise MOE_ERR_WORKSPACE; calls that
    overlap on one GPU race)."""
    dt = _TORCH_DTYPE[cfg.dtype]
    w = _weights(cfg, weights)
    r = _routing(cfg, logits, topk_idx, topk_gate, counts, prob_sum, f, P, aux, alpha)
    td = cfg.T * cfg.d_model
    _check(lib().moe_layer_forward_noalloc(ctypes.byref(cfg), _ptr(x, dt, "x", td),
                                           ctypes.byref(w), _ptr(y, dt, "y", td),
                                           ctypes.byref(r), _stream(stream)))


def moe_balance_stats(T: int, N: int, k: int, counts: torch.Tensor, prob_sum: torch.Tensor,
                      alpha: float, f: torch.Tensor, P: torch.Tensor, aux: torch.Tensor,
                      stream=None) -> None:
    """f = counts / (T k), P = prob_sum / T, aux = [N sum f P, alpha N sum f P]."""
    _check(lib().moe_balance_stats(
        int(T), int(N), int(k), _ptr(counts, torch.int32, "counts", N),
        _ptr(prob_sum, torch.float32, "prob_sum", N), float(alpha),
        _ptr(f, torch.float32, "f", N), _ptr(P, torch.float32, "P", N),
        _ptr(aux, torch.float32, "aux", 2), _stream(stream)))


def moe_backward_workspace_size(cfg: MoEConfig) -> int:
    return int(lib().moe_backward_workspace_size(ctypes.byref(cfg)))


def alloc_backward_workspace(cfg: MoEConfig, device="cuda") -> torch.Tensor:
    n = moe_backward_workspace_size(cfg)
    if n == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "configuration rejected")
    return torch.empty(n, dtype=torch.uint8, device=device)


_GRADS = ("dx", "dw_router", "dlogit_bias", "dw_gate", "dw_up", "dw_down", "dws_gate", "dws_up",
          "dws_down")


def _event_array(stage_events, n, stream):
    if len(stage_events) != n + 1:
        raise ValueError("need one event per stage plus one")
    s = torch.cuda.current_stream() if stream is None else stream
    for ev in stage_events:      # torch creates the HIP event on first record
        if ev is not None and not ev.cuda_event:
            ev.record(s)
    return (ctypes.c_void_p * len(stage_events))(
        *[None if ev is None else ev.cuda_event for ev in stage_events])


def moe_layer_backward(cfg: MoEConfig, x: torch.Tensor, weights: Dict[str, Optional[torch.Tensor]],
                       dy: torch.Tensor, grads: Dict[str, Optional[torch.Tensor]], *,
                       workspace: torch.Tensor, alpha: float = 0.01, aux_grad: float = 1.0,
                       stream=None,
                       stage_events: Optional[Sequence[torch.cuda.Event]] = None) -> None:
    """Gradients of sum(y * dy) + aux_grad * aux into ``grads`` (keys dx,
    dw_router, dlogit_bias, dw_gate, dw_up, dw_down, dws_*); see
    ``moe_layer_backward`` in include/moe.h.  ``stage_events``: as for
    moe_layer_forward, one per BACKWARD_STAGES entry plus one."""
    dt = _TORCH_DTYPE[cfg.dtype]
    w = _weights(cfg, weights)
    wn = _weight_numels(cfg)
    td = cfg.T * cfg.d_model
    gn = {"dx": td, "dw_router": wn["w_router"], "dlogit_bias": cfg.n_experts,
          "dw_gate": wn["w_gate"], "dw_up": wn["w_up"], "dw_down": wn["w_down"],
          "dws_gate": wn["ws_gate"], "dws_up": wn["ws_up"], "dws_down": wn["ws_down"]}
    g = MoEGrads(**{n: _ptr(grads.get(n), torch.float32 if n == "dlogit_bias" else dt, n, gn[n])
                    for n in _GRADS})
    args = (ctypes.byref(cfg), _ptr(x, dt, "x", td), ctypes.byref(w), _ptr(dy, dt, "dy", td),
            float(alpha), float(aux_grad), ctypes.byref(g), _ptr(workspace, None, "workspace"),
            workspace.numel(), _stream(stream))
    if stage_events is None:
        _check(lib().moe_layer_backward(*args))
    else:
        _check(lib().moe_layer_backward_timed(
            *args, _event_array(stage_events, len(BACKWARD_STAGES), stream)))


def moe_update_select_bias(counts: torch.Tensor, rate: float, select_bias: torch.Tensor,
                           stream=None) -> None:
    """select_bias += rate * sign(mean(counts) - counts), in place (fp32)."""
    n = int(counts.numel())
    _check(lib().moe_update_select_bias(
        n, _ptr(counts, torch.int32, "counts"), float(rate),
        _ptr(select_bias, torch.float32, "select_bias", n), _stream(stream)))


# ---------------------------------------------------------------- experts of one's own
_CODE = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}


def _dtype_code(t: torch.Tensor, name: str) -> int:
    try:
        return _CODE[t.dtype]
    except KeyError:
        raise ValueError(f"{name} has dtype {t.dtype}, expected bfloat16 or float32") from None


class _Call:
    """Marshals the tensors of one call, all on one device, and makes it there:
    the C ABI launches on the current device, which may be another one.

    A decode step makes several of these calls, each a few microseconds of GPU
    time, so this path is kept short: the raw handle of the current stream
    costs 0.1 us, ``torch.cuda.current_stream()`` 2.6 (of 8.5 for a call)."""

    __slots__ = ("device",)

    def __init__(self, first: torch.Tensor):
        self.device = first.get_device()   # -1: not on a GPU

    def ptr(self, t: Optional[torch.Tensor], dtype, name: str, shape) -> Optional[int]:
        if t is None:
            return None
        device = t.get_device()
        if device != self.device or device < 0:
            if device < 0:
                raise ValueError(f"{name} must be a device tensor")
            raise ValueError(f"{name} is on device {device}, expected {self.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def workspace(self, t: torch.Tensor) -> int:
        if t.get_device() != self.device or not t.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on device {self.device}")
        return t.data_ptr()

    def run(self, fn, stream, *args):
        if self.device < 0:
            raise ValueError("tensors must be device tensors")
        if torch._C._cuda_getDevice() == self.device:
            _check(fn(*args, self._stream(stream)))
            return
        with torch.cuda.device(self.device):
            _check(fn(*args, self._stream(stream)))

    def _stream(self, stream) -> int:
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device)
        return stream.cuda_stream


def _int32(sizes: int) -> None:
    """Refuses sizes, given or-ed together, that do not fit 32 bits: ctypes
    would take their low bits without a word (the library refuses negative
    ones)."""
    if sizes > 0x7FFFFFFF:
        raise ValueError("a size does not fit 32 bits")


def _nbytes(workspace: torch.Tensor) -> int:
    return workspace.numel() * workspace.element_size()


def moe_group_workspace_size(T: int, n_experts: int, top_k: int) -> int:
    _int32(int(T) | int(n_experts) | int(top_k))
    return int(lib().moe_group_workspace_size(int(T), int(n_experts), int(top_k)))


def _alloc(n: int, device) -> torch.Tensor:
    if n == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "configuration rejected")
    return torch.empty(n, dtype=torch.uint8, device=device)


def alloc_group_workspace(T: int, n_experts: int, top_k: int, device="cuda") -> torch.Tensor:
    return _alloc(moe_group_workspace_size(T, n_experts, top_k), device)


def moe_group_rows(topk_idx: torch.Tensor, n_experts: int, offsets: torch.Tensor,
                   row_token: torch.Tensor, slot_row: torch.Tensor, *, workspace: torch.Tensor,
                   capacity: int = 0, stream=None) -> None:
    """(token, slot) pairs grouped by expert: ``offsets`` [N + 1], ``row_token``
    [T k] and ``slot_row`` [T, k] from ``topk_idx`` [T, k] (all int32); see
    ``moe_group_rows`` in include/moe.h."""
    T, k = topk_idx.shape
    _int32(T | k | int(n_experts) | int(capacity))
    c = _Call(topk_idx)
    i32 = torch.int32
    c.run(lib().moe_group_rows, stream, T, int(n_experts), k, int(capacity),
          c.ptr(topk_idx, i32, "topk_idx", (T, k)),
          c.ptr(offsets, i32, "offsets", (int(n_experts) + 1,)),
          c.ptr(row_token, i32, "row_token", (T * k,)), c.ptr(slot_row, i32, "slot_row", (T, k)),
          c.workspace(workspace), _nbytes(workspace))


def make_linear_config(rows: int, groups: int, in_dim: int, out_dim: int, *,
                       dtype=torch.bfloat16, activation: str = "none", x_rows: int = 0,
                       weight_format: int = MOE_WEIGHTS_DTYPE) -> MoELinearConfig:
    """``activation``: one of ACTIVATIONS.  ``x_rows``: rows of x when a call
    gives ``row_index``, else 0 (x has ``rows`` rows)."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is none of {ACTIVATIONS}")
    if dtype not in (torch.bfloat16, torch.float32, "bf16", "f32", MOE_BF16, MOE_F32):
        raise ValueError(f"dtype {dtype}, expected bfloat16 or float32")
    _int32(int(rows) | int(x_rows) | int(groups) | int(in_dim) | int(out_dim))
    code = MOE_BF16 if dtype in (torch.bfloat16, "bf16", MOE_BF16) else MOE_F32
    return MoELinearConfig(int(rows), int(x_rows), int(groups), int(in_dim), int(out_dim), code,
                           int(weight_format), ACTIVATIONS.index(activation))


def _z_dim(cfg: MoELinearConfig) -> int:
    return cfg.out_dim * (2 if cfg.activation == ACTIVATIONS.index("swiglu") else 1)


def _x_shape(cfg: MoELinearConfig):
    return (cfg.x_rows if cfg.x_rows > 0 else cfg.rows, cfg.in_dim)


def moe_linear_workspace_size(cfg: MoELinearConfig) -> int:
    return int(lib().moe_linear_workspace_size(ctypes.byref(cfg)))


def alloc_linear_workspace(cfg: MoELinearConfig, device="cuda") -> torch.Tensor:
    return _alloc(moe_linear_workspace_size(cfg), device)


def moe_grouped_linear(cfg: MoELinearConfig, x: torch.Tensor, offsets: torch.Tensor,
                       w: torch.Tensor, y: torch.Tensor, *, workspace: torch.Tensor,
                       row_index: Optional[torch.Tensor] = None,
                       w_scale: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None,
                       residual: Optional[torch.Tensor] = None,
                       z_codes: Optional[torch.Tensor] = None,
                       z_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """y[r] = act(x[src(r)] W_e^T + bias[e]) + residual[r] for the rows of every
    group, and the 8-bit checkpoint of the pre-activations when ``z_codes``
    (uint8) and ``z_scale`` are given; see ``moe_grouped_linear`` in
    include/moe.h."""
    dt, z, f32 = _TORCH_DTYPE[cfg.dtype], _z_dim(cfg), torch.float32
    wt = torch.uint8 if cfg.weight_format == MOE_WEIGHTS_FP8_E4M3 else dt
    c = _Call(y)
    a = MoELinearArgs(
        c.ptr(x, dt, "x", _x_shape(cfg)),
        c.ptr(row_index, torch.int32, "row_index", (cfg.rows,)),
        c.ptr(offsets, torch.int32, "offsets", (cfg.groups + 1,)),
        c.ptr(w, wt, "w", (cfg.groups, z, cfg.in_dim)),
        c.ptr(w_scale, f32, "w_scale", (cfg.groups, z)),
        c.ptr(bias, f32, "bias", (cfg.groups, z)),
        c.ptr(residual, dt, "residual", (cfg.rows, cfg.out_dim)),
        c.ptr(y, dt, "y", (cfg.rows, cfg.out_dim)),
        c.ptr(z_codes, torch.uint8, "z_codes", (cfg.rows, z)),
        c.ptr(z_scale, f32, "z_scale", (cfg.rows, z // CHECKPOINT_BLOCK)))
    c.run(lib().moe_grouped_linear, stream, ctypes.byref(cfg), ctypes.byref(a),
          c.workspace(workspace), _nbytes(workspace))


def moe_linear_backward_workspace_size(cfg: MoELinearConfig) -> int:
    return int(lib().moe_linear_backward_workspace_size(ctypes.byref(cfg)))


def alloc_linear_backward_workspace(cfg: MoELinearConfig, device="cuda") -> torch.Tensor:
    return _alloc(moe_linear_backward_workspace_size(cfg), device)


def moe_grouped_linear_backward(cfg: MoELinearConfig, x: Optional[torch.Tensor],
                                offsets: torch.Tensor, w: Optional[torch.Tensor],
                                dy: torch.Tensor, *, workspace: torch.Tensor,
                                row_index: Optional[torch.Tensor] = None,
                                z_codes: Optional[torch.Tensor] = None,
                                z_scale: Optional[torch.Tensor] = None,
                                dx: Optional[torch.Tensor] = None,
                                dw: Optional[torch.Tensor] = None,
                                dbias: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of moe_grouped_linear into ``dx`` [rows, in_dim], ``dw`` and
    ``dbias`` (fp32), those that are given; the pre-activations come from their
    8-bit checkpoint; see ``moe_grouped_linear_backward`` in include/moe.h."""
    dt, z, f32 = _TORCH_DTYPE[cfg.dtype], _z_dim(cfg), torch.float32
    c = _Call(dy)
    a = MoELinearGradArgs(
        c.ptr(x, dt, "x", _x_shape(cfg)),
        c.ptr(row_index, torch.int32, "row_index", (cfg.rows,)),
        c.ptr(offsets, torch.int32, "offsets", (cfg.groups + 1,)),
        c.ptr(w, dt, "w", (cfg.groups, z, cfg.in_dim)),
        c.ptr(dy, dt, "dy", (cfg.rows, cfg.out_dim)),
        c.ptr(z_codes, torch.uint8, "z_codes", (cfg.rows, z)),
        c.ptr(z_scale, f32, "z_scale", (cfg.rows, z // CHECKPOINT_BLOCK)),
        c.ptr(dx, dt, "dx", (cfg.rows, cfg.in_dim)),
        c.ptr(dw, dt, "dw", (cfg.groups, z, cfg.in_dim)),
        c.ptr(dbias, f32, "dbias", (cfg.groups, z)))
    c.run(lib().moe_grouped_linear_backward, stream, ctypes.byref(cfg), ctypes.byref(a),
          c.workspace(workspace), _nbytes(workspace))


def moe_checkpoint_pack(x: torch.Tensor, codes: torch.Tensor, scale: torch.Tensor,
                        stream=None) -> None:
    """x [rows, cols] as E4M3 ``codes`` (uint8) and one fp32 ``scale`` for each
    64 columns of a row; see ``moe_checkpoint_pack`` in include/moe.h."""
    rows, cols = x.shape
    _int32(cols)
    c = _Call(x)
    c.run(lib().moe_checkpoint_pack, stream, rows, cols, _dtype_code(x, "x"),
          c.ptr(x, x.dtype, "x", (rows, cols)), c.ptr(codes, torch.uint8, "codes", (rows, cols)),
          c.ptr(scale, torch.float32, "scale", (rows, cols // CHECKPOINT_BLOCK)))


def moe_checkpoint_unpack(codes: torch.Tensor, scale: torch.Tensor, x: torch.Tensor,
                          stream=None) -> None:
    """x [rows, cols] = codes * scale; see ``moe_checkpoint_unpack`` in include/moe.h."""
    rows, cols = x.shape
    _int32(cols)
    c = _Call(x)
    c.run(lib().moe_checkpoint_unpack, stream, rows, cols, _dtype_code(x, "x"),
          c.ptr(codes, torch.uint8, "codes", (rows, cols)),
          c.ptr(scale, torch.float32, "scale", (rows, cols // CHECKPOINT_BLOCK)),
          c.ptr(x, x.dtype, "x", (rows, cols)))


def moe_combine(rows: torch.Tensor, slot_row: torch.Tensor, y: torch.Tensor, *,
                gate: Optional[torch.Tensor] = None, stream=None) -> None:
    """y[t] = sum_s gate[t, s] rows[slot_row[t, s]] (no gate: 1); see
    ``moe_combine`` in include/moe.h."""
    (n_rows, d), (T, k) = rows.shape, slot_row.shape
    _int32(n_rows | d | T | k)
    c = _Call(y)
    c.run(lib().moe_combine, stream, T, k, n_rows, d, _dtype_code(rows, "rows"),
          c.ptr(rows, rows.dtype, "rows", (n_rows, d)),
          c.ptr(slot_row, torch.int32, "slot_row", (T, k)),
          c.ptr(gate, torch.float32, "gate", (T, k)), c.ptr(y, rows.dtype, "y", (T, d)))


def moe_combine_backward(rows: torch.Tensor, slot_row: torch.Tensor,
                         gate: Optional[torch.Tensor], dy: torch.Tensor,
                         drows: Optional[torch.Tensor], dgate: Optional[torch.Tensor],
                         stream=None) -> None:
    """Gradients of moe_combine with respect to its rows and gates; see
    ``moe_combine_backward`` in include/moe.h."""
    (n_rows, d), (T, k) = rows.shape, slot_row.shape
    _int32(n_rows | d | T | k)
    c = _Call(dy)
    c.run(lib().moe_combine_backward, stream, T, k, n_rows, d, _dtype_code(rows, "rows"),
          c.ptr(rows, rows.dtype, "rows", (n_rows, d)),
          c.ptr(slot_row, torch.int32, "slot_row", (T, k)),
          c.ptr(gate, torch.float32, "gate", (T, k)), c.ptr(dy, rows.dtype, "dy", (T, d)),
          c.ptr(drows, rows.dtype, "drows", (n_rows, d)),
          c.ptr(dgate, torch.float32, "dgate", (T, k)))


class MoELayer:
    """Convenience holder: config, device weights and a workspace sized once.

    ``forward(x)`` allocates the outputs with torch (device memory only) and
    calls ``moe_layer_forward``, which also writes the balance statistics.
    """

    def __init__(self, weights: Dict[str, Optional[torch.Tensor]], top_k: int,
                 alpha: float = 0.01):
        wg = weights["w_gate"]
        self.weights = weights
        self.N, self.F, self.d = wg.shape
        self.S = 0 if weights.get("ws_gate") is None else weights["ws_gate"].shape[0]
        self.k = int(top_k)
        self.dtype = wg.dtype
        self.alpha = alpha
        self._ws = None
        self._ws_T = -1

    def config(self, T: int) -> MoEConfig:
        return make_config(T, self.d, self.N, self.k, self.F, self.S, self.dtype)

    def forward(self, x: torch.Tensor, want_logits: bool = False):
        T = x.shape[0]
        cfg = self.config(T)
        if self._ws is None or self._ws_T < T:
            self._ws = alloc_workspace(cfg, x.device)
            self._ws_T = T
        dev = x.device
        out = {
            "y": torch.empty_like(x),
            "topk_idx": torch.empty((T, self.k), dtype=torch.int32, device=dev),
            "topk_gate": torch.empty((T, self.k), dtype=torch.float32, device=dev),
            "counts": torch.zeros(self.N, dtype=torch.int32, device=dev),
            "prob_sum": torch.zeros(self.N, dtype=torch.float32, device=dev),
            "logits": (torch.empty((T, self.N), dtype=torch.float32, device=dev)
                       if want_logits else None),
            "f": torch.empty(self.N, dtype=torch.float32, device=dev),
            "P": torch.empty(self.N, dtype=torch.float32, device=dev),
            "aux": torch.empty(2, dtype=torch.float32, device=dev),
        }
        moe_layer_forward(cfg, x, self.weights, out["y"], workspace=self._ws,
                          logits=out["logits"], topk_idx=out["topk_idx"],
                          topk_gate=out["topk_gate"], counts=out["counts"],
                          prob_sum=out["prob_sum"], f=out["f"], P=out["P"], aux=out["aux"],
                          alpha=self.alpha)
        return out

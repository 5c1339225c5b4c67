"""MI355X (gfx950) sparse-MoE FFN forward of GLM-4.5 / GLM-5: Python binding of libmoe.so.

Argument marshalling only: every step of the layer, of the operators around it and of those of a training step runs
in the HIP kernels behind the C ABI declared in include/moe.h, under its names. Tensors are
torch device tensors; the binding checks their device, dtype, shape and contiguity, passes raw pointers
and the current HIP stream, and raises MoeError on any status other than MOE_OK. There is no fallback:
without the built library every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
MOE_F32, MOE_BF16 = 0, 1
MOE_ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
MOE_ROUTE_SCORES_IN, MOE_ROUTE_SCORES_OUT, MOE_ROUTE_PREPARED = 1, 2, 4

EXPORTED = ["moe_check_config", "moe_workspace_size", "moe_dispatch_workspace_size", "moe_router_prepared_size",
            "moe_router_prepare", "moe_route", "moe_dispatch", "moe_forward", "moe_forward_routed",
            "moe_forward_noalloc", "moe_noalloc_scratch_bytes", "moe_dense_workspace_size", "moe_dense_forward",
            "moe_block_norm", "moe_block_norm_backward", "moe_block_norm_workspace_size", "moe_combine",
            "moe_combine_backward", "moe_grouped_workspace_size", "moe_grouped_linear", "moe_grouped_linear_dgrad",
            "moe_grouped_linear_wgrad", "moe_qlinear", "moe_quantize", "moe_layer_norm",
            "moe_layer_norm_workspace_size", "moe_layer_norm_backward", "moe_linear_workspace_size", "moe_linear",
            "moe_linear_backward_workspace_size", "moe_linear_backward", "moe_balance_workspace_size",
            "moe_balance_loss", "moe_route_backward", "moe_grad_norm_workspace_size", "moe_grad_norm",
            "moe_grad_clip", "moe_status_str", "moe_profile_begin",
            "moe_profile_begin_mask", "moe_profile_end", "moe_stage_name", "moe_stage_count"]


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {moe_status_str(status)}")
        self.status = status


class MoeConfig(ctypes.Structure):
    _fields_ = [
        ("hidden_size", ctypes.c_int32),
        ("n_routed_experts", ctypes.c_int32),
        ("n_group", ctypes.c_int32),
        ("topk_group", ctypes.c_int32),
        ("num_experts_per_tok", ctypes.c_int32),
        ("moe_intermediate_size", ctypes.c_int32),
        ("n_shared_experts", ctypes.c_int32),
        ("routed_scaling_factor", ctypes.c_float),
        ("norm_topk_prob", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("dtype", ctypes.c_int32),
        ("alpha_on_output", ctypes.c_int32),
        ("swiglu_limit", ctypes.c_float),
    ]


class MoeWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_router", "e_bias", "gate_up", "down", "sh_gate", "sh_up", "sh_down",
                                               "w_router_prepared")]


class MoeTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32)]


_lib = None


def lib():
    """The loaded libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
        cp = ctypes.POINTER(MoeConfig)
        L.moe_check_config.argtypes = [cp]
        L.moe_check_config.restype = ctypes.c_int
        L.moe_workspace_size.argtypes = [cp, i64]
        L.moe_workspace_size.restype = ctypes.c_size_t
        L.moe_dispatch_workspace_size.argtypes = [cp, i64]
        L.moe_dispatch_workspace_size.restype = ctypes.c_size_t
        L.moe_router_prepared_size.argtypes = [cp]
        L.moe_router_prepared_size.restype = ctypes.c_size_t
        L.moe_router_prepare.argtypes = [cp, vp, vp, ctypes.c_size_t, vp]
        L.moe_router_prepare.restype = ctypes.c_int
        L.moe_route.argtypes = [cp, i64, vp, vp, vp, vp, u32, vp, vp, vp, ctypes.c_size_t, vp]
        L.moe_route.restype = ctypes.c_int
        L.moe_dispatch.argtypes = [cp, i64, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.moe_dispatch.restype = ctypes.c_int
        L.moe_forward.argtypes = [cp, i64, vp, ctypes.POINTER(MoeWeights), vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.moe_forward_routed.argtypes = [cp, i64, vp, ctypes.POINTER(MoeWeights), vp, vp, vp, vp, vp,
                                         ctypes.c_size_t, vp]
        L.moe_forward_noalloc.argtypes = [cp, i64, vp, ctypes.POINTER(MoeWeights), vp, vp, vp, vp, vp]
        L.moe_forward_noalloc.restype = ctypes.c_int
        L.moe_noalloc_scratch_bytes.argtypes = []
        L.moe_noalloc_scratch_bytes.restype = ctypes.c_size_t
        L.moe_dense_workspace_size.argtypes = [i64, i32, i32, i32]
        L.moe_dense_workspace_size.restype = ctypes.c_size_t
        L.moe_dense_forward.argtypes = [i64, i32, i32, i32, ctypes.c_float, vp, vp, vp, vp, vp, vp, ctypes.c_size_t,
                                        vp]
        L.moe_forward.restype = ctypes.c_int
        f32, sz = ctypes.c_float, ctypes.c_size_t
        L.moe_block_norm_workspace_size.argtypes = [i64, i32, i32, i64]
        L.moe_block_norm_workspace_size.restype = sz
        L.moe_block_norm.argtypes = [i64, i32, i32, f32, f32, vp, vp, vp, vp, i64, vp, vp, vp, vp]
        L.moe_block_norm_backward.argtypes = [i64, i32, i32, f32, f32, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp,
                                              vp, vp, sz, vp]
        L.moe_combine.argtypes = [i64, i32, i32, i32, vp, i64, vp, vp, vp, f32, vp, vp]
        L.moe_combine_backward.argtypes = [i64, i32, i32, i32, vp, vp, i64, vp, vp, f32, vp, vp, vp]
        L.moe_grouped_workspace_size.argtypes = [i32, i64, i32]
        L.moe_grouped_workspace_size.restype = sz
        L.moe_grouped_linear.argtypes = [i32, i64, i32, i32, i32, vp, i64, vp, i32, vp, vp, vp, vp, sz, vp]
        L.moe_grouped_linear_dgrad.argtypes = [i32, i64, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_grouped_linear_wgrad.argtypes = [i32, i64, i32, i32, i32, vp, vp, i64, vp, i32, vp, vp, vp, sz, vp]
        L.moe_qlinear.argtypes = [i32, i64, i32, i32, i32, vp, i64, vp, i32, vp, vp, vp, i32, f32, vp, vp]
        L.moe_quantize.argtypes = [i32, i64, i32, i32, vp, vp, vp, vp]
        tp = ctypes.POINTER(MoeTensor)
        L.moe_layer_norm_workspace_size.argtypes = [i64, i32, i32]
        L.moe_layer_norm.argtypes = [i64, i32, i32, f32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_layer_norm_backward.argtypes = [i64, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_linear_workspace_size.argtypes = [i64, i32, i32, i32]
        L.moe_linear.argtypes = [i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_linear_backward_workspace_size.argtypes = [i64, i32, i32]
        L.moe_linear_backward.argtypes = [i64, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_balance_workspace_size.argtypes = [cp, i64, i64]
        L.moe_balance_loss.argtypes = [cp, i64, i64, f32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_route_backward.argtypes = [cp, i64, vp, vp, vp, i64, vp, vp, vp, vp, vp]
        L.moe_grad_norm_workspace_size.argtypes = [tp, i32]
        L.moe_grad_norm.argtypes = [tp, i32, vp, vp, sz, vp]
        L.moe_grad_clip.argtypes = [tp, tp, i32, vp, f32, f32, vp]
        for fn in (L.moe_layer_norm_workspace_size, L.moe_linear_workspace_size, L.moe_linear_backward_workspace_size,
                   L.moe_balance_workspace_size, L.moe_grad_norm_workspace_size):
            fn.restype = sz
        for fn in (L.moe_layer_norm, L.moe_layer_norm_backward, L.moe_linear, L.moe_linear_backward,
                   L.moe_balance_loss, L.moe_route_backward, L.moe_grad_norm, L.moe_grad_clip):
            fn.restype = ctypes.c_int
        for fn in (L.moe_block_norm, L.moe_block_norm_backward, L.moe_combine, L.moe_combine_backward,
                   L.moe_grouped_linear, L.moe_grouped_linear_dgrad, L.moe_grouped_linear_wgrad, L.moe_qlinear,
                   L.moe_quantize):
            fn.restype = ctypes.c_int
        L.moe_status_str.argtypes = [ctypes.c_int]
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_profile_begin.argtypes = []
        L.moe_profile_begin_mask.argtypes = [u32]
        L.moe_profile_begin.restype = ctypes.c_int
        L.moe_profile_end.argtypes = [vp, vp, i32]
        L.moe_profile_end.restype = ctypes.c_int
        L.moe_stage_name.argtypes = [i32]
        L.moe_stage_name.restype = ctypes.c_char_p
        L.moe_stage_count.argtypes = []
        L.moe_stage_count.restype = i32
        _lib = L
    return _lib


def make_config(D, E, G, TG, k, d, n_shared=1, alpha=1.0, norm=True, eps=1e-20, dtype="bf16",
                alpha_on_output=False, limit=0.0) -> MoeConfig:
    """moe_config from the pages' config fields (hidden_size, n_routed_experts, n_group, topk_group,
    num_experts_per_tok, moe_intermediate_size, n_shared_experts, routed_scaling_factor, norm_topk_prob),
    where alpha goes, and the SwiGLU clamp bound (0: none)."""
    dt = {"bf16": MOE_BF16, "f32": MOE_F32}[dtype] if isinstance(dtype, str) else int(dtype)
    return MoeConfig(D, E, G, TG, k, d, n_shared, float(alpha), int(bool(norm)), float(eps), dt,
                     int(bool(alpha_on_output)), float(limit))


def config_of(w) -> MoeConfig:
    """moe_config from an object with fields D, E, G, TG, k, d, n_shared, alpha, norm, eps, dtype (and
    optionally alpha_on_output, limit)."""
    return make_config(w.D, w.E, w.G, w.TG, w.k, w.d, w.n_shared, w.alpha, w.norm, w.eps, w.dtype,
                       getattr(w, "alpha_on_output", False), getattr(w, "limit", 0.0))


def moe_status_str(status: int) -> str:
    return lib().moe_status_str(int(status)).decode()


_torch = None  # the torch module, from the first call that needs it (an import statement costs 0.2 us a time)


def _import_torch():
    global _torch
    import torch

    _torch = torch
    return torch


def _ptr(t, name, dtype=None, shape=None, required=True):
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return None
    torch = _torch or _import_torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _device() -> int:
    """The current device's index, without the checks of torch.cuda.current_device()."""
    torch = _torch or _import_torch()
    get = getattr(torch._C, "_cuda_getDevice", None)
    return get() if get and torch.cuda.is_initialized() else torch.cuda.current_device()


def _stream(stream):
    if stream is None:
        torch = _torch or _import_torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # no Stream object: a third of the time
        return raw(_device()) if raw else torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _act_dtype(cfg: MoeConfig):
    import torch

    return torch.float32 if cfg.dtype == MOE_F32 else torch.bfloat16


def _check(status, what):
    if status != MOE_OK:
        raise MoeError(status, what)


def moe_check_config(cfg: MoeConfig) -> int:
    return lib().moe_check_config(ctypes.byref(cfg))


def moe_workspace_size(cfg: MoeConfig, N: int) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(cfg), int(N)))


def alloc_workspace(cfg: MoeConfig, N: int, device="cuda"):
    import torch

    n = moe_workspace_size(cfg, N)
    if n == 0 and N > 0:
        _check(moe_check_config(cfg) or MOE_ERR_INVALID_ARG, "moe_workspace_size")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def moe_dispatch_workspace_size(cfg: MoeConfig, N: int) -> int:
    return int(lib().moe_dispatch_workspace_size(ctypes.byref(cfg), int(N)))


def moe_router_prepared_size(cfg: MoeConfig) -> int:
    return int(lib().moe_router_prepared_size(ctypes.byref(cfg)))


def moe_router_prepare(cfg: MoeConfig, w_router, prepared=None, stream=None):
    """The [3, E, D] bf16 pieces of w_router (bf16 layers), for moe_weights.w_router_prepared or moe_route
    with MOE_ROUTE_PREPARED. Returns `prepared` (allocated here as a bf16 tensor when None)."""
    import torch

    E, D = cfg.n_routed_experts, cfg.hidden_size
    if prepared is None:
        prepared = torch.empty((3, E, D), dtype=torch.bfloat16, device=w_router.device)
    st = lib().moe_router_prepare(ctypes.byref(cfg), _ptr(w_router, "w_router", torch.float32, (E, D)),
                                  _ptr(prepared, "prepared"), prepared.numel() * prepared.element_size(),
                                  _stream(stream))
    _check(st, "moe_router_prepare")
    return prepared


def moe_route(cfg: MoeConfig, N: int, x, w_router, e_bias, scores, topk_idx, topk_w, flags: int = 0,
              workspace=None, stream=None):
    """Router on the GPU. With flags = MOE_ROUTE_SCORES_IN, `scores` [N, E] is read and x / w_router /
    workspace are ignored; otherwise `workspace` (uint8, moe_workspace_size bytes) is required, `scores`
    is written with MOE_ROUTE_SCORES_OUT (else it may be None), and with MOE_ROUTE_PREPARED `w_router` is
    the output of moe_router_prepare."""
    import torch

    E, D, k = cfg.n_routed_experts, cfg.hidden_size, cfg.num_experts_per_tok
    scores_in = bool(flags & MOE_ROUTE_SCORES_IN)
    prepared = bool(flags & MOE_ROUTE_PREPARED)
    need_scores = scores_in or bool(flags & MOE_ROUTE_SCORES_OUT)
    st = lib().moe_route(
        ctypes.byref(cfg), int(N),
        _ptr(x, "x", _act_dtype(cfg), (N, D), required=not scores_in),
        _ptr(w_router, "w_router", torch.bfloat16 if prepared else torch.float32, (3, E, D) if prepared else (E, D),
             required=not scores_in),
        _ptr(e_bias, "e_bias", torch.float32, (E,)),
        _ptr(scores, "scores", torch.float32, (N, E), required=need_scores),
        int(flags),
        _ptr(topk_idx, "topk_idx", torch.int32, (N, k)),
        _ptr(topk_w, "topk_w", torch.float32, (N, k)),
        _ptr(workspace, "workspace", torch.uint8, required=not scores_in),
        0 if workspace is None else workspace.numel(),
        _stream(stream))
    _check(st, "moe_route")


def moe_dispatch(cfg: MoeConfig, N: int, topk_idx, counts, offsets, sorted_pair, inv_row, workspace=None,
                 stream=None):
    """Dispatch on the GPU; `workspace` (uint8, moe_dispatch_workspace_size bytes) may be None when that
    size is 0."""
    import torch

    E, k = cfg.n_routed_experts, cfg.num_experts_per_tok
    st = lib().moe_dispatch(
        ctypes.byref(cfg), int(N),
        _ptr(topk_idx, "topk_idx", torch.int32, (N, k)),
        _ptr(counts, "counts", torch.int32, (E,)),
        _ptr(offsets, "offsets", torch.int32, (E + 1,)),
        _ptr(sorted_pair, "sorted_pair", torch.int32, (N * k,)),
        _ptr(inv_row, "inv_row", torch.int32, (N * k,)),
        _ptr(workspace, "workspace", torch.uint8, required=False),
        0 if workspace is None else workspace.numel(),
        _stream(stream))
    _check(st, "moe_dispatch")


def weights_struct(cfg: MoeConfig, w: dict) -> MoeWeights:
    """MoeWeights from a dict of device tensors: w_router, e_bias, gate_up, down, sh_gate, sh_up, sh_down and
    optionally w_router_prepared (the router pair may be absent for moe_forward_routed)."""
    import torch

    E, D, d = cfg.n_routed_experts, cfg.hidden_size, cfg.moe_intermediate_size
    dsh = d * cfg.n_shared_experts
    adt = _act_dtype(cfg)
    sh = cfg.n_shared_experts > 0
    prep = w.get("w_router_prepared")
    return MoeWeights(
        _ptr(w.get("w_router"), "w_router", torch.float32, (E, D), required=False),
        _ptr(w.get("e_bias"), "e_bias", torch.float32, (E,), required=False),
        _ptr(w["gate_up"], "gate_up", adt, (E, 2 * d, D)),
        _ptr(w["down"], "down", adt, (E, D, d)),
        _ptr(w.get("sh_gate"), "sh_gate", adt, (dsh, D), required=sh) if sh else None,
        _ptr(w.get("sh_up"), "sh_up", adt, (dsh, D), required=sh) if sh else None,
        _ptr(w.get("sh_down"), "sh_down", adt, (D, dsh), required=sh) if sh else None,
        _ptr(prep, "w_router_prepared", torch.bfloat16, (3, E, D), required=False),
    )


def moe_forward(cfg: MoeConfig, N: int, x, weights, y, workspace, topk_idx_out=None, topk_w_out=None,
                counts_out=None, stream=None):
    """The whole layer on the GPU; `weights` is a MoeWeights or a dict accepted by weights_struct."""
    import torch

    E, D, k = cfg.n_routed_experts, cfg.hidden_size, cfg.num_experts_per_tok
    ws = weights if isinstance(weights, MoeWeights) else weights_struct(cfg, weights)
    adt = _act_dtype(cfg)
    st = lib().moe_forward(
        ctypes.byref(cfg), int(N),
        _ptr(x, "x", adt, (N, D)),
        ctypes.byref(ws),
        _ptr(y, "y", adt, (N, D)),
        _ptr(topk_idx_out, "topk_idx_out", torch.int32, (N, k), required=False),
        _ptr(topk_w_out, "topk_w_out", torch.float32, (N, k), required=False),
        _ptr(counts_out, "counts_out", torch.int32, (E,), required=False),
        _ptr(workspace, "workspace", torch.uint8),
        workspace.numel(),
        _stream(stream))
    _check(st, "moe_forward")


def moe_forward_routed(cfg: MoeConfig, N: int, x, weights, topk_idx, topk_w, y, workspace, counts_out=None,
                       stream=None):
    """The layer with routing given by the caller: topk_idx [N, k] int32 (id E = empty slot), topk_w [N, k]
    float32 used as given."""
    import torch

    E, D, k = cfg.n_routed_experts, cfg.hidden_size, cfg.num_experts_per_tok
    ws = weights if isinstance(weights, MoeWeights) else weights_struct(cfg, weights)
    adt = _act_dtype(cfg)
    st = lib().moe_forward_routed(
        ctypes.byref(cfg), int(N),
        _ptr(x, "x", adt, (N, D)),
        ctypes.byref(ws),
        _ptr(topk_idx, "topk_idx", torch.int32, (N, k)),
        _ptr(topk_w, "topk_w", torch.float32, (N, k)),
        _ptr(y, "y", adt, (N, D)),
        _ptr(counts_out, "counts_out", torch.int32, (E,), required=False),
        _ptr(workspace, "workspace", torch.uint8),
        workspace.numel(),
        _stream(stream))
    _check(st, "moe_forward_routed")


def _dtype_code(dtype) -> int:
    return {"bf16": MOE_BF16, "f32": MOE_F32}[dtype] if isinstance(dtype, str) else int(dtype)


def moe_dense_workspace_size(N: int, D: int, dff: int, dtype="bf16") -> int:
    return int(lib().moe_dense_workspace_size(int(N), int(D), int(dff), _dtype_code(dtype)))


def moe_dense_forward(N: int, x, gate, up, down, y, workspace, limit: float = 0.0, stream=None):
    """Dense SwiGLU FFN y = down (SiLU(gate x) * up x); gate, up [dff, D], down [D, dff]."""
    import torch

    dff, D = gate.shape
    dt = _dtype_code("f32" if x.dtype == torch.float32 else "bf16")
    adt = torch.float32 if dt == MOE_F32 else torch.bfloat16
    st = lib().moe_dense_forward(
        int(N), int(D), int(dff), dt, float(limit),
        _ptr(x, "x", adt, (N, D)), _ptr(gate, "gate", adt, (dff, D)), _ptr(up, "up", adt, (dff, D)),
        _ptr(down, "down", adt, (D, dff)), _ptr(y, "y", adt, (N, D)),
        _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check(st, "moe_dense_forward")


# ---- the operators around the experts ----
def _tensor_dtype(t, name) -> int:
    torch = _torch or _import_torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype is torch.bfloat16:
        return MOE_BF16
    if t.dtype is torch.float32:
        return MOE_F32
    raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")


_NO_CHANGE = contextlib.nullcontext()


def _same_device(what, *tensors):
    """The tensors' one device, made the current one for the launch (and its current stream the default)."""
    index = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise TypeError(f"{what}: every tensor must be a device tensor")
        i = t.get_device()
        if index is not None and i != index:
            raise ValueError(f"{what}: tensors on more than one device: {index} and {i}")
        index = i
    if index is None or index == _device():
        return _NO_CHANGE
    return _torch.cuda.device(index)


def _ws(workspace):
    if workspace is None:
        return None, 0
    return _ptr(workspace, "workspace", (_torch or _import_torch()).uint8), workspace.numel()


def moe_block_norm_workspace_size(N: int, D: int, dtype="bf16", gate_rows: int = 0) -> int:
    """Bytes of workspace of moe_block_norm_backward (gate_rows 0: no gate)."""
    return int(lib().moe_block_norm_workspace_size(int(N), int(D), _dtype_code(dtype), int(gate_rows)))


def moe_block_norm(N: int, h, o, w_post, gate, gate_rows, w_pre, h_out, u, residual_scale: float = 1.0,
                   eps: float = 1e-5, stream=None):
    """h_out = residual_scale h + gate (o / rms(o)) w_post and u = (h_out / rms(h_out)) w_pre. Without o (None)
    u is the norm of h; without w_pre only h_out is written; w_post and gate may be None. Row n uses row
    n // gate_rows of gate [ceil(N / gate_rows), D]."""
    dt = _tensor_dtype(h, "h")
    t, D, T = h.dtype, h.shape[-1], int(gate_rows or 0)
    groups = (N + T - 1) // T if T > 0 else 0
    with _same_device("moe_block_norm", h, o, w_post, gate, w_pre, h_out, u):
        st = lib().moe_block_norm(
            int(N), int(D), dt, float(eps), float(residual_scale),
            _ptr(h, "h", t, (N, D)), _ptr(o, "o", t, (N, D), required=False),
            _ptr(w_post, "w_post", t, (D,), required=False),
            _ptr(gate, "gate", t, (groups, D), required=False), T,
            _ptr(w_pre, "w_pre", t, (D,), required=False),
            _ptr(h_out, "h_out", t, (N, D), required=False), _ptr(u, "u", t, (N, D), required=False),
            _stream(stream))
    _check(st, "moe_block_norm")


def moe_block_norm_backward(N: int, h_out, o, w_post, gate, gate_rows, w_pre, dh_out, du, dh, d_o, dw_post, dgate,
                            dw_pre, workspace, residual_scale: float = 1.0, eps: float = 1e-5, stream=None):
    """Gradients of moe_block_norm from its tensors (h_out: the forward's h when o is None) and the gradients
    dh_out (or None) and du. Writes dh, d_o and, where given, the float32 sums dw_post, dgate, dw_pre;
    workspace: moe_block_norm_workspace_size(N, D, dtype, gate_rows) bytes, or None without sums."""
    torch = _torch or _import_torch()
    dt = _tensor_dtype(dh, "dh")
    t, f, D, T = dh.dtype, torch.float32, dh.shape[-1], int(gate_rows or 0)
    groups = (N + T - 1) // T if T > 0 else 0
    ws, ws_bytes = _ws(workspace)
    with _same_device("moe_block_norm_backward", h_out, o, w_post, gate, w_pre, dh_out, du, dh, d_o, dw_post, dgate,
                      dw_pre, workspace):
        st = lib().moe_block_norm_backward(
            int(N), int(D), dt, float(eps), float(residual_scale),
            _ptr(h_out, "h_out", t, (N, D), required=False), _ptr(o, "o", t, (N, D), required=False),
            _ptr(w_post, "w_post", t, (D,), required=False),
            _ptr(gate, "gate", t, (groups, D), required=False), T,
            _ptr(w_pre, "w_pre", t, (D,), required=False),
            _ptr(dh_out, "dh_out", t, (N, D), required=False), _ptr(du, "du", t, (N, D), required=False),
            _ptr(dh, "dh", t, (N, D)), _ptr(d_o, "d_o", t, (N, D), required=False),
            _ptr(dw_post, "dw_post", f, (D,), required=False), _ptr(dgate, "dgate", f, (groups, D), required=False),
            _ptr(dw_pre, "dw_pre", f, (D,), required=False), ws, ws_bytes, _stream(stream))
    _check(st, "moe_block_norm_backward")


def moe_combine(N: int, k: int, rows, inv_row, topk_w, shared, y, alpha: float = 1.0, stream=None):
    """y[n] = alpha sum_s topk_w[n, s] rows[inv_row[n, s]] + shared[n]; topk_w None: ones, shared None: nothing
    added. inv_row (N * k int32) as moe_dispatch writes it; entries outside rows are empty slots."""
    torch = _torch or _import_torch()
    dt = _tensor_dtype(rows, "rows")
    t, (R, D) = rows.dtype, rows.shape
    with _same_device("moe_combine", rows, inv_row, topk_w, shared, y):
        st = lib().moe_combine(
            int(N), int(k), int(D), dt, _ptr(rows, "rows", t), int(R),
            _ptr(inv_row, "inv_row", torch.int32, (N * k,)),
            _ptr(topk_w, "topk_w", torch.float32, (N, k), required=False),
            _ptr(shared, "shared", t, (N, D), required=False), float(alpha), _ptr(y, "y", t, (N, D)),
            _stream(stream))
    _check(st, "moe_combine")


def moe_combine_backward(N: int, k: int, dy, rows, inv_row, topk_w, drows, dtopk_w, alpha: float = 1.0, stream=None):
    """drows[inv_row[n, s]] = alpha topk_w[n, s] dy[n] and dtopk_w[n, s] = alpha <dy[n], rows[inv_row[n, s]]>.
    dtopk_w (and with it rows) may be None; rows that no slot names keep what they held in drows."""
    torch = _torch or _import_torch()
    dt = _tensor_dtype(drows, "drows")
    t, (R, D) = drows.dtype, drows.shape
    with _same_device("moe_combine_backward", dy, rows, inv_row, topk_w, drows, dtopk_w):
        st = lib().moe_combine_backward(
            int(N), int(k), int(D), dt, _ptr(dy, "dy", t, (N, D)), _ptr(rows, "rows", t, (R, D), required=False),
            int(R), _ptr(inv_row, "inv_row", torch.int32, (N * k,)),
            _ptr(topk_w, "topk_w", torch.float32, (N, k), required=False), float(alpha), _ptr(drows, "drows", t),
            _ptr(dtopk_w, "dtopk_w", torch.float32, (N, k), required=False), _stream(stream))
    _check(st, "moe_combine_backward")


def moe_grouped_workspace_size(E: int, R: int, dtype="bf16") -> int:
    return int(lib().moe_grouped_workspace_size(int(E), int(R), _dtype_code(dtype)))


def moe_grouped_linear(x, w, offsets, y, workspace, row_index=None, index_div: int = 1, stream=None):
    """y[r] = w[e] x[src(r)] for the rows r in [offsets[e], offsets[e + 1]); w [E, out, in], y [R, out].
    src(r) = row_index[r] // index_div (moe_dispatch's sorted_pair and k), or r without row_index."""
    torch = _torch or _import_torch()
    dt = _tensor_dtype(x, "x")
    t, (E, M, K), R = x.dtype, w.shape, y.shape[0]
    ws, ws_bytes = _ws(workspace)
    with _same_device("moe_grouped_linear", x, w, offsets, y, workspace, row_index):
        st = lib().moe_grouped_linear(
            int(E), int(R), int(K), int(M), dt, _ptr(x, "x", t, (x.shape[0], K)), int(x.shape[0]),
            _ptr(row_index, "row_index", torch.int32, (R,), required=False), int(index_div), _ptr(w, "w", t),
            _ptr(offsets, "offsets", torch.int32, (E + 1,)), _ptr(y, "y", t, (R, M)), ws, ws_bytes,
            _stream(stream))
    _check(st, "moe_grouped_linear")


def moe_grouped_linear_dgrad(dy, w, offsets, dx, workspace, stream=None):
    """dx[r] = w[e]^T dy[r], one row per grouped row."""
    torch = _torch or _import_torch()
    dt = _tensor_dtype(dy, "dy")
    t, (E, M, K), R = dy.dtype, w.shape, dx.shape[0]
    ws, ws_bytes = _ws(workspace)
    with _same_device("moe_grouped_linear_dgrad", dy, w, offsets, dx, workspace):
        st = lib().moe_grouped_linear_dgrad(
            int(E), int(R), int(K), int(M), dt, _ptr(dy, "dy", t, (R, M)), _ptr(w, "w", t),
            _ptr(offsets, "offsets", torch.int32, (E + 1,)), _ptr(dx, "dx", t, (R, K)), ws, ws_bytes,
            _stream(stream))
    _check(st, "moe_grouped_linear_dgrad")


def moe_grouped_linear_wgrad(dy, x, offsets, dw, workspace, row_index=None, index_div: int = 1, stream=None):
    """dw[e] = sum of dy[r] x[src(r)]^T over the rows of expert e (zeros without rows)."""
    torch = _torch or _import_torch()
    dt = _tensor_dtype(dy, "dy")
    t, (E, M, K), R = dy.dtype, dw.shape, dy.shape[0]
    ws, ws_bytes = _ws(workspace)
    with _same_device("moe_grouped_linear_wgrad", dy, x, offsets, dw, workspace, row_index):
        st = lib().moe_grouped_linear_wgrad(
            int(E), int(R), int(K), int(M), dt, _ptr(dy, "dy", t, (R, M)), _ptr(x, "x", t, (x.shape[0], K)),
            int(x.shape[0]), _ptr(row_index, "row_index", torch.int32, (R,), required=False), int(index_div),
            _ptr(offsets, "offsets", torch.int32, (E + 1,)), _ptr(dw, "dw", t), ws, ws_bytes, _stream(stream))
    _check(st, "moe_grouped_linear_wgrad")


def moe_qlinear(x, wq, scales, y, offsets=None, row_index=None, index_div: int = 1, swiglu: bool = False,
                limit: float = 0.0, stream=None):
    """moe_grouped_linear with 4-bit weights: wq [E, out, in / 2] uint8, scales [E, out, in / group] bf16
    (moe_quantize). offsets None (E = 1): all rows. swiglu: y [R, out / 2] = SiLU(gate half) * up half."""
    torch = _torch or _import_torch()
    E, M, half = wq.shape
    K = 2 * half
    if scales.dim() != 3 or scales.shape[2] < 1 or K % scales.shape[2]:
        raise ValueError(f"scales must have shape (E, out, in / group), got {tuple(scales.shape)}")
    groups, R, bf = scales.shape[2], y.shape[0], torch.bfloat16
    with _same_device("moe_qlinear", x, wq, scales, y, offsets, row_index):
        st = lib().moe_qlinear(
            int(E), int(R), int(K), int(M), K // groups, _ptr(x, "x", bf, (x.shape[0], K)), int(x.shape[0]),
            _ptr(row_index, "row_index", torch.int32, (R,), required=False), int(index_div),
            _ptr(wq, "wq", torch.uint8), _ptr(scales, "scales", bf, (E, M, groups)),
            _ptr(offsets, "offsets", torch.int32, (E + 1,), required=False), int(bool(swiglu)), float(limit),
            _ptr(y, "y", bf, (R, M // 2 if swiglu else M)), _stream(stream))
    _check(st, "moe_qlinear")


def moe_quantize(w, group: int, wq=None, scales=None, stream=None):
    """(wq, scales) of w [..., in] for moe_qlinear: uint8 [..., in / 2] and bf16 [..., in / group], allocated here
    when None."""
    torch = _torch or _import_torch()
    dt = _tensor_dtype(w, "w")
    K, lead = w.shape[-1], tuple(w.shape[:-1])
    if group < 1 or K % group:
        raise ValueError(f"group {group} does not divide {K}")
    if wq is None:
        wq = torch.empty(lead + (K // 2,), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(lead + (K // group,), dtype=torch.bfloat16, device=w.device)
    rows = w.numel() // K if K else 0
    with _same_device("moe_quantize", w, wq, scales):
        st = lib().moe_quantize(dt, rows, int(K), int(group), _ptr(w, "w"),
                                _ptr(wq, "wq", torch.uint8, lead + (K // 2,)),
                                _ptr(scales, "scales", torch.bfloat16, lead + (K // group,)), _stream(stream))
    _check(st, "moe_quantize")
    return wq, scales


# ---- a training step around the layer ----
def moe_layer_norm_workspace_size(N: int, D: int, dtype="bf16") -> int:
    """Bytes of workspace of moe_layer_norm_backward."""
    return int(lib().moe_layer_norm_workspace_size(int(N), int(D), _dtype_code(dtype)))


def moe_layer_norm(N: int, x, residual, w, b, h_out, y, stats=None, eps: float = 1e-5, stream=None):
    """h = x + residual and y = (h - mean(h)) / std(h) * w + b over each row; std with eps under the root. residual
    (and with it h_out, which receives h), w and b may be None; stats [N, 2] float32 receives mean and 1 / std for
    moe_layer_norm_backward."""
    torch = _torch or _import_torch()
    dt = _tensor_dtype(x, "x")
    t, D = x.dtype, x.shape[-1]
    with _same_device("moe_layer_norm", x, residual, w, b, h_out, y, stats):
        st = lib().moe_layer_norm(
            int(N), int(D), dt, float(eps), _ptr(x, "x", t, (N, D)),
            _ptr(residual, "residual", t, (N, D), required=False), _ptr(w, "w", t, (D,), required=False),
            _ptr(b, "b", t, (D,), required=False), _ptr(h_out, "h_out", t, (N, D), required=False),
            _ptr(y, "y", t, (N, D)), _ptr(stats, "stats", torch.float32, (N, 2), required=False), _stream(stream))
    _check(st, "moe_layer_norm")


def moe_layer_norm_backward(N: int, h, stats, w, dh_out, dy, dh, dw, db, workspace, stream=None):
    """Gradients of moe_layer_norm from its h (h_out, or x without a residual) and stats: dh [N, D] (of x and residual
    alike, dh_out added when given) and, where given, the float32 sums dw and db; workspace:
    moe_layer_norm_workspace_size(N, D, dtype) bytes, or None without sums."""
    torch = _torch or _import_torch()
    dt = _tensor_dtype(h, "h")
    t, f, D = h.dtype, torch.float32, h.shape[-1]
    ws, ws_bytes = _ws(workspace)
    with _same_device("moe_layer_norm_backward", h, stats, w, dh_out, dy, dh, dw, db, workspace):
        st = lib().moe_layer_norm_backward(
            int(N), int(D), dt, _ptr(h, "h", t, (N, D)), _ptr(stats, "stats", f, (N, 2)),
            _ptr(w, "w", t, (D,), required=False), _ptr(dh_out, "dh_out", t, (N, D), required=False),
            _ptr(dy, "dy", t, (N, D)), _ptr(dh, "dh", t, (N, D)), _ptr(dw, "dw", f, (D,), required=False),
            _ptr(db, "db", f, (D,), required=False), ws, ws_bytes, _stream(stream))
    _check(st, "moe_layer_norm_backward")


def _activation(act) -> int:
    code = MOE_ACTIVATIONS.get(act) if isinstance(act, str) else act
    if code is None:
        raise ValueError(f"act must be one of {', '.join(MOE_ACTIVATIONS)}, got {act!r}")
    return int(code)


def _rows_columns(t, name):
    shape = getattr(t, "shape", ())
    if len(shape) != 2:
        raise ValueError(f"{name} must be a tensor of two dimensions")
    return shape


def moe_linear_workspace_size(R: int, K: int, M: int, dtype="bf16") -> int:
    """Bytes of workspace of moe_linear for R rows, K input and M output features."""
    return int(lib().moe_linear_workspace_size(int(R), int(K), int(M), _dtype_code(dtype)))


def moe_linear(x, w, y, workspace=None, bias=None, residual=None, act="none", z=None, stream=None):
    """y = act(x w^T + bias) + residual; x [R, in], w [out, in], y [R, out]. z [R, out] receives x w^T + bias for
    moe_linear_backward. act: a key of MOE_ACTIVATIONS. workspace: moe_linear_workspace_size(R, in, out, dtype) bytes."""
    dt = _tensor_dtype(x, "x")
    t, (R, M), K = x.dtype, _rows_columns(y, "y"), x.shape[-1]
    ws, ws_bytes = _ws(workspace)
    with _same_device("moe_linear", x, w, y, workspace, bias, residual, z):
        st = lib().moe_linear(
            int(R), int(K), int(M), dt, _activation(act), _ptr(x, "x", t, (R, K)), _ptr(w, "w", t, (M, K)),
            _ptr(bias, "bias", t, (M,), required=False), _ptr(residual, "residual", t, (R, M), required=False),
            _ptr(z, "z", t, (R, M), required=False), _ptr(y, "y", t, (R, M)), ws, ws_bytes, _stream(stream))
    _check(st, "moe_linear")


def moe_linear_backward_workspace_size(R: int, M: int, dtype="bf16") -> int:
    """Bytes of workspace of moe_linear_backward with dbias."""
    return int(lib().moe_linear_backward_workspace_size(int(R), int(M), _dtype_code(dtype)))


def moe_linear_backward(dy, z, dz, dbias, workspace=None, act="none", stream=None):
    """dz = dy * act'(z) and the float32 dbias = sum of its rows, each where given; z may be None for act "none". dx and
    dw follow from dz with moe_grouped_linear_dgrad and moe_grouped_linear_wgrad (one expert, offsets [0, R])."""
    torch = _torch or _import_torch()
    dt = _tensor_dtype(dy, "dy")
    t, (R, M) = dy.dtype, _rows_columns(dy, "dy")
    ws, ws_bytes = _ws(workspace)
    with _same_device("moe_linear_backward", dy, z, dz, dbias, workspace):
        st = lib().moe_linear_backward(
            int(R), int(M), dt, _activation(act), _ptr(dy, "dy", t, (R, M)), _ptr(z, "z", t, (R, M), required=False),
            _ptr(dz, "dz", t, (R, M), required=False), _ptr(dbias, "dbias", torch.float32, (M,), required=False), ws,
            ws_bytes, _stream(stream))
    _check(st, "moe_linear_backward")


def moe_balance_workspace_size(cfg: MoeConfig, N: int, seq_rows: int) -> int:
    return int(lib().moe_balance_workspace_size(ctypes.byref(cfg), int(N), int(seq_rows)))


def moe_balance_loss(cfg: MoeConfig, N: int, scores, topk_idx, seq_rows: int, weight: float, counts, coef, loss,
                     workspace, token_mask=None, stream=None):
    """loss[0] = weight * mean over sequences (runs of seq_rows rows) of sum_i f_i P_i, f_i = E / (k V) times the slots
    that name expert i, P_i the mean of the normalised scores, over the V live tokens (token_mask [N] uint8 or bool).
    counts [S, E] int32 and coef [S, E] float32 (d loss / d normalised score, for moe_route_backward) may be None."""
    torch = _torch or _import_torch()
    E, k, f = cfg.n_routed_experts, cfg.num_experts_per_tok, torch.float32
    S = (N + seq_rows - 1) // seq_rows if seq_rows > 0 else 0
    mask = _token_mask(token_mask, N)
    ws, ws_bytes = _ws(workspace)
    with _same_device("moe_balance_loss", scores, topk_idx, token_mask, counts, coef, loss, workspace):
        st = lib().moe_balance_loss(
            ctypes.byref(cfg), int(N), int(seq_rows), float(weight), _ptr(scores, "scores", f, (N, E)),
            _ptr(topk_idx, "topk_idx", torch.int32, (N, k)), mask,
            _ptr(counts, "counts", torch.int32, (S, E), required=False), _ptr(coef, "coef", f, (S, E), required=False),
            _ptr(loss, "loss", f, (1,)), ws, ws_bytes, _stream(stream))
    _check(st, "moe_balance_loss")


def _token_mask(t, N):
    torch = _torch or _import_torch()
    return _ptr(t, "token_mask", torch.bool if getattr(t, "dtype", None) is torch.bool else torch.uint8, (N,),
                required=False)


def moe_route_backward(cfg: MoeConfig, N: int, scores, topk_idx, dtopk_w, dlogits, seq_rows: int = 0, coef=None,
                       dloss=None, token_mask=None, stream=None):
    """dlogits [N, E] float32 of the router from the gradient of the mixture weights (dtopk_w [N, k], or None) and of the
    balance loss (coef [S, E] of moe_balance_loss with its seq_rows and token_mask, or None; dloss [1] float32, None: 1)."""
    torch = _torch or _import_torch()
    E, k, f = cfg.n_routed_experts, cfg.num_experts_per_tok, torch.float32
    S = (N + seq_rows - 1) // seq_rows if seq_rows > 0 else 0
    mask = _token_mask(token_mask, N)
    with _same_device("moe_route_backward", scores, topk_idx, dtopk_w, coef, dloss, token_mask, dlogits):
        st = lib().moe_route_backward(
            ctypes.byref(cfg), int(N), _ptr(scores, "scores", f, (N, E)),
            _ptr(topk_idx, "topk_idx", torch.int32, (N, k), required=False),
            _ptr(dtopk_w, "dtopk_w", f, (N, k), required=False), int(seq_rows),
            _ptr(coef, "coef", f, (S, E), required=False), _ptr(dloss, "dloss", f, (1,), required=False), mask,
            _ptr(dlogits, "dlogits", f, (N, E)), _stream(stream))
    _check(st, "moe_route_backward")


class MoeTensorList:
    """Tensors for moe_grad_norm and moe_grad_clip, described once: calls with the list then cost no walk over it.
    Holds the tensors, so their memory stays theirs; build it anew when gradients move to other memory."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        for i, t in enumerate(self.tensors):
            _tensor_dtype(t, f"tensors[{i}]")
        self.array = (MoeTensor * max(1, len(self.tensors)))(
            *(MoeTensor(_ptr(t, f"tensors[{i}]"), t.numel(), _tensor_dtype(t, f"tensors[{i}]"))
              for i, t in enumerate(self.tensors)))
        _same_device("moe_tensor_list", *self.tensors)

    def __len__(self):
        return len(self.tensors)


def moe_tensor_list(tensors) -> MoeTensorList:
    """A MoeTensorList of contiguous bfloat16 or float32 device tensors of one device (any length; views into a buffer
    need the alignment of their type alone)."""
    return tensors if isinstance(tensors, MoeTensorList) else MoeTensorList(tensors)


def moe_grad_norm_workspace_size(tensors) -> int:
    t = moe_tensor_list(tensors)
    return int(lib().moe_grad_norm_workspace_size(t.array, len(t)))


def moe_grad_norm(tensors, norm, workspace, stream=None):
    """norm[0] = the 2-norm over all values of the tensors (a sequence or a MoeTensorList); workspace:
    moe_grad_norm_workspace_size(tensors) bytes."""
    torch = _torch or _import_torch()
    t = moe_tensor_list(tensors)
    ws, ws_bytes = _ws(workspace)
    with _same_device("moe_grad_norm", *t.tensors[:1], norm, workspace):
        st = lib().moe_grad_norm(t.array, len(t), _ptr(norm, "norm", torch.float32, (1,)), ws, ws_bytes,
                                 _stream(stream))
    _check(st, "moe_grad_norm")


def moe_grad_clip(tensors, norm, max_norm: float, out=None, eps: float = 1e-6, stream=None):
    """out[i] = tensors[i] * min(1, max_norm / (norm[0] + eps)), read on the device; out None: in place. out may have
    types of its own (bfloat16 gradients clipped into float32 ones)."""
    torch = _torch or _import_torch()
    t = moe_tensor_list(tensors)
    o = None if out is None else moe_tensor_list(out)
    if o is not None and len(o) != len(t):
        raise ValueError(f"out must have {len(t)} tensors, got {len(o)}")
    with _same_device("moe_grad_clip", *t.tensors[:1], *(o.tensors[:1] if o is not None else ()), norm):
        st = lib().moe_grad_clip(t.array, None if o is None else o.array, len(t),
                                 _ptr(norm, "norm", torch.float32, (1,)), float(max_norm), float(eps), _stream(stream))
    _check(st, "moe_grad_clip")


def stage_names() -> list:
    L = lib()
    return [L.moe_stage_name(i).decode() for i in range(L.moe_stage_count())]


def profile_begin(stages=None) -> None:
    """Start per-stage timing; `stages` (stage names) limits it to those stages."""
    if stages is None:
        _check(lib().moe_profile_begin(), "moe_profile_begin")
        return
    names = stage_names()
    mask = 0
    for st in stages:
        mask |= 1 << names.index(st)
    _check(lib().moe_profile_begin_mask(mask), "moe_profile_begin_mask")


def profile_end() -> dict:
    """{stage name: (total ms, launches)} for the launches since profile_begin()."""
    import numpy as np

    names = stage_names()
    ms = np.zeros(len(names), np.float64)
    n = np.zeros(len(names), np.int32)
    _check(lib().moe_profile_end(ms.ctypes.data, n.ctypes.data, len(names)), "moe_profile_end")
    return {names[i]: (float(ms[i]), int(n[i])) for i in range(len(names))}

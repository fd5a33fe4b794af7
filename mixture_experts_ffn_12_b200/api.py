"""Python binding of libmoe: argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; this module turns
torch CUDA tensors into the pointers and sizes of the C ABI (include/moe.h),
allocates outputs and workspaces with torch, and passes torch's current
stream.  There is no fallback: without the library or a CUDA device the calls
raise.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
from typing import Dict, Optional, Tuple

import numpy as np
import torch

from . import _lib
from ._lib import MoeConfig, MoeExpertWeights


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {_lib.status_string(code)}" if what else _lib.status_string(code))


def _check(code: int, what: str) -> None:
    if code != _lib.MOE_OK:
        raise MoeError(code, what)


_DT = {"bf16": (_lib.MOE_BF16, torch.bfloat16), "f32": (_lib.MOE_F32, torch.float32)}
# expert-weight formats: dense, MXFP4 (decoded to bf16 in the GEMM mainloop), MXFP4 with MXFP8
# activations on the block-scaled tensor cores
_WF = {"dense": _lib.MOE_W_DENSE, "mxfp4": _lib.MOE_W_MXFP4, "mxfp4_a8": _lib.MOE_W_MXFP4_A8}


def make_config(hidden_size: int, intermediate_size: int, num_local_experts: int, num_experts_per_tok: int,
                swiglu_limit: float = 7.0, swiglu_alpha: float = 1.702, dtype: str = "bf16",
                wfmt: str = "dense", y_f32: bool = False, h_split: bool = False) -> MoeConfig:
    """y_f32: the layer output y is stored in fp32 (the sums before their rounding to dtype).
    h_split: the SwiGLU output is kept as two bf16 halves (hi + lo) between the expert GEMMs."""
    return MoeConfig(hidden_size, intermediate_size, num_local_experts, num_experts_per_tok, swiglu_limit,
                     swiglu_alpha, _DT[dtype][0], _WF[wfmt], 1 if y_f32 else 0, 1 if h_split else 0)


def config_from_spec(spec, y_f32: bool = False, h_split: bool = False, wfmt: Optional[str] = None) -> MoeConfig:
    """Config of a ``workloads.LayerSpec``; `wfmt` overrides the spec's weight format (the MXFP4
    weights of a spec also run as "mxfp4_a8")."""
    return make_config(spec.D, spec.F, spec.E, spec.k, spec.limit, spec.alpha, spec.dtype, wfmt or spec.wfmt,
                       y_f32, h_split)


def torch_dtype(cfg: MoeConfig) -> torch.dtype:
    return torch.bfloat16 if cfg.dtype == _lib.MOE_BF16 else torch.float32


def out_dtype(cfg: MoeConfig) -> torch.dtype:
    """dtype of the layer output y: fp32 when cfg.y_f32 is set, else the layer dtype."""
    return torch.float32 if cfg.y_f32 else torch_dtype(cfg)


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libmoe takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("libmoe takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


# --------------------------------------------------------------------------- #
# argument checks: the C ABI sees pointers only, so shapes and dtypes are checked
# here, against the layouts include/moe.h documents, before any pointer is passed
# (a bf16 buffer passed where fp32 is declared would be read past its end).
# These checks touch no device and run on CPU tensors too.
# --------------------------------------------------------------------------- #
def _want(name: str, t: Optional[torch.Tensor], shape, dtype: torch.dtype,
          device: Optional[torch.device] = None) -> None:
    if (t is not None and t.shape == shape and t.dtype is dtype and t.is_contiguous()
            and (device is None or t.device == device)):
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _rows(name: str, t: Optional[torch.Tensor]) -> int:
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dim() == 0:
        raise ValueError(f"{name} must have a leading token dimension")
    return int(t.shape[0])


def check_expert_weights(cfg: MoeConfig, w: "ExpertWeights", device: Optional[torch.device] = None) -> None:
    """Dense: W_g, W_u [E, F, D], W_d [E, D, F] in the layer dtype.  MXFP4: packed E2M1
    codes [E, F, D/2], [E, F, D/2], [E, D, F/2] and E8M0 scales [E, F, D/32], [E, F, D/32],
    [E, D, F/32], all uint8.  Biases [E, F], [E, F], [E, D] in the layer dtype."""
    D, F, E = cfg.hidden_size, cfg.intermediate_size, cfg.num_local_experts
    dt = torch_dtype(cfg)
    if cfg.wfmt in (_lib.MOE_W_MXFP4, _lib.MOE_W_MXFP4_A8):
        if D % 32 or F % 32:
            raise ValueError(f"MXFP4 weights need D and F divisible by 32 (D={D}, F={F})")
        _want("w_gate", w.w_gate, (E, F, D // 2), torch.uint8, device)
        _want("w_up", w.w_up, (E, F, D // 2), torch.uint8, device)
        _want("w_down", w.w_down, (E, D, F // 2), torch.uint8, device)
        _want("s_gate", w.s_gate, (E, F, D // 32), torch.uint8, device)
        _want("s_up", w.s_up, (E, F, D // 32), torch.uint8, device)
        _want("s_down", w.s_down, (E, D, F // 32), torch.uint8, device)
    else:
        _want("w_gate", w.w_gate, (E, F, D), dt, device)
        _want("w_up", w.w_up, (E, F, D), dt, device)
        _want("w_down", w.w_down, (E, D, F), dt, device)
    _want("b_gate", w.b_gate, (E, F), dt, device)
    _want("b_up", w.b_up, (E, F), dt, device)
    _want("b_down", w.b_down, (E, D), dt, device)


def check_router_args(cfg: MoeConfig, x, w_router, b_router, topk_ids=None, topk_w=None) -> int:
    """x [T, D], W_r [E, D], b_r [E] in the layer dtype; topk_ids [T, k] int32 and
    topk_w [T, k] fp32 when given.  Returns T."""
    D, E, k = cfg.hidden_size, cfg.num_local_experts, cfg.num_experts_per_tok
    dt = torch_dtype(cfg)
    T = _rows("x", x)
    _want("x", x, (T, D), dt)
    _want("w_router", w_router, (E, D), dt, x.device)
    _want("b_router", b_router, (E,), dt, x.device)
    if topk_ids is not None:
        _want("topk_ids", topk_ids, (T, k), torch.int32, x.device)
    if topk_w is not None:
        _want("topk_w", topk_w, (T, k), torch.float32, x.device)
    return T


def check_permute_args(cfg: MoeConfig, topk_ids, x=None) -> int:
    """topk_ids [T, k] int32; x [T, D] in the layer dtype when given.  Returns T."""
    T = _rows("topk_ids", topk_ids)
    _want("topk_ids", topk_ids, (T, cfg.num_experts_per_tok), torch.int32)
    if x is not None:
        _want("x", x, (T, cfg.hidden_size), torch_dtype(cfg), topk_ids.device)
    return T


def check_expert_ffn_args(cfg: MoeConfig, x_perm, expert_off, weights: "ExpertWeights") -> int:
    """x_perm [R, D] in the layer dtype with R = T·k; expert_off [E+1] int32.  Returns T."""
    R, k = _rows("x_perm", x_perm), cfg.num_experts_per_tok
    if R % k:
        raise ValueError(f"x_perm has {R} rows, not a multiple of k = {k}")
    _want("x_perm", x_perm, (R, cfg.hidden_size), torch_dtype(cfg))
    _want("expert_off", expert_off, (cfg.num_local_experts + 1,), torch.int32, x_perm.device)
    check_expert_weights(cfg, weights, x_perm.device)
    return R // k


def check_combine_args(cfg: MoeConfig, y_perm, row_of_slot, topk_w) -> int:
    """y_perm [T·k, D] in the layer dtype; row_of_slot [T, k] int32; topk_w [T, k] fp32.  Returns T."""
    k = cfg.num_experts_per_tok
    T = _rows("row_of_slot", row_of_slot)
    _want("row_of_slot", row_of_slot, (T, k), torch.int32)
    _want("y_perm", y_perm, (T * k, cfg.hidden_size), torch_dtype(cfg), row_of_slot.device)
    _want("topk_w", topk_w, (T, k), torch.float32, row_of_slot.device)
    return T


def check_layer_args(cfg: MoeConfig, x, w_router, b_router, weights: Optional["ExpertWeights"], y=None,
                     topk_ids=None, topk_w=None) -> int:
    """The router's arguments, the expert weights (skipped when None: already checked)
    and y [T, D] in the output dtype (``out_dtype``) when given.  Returns T."""
    T = check_router_args(cfg, x, w_router, b_router, topk_ids, topk_w)
    if weights is not None:
        check_expert_weights(cfg, weights, x.device)
    if y is not None:
        _want("y", y, (T, cfg.hidden_size), out_dtype(cfg), x.device)
    return T


def _stream(device: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _new(shape, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    """A new contiguous tensor (torch.empty takes 0.8 us longer to read its arguments)."""
    if len(shape) == 2:
        return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def _workspace(ws: Optional[torch.Tensor], n: int, device: torch.device) -> torch.Tensor:
    """`ws` (checked) or a new workspace of n bytes."""
    if ws is None:
        return torch.empty_strided((max(n, 16),), (1,), dtype=torch.uint8, device=device)
    if ws.device != device:
        raise ValueError(f"ws is on {ws.device}, expected {device}")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws


def _launch(what: str, device: torch.device, *args) -> None:
    """Calls the library function `what` with torch's current stream of `device` behind args, that device
    current.  Tensors in args are checked ones (``_want``): their addresses are passed."""
    if device.type != "cuda":
        raise ValueError("libmoe takes CUDA tensors")
    fn = getattr(_lib.load(), what)
    args = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    if torch.cuda.current_device() == device.index:
        code = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            code = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if code != _lib.MOE_OK:
        raise MoeError(code, what)


@dataclasses.dataclass
class ExpertWeights:
    """Device expert parameters: dense (dtype) or MXFP4 (uint8 codes + E8M0 scales)."""
    w_gate: torch.Tensor
    w_up: torch.Tensor
    w_down: torch.Tensor
    b_gate: torch.Tensor
    b_up: torch.Tensor
    b_down: torch.Tensor
    s_gate: Optional[torch.Tensor] = None
    s_up: Optional[torch.Tensor] = None
    s_down: Optional[torch.Tensor] = None

    def c_struct(self) -> MoeExpertWeights:
        return MoeExpertWeights(*(None if t is None else t.data_ptr() for t in (
            self.w_gate, self.w_up, self.w_down, self.s_gate, self.s_up, self.s_down,
            self.b_gate, self.b_up, self.b_down)))


def to_torch(a: np.ndarray) -> torch.Tensor:
    """Host array from ``workloads`` -> torch CPU tensor (uint16 bits -> bfloat16)."""
    if a.dtype == np.uint16:
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(a))


def upload_layer(layer: Dict[str, np.ndarray], device="cuda") -> Dict[str, torch.Tensor]:
    return {k: to_torch(v).to(device) for k, v in layer.items()}


def expert_weights_from(d: Dict[str, torch.Tensor]) -> ExpertWeights:
    return ExpertWeights(d["w_gate"], d["w_up"], d["w_down"], d["b_gate"], d["b_up"], d["b_down"],
                         d.get("s_gate"), d.get("s_up"), d.get("s_down"))


# --------------------------------------------------------------------------- #
# the five calls (each on torch's current stream of the tensors' device)
# --------------------------------------------------------------------------- #
def _size(n: int, what: str) -> int:
    if n == _lib.SIZE_INVALID:
        raise MoeError(_lib.MOE_ERR_INVALID_ARG, what)
    return n


def router_topk(cfg: MoeConfig, x: torch.Tensor, w_router: torch.Tensor, b_router: torch.Tensor,
                topk_ids: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None
                ) -> Tuple[torch.Tensor, torch.Tensor]:
    T = check_router_args(cfg, x, w_router, b_router, topk_ids, topk_w)
    k = cfg.num_experts_per_tok
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    with torch.cuda.device(x.device):
        _check(_lib.load().moe_router_topk(ctypes.byref(cfg), T, _p(x), _p(w_router), _p(b_router), _p(topk_ids),
                                           _p(topk_w), _stream(x.device)), "moe_router_topk")
    return topk_ids, topk_w


def permute(cfg: MoeConfig, topk_ids: torch.Tensor, x: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    T = check_permute_args(cfg, topk_ids, x)
    L = _lib.load()
    k, dev = cfg.num_experts_per_tok, topk_ids.device
    R = T * k
    out = dict(
        expert_off=torch.empty(cfg.num_local_experts + 1, dtype=torch.int32, device=dev),
        row_of_slot=torch.empty((T, k), dtype=torch.int32, device=dev),
        slot_of_row=torch.empty(R, dtype=torch.int32, device=dev),
    )
    out["x_perm"] = None if x is None else torch.empty((R, cfg.hidden_size), dtype=x.dtype, device=dev)
    nws = _size(L.moe_permute_workspace_size(ctypes.byref(cfg), T), "moe_permute_workspace_size")
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check(L.moe_permute(ctypes.byref(cfg), T, _p(topk_ids), _p(x), _p(out["expert_off"]),
                             _p(out["row_of_slot"]), _p(out["slot_of_row"]), _p(out["x_perm"]), _p(ws), ws.numel(),
                             _stream(dev)), "moe_permute")
    return out


def expert_ffn(cfg: MoeConfig, x_perm: torch.Tensor, expert_off: torch.Tensor, weights: ExpertWeights
               ) -> Tuple[torch.Tensor, torch.Tensor]:
    T = check_expert_ffn_args(cfg, x_perm, expert_off, weights)
    L = _lib.load()
    R, dev = x_perm.shape[0], x_perm.device
    dt = torch_dtype(cfg)
    # with h_split (bf16) each row of h holds the bf16 halves hi and lo: [R, 2, F]
    halves = 2 if (cfg.h_split and cfg.dtype == _lib.MOE_BF16) else 1
    h = torch.empty((R, halves * cfg.intermediate_size), dtype=dt, device=dev)
    y_perm = torch.empty((R, cfg.hidden_size), dtype=dt, device=dev)
    nws = _size(L.moe_expert_ffn_workspace_size(ctypes.byref(cfg), T), "moe_expert_ffn_workspace_size")
    ws = torch.empty(nws, dtype=torch.uint8, device=dev) if nws else None
    ws_struct = weights.c_struct()
    with torch.cuda.device(dev):
        _check(L.moe_expert_ffn(ctypes.byref(cfg), T, _p(x_perm), _p(expert_off), ctypes.byref(ws_struct), _p(h),
                                _p(y_perm), _p(ws), nws, _stream(dev)), "moe_expert_ffn")
    return h, y_perm


def combine(cfg: MoeConfig, y_perm: torch.Tensor, row_of_slot: torch.Tensor, topk_w: torch.Tensor) -> torch.Tensor:
    T = check_combine_args(cfg, y_perm, row_of_slot, topk_w)
    dev = y_perm.device
    y = torch.empty((T, cfg.hidden_size), dtype=out_dtype(cfg), device=dev)
    with torch.cuda.device(dev):
        _check(_lib.load().moe_combine(ctypes.byref(cfg), T, _p(y_perm), _p(row_of_slot), _p(topk_w), _p(y),
                                       _stream(dev)), "moe_combine")
    return y


def workspace_size(cfg: MoeConfig, T: int) -> int:
    return _size(_lib.load().moe_workspace_size(ctypes.byref(cfg), T), "moe_workspace_size")


def layer_forward(cfg: MoeConfig, x: torch.Tensor, w_router: torch.Tensor, b_router: torch.Tensor,
                  weights: ExpertWeights, y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                  topk_ids: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                  _weights_checked: bool = False) -> torch.Tensor:
    T = check_layer_args(cfg, x, w_router, b_router, None if _weights_checked else weights, y, topk_ids, topk_w)
    dev = x.device
    if y is None:
        y = torch.empty((T, cfg.hidden_size), dtype=out_dtype(cfg), device=dev)
    if ws is None:
        ws = torch.empty(max(workspace_size(cfg, T), 16), dtype=torch.uint8, device=dev)
    elif ws.device != dev:
        raise ValueError(f"ws is on {ws.device}, expected {dev}")
    wst = weights.c_struct()
    with torch.cuda.device(dev):
        _check(_lib.load().moe_layer_forward(ctypes.byref(cfg), T, _p(x), _p(w_router), _p(b_router),
                                             ctypes.byref(wst), _p(y), _p(topk_ids), _p(topk_w), _p(ws),
                                             ws.numel() * ws.element_size(), _stream(dev)), "moe_layer_forward")
    return y


# --------------------------------------------------------------------------- #
# the GLM4-MoE-Lite variant (moe_glm_*)
# --------------------------------------------------------------------------- #
@dataclasses.dataclass
class GlmParams:
    """Router and shared-expert parameters of the GLM4-MoE-Lite variant (moe_glm_params_t):
    e_score_correction_bias [E] and the shared expert ws_gate / ws_up [Fs, D], ws_down [D, Fs],
    all in the layer dtype and optional."""
    norm_topk_prob: bool = True
    routed_scaling_factor: float = 1.0
    e_score_correction_bias: Optional[torch.Tensor] = None
    ws_gate: Optional[torch.Tensor] = None
    ws_up: Optional[torch.Tensor] = None
    ws_down: Optional[torch.Tensor] = None

    @property
    def shared_intermediate_size(self) -> int:
        return 0 if self.ws_gate is None else int(self.ws_gate.shape[0])

    def c_struct(self) -> _lib.MoeGlmParams:
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        return _lib.MoeGlmParams(1 if self.norm_topk_prob else 0, float(self.routed_scaling_factor),
                                 ptr(self.e_score_correction_bias), ptr(self.ws_gate), ptr(self.ws_up),
                                 ptr(self.ws_down), self.shared_intermediate_size)


def glm_params_from(spec, d: Dict[str, torch.Tensor]) -> GlmParams:
    """Parameters of a ``workloads.GlmLayerSpec`` layer uploaded with ``upload_layer``."""
    return GlmParams(spec.norm_topk_prob, spec.routed_scaling_factor, d.get("e_score_correction_bias"),
                     d.get("ws_gate"), d.get("ws_up"), d.get("ws_down"))


def glm_expert_weights_from(d: Dict[str, torch.Tensor]) -> ExpertWeights:
    """The variant's expert weights (no biases)."""
    return ExpertWeights(d["w_gate"], d["w_up"], d["w_down"], None, None, None)


def glm_config_from_spec(spec, y_f32: bool = False, h_split: bool = False) -> MoeConfig:
    """Config of a ``workloads.GlmLayerSpec`` (the SwiGLU limit and alpha are not used by the variant)."""
    return make_config(spec.D, spec.F, spec.E, spec.k, dtype=spec.dtype, y_f32=y_f32, h_split=h_split)


def check_glm_args(cfg: MoeConfig, params: GlmParams, x, w_router, weights: Optional[ExpertWeights] = None,
                   y=None, topk_ids=None, topk_w=None) -> int:
    """x [T, D], W_r [E, D], e_score_correction_bias [E], the shared expert (all three or none:
    [Fs, D], [Fs, D], [D, Fs]) and, when given, the expert weights (dense, no biases) and
    y [T, D], in the layer dtype; topk_ids [T, k] int32 and topk_w [T, k] fp32.  Returns T."""
    D, F, E, k = cfg.hidden_size, cfg.intermediate_size, cfg.num_local_experts, cfg.num_experts_per_tok
    dt = torch_dtype(cfg)
    if cfg.wfmt != _lib.MOE_W_DENSE:
        raise ValueError("the GLM4-MoE-Lite variant takes dense expert weights")
    T = _rows("x", x)
    dev = x.device
    _want("x", x, (T, D), dt)
    _want("w_router", w_router, (E, D), dt, dev)
    if params.e_score_correction_bias is not None:
        _want("e_score_correction_bias", params.e_score_correction_bias, (E,), dt, dev)
    shared = [params.ws_gate, params.ws_up, params.ws_down]
    if any(t is not None for t in shared):
        Fs = _rows("ws_gate", params.ws_gate)
        _want("ws_gate", params.ws_gate, (Fs, D), dt, dev)
        _want("ws_up", params.ws_up, (Fs, D), dt, dev)
        _want("ws_down", params.ws_down, (D, Fs), dt, dev)
    if weights is not None:
        _want("w_gate", weights.w_gate, (E, F, D), dt, dev)
        _want("w_up", weights.w_up, (E, F, D), dt, dev)
        _want("w_down", weights.w_down, (E, D, F), dt, dev)
    if y is not None:
        _want("y", y, (T, D), out_dtype(cfg), dev)
    if topk_ids is not None:
        _want("topk_ids", topk_ids, (T, k), torch.int32, dev)
    if topk_w is not None:
        _want("topk_w", topk_w, (T, k), torch.float32, dev)
    return T


def glm_router_topk(cfg: MoeConfig, params: GlmParams, x: torch.Tensor, w_router: torch.Tensor,
                    topk_ids: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None
                    ) -> Tuple[torch.Tensor, torch.Tensor]:
    T = check_glm_args(cfg, params, x, w_router, topk_ids=topk_ids, topk_w=topk_w)
    L = _lib.load()
    k, dev = cfg.num_experts_per_tok, x.device
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
    nws = _size(L.moe_glm_router_workspace_size(ctypes.byref(cfg), T), "moe_glm_router_workspace_size")
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev)
    gp = params.c_struct()
    with torch.cuda.device(dev):
        _check(L.moe_glm_router_topk(ctypes.byref(cfg), ctypes.byref(gp), T, _p(x), _p(w_router), _p(topk_ids),
                                     _p(topk_w), _p(ws), ws.numel(), _stream(dev)), "moe_glm_router_topk")
    return topk_ids, topk_w


def glm_workspace_size(cfg: MoeConfig, params: GlmParams, T: int) -> int:
    gp = params.c_struct()
    return _size(_lib.load().moe_glm_workspace_size(ctypes.byref(cfg), ctypes.byref(gp), T), "moe_glm_workspace_size")


def glm_layer_forward(cfg: MoeConfig, params: GlmParams, x: torch.Tensor, w_router: torch.Tensor,
                      weights: ExpertWeights, y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                      topk_ids: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None
                      ) -> torch.Tensor:
    T = check_glm_args(cfg, params, x, w_router, weights, y, topk_ids, topk_w)
    dev = x.device
    if y is None:
        y = torch.empty((T, cfg.hidden_size), dtype=out_dtype(cfg), device=dev)
    if ws is None:
        ws = torch.empty(max(glm_workspace_size(cfg, params, T), 16), dtype=torch.uint8, device=dev)
    elif ws.device != dev:
        raise ValueError(f"ws is on {ws.device}, expected {dev}")
    wst = weights.c_struct()
    gp = params.c_struct()
    with torch.cuda.device(dev):
        _check(_lib.load().moe_glm_layer_forward(ctypes.byref(cfg), ctypes.byref(gp), T, _p(x), _p(w_router),
                                                 ctypes.byref(wst), _p(y), _p(topk_ids), _p(topk_w), _p(ws),
                                                 ws.numel() * ws.element_size(), _stream(dev)),
               "moe_glm_layer_forward")
    return y


def quantize_mxfp8(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [rows, K] bf16 -> (E4M3 codes [rows, K] uint8, E8M0 scale rows [rows, stride] uint8)."""
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        raise ValueError("quantize_mxfp8 takes a 2-D bf16 tensor")
    L = _lib.load()
    rows, K = x.shape
    stride = L.moe_mxfp8_scale_stride(K)
    xq = torch.empty((rows, K), dtype=torch.uint8, device=x.device)
    sf = torch.empty((rows, max(stride, 1)), dtype=torch.uint8, device=x.device)
    with torch.cuda.device(x.device):
        _check(L.moe_quantize_mxfp8(rows, K, _p(x), _p(xq), _p(sf), _stream(x.device)), "moe_quantize_mxfp8")
    return xq, sf


# --------------------------------------------------------------------------- #
# MXFP4 quantization and the MXFP4 x MXFP4 linear layer
# --------------------------------------------------------------------------- #
_DT_OF = {torch.bfloat16: _lib.MOE_BF16, torch.float32: _lib.MOE_F32}


def quantize_mxfp4(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [..., K] bf16 or fp32 -> (E2M1 codes [..., K/2] uint8, E8M0 scales [..., K/32] uint8), the
    layout of MXFP4 expert weights (moe_quantize_mxfp4)."""
    if x.dim() < 1 or x.dtype not in _DT_OF:
        raise ValueError("quantize_mxfp4 takes a bf16 or fp32 tensor of at least one dimension")
    if not x.is_contiguous():
        raise ValueError("quantize_mxfp4: x must be contiguous")
    K = x.shape[-1]
    if K == 0 or K % 32:
        raise ValueError(f"quantize_mxfp4: the last dimension ({K}) must be a positive multiple of 32")
    lead = x.shape[:-1]
    codes = _new((*lead, K // 2), torch.uint8, x.device)
    scales = _new((*lead, K // 32), torch.uint8, x.device)
    _launch("moe_quantize_mxfp4", x.device, x.numel() // K, K, _DT_OF[x.dtype], x, codes, scales)
    return codes, scales


def dequantize_mxfp4(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values of quantize_mxfp4's codes and scales, [..., K] in dtype (exact; NaN for scale byte 255)."""
    if codes.dim() < 1 or codes.dtype != torch.uint8:
        raise ValueError("dequantize_mxfp4 takes uint8 codes [..., K/2]")
    if not codes.is_contiguous():
        raise ValueError("dequantize_mxfp4: codes must be contiguous")
    if dtype not in _DT_OF:
        raise ValueError("dequantize_mxfp4 gives bf16 or fp32")
    K = 2 * codes.shape[-1]
    if K == 0 or K % 32:
        raise ValueError(f"dequantize_mxfp4: K = {K} must be a positive multiple of 32")
    lead = codes.shape[:-1]
    _want("scales", scales, (*lead, K // 32), torch.uint8, codes.device)
    out = _new((*lead, K), dtype, codes.device)
    _launch("moe_dequantize_mxfp4", codes.device, out.numel() // K, K, codes, scales, _DT_OF[dtype], out)
    return out


@dataclasses.dataclass
class Mxfp4Weights:
    """Weights of ``mxfp4_linear``: E2M1 codes [G, N, K/2] and the scales as moe_mxfp4_weight_tiles lays
    them out (flat uint8).  ``mxfp4_weights`` makes them from codes and scales."""
    codes: torch.Tensor
    tiles: torch.Tensor


def _mxfp4_sizes(codes: torch.Tensor) -> Tuple[int, int, int]:
    if codes.dim() != 3 or codes.dtype != torch.uint8:
        raise ValueError("MXFP4 weight codes are uint8 [G, N, K/2]")
    return codes.shape[0], codes.shape[1], 2 * codes.shape[2]


def mxfp4_weights(codes: torch.Tensor, scales: torch.Tensor) -> Mxfp4Weights:
    """codes [G, N, K/2], scales [G, N, K/32] (quantize_mxfp4's, or MXFP4 expert weights) -> Mxfp4Weights."""
    G, N, K = _mxfp4_sizes(codes)
    L = _lib.load()
    _want("codes", codes, (G, N, K // 2), torch.uint8)
    _want("scales", scales, (G, N, K // 32), torch.uint8, codes.device)
    n = _size(L.moe_mxfp4_weight_tiles_size(G, N, K), "moe_mxfp4_weight_tiles_size")
    tiles = torch.empty(n, dtype=torch.uint8, device=codes.device)
    _launch("moe_mxfp4_weight_tiles", codes.device, G, N, K, scales, tiles)
    return Mxfp4Weights(codes, tiles)


def check_mxfp4_linear_args(x, w: Mxfp4Weights, bias=None, group_off=None, y=None, out_f32: bool = False) -> int:
    """x [R, K] bf16, w from ``mxfp4_weights``, bias [G, N] bf16 and group_off [G+1] int32 when given
    (group_off is required for G > 1), y [R, N] bf16 (fp32 with out_f32) when given.  Returns R."""
    G, N, K = _mxfp4_sizes(w.codes)
    R = _rows("x", x)
    dev = x.device
    _want("x", x, (R, K), torch.bfloat16)
    _want("w.codes", w.codes, w.codes.shape, torch.uint8, dev)
    n = _size(_lib.load().moe_mxfp4_weight_tiles_size(G, N, K), "moe_mxfp4_weight_tiles_size")
    _want("w.tiles", w.tiles, (n,), torch.uint8, dev)
    if bias is not None:
        _want("bias", bias, (G, N), torch.bfloat16, dev)
    if group_off is not None:
        _want("group_off", group_off, (G + 1,), torch.int32, dev)
    elif G != 1:
        raise ValueError("group_off is required for more than one group of weights")
    if y is not None:
        _want("y", y, (R, N), torch.float32 if out_f32 else torch.bfloat16, dev)
    return R


def mxfp4_linear(x: torch.Tensor, w: Mxfp4Weights, bias: Optional[torch.Tensor] = None,
                 group_off: Optional[torch.Tensor] = None, out_f32: bool = False, y: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[r] = q(x)[r] W_g^T + bias_g for the rows r of group g (group_off as expert_off; all rows if None),
    x quantized to MXFP4 in the call: 4-bit x 4-bit products on the block-scaled tensor cores
    (moe_mxfp4_linear).  Rows of no group are not written: those of a new y hold anything."""
    R = check_mxfp4_linear_args(x, w, bias, group_off, y, out_f32)
    G, N, K = _mxfp4_sizes(w.codes)
    L, dev = _lib.load(), x.device
    if y is None:
        y = _new((R, N), torch.float32 if out_f32 else torch.bfloat16, dev)
    ws = _workspace(ws, _size(L.moe_mxfp4_linear_workspace_size(G, R, N, K), "moe_mxfp4_linear_workspace_size"), dev)
    _launch("moe_mxfp4_linear", dev, G, R, N, K, x, group_off, w.codes, w.tiles, bias, 1 if out_f32 else 0, y, ws,
            ws.numel() * ws.element_size())
    return y


def quantize_experts(cfg: MoeConfig, w: ExpertWeights, wfmt: str = "mxfp4") -> Tuple[MoeConfig, ExpertWeights]:
    """Dense bf16 expert weights -> (config, weights) of the same layer with MXFP4 weights (wfmt "mxfp4"
    or "mxfp4_a8"); biases stay as they are.  h_split does not carry over: layers with MXFP4 weights keep
    h in bf16 ("mxfp4") or MXFP8 ("mxfp4_a8")."""
    if cfg.wfmt != _lib.MOE_W_DENSE or cfg.dtype != _lib.MOE_BF16:
        raise ValueError("quantize_experts takes dense bf16 expert weights")
    if wfmt not in ("mxfp4", "mxfp4_a8"):
        raise ValueError(f"wfmt {wfmt!r}: 'mxfp4' or 'mxfp4_a8'")
    check_expert_weights(cfg, w)
    new = MoeConfig(cfg.hidden_size, cfg.intermediate_size, cfg.num_local_experts, cfg.num_experts_per_tok,
                    cfg.swiglu_limit, cfg.swiglu_alpha, cfg.dtype, _WF[wfmt], cfg.y_f32, 0)
    _check(_lib.load().moe_config_check(ctypes.byref(new)), "moe_config_check")
    (cg, sg), (cu, su), (cd, sd) = (quantize_mxfp4(t) for t in (w.w_gate, w.w_up, w.w_down))
    return new, ExpertWeights(cg, cu, cd, w.b_gate, w.b_up, w.b_down, sg, su, sd)


# --------------------------------------------------------------------------- #
# training pass of the expert block
# --------------------------------------------------------------------------- #
_ACT = {"swiglu": _lib.MOE_ACT_SWIGLU, "silu": _lib.MOE_ACT_SILU}


def _act_code(act: str) -> int:
    if act not in _ACT:
        raise ValueError(f"act {act!r}: 'swiglu' (the layer's clipped SwiGLU) or 'silu'")
    return _ACT[act]


def check_ffn_train_args(cfg: MoeConfig, x_perm, expert_off, w: ExpertWeights, gu=None, h=None, dy_perm=None) -> int:
    """x_perm [R, D] with R = T*k, expert_off [E+1] int32, dense weights in the layer dtype (each bias
    may be None); for the backward pass gu [R, 2, F], h [R, F] and dy_perm [R, D].  Returns T."""
    D, F, E, k = cfg.hidden_size, cfg.intermediate_size, cfg.num_local_experts, cfg.num_experts_per_tok
    dt = torch_dtype(cfg)
    if cfg.wfmt != _lib.MOE_W_DENSE:
        raise ValueError("the training pass takes dense expert weights")
    R = _rows("x_perm", x_perm)
    if R % k:
        raise ValueError(f"x_perm has {R} rows, not a multiple of k = {k}")
    dev = x_perm.device
    _want("x_perm", x_perm, (R, D), dt)
    _want("expert_off", expert_off, (E + 1,), torch.int32, dev)
    _want("w_gate", w.w_gate, (E, F, D), dt, dev)
    _want("w_up", w.w_up, (E, F, D), dt, dev)
    _want("w_down", w.w_down, (E, D, F), dt, dev)
    for name, t, n in (("b_gate", w.b_gate, F), ("b_up", w.b_up, F), ("b_down", w.b_down, D)):
        if t is not None:
            _want(name, t, (E, n), dt, dev)
    if dy_perm is not None:
        _want("gu", gu, (R, 2, F), dt, dev)
        _want("h", h, (R, F), dt, dev)
        _want("dy_perm", dy_perm, (R, D), dt, dev)
    return R // k


def expert_ffn_train(cfg: MoeConfig, x_perm: torch.Tensor, expert_off: torch.Tensor, weights: ExpertWeights,
                     act: str = "swiglu") -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """expert_ffn that also keeps the pre-activations: (gu [R, 2, F], h [R, F], y_perm [R, D]).
    act: "swiglu" (the layer's clipped SwiGLU) or "silu"; biases may be None.  Rows of no expert are not
    written and hold anything.  A call of its own, which autograd does not see: expert_ffn_backward is its
    backward pass."""
    code = _act_code(act)
    T = check_ffn_train_args(cfg, x_perm, expert_off, weights)
    R, dev, dt = x_perm.shape[0], x_perm.device, x_perm.dtype
    F = cfg.intermediate_size
    gu = torch.empty_strided((R, 2, F), (2 * F, F, 1), dtype=dt, device=dev)
    h = _new((R, F), dt, dev)
    y = torch.empty_like(x_perm)
    wst = weights.c_struct()
    _launch("moe_expert_ffn_train", dev, ctypes.byref(cfg), code, T, x_perm, expert_off, ctypes.byref(wst), gu, h, y)
    return gu, h, y


@dataclasses.dataclass
class ExpertGrads:
    """Gradients of the expert parameters, laid out as the parameters (moe_expert_grads_t); None: not wanted."""
    w_gate: Optional[torch.Tensor]
    w_up: Optional[torch.Tensor]
    w_down: Optional[torch.Tensor]
    b_gate: Optional[torch.Tensor] = None
    b_up: Optional[torch.Tensor] = None
    b_down: Optional[torch.Tensor] = None

    def c_struct(self) -> _lib.MoeExpertGrads:
        ts = (self.w_gate, self.w_up, self.w_down, self.b_gate, self.b_up, self.b_down)
        f32 = any(t is not None and t.dtype == torch.float32 for t in ts)
        return _lib.MoeExpertGrads(*(None if t is None else t.data_ptr() for t in ts), 1 if f32 else 0)


def expert_ffn_backward(cfg: MoeConfig, x_perm: torch.Tensor, expert_off: torch.Tensor, weights: ExpertWeights,
                        gu: torch.Tensor, h: torch.Tensor, dy_perm: torch.Tensor, act: str = "swiglu",
                        grad_f32: bool = False, need_dx: bool = True, grads: Optional[ExpertGrads] = None,
                        ws: Optional[torch.Tensor] = None) -> Tuple[Optional[torch.Tensor], ExpertGrads]:
    """Backward pass of expert_ffn_train: (dx_perm [R, D] or None, ExpertGrads).  Bias gradients come for
    the biases that `weights` has.  grad_f32: the parameters' gradients in fp32.  `grads` are buffers to
    overwrite (same layouts, one dtype; a weight's or bias's may be None: not computed, as for frozen experts; a
    bias's comes with its weight's), else new ones.  dx_perm's rows of no expert are not written and hold
    anything."""
    code = _act_code(act)
    if dy_perm is None:
        raise ValueError("dy_perm is required")
    T = check_ffn_train_args(cfg, x_perm, expert_off, weights, gu, h, dy_perm)
    L, dev = _lib.load(), x_perm.device
    D, F, E = cfg.hidden_size, cfg.intermediate_size, cfg.num_local_experts
    gdt = torch.float32 if grad_f32 else torch_dtype(cfg)
    if grads is None:
        like = torch.empty_like if gdt == x_perm.dtype else functools.partial(torch.empty_like, dtype=gdt)
        grads = ExpertGrads(*(None if p is None else like(p) for p in (
            weights.w_gate, weights.w_up, weights.w_down, weights.b_gate, weights.b_up, weights.b_down)))
    else:
        for name, t, bias, shape in (("gate", grads.w_gate, grads.b_gate, (E, F, D)),
                                     ("up", grads.w_up, grads.b_up, (E, F, D)),
                                     ("down", grads.w_down, grads.b_down, (E, D, F))):
            if t is not None:
                _want("grads.w_" + name, t, shape, gdt, dev)
            if bias is not None:
                if t is None:
                    raise ValueError(f"grads.b_{name} is given without grads.w_{name}")
                _want("grads.b_" + name, bias, shape[:2], gdt, dev)
    dx = torch.empty_like(x_perm) if need_dx else None
    ws = _workspace(ws, _size(L.moe_expert_ffn_backward_workspace_size(ctypes.byref(cfg), T),
                              "moe_expert_ffn_backward_workspace_size"), dev)
    wst, gst = weights.c_struct(), grads.c_struct()
    _launch("moe_expert_ffn_backward", dev, ctypes.byref(cfg), code, T, x_perm, expert_off, ctypes.byref(wst), gu, h,
            dy_perm, dx, ctypes.byref(gst), ws, ws.numel() * ws.element_size())
    return dx, grads


def combine_backward(cfg: MoeConfig, dy: torch.Tensor, y_perm: torch.Tensor, row_of_slot: torch.Tensor,
                     topk_w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Backward pass of combine: dy [T, D] (layer dtype, with y_f32 too) -> (dy_perm [T*k, D], dtopk_w [T, k]
    fp32).  row_of_slot names every row once, as permute leaves it."""
    T = check_combine_args(cfg, y_perm, row_of_slot, topk_w)
    dev = y_perm.device
    _want("dy", dy, (T, cfg.hidden_size), torch_dtype(cfg), dev)
    dy_perm = torch.empty_like(y_perm)
    dw = torch.empty_like(topk_w)
    _launch("moe_combine_backward", dev, ctypes.byref(cfg), T, dy, y_perm, row_of_slot, topk_w, dy_perm, dw)
    return dy_perm, dw


def last_device_error() -> int:
    """Reads and clears the device error word (synchronises); returns a status code."""
    return _lib.load().moe_last_device_error()


def set_expert_gemm_variant(variant: int) -> None:
    """Expert-GEMM kernel choice for bf16 dense weights: 0 = by size (the default), 1 = single-CTA
    128-row tiles, 2 = CTA-pair 256-row tiles, 3 = the weight-stationary decode kernel,
    4 = CTA pairs with the weights in M, 5 = layer_forward as the two-kernel decode layer
    wherever it applies, 6 = by size with the layer's gate/up rows gathered from x (TMA gather4)
    rather than read from x_perm, 7 = by size, with the MXFP4 x MXFP8 GEMMs widening every E2M1
    stage in their converter warps (no TMA 4-bit unpacking).  Process-wide; other MXFP4 layers
    ignore it."""
    _check(_lib.load().moe_set_expert_gemm_variant(variant), "moe_set_expert_gemm_variant")


def set_wait_limit_ns(ns: int) -> None:
    _lib.load().moe_set_wait_limit_ns(ns)


class MoELayer:
    """A GPT-OSS MoE FFN layer resident on one GPU: weights, config and a reusable workspace."""

    def __init__(self, cfg: MoeConfig, w_router: torch.Tensor, b_router: torch.Tensor, experts: ExpertWeights):
        _check(_lib.load().moe_config_check(ctypes.byref(cfg)), "moe_config_check")
        check_expert_weights(cfg, experts, w_router.device)
        self.cfg, self.w_router, self.b_router, self.experts = cfg, w_router, b_router, experts
        self._ws: Optional[torch.Tensor] = None

    def workspace(self, T: int) -> torch.Tensor:
        n = max(workspace_size(self.cfg, T), 16)
        if self._ws is None or self._ws.numel() < n:
            self._ws = torch.empty(n, dtype=torch.uint8, device=self.w_router.device)
        return self._ws

    def __call__(self, x: torch.Tensor, y: Optional[torch.Tensor] = None, topk_ids=None, topk_w=None) -> torch.Tensor:
        return layer_forward(self.cfg, x, self.w_router, self.b_router, self.experts, y=y,
                             ws=self.workspace(_rows("x", x)), topk_ids=topk_ids, topk_w=topk_w,
                             _weights_checked=True)

    def graphed(self, x: torch.Tensor, y: Optional[torch.Tensor] = None, topk_ids=None, topk_w=None):
        """Capture one forward on these fixed buffers into a CUDA graph; returns (replay, y).

        The library makes no host synchronisation and allocates nothing, so its
        launches are captured as they are; ``replay()`` re-runs them on whatever
        ``x`` holds at that time.  Removes host launch overhead (decode sizes).
        """
        if y is None:
            y = torch.empty((x.shape[0], self.cfg.hidden_size), dtype=out_dtype(self.cfg), device=x.device)
        ws = self.workspace(x.shape[0])
        self(x, y=y, topk_ids=topk_ids, topk_w=topk_w)          # warm: per-device set-up outside capture
        torch.cuda.synchronize(x.device)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer_forward(self.cfg, x, self.w_router, self.b_router, self.experts, y=y, ws=ws,
                          topk_ids=topk_ids, topk_w=topk_w, _weights_checked=True)
        return g.replay, y

    def quantized(self, wfmt: str = "mxfp4") -> "MoELayer":
        """The same layer with its dense bf16 expert weights quantized to MXFP4 (``quantize_experts``)."""
        cfg, experts = quantize_experts(self.cfg, self.experts, wfmt)
        return MoELayer(cfg, self.w_router, self.b_router, experts)

    def run_host_batches(self, xs_host, ys_host) -> None:
        """Run the layer on a sequence of pinned host batches, results into pinned host buffers.

        Batch i's host->device copy, forward and device->host copy go on three
        streams with two device buffers each way, so the copies of neighbouring
        batches overlap this batch's forward (PCIe is full duplex).  Ordering:
        copy-in(i) after forward(i-2) released its input buffer; forward(i) after
        copy-in(i) and after copy-out(i-2) released its output buffer; copy-out(i)
        after forward(i).  Returns when everything has been queued; the caller
        synchronises.  All batches must have the same shape.
        """
        if len(xs_host) == 0:
            return
        dev = self.w_router.device
        T, D = xs_host[0].shape
        xd = [torch.empty((T, D), dtype=xs_host[0].dtype, device=dev) for _ in range(2)]
        yd = [torch.empty((T, self.cfg.hidden_size), dtype=out_dtype(self.cfg), device=dev) for _ in range(2)]
        s_in, s_run, s_out = torch.cuda.Stream(dev), torch.cuda.Stream(dev), torch.cuda.Stream(dev)
        cur = torch.cuda.current_stream(dev)
        for st in (s_in, s_run, s_out):
            st.wait_stream(cur)
        copied = [torch.cuda.Event() for _ in range(2)]
        ran = [torch.cuda.Event() for _ in range(2)]
        drained = [torch.cuda.Event() for _ in range(2)]
        self.workspace(T)
        for i, (xh, yh) in enumerate(zip(xs_host, ys_host)):
            b = i % 2
            with torch.cuda.stream(s_in):
                if i >= 2:
                    s_in.wait_event(ran[b])
                xd[b].copy_(xh, non_blocking=True)
                copied[b].record(s_in)
            with torch.cuda.stream(s_run):
                s_run.wait_event(copied[b])
                if i >= 2:
                    s_run.wait_event(drained[b])
                self(xd[b], y=yd[b])
                ran[b].record(s_run)
            with torch.cuda.stream(s_out):
                s_out.wait_event(ran[b])
                yh.copy_(yd[b], non_blocking=True)
                drained[b].record(s_out)
        for st in (s_in, s_run, s_out):
            cur.wait_stream(st)
        for t in xd + yd:
            t.record_stream(s_in)
            t.record_stream(s_run)
            t.record_stream(s_out)

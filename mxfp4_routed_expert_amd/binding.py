"""ctypes binding of libmoe.so: one Python function per C entry point, same names.

Argument marshalling only: tensors are checked for device, dtype and layout, outputs and
workspaces are allocated with torch (device memory plumbing), and every computation runs
in the HIP library on torch's current stream.  If the library is missing, importing this
module raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import warnings
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 0, 1, 2, 3, 4
SCORE = {"softmax": 0, "sigmoid": 1}
WFMT = {"mxfp4": 0, "fp8b128": 1}
ACT = {"float": 0, "mxfp4": 1, "fp8": 2}
DT = {torch.bfloat16: 0, torch.float32: 1}
DT_MXFP8 = 2
DT_FP8 = 3
FP8_SCALE_F32, FP8_SCALE_E8M0, FP8_SCALE_E8M0_ROW = 0, 1, 2
GATE_NONE, GATE_TOKEN, GATE_CHANNEL = 0, 1, 2
ACT_FN = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"[status {status}] {msg}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"HIP library not built: {LIB_PATH} is missing "
                          "(run `python mxfp4_routed_expert_amd/build.py`)")
    return ctypes.CDLL(LIB_PATH)


lib = _load()

_p, _i32, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float


class RouteDesc(ctypes.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("E", _i32), ("k", _i32), ("score", _i32),
                ("renormalize", _i32), ("routed_scaling", _f32), ("n_group", _i32), ("topk_group", _i32)]


class ExpertWeightsC(ctypes.Structure):
    _fields_ = [("format", _i32), ("num_experts", _i32), ("d_model", _i32), ("d_ff", _i32),
                ("gate", _p), ("up", _p), ("down", _p), ("gate_s", _p), ("up_s", _p), ("down_s", _p)]


class LinearDesc(ctypes.Structure):
    _fields_ = [("T", _i32), ("n", _i32), ("kdim", _i32), ("fn", _i32), ("x_dtype", _i32), ("y_dtype", _i32),
                ("dx_dtype", _i32)]


class GateupDesc(ctypes.Structure):
    _fields_ = [("T", _i32), ("d_model", _i32), ("d_ff", _i32), ("fn", _i32), ("x_dtype", _i32), ("h_dtype", _i32),
                ("dh_dtype", _i32)]


class Fp8LinearDesc(ctypes.Structure):
    _fields_ = [("T", _i32), ("n", _i32), ("kdim", _i32), ("x_dtype", _i32), ("y_dtype", _i32), ("w_scale", _i32)]


class BlockNormDesc(ctypes.Structure):
    _fields_ = [("T", _i32), ("d", _i32), ("z_dtype", _i32), ("y_dtype", _i32), ("gate", _i32), ("eps", _f32),
                ("residual_scale", _f32), ("dropout", _f32)]


def _sig(name, res, *args):
    f = getattr(lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_sig("moe_last_error", ctypes.c_char_p)
_sig("moe_abi_version", _i32)
_sig("moe_route", _i32, ctypes.POINTER(RouteDesc), _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p)
_sig("moe_route_workspace", _sz, ctypes.POINTER(RouteDesc))
_sig("moe_permute", _i32, _i32, _i32, _i32, _p, _p, _p, _p, _p, _sz, _p)
_sig("moe_route_permute", _i32, ctypes.POINTER(RouteDesc), _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p)
_sig("moe_permute_workspace", _sz, _i32, _i32, _i32)
_sig("moe_route_permute_noalloc", _i32, ctypes.POINTER(RouteDesc), _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p)
_sig("moe_expert_ffn", _i32, ctypes.POINTER(ExpertWeightsC), _i32, _i32, _i32, _p, _i32, _p, _p, _p, _p, _sz, _p)
_sig("moe_expert_ffn_workspace", _sz, ctypes.POINTER(ExpertWeightsC), _i32, _i32, _i32)
_sig("moe_expert_gateup", _i32, ctypes.POINTER(ExpertWeightsC), _i32, _i32, _i32, _p, _i32, _p, _p, _p, _p, _p,
     _p, _sz, _p)
_sig("moe_expert_gateup_workspace", _sz, ctypes.POINTER(ExpertWeightsC), _i32, _i32, _i32)
_sig("moe_expert_down", _i32, ctypes.POINTER(ExpertWeightsC), _i32, _i32, _i32, _p, _p, _p, _p, _p, _p)
_sig("moe_expert_gateup_shared", _i32, ctypes.POINTER(ExpertWeightsC), ctypes.POINTER(ExpertWeightsC), _i32, _i32, _p,
     _i32, _p, _p, _p, _p, _p)
_sig("moe_router_logits", _i32, ctypes.POINTER(RouteDesc), _p, _p, _p, _p, _p, _sz, _p)
_sig("moe_topk_gateup_shared", _i32, ctypes.POINTER(RouteDesc), _p, _p, _p, _i32, ctypes.POINTER(ExpertWeightsC),
     ctypes.POINTER(ExpertWeightsC), _p, _p, _p, _p, _p, _p, _p, _p, _p, _p)
_sig("moe_expert_down_combine", _i32, ctypes.POINTER(ExpertWeightsC), ctypes.POINTER(ExpertWeightsC), _i32, _i32, _p,
     _p, _p, _p, _p, _p, _p, _p)
_sig("moe_decode_step_sync_bytes", _sz)
_sig("moe_decode_step", _i32, ctypes.POINTER(RouteDesc), _p, _p, _p, _p, _p, ctypes.POINTER(ExpertWeightsC),
     ctypes.POINTER(ExpertWeightsC), _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p)
_sig("moe_combine", _i32, _i32, _i32, _i32, _p, _p, _p, _p, _p, _p, _p)
_sig("moe_dense_bf16", _i32, _i32, _i32, _i32, _p, _i32, _p, _p, _p, _p)
_sig("moe_dequant_bf16", _i32, _i32, _i32, _p, _p, _p, _p)
_sig("moe_dequant", _i32, _i32, _i32, _i32, _p, _p, _p, _p)
_sig("moe_mx_quantize", _i32, _i32, _i32, _p, _i32, _p, _p, _p)
_sig("moe_dense_linear", _i32, ctypes.POINTER(LinearDesc), _p, _p, _p, _p, _p, _p, _sz, _p)
_sig("moe_dense_linear_workspace", _sz, ctypes.POINTER(LinearDesc))
_sig("moe_dense_linear_backward", _i32, ctypes.POINTER(LinearDesc), _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p)
_sig("moe_dense_linear_backward_workspace", _sz, ctypes.POINTER(LinearDesc))
_sig("moe_dense_gateup", _i32, ctypes.POINTER(GateupDesc), _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p)
_sig("moe_dense_gateup_workspace", _sz, ctypes.POINTER(GateupDesc))
_sig("moe_dense_gateup_backward", _i32, ctypes.POINTER(GateupDesc), _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p,
     _p, _p, _sz, _p)
_sig("moe_dense_gateup_backward_workspace", _sz, ctypes.POINTER(GateupDesc))
_sig("moe_mxfp8_quantize", _i32, _i32, _i32, _p, _i32, _p, _p, _p)
_sig("moe_mxfp8_dequant", _i32, _i32, _i32, _p, _p, _p, _i32, _p)
_sig("moe_fp8_quantize", _i32, _i32, _i32, _p, _i32, _p, _p, _p, _p, _p)
_sig("moe_fp8_quantize_weight", _i32, _i32, _i32, _p, _i32, _i32, _p, _p, _p, _p, _p)
_sig("moe_fp8_dequant", _i32, _i32, _i32, _p, _p, _p, _i32, _p)
_sig("moe_fp8_linear", _i32, ctypes.POINTER(Fp8LinearDesc), _p, _p, _p, _p, _p, _p, _p, _sz, _p)
_sig("moe_fp8_linear_workspace", _sz, ctypes.POINTER(Fp8LinearDesc))
_sig("moe_block_norm", _i32, ctypes.POINTER(BlockNormDesc), _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p)
_sig("moe_block_norm_backward", _i32, ctypes.POINTER(BlockNormDesc), _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p,
     _p, _sz, _p)
_sig("moe_block_norm_backward_workspace", _sz, ctypes.POINTER(BlockNormDesc))

EXPORTS = ["moe_route", "moe_route_workspace", "moe_permute", "moe_permute_workspace", "moe_route_permute",
           "moe_route_permute_noalloc",
           "moe_expert_ffn", "moe_expert_gateup_shared", "moe_router_logits", "moe_topk_gateup_shared",
           "moe_expert_down_combine", "moe_decode_step", "moe_decode_step_sync_bytes",
           "moe_expert_ffn_workspace", "moe_expert_gateup", "moe_expert_gateup_workspace", "moe_expert_down",
           "moe_combine", "moe_dense_bf16", "moe_dequant", "moe_dequant_bf16", "moe_mx_quantize", "moe_last_error",
           "moe_abi_version", "moe_dense_linear", "moe_dense_linear_workspace", "moe_dense_linear_backward",
           "moe_dense_linear_backward_workspace", "moe_dense_gateup", "moe_dense_gateup_workspace",
           "moe_dense_gateup_backward", "moe_dense_gateup_backward_workspace", "moe_mxfp8_quantize",
           "moe_mxfp8_dequant", "moe_fp8_quantize", "moe_fp8_quantize_weight", "moe_fp8_dequant", "moe_fp8_linear",
           "moe_fp8_linear_workspace", "moe_block_norm", "moe_block_norm_backward", "moe_block_norm_backward_workspace"]


def last_error() -> str:
    return (lib.moe_last_error() or b"").decode()


def check(status: int):
    if status != MOE_OK:
        raise MoeError(status, last_error())


def abi_version() -> int:
    return lib.moe_abi_version()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need(t, dtype, name, shape=None):
    # (one expression a tensor when all is well: a decoded token's step is a few dozen microseconds of the host)
    if t is None or (type(t) is torch.Tensor and t.is_cuda and (dtype is None or t.dtype is dtype) and t.is_contiguous()
                     and (shape is None or t.shape == shape)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live in device memory (got {t.device})")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _room(t, dtype, name, n):
    """An optional tensor that a call reads or writes n elements of: of dtype, contiguous, no shorter, in device memory."""
    if t is None or (type(t) is torch.Tensor and t.dtype is dtype and t.numel() >= n and t.is_cuda and t.is_contiguous()):
        return
    if isinstance(t, torch.Tensor) and t.dtype == dtype and t.numel() < n:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, room for {n} values is needed")
    _need(t, dtype, name)


def _workspace(nbytes: int, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ router

def moe_route(x, w_router, k, score="softmax", renormalize=True, routed_scaling=1.0, logit_bias=None,
              select_bias=None, w_shared_gate=None, out=None, ws=None, n_group=1, topk_group=1):
    """Returns (topk_ids int32 [T][k], topk_w float32 [T][k], shared_gate float32 [T] or None).
    n_group > 1 selects among the topk_group best expert groups only (see moe.h)."""
    T, H = x.shape
    E = w_router.shape[0]
    _need(x, torch.bfloat16, "x")
    _need(w_router, torch.bfloat16, "w_router", (E, H))
    _need(logit_bias, torch.float32, "logit_bias", (E,))
    _need(select_bias, torch.float32, "select_bias", (E,))
    _need(w_shared_gate, torch.bfloat16, "w_shared_gate", (H,))
    d = RouteDesc(T, H, E, k, SCORE[score], 1 if renormalize else 0, routed_scaling, n_group, topk_group)
    dev = x.device
    if out is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        w = torch.empty((T, k), dtype=torch.float32, device=dev)
        sg = torch.empty((T,), dtype=torch.float32, device=dev) if w_shared_gate is not None else None
    else:
        ids, w, sg = out
    if ws is None:
        ws = _workspace(lib.moe_route_workspace(ctypes.byref(d)), dev)
    check(lib.moe_route(ctypes.byref(d), _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(select_bias),
                        _ptr(w_shared_gate), _ptr(ids), _ptr(w), _ptr(sg), _ptr(ws), ws.numel(), _stream()))
    return ids, w, sg


def moe_permute(topk_ids, E, out=None):
    """Returns (expert_offsets [E+1], sorted_pairs [T*k], pair_to_row [T*k]), int32."""
    T, k = topk_ids.shape
    _need(topk_ids, torch.int32, "topk_ids")
    dev = topk_ids.device
    if out is None:
        offs = torch.empty((E + 1,), dtype=torch.int32, device=dev)
        sp = torch.empty((T * k,), dtype=torch.int32, device=dev)
        p2r = torch.empty((T * k,), dtype=torch.int32, device=dev)
    else:
        offs, sp, p2r = out
    check(lib.moe_permute(T, k, E, _ptr(topk_ids), _ptr(offs), _ptr(sp), _ptr(p2r), None, 0, _stream()))
    return offs, sp, p2r


def moe_route_permute(x, w_router, k, score="softmax", renormalize=True, routed_scaling=1.0, logit_bias=None,
                      select_bias=None, w_shared_gate=None, out=None, ws=None, n_group=1, topk_group=1):
    """moe_route then moe_permute in one call.  Returns (topk_ids, topk_w, shared_gate or None,
    expert_offsets, sorted_pairs, pair_to_row)."""
    T, H = x.shape
    E = w_router.shape[0]
    _need(x, torch.bfloat16, "x")
    _need(w_router, torch.bfloat16, "w_router", (E, H))
    _need(logit_bias, torch.float32, "logit_bias", (E,))
    _need(select_bias, torch.float32, "select_bias", (E,))
    _need(w_shared_gate, torch.bfloat16, "w_shared_gate", (H,))
    d = RouteDesc(T, H, E, k, SCORE[score], 1 if renormalize else 0, routed_scaling, n_group, topk_group)
    dev = x.device
    if out is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        w = torch.empty((T, k), dtype=torch.float32, device=dev)
        sg = torch.empty((T,), dtype=torch.float32, device=dev) if w_shared_gate is not None else None
        offs = torch.empty((E + 1,), dtype=torch.int32, device=dev)
        sp = torch.empty((T * k,), dtype=torch.int32, device=dev)
        p2r = torch.empty((T * k,), dtype=torch.int32, device=dev)
    else:
        ids, w, sg, offs, sp, p2r = out
    if ws is None:
        ws = _workspace(lib.moe_route_workspace(ctypes.byref(d)), dev)
    check(lib.moe_route_permute(ctypes.byref(d), _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(select_bias),
                                _ptr(w_shared_gate), _ptr(ids), _ptr(w), _ptr(sg), _ptr(offs), _ptr(sp), _ptr(p2r),
                                _ptr(ws), ws.numel(), _stream()))
    return ids, w, sg, offs, sp, p2r


def moe_route_permute_noalloc(x, w_router, k, score="softmax", renormalize=True, routed_scaling=1.0,
                              logit_bias=None, select_bias=None, w_shared_gate=None, out=None, n_group=1,
                              topk_group=1):
    """moe_route_permute with the library's static scratch instead of a workspace.  `out` as for
    moe_route_permute (allocated here, by torch, when None)."""
    T, H = x.shape
    E = w_router.shape[0]
    _need(x, torch.bfloat16, "x")
    _need(w_router, torch.bfloat16, "w_router", (E, H))
    _need(logit_bias, torch.float32, "logit_bias", (E,))
    _need(select_bias, torch.float32, "select_bias", (E,))
    _need(w_shared_gate, torch.bfloat16, "w_shared_gate", (H,))
    d = RouteDesc(T, H, E, k, SCORE[score], 1 if renormalize else 0, routed_scaling, n_group, topk_group)
    dev = x.device
    if out is None:
        out = (torch.empty((T, k), dtype=torch.int32, device=dev), torch.empty((T, k), dtype=torch.float32, device=dev),
               torch.empty((T,), dtype=torch.float32, device=dev) if w_shared_gate is not None else None,
               torch.empty((E + 1,), dtype=torch.int32, device=dev), torch.empty((T * k,), dtype=torch.int32, device=dev),
               torch.empty((T * k,), dtype=torch.int32, device=dev))
    ids, w, sg, offs, sp, p2r = out
    check(lib.moe_route_permute_noalloc(ctypes.byref(d), _ptr(x), _ptr(w_router), _ptr(logit_bias),
                                        _ptr(select_bias), _ptr(w_shared_gate), _ptr(ids), _ptr(w), _ptr(sg),
                                        _ptr(offs), _ptr(sp), _ptr(p2r), _stream()))
    return ids, w, sg, offs, sp, p2r


# ------------------------------------------------------------------ experts

@dataclass
class ExpertWeights:
    """Device tensors of an expert stack in the storage layout of moe.h."""
    fmt: str
    d_model: int
    d_ff: int
    gate: torch.Tensor
    gate_s: torch.Tensor
    up: torch.Tensor
    up_s: torch.Tensor
    down: torch.Tensor
    down_s: torch.Tensor

    @property
    def num_experts(self):
        return self.gate.shape[0]

    def c_struct(self):
        E, K, I = self.num_experts, self.d_model, self.d_ff
        if self.fmt == "mxfp4":
            shapes = {"gate": (E, I, K // 2), "up": (E, I, K // 2), "down": (E, K, I // 2),
                      "gate_s": (E, I, K // 32), "up_s": (E, I, K // 32), "down_s": (E, K, I // 32)}
            sdt = torch.uint8
        else:
            shapes = {"gate": (E, I, K), "up": (E, I, K), "down": (E, K, I),
                      "gate_s": (E, I // 128, K // 128), "up_s": (E, I // 128, K // 128),
                      "down_s": (E, K // 128, I // 128)}
            sdt = torch.float32
        for n, s in shapes.items():
            _need(getattr(self, n), sdt if n.endswith("_s") else torch.uint8, n, s)
        return ExpertWeightsC(WFMT[self.fmt], E, K, I, self.gate.data_ptr(), self.up.data_ptr(),
                              self.down.data_ptr(), self.gate_s.data_ptr(), self.up_s.data_ptr(),
                              self.down_s.data_ptr())

    @staticmethod
    def from_arrays(es, device=None):
        t = lambda a: a if isinstance(a, torch.Tensor) else torch.from_numpy(a).to(device)
        return ExpertWeights(es.fmt, es.d_model, es.d_ff, t(es.gate), t(es.gate_s), t(es.up), t(es.up_s),
                             t(es.down), t(es.down_s))


@dataclass
class DenseWeights:
    """Device tensors of one expert with bf16 weights: gate, up [d_ff][d_model], down [d_model][d_ff]."""
    gate: torch.Tensor
    up: torch.Tensor
    down: torch.Tensor

    @property
    def d_model(self):
        return self.gate.shape[1]

    @property
    def d_ff(self):
        return self.gate.shape[0]


def moe_expert_ffn(w: ExpertWeights, x, act="float", k=1, expert_offsets=None, sorted_pairs=None, out=None,
                   ws=None):
    """y_rows [R][d_model] float32; R = T*k (routed) or T (expert_offsets None, one expert)."""
    T = x.shape[0]
    _need(x, None, "x", (T, w.d_model))
    _need(expert_offsets, torch.int32, "expert_offsets", (w.num_experts + 1,))
    c = w.c_struct()
    R = T * k if expert_offsets is not None else T
    _room(sorted_pairs, torch.int32, "sorted_pairs", R)
    _need(ws, None, "ws")
    y = out if out is not None else torch.empty((R, w.d_model), dtype=torch.float32, device=x.device)
    _need(y, torch.float32, "y_rows", (R, w.d_model))
    kk = k if expert_offsets is not None else 1
    if ws is None:
        ws = _workspace(lib.moe_expert_ffn_workspace(ctypes.byref(c), ACT[act], T, kk), x.device)
    check(lib.moe_expert_ffn(ctypes.byref(c), ACT[act], T, kk, _ptr(x), DT[x.dtype], _ptr(expert_offsets),
                             _ptr(sorted_pairs), _ptr(y), _ptr(ws), ws.numel(), _stream()))
    return y


def moe_expert_ffn_workspace(w: ExpertWeights, act, T, k):
    return lib.moe_expert_ffn_workspace(ctypes.byref(w.c_struct()), ACT[act], T, k)


def moe_expert_gateup_workspace(w: ExpertWeights, act, T, k):
    return lib.moe_expert_gateup_workspace(ctypes.byref(w.c_struct()), ACT[act], T, k)


def _expert_rows(w, act, R, expert_offsets, h, h_codes, h_scales):
    """Room for R rows of h in the forms that `act` reads and writes (the codes' width depends on it)."""
    _room(expert_offsets, torch.int32, "expert_offsets", w.num_experts + 1)
    _room(h, torch.float32, "h", R * w.d_ff)
    if act != "float":
        fp8 = act == "fp8"
        _room(h_codes, torch.uint8, "h_codes", R * (w.d_ff if fp8 else w.d_ff // 2))
        _room(h_scales, torch.uint8, "h_scales", R * (w.d_ff // (128 if fp8 else 32)))


def moe_expert_gateup(w: ExpertWeights, x, act="float", k=1, expert_offsets=None, sorted_pairs=None,
                      want_h=True, out=None, ws=None):
    """Returns (h float32 [R][d_ff] or None, h_codes or None, h_scales or None): codes [R][d_ff/2] with scales [R][d_ff/32]
    (act "mxfp4") or [R][d_ff] with [R][d_ff/128] ("fp8")."""
    T = x.shape[0]
    _need(x, None, "x", (T, w.d_model))
    c = w.c_struct()
    kk = k if expert_offsets is not None else 1
    R = T * kk
    dev = x.device
    if out is not None:
        h, hq, hs = out
    else:
        h = torch.empty((R, w.d_ff), dtype=torch.float32, device=dev) if (want_h or act == "float") else None
        hq = hs = None
        if act == "mxfp4":
            hq = torch.empty((R, w.d_ff // 2), dtype=torch.uint8, device=dev)
            hs = torch.empty((R, w.d_ff // 32), dtype=torch.uint8, device=dev)
        elif act == "fp8":
            hq = torch.empty((R, w.d_ff), dtype=torch.uint8, device=dev)
            hs = torch.empty((R, w.d_ff // 128), dtype=torch.uint8, device=dev)
    _expert_rows(w, act, R, expert_offsets, h, hq, hs)
    _room(sorted_pairs, torch.int32, "sorted_pairs", R)
    _need(ws, None, "ws")
    if ws is None:
        ws = _workspace(lib.moe_expert_gateup_workspace(ctypes.byref(c), ACT[act], T, kk), dev)
    check(lib.moe_expert_gateup(ctypes.byref(c), ACT[act], T, kk, _ptr(x), DT[x.dtype], _ptr(expert_offsets),
                                _ptr(sorted_pairs), _ptr(h), _ptr(hq), _ptr(hs), _ptr(ws), ws.numel(), _stream()))
    return h, hq, hs


def moe_expert_down(w: ExpertWeights, T, act="float", k=1, expert_offsets=None, h=None, h_codes=None,
                    h_scales=None, out=None):
    c = w.c_struct()
    kk = k if expert_offsets is not None else 1
    R = T * kk
    dev = (h if h is not None else h_codes).device
    y = out if out is not None else torch.empty((R, w.d_model), dtype=torch.float32, device=dev)
    _expert_rows(w, act, R, expert_offsets, h if act == "float" else None, h_codes, h_scales)
    _room(y, torch.float32, "y_rows", R * w.d_model)
    check(lib.moe_expert_down(ctypes.byref(c), ACT[act], T, kk, _ptr(h), _ptr(h_codes), _ptr(h_scales),
                              _ptr(expert_offsets), _ptr(y), _stream()))
    return y


def moe_expert_gateup_shared(w: ExpertWeights, shared, x, k, expert_offsets, sorted_pairs, out=None):
    """Routed gate/up (FLOAT activations) and, when `shared` is given, the shared expert's
    gate/up over every token, in one launch.  Returns (h [T*k][d_ff], h_shared [T][d_ff_s] or None)."""
    T = x.shape[0]
    _need(x, None, "x", (T, w.d_model))
    dev = x.device
    if out is not None:
        h, hsh = out
    else:
        h = torch.empty((T * k, w.d_ff), dtype=torch.float32, device=dev)
        hsh = torch.empty((T, shared.d_ff), dtype=torch.float32, device=dev) if shared is not None else None
    c = w.c_struct()
    cs = shared.c_struct() if shared is not None else None
    check(lib.moe_expert_gateup_shared(ctypes.byref(c), ctypes.byref(cs) if cs is not None else None, T, k, _ptr(x),
                                       DT[x.dtype], _ptr(expert_offsets), _ptr(sorted_pairs), _ptr(h), _ptr(hsh),
                                       _stream()))
    return h, hsh


def moe_router_logits(x, w_router, k, score="softmax", w_shared_gate=None, out=None, ws=None, n_group=1,
                      topk_group=1):
    """float32 router logits [T][E (+1 with the shared gate)]."""
    T, H = x.shape
    E = w_router.shape[0]
    _need(x, torch.bfloat16, "x")
    _need(w_router, torch.bfloat16, "w_router", (E, H))
    _need(w_shared_gate, torch.bfloat16, "w_shared_gate", (H,))
    d = RouteDesc(T, H, E, k, SCORE[score], 1, 1.0, n_group, topk_group)
    rows = E + (1 if w_shared_gate is not None else 0)
    lg = out if out is not None else torch.empty((T, rows), dtype=torch.float32, device=x.device)
    _need(lg, torch.float32, "logits", (T, rows))
    if ws is None:
        ws = _workspace(lib.moe_route_workspace(ctypes.byref(d)), x.device)
    check(lib.moe_router_logits(ctypes.byref(d), _ptr(x), _ptr(w_router), _ptr(w_shared_gate), _ptr(lg), _ptr(ws),
                                ws.numel(), _stream()))
    return lg


def moe_topk_gateup_shared(logits, x, k, w: ExpertWeights, shared=None, score="softmax", renormalize=True,
                           routed_scaling=1.0, logit_bias=None, select_bias=None, has_shared_gate=False, out=None,
                           n_group=1, topk_group=1):
    """Routing of `logits` (moe_route_permute's selection) and the routed + shared gate/up on it,
    in one launch.  Returns (topk_ids, topk_w, shared_gate or None, expert_offsets, sorted_pairs,
    pair_to_row, h [T*k][d_ff], h_shared [T][d_ff_s] or None)."""
    T, H = x.shape
    E = w.num_experts
    _need(x, torch.bfloat16, "x")
    _need(logits, torch.float32, "logits", (T, E + (1 if has_shared_gate else 0)))
    _need(logit_bias, torch.float32, "logit_bias", (E,))
    _need(select_bias, torch.float32, "select_bias", (E,))
    d = RouteDesc(T, H, E, k, SCORE[score], 1 if renormalize else 0, routed_scaling, n_group, topk_group)
    dev = x.device
    if out is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        tw = torch.empty((T, k), dtype=torch.float32, device=dev)
        sg = torch.empty((T,), dtype=torch.float32, device=dev) if has_shared_gate else None
        offs = torch.empty((E + 1,), dtype=torch.int32, device=dev)
        sp = torch.empty((T * k,), dtype=torch.int32, device=dev)
        p2r = torch.empty((T * k,), dtype=torch.int32, device=dev)
        h = torch.empty((T * k, w.d_ff), dtype=torch.float32, device=dev)
        hsh = torch.empty((T, shared.d_ff), dtype=torch.float32, device=dev) if shared is not None else None
    else:
        ids, tw, sg, offs, sp, p2r, h, hsh = out
    c = w.c_struct()
    cs = shared.c_struct() if shared is not None else None
    check(lib.moe_topk_gateup_shared(ctypes.byref(d), _ptr(logits), _ptr(logit_bias), _ptr(select_bias),
                                     1 if has_shared_gate else 0, ctypes.byref(c),
                                     ctypes.byref(cs) if cs is not None else None, _ptr(x), _ptr(ids), _ptr(tw),
                                     _ptr(sg), _ptr(offs), _ptr(sp), _ptr(p2r), _ptr(h), _ptr(hsh), _stream()))
    return ids, tw, sg, offs, sp, p2r, h, hsh


def moe_expert_down_combine(w: ExpertWeights, shared, h, h_shared, topk_ids, topk_w, pair_to_row, shared_gate=None,
                            out=None):
    """out[t] = sum_j topk_w[t][j] * down_{e_j}(h[pair_to_row[t*k+j]]) + g_t * shared_down(h_shared[t]),
    float32 [T][d_model], in one launch."""
    T, k = topk_w.shape
    _need(topk_ids, torch.int32, "topk_ids", (T, k))
    o = out if out is not None else torch.empty((T, w.d_model), dtype=torch.float32, device=topk_w.device)
    c = w.c_struct()
    cs = shared.c_struct() if shared is not None else None
    check(lib.moe_expert_down_combine(ctypes.byref(c), ctypes.byref(cs) if cs is not None else None, T, k, _ptr(h),
                                      _ptr(h_shared), _ptr(topk_ids), _ptr(topk_w), _ptr(pair_to_row),
                                      _ptr(shared_gate), _ptr(o), _stream()))
    return o


def decode_step_sync(device):
    """A zero-filled sync buffer for moe_decode_step (one per stream that runs steps)."""
    return torch.zeros((lib.moe_decode_step_sync_bytes() // 4,), dtype=torch.int32, device=device)


def moe_decode_step(x, w_router, k, w: ExpertWeights, shared=None, score="softmax", renormalize=True,
                    routed_scaling=1.0, logit_bias=None, select_bias=None, w_shared_gate=None, sync=None, out=None,
                    n_group=1, topk_group=1):
    """A whole decode layer step (router logits, top-k with the routed and shared gate/up, down
    with the weighted combine) in one launch when the shapes allow it.  `sync`: a buffer from
    decode_step_sync(), kept across calls.  Returns (logits, topk_ids, topk_w, shared_gate or
    None, expert_offsets, sorted_pairs, pair_to_row, h, h_shared or None, out [T][d_model])."""
    T, H = x.shape
    E = w.num_experts
    _need(x, torch.bfloat16, "x")
    _need(w_router, torch.bfloat16, "w_router", (E, H))
    _need(w_shared_gate, torch.bfloat16, "w_shared_gate", (H,))
    _need(logit_bias, torch.float32, "logit_bias", (E,))
    _need(select_bias, torch.float32, "select_bias", (E,))
    if sync is None:
        raise MoeError(1, "moe_decode_step: a sync buffer (decode_step_sync) is required")
    _need(sync, torch.int32, "sync", (lib.moe_decode_step_sync_bytes() // 4,))
    d = RouteDesc(T, H, E, k, SCORE[score], 1 if renormalize else 0, routed_scaling, n_group, topk_group)
    dev = x.device
    has_sg = w_shared_gate is not None
    if out is None:
        lg = torch.empty((T, E + (1 if has_sg else 0)), dtype=torch.float32, device=dev)
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        tw = torch.empty((T, k), dtype=torch.float32, device=dev)
        sg = torch.empty((T,), dtype=torch.float32, device=dev) if has_sg else None
        offs = torch.empty((E + 1,), dtype=torch.int32, device=dev)
        sp = torch.empty((T * k,), dtype=torch.int32, device=dev)
        p2r = torch.empty((T * k,), dtype=torch.int32, device=dev)
        h = torch.empty((T * k, w.d_ff), dtype=torch.float32, device=dev)
        hsh = torch.empty((T, shared.d_ff), dtype=torch.float32, device=dev) if shared is not None else None
        o = torch.empty((T, w.d_model), dtype=torch.float32, device=dev)
    else:
        lg, ids, tw, sg, offs, sp, p2r, h, hsh, o = out
    c = w.c_struct()
    cs = shared.c_struct() if shared is not None else None
    check(lib.moe_decode_step(ctypes.byref(d), _ptr(x), _ptr(w_router), _ptr(w_shared_gate), _ptr(logit_bias),
                              _ptr(select_bias), ctypes.byref(c), ctypes.byref(cs) if cs is not None else None,
                              _ptr(lg), _ptr(ids), _ptr(tw), _ptr(sg), _ptr(offs), _ptr(sp), _ptr(p2r), _ptr(h),
                              _ptr(hsh), _ptr(o), _ptr(sync), _stream()))
    return lg, ids, tw, sg, offs, sp, p2r, h, hsh, o


# ------------------------------------------------------------------ combine, dense, formats

def moe_route_workspace(T, H, E, k, score="softmax"):
    d = RouteDesc(T, H, E, k, SCORE[score], 1, 1.0, 1, 1)
    return lib.moe_route_workspace(ctypes.byref(d))


def moe_combine(y_rows, pair_to_row, topk_w, y_shared=None, shared_gate=None, out=None):
    T, k = topk_w.shape
    d = y_rows.shape[1] if y_rows is not None else y_shared.shape[1]
    _need(y_rows, torch.float32, "y_rows")
    _need(pair_to_row, torch.int32, "pair_to_row", (T * k,))
    _need(topk_w, torch.float32, "topk_w")
    _need(y_shared, torch.float32, "y_shared", (T, d))
    _need(shared_gate, torch.float32, "shared_gate", (T,))
    o = out if out is not None else torch.empty((T, d), dtype=torch.float32, device=topk_w.device)
    check(lib.moe_combine(T, k, d, _ptr(y_rows), _ptr(pair_to_row), _ptr(topk_w), _ptr(y_shared),
                          _ptr(shared_gate), _ptr(o), _stream()))
    return o


def moe_dense_bf16(x, w, residual=None, out=None):
    T, kdim = x.shape
    n = w.shape[0]
    _need(x, None, "x")
    _need(w, torch.bfloat16, "w", (n, kdim))
    _need(residual, torch.float32, "residual", (T, n))
    y = out if out is not None else torch.empty((T, n), dtype=torch.float32, device=x.device)
    check(lib.moe_dense_bf16(T, n, kdim, _ptr(x), DT[x.dtype], _ptr(w), _ptr(residual), _ptr(y), _stream()))
    return y


def moe_dequant(fmt, codes, scales):
    _need(codes, torch.uint8, "codes")
    _need(scales, None, "scales")
    n = codes.shape[0]
    kdim = codes.shape[1] * (2 if fmt == "mxfp4" else 1)
    out = torch.empty((n, kdim), dtype=torch.float32, device=codes.device)
    check(lib.moe_dequant(WFMT[fmt], n, kdim, _ptr(codes), _ptr(scales), _ptr(out), _stream()))
    return out


def moe_dequant_bf16(codes, scales):
    """MXFP4 codes [n][kdim/2] + E8M0 scales [n][kdim/32] -> bf16 [n][kdim] (the matrix-core decode)."""
    _need(codes, torch.uint8, "codes")
    n = codes.shape[0]
    kdim = codes.shape[1] * 2
    _need(scales, torch.uint8, "scales", (n, kdim // 32))
    out = torch.empty((n, kdim), dtype=torch.bfloat16, device=codes.device)
    check(lib.moe_dequant_bf16(n, kdim, _ptr(codes), _ptr(scales), _ptr(out), _stream()))
    return out


def moe_mx_quantize(x):
    rows, cols = x.shape
    _need(x, None, "x")
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
    check(lib.moe_mx_quantize(rows, cols, _ptr(x), DT[x.dtype], _ptr(codes), _ptr(scales), _stream()))
    return codes, scales


# ------------------------------------------------------------------ dense bf16 layers

def _operands(dev, *items):
    """items: (tensor or None, dtype or tuple of dtypes, name, shape or None).  Each on `dev`, of its dtype and shape,
    contiguous.  (One expression a tensor when all is well: a decoded token's call is a few microseconds.)"""
    if dev.type != "cuda":
        raise ValueError(f"{items[0][2]} must live in device memory (got {dev})")
    for t, dtype, name, shape in items:
        if t is None or (isinstance(t, torch.Tensor) and (t.dtype is dtype) and t.device == dev and t.is_contiguous()
                         and (shape is None or t.shape == shape)):
            continue
        if isinstance(dtype, tuple):
            if isinstance(t, torch.Tensor) and t.dtype not in dtype:
                raise TypeError(f"{name} must be one of {dtype} (got {t.dtype})")
            dtype = None
        _need(t, dtype, name, shape)
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _launch(dev, fn, *args):
    """fn(*args, stream) on dev's current stream, with dev the current device for the call."""
    i = dev.index
    if i == torch.cuda.current_device():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(i):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    if status != MOE_OK:
        check(status)


def _at(t):
    return None if t is None else t.data_ptr()


def _one_of(t, types):
    """t's dtype when it is one of `types`, else `types` (refused by _operands)."""
    dt = getattr(t, "dtype", None)
    return dt if dt in types else tuple(types)


def _matrix(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions (got shape {tuple(t.shape)})")
    return t.shape


def _act_fn(name):
    if name not in ACT_FN:
        raise ValueError(f"act_fn must be one of {sorted(ACT_FN)} (got {name!r})")
    return ACT_FN[name]


def _int32(*sizes):
    """Refuses what the C side's int32 cannot hold (ctypes would cut it off without a word)."""
    if max(sizes) > 2 ** 31 - 1 or min(sizes) < -2 ** 31:
        raise MoeError(MOE_ERR_INVALID_ARG, f"sizes overflow int32 {sizes}")


@functools.lru_cache(maxsize=4096)
def _dense_plan(kind, *sizes):
    """(descriptor, workspace bytes) of a dense call: a function of its sizes and types alone."""
    _int32(*sizes)
    d = ctypes.byref((LinearDesc if kind.startswith("linear") else GateupDesc)(*sizes))
    return d, getattr(lib, f"moe_dense_{kind}_workspace")(d)


def moe_dense_linear_workspace(T, n, kdim, act_fn="none", x_dtype=torch.bfloat16, out_dtype=torch.bfloat16):
    return _dense_plan("linear", T, n, kdim, _act_fn(act_fn), DT[x_dtype], DT[out_dtype], 0)[1]


def moe_dense_linear_backward_workspace(T, n, kdim, act_fn="none", x_dtype=torch.bfloat16, mxfp8=False):
    return _dense_plan("linear_backward", T, n, kdim, _act_fn(act_fn), DT_MXFP8 if mxfp8 else DT[x_dtype], 0, 0)[1]


def moe_dense_gateup_workspace(T, d_model, d_ff, act_fn="silu", out_dtype=torch.bfloat16):
    return _dense_plan("gateup", T, d_model, d_ff, _act_fn(act_fn), 0, DT[out_dtype], 0)[1]


def moe_dense_gateup_backward_workspace(T, d_model, d_ff, act_fn="silu", mxfp8=False):
    return _dense_plan("gateup_backward", T, d_model, d_ff, _act_fn(act_fn), DT_MXFP8 if mxfp8 else 0, 0, 0)[1]


def _ws_for(ws, need, dev):
    if need == 0:
        return None, 0
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=dev), need
    _operands(dev, (ws, torch.uint8, "ws", None))
    return ws, ws.numel()


def _outside_graph(who, backward=None):
    warnings.warn(f"{who}: an operand requires grad, but the result is not part of autograd's graph; its gradients come from "
                  f"{backward or who + '_backward'} (under torch.no_grad() this is not said)", stacklevel=3)


def moe_dense_linear(x, w, bias=None, act_fn="none", residual=None, out=None, out_dtype=None, ws=None):
    """y = act_fn(x w^T + bias) + residual.  x [T][kdim] bf16 or float32, w bf16 [n][kdim], bias float32 [n],
    residual [T][n] of y's type; y [T][n] of out_dtype (x's type when None), bf16 or float32.  Autograd does not see the
    call (it warns of operands that require grad): moe_dense_linear_backward forms the gradients."""
    T, kdim = _matrix(x, "x")
    n = _matrix(w, "w")[0]
    dt = out.dtype if out is not None else (out_dtype or x.dtype)
    if dt not in DT:
        raise TypeError(f"y must be bfloat16 or float32 (got {dt})")
    dev = x.device
    _operands(dev, (x, _one_of(x, DT), "x", None), (w, torch.bfloat16, "w", (n, kdim)), (bias, torch.float32, "bias", (n,)),
              (residual, dt, "residual", (T, n)), (out, dt, "out", (T, n)))
    if (x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad)
            or (residual is not None and residual.requires_grad)) and torch.is_grad_enabled():
        _outside_graph("moe_dense_linear")
    d, need = _dense_plan("linear", T, n, kdim, _act_fn(act_fn), DT[x.dtype], DT[dt], 0)
    y = out if out is not None else torch.empty((T, n), dtype=dt, device=dev)
    ws, nws = _ws_for(ws, need, dev)
    _launch(dev, lib.moe_dense_linear, d, _at(x), _at(w), _at(bias), _at(residual), _at(y), _at(ws), nws)
    return y


def _wanted(want, names):
    unknown = set(want) - set(names)
    if unknown or not want:
        raise ValueError(f"want must name some of {names} (got {tuple(want)})")
    return [n in want for n in names]


def _saved_input(x, x_scales, T, width, types):
    """(x_dtype, operand rows) of an input kept as it is (one of `types`) or as MXFP8 codes with their scales."""
    mx = x_scales is not None
    dt = DT_MXFP8 if mx else (DT.get(x.dtype, 0) if isinstance(x, torch.Tensor) else 0)
    return dt, ((x, torch.uint8 if mx else _one_of(x, types), "x", (T, width)), (x_scales, torch.uint8, "x_scales", (T, width // 32)))


def moe_dense_linear_backward(dy, x, w, bias=None, act_fn="none", x_scales=None, want=("dx", "dw", "dbias"), out=None,
                              dx_dtype=None, ws=None):
    """Gradients of moe_dense_linear at dy (bf16 [T][n]): (dx [T][kdim] of dx_dtype (bf16 when None, or float32), dw bf16
    [n][kdim], dbias float32 [n]), None for what `want` does not name.  x: bf16 or float32, or the codes of
    moe_mxfp8_quantize with their x_scales.  out: the three results' tensors (None where not wanted)."""
    T, n = _matrix(dy, "dy")
    kdim = _matrix(w, "w")[1]
    fx, fw, fb = _wanted(want, ("dx", "dw", "dbias"))
    xdt, xitems = _saved_input(x, x_scales, T, kdim, tuple(DT))
    dev = dy.device
    ox, ow, ob = out if out is not None else (None, None, None)
    bf = torch.bfloat16
    xt = ox.dtype if ox is not None else (dx_dtype or bf)
    if xt not in DT:
        raise TypeError(f"dx must be bfloat16 or float32 (got {xt})")
    _operands(dev, (dy, bf, "dy", None), *xitems, (w, bf, "w", (n, kdim)), (bias, torch.float32, "bias", (n,)),
              (ox, xt, "dx", (T, kdim)), (ow, bf, "dw", (n, kdim)), (ob, torch.float32, "dbias", (n,)))
    d, need = _dense_plan("linear_backward", T, n, kdim, _act_fn(act_fn), xdt, 0, DT[xt])
    e = lambda o, on, shape, dt: None if not on else (o if o is not None else torch.empty(shape, dtype=dt, device=dev))
    dx, dw, db = e(ox, fx, (T, kdim), xt), e(ow, fw, (n, kdim), bf), e(ob, fb, (n,), torch.float32)
    ws, nws = _ws_for(ws, need, dev)
    _launch(dev, lib.moe_dense_linear_backward, d, _at(dy), _at(x), _at(x_scales), _at(w), _at(bias), _at(dx), _at(dw),
            _at(db), _at(ws), nws)
    return dx, dw, db


def moe_dense_gateup(x, w_gate, w_up, b_gate=None, b_up=None, act_fn="silu", out=None, out_dtype=None, want_pre=False,
                     pre=None, ws=None):
    """h = act_fn(x w_gate^T + b_gate) * (x w_up^T + b_up), both products in one kernel.  x bf16 [T][d_model], weights
    bf16 [d_ff][d_model], biases float32 [d_ff].  Returns (h [T][d_ff] of out_dtype (bf16 when None), the bf16
    pre-activations [2][T][d_ff] for the backward call, or None).  Autograd does not see the call (it warns of operands that
    require grad): moe_dense_gateup_backward forms the gradients."""
    T, dm = _matrix(x, "x")
    f = _matrix(w_gate, "w_gate")[0]
    bf = torch.bfloat16
    dt = out.dtype if out is not None else (out_dtype or bf)
    if dt not in DT:
        raise TypeError(f"h must be bfloat16 or float32 (got {dt})")
    dev = x.device
    _operands(dev, (x, bf, "x", None), (w_gate, bf, "w_gate", (f, dm)), (w_up, bf, "w_up", (f, dm)),
              (b_gate, torch.float32, "b_gate", (f,)), (b_up, torch.float32, "b_up", (f,)), (out, dt, "out", (T, f)),
              (pre, bf, "pre", (2, T, f)))
    if (x.requires_grad or w_gate.requires_grad or w_up.requires_grad or (b_gate is not None and b_gate.requires_grad)
            or (b_up is not None and b_up.requires_grad)) and torch.is_grad_enabled():
        _outside_graph("moe_dense_gateup")
    d, need = _dense_plan("gateup", T, dm, f, _act_fn(act_fn), 0, DT[dt])
    h = out if out is not None else torch.empty((T, f), dtype=dt, device=dev)
    if pre is None and want_pre:
        pre = torch.empty((2, T, f), dtype=bf, device=dev)
    ws, nws = _ws_for(ws, need, dev)
    _launch(dev, lib.moe_dense_gateup, d, _at(x), _at(w_gate), _at(w_up), _at(b_gate), _at(b_up), _at(h), _at(pre), _at(ws),
            nws)
    return h, pre


def moe_dense_gateup_backward(dh, x, w_gate, w_up, b_gate=None, b_up=None, act_fn="silu", x_scales=None, pre=None,
                              want=("dx", "dw", "db"), want_h=False, h_dtype=None, out=None, ws=None):
    """Gradients of moe_dense_gateup at dh (bf16 or float32 [T][d_ff]): (dx, dw_gate, dw_up, db_gate, db_up, h), None for
    what was not asked for; the weights' gradients and dx are bf16, the biases' float32.  h (of h_dtype, bf16 when None,
    or float32) is the forward result again, for the down projection's weight gradient.  x: bf16, or MXFP8
    codes with x_scales; pre: the forward call's pre-activations (recomputed from x when None).  out: the six results'
    tensors."""
    T, f = _matrix(dh, "dh")
    dm = _matrix(w_gate, "w_gate")[1]
    fx, fw, fb = _wanted(want, ("dx", "dw", "db")) if want or not want_h else (False, False, False)
    xdt, xitems = _saved_input(x, x_scales, T, dm, (torch.bfloat16,))
    dev = dh.device
    bf, f32 = torch.bfloat16, torch.float32
    o = out if out is not None else (None,) * 6
    ht = o[5].dtype if o[5] is not None else (h_dtype or bf)
    if ht not in DT:
        raise TypeError(f"h must be bfloat16 or float32 (got {ht})")
    names = ("dx", "dw_gate", "dw_up", "db_gate", "db_up", "h")
    shapes = ((T, dm), (f, dm), (f, dm), (f,), (f,), (T, f))
    types = (bf, bf, bf, f32, f32, ht)
    _operands(dev, (dh, _one_of(dh, DT), "dh", None), *xitems, (w_gate, bf, "w_gate", (f, dm)), (w_up, bf, "w_up", (f, dm)),
              (b_gate, f32, "b_gate", (f,)), (b_up, f32, "b_up", (f,)), (pre, bf, "pre", (2, T, f)),
              *((t, dt, nm, sh) for t, dt, nm, sh in zip(o, types, names, shapes)))
    d, need = _dense_plan("gateup_backward", T, dm, f, _act_fn(act_fn), xdt, DT[ht], DT[dh.dtype])
    r = [None if not on else (t if t is not None else torch.empty(sh, dtype=dt, device=dev))
         for t, dt, sh, on in zip(o, types, shapes, (fx, fw, fw, fb, fb, want_h))]
    ws, nws = _ws_for(ws, need, dev)
    _launch(dev, lib.moe_dense_gateup_backward, d, _at(dh), _at(x), _at(x_scales), _at(w_gate), _at(w_up), _at(b_gate),
            _at(b_up), _at(pre), *map(_at, r), _at(ws), nws)
    return tuple(r)


def moe_mxfp8_quantize(x, out=None):
    """Rows of x (bf16 or float32, a multiple of 32 wide) as OCP MXFP8: (codes uint8 [rows][cols], E8M0 scales uint8
    [rows][cols/32]).  out: the two tensors."""
    rows, cols = _matrix(x, "x")
    _int32(rows, cols)
    dev = x.device
    codes, scales = out if out is not None else (None, None)
    _operands(dev, (x, _one_of(x, DT), "x", None), (codes, torch.uint8, "codes", (rows, cols)),
              (scales, torch.uint8, "scales", (rows, cols // 32)))
    if out is None:
        codes = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev)
    _launch(dev, lib.moe_mxfp8_quantize, rows, cols, _at(x), DT[x.dtype], _at(codes), _at(scales))
    return codes, scales


def moe_mxfp8_dequant(codes, scales, out=None, out_dtype=torch.bfloat16):
    """The values of moe_mxfp8_quantize's codes and scales, bf16 or float32."""
    rows, cols = _matrix(codes, "codes")
    _int32(rows, cols)
    dev = codes.device
    dt = out.dtype if out is not None else out_dtype
    if dt not in DT:
        raise TypeError(f"values must be bfloat16 or float32 (got {dt})")
    _operands(dev, (codes, torch.uint8, "codes", None), (scales, torch.uint8, "scales", (rows, cols // 32)),
              (out, dt, "out", (rows, cols)))
    o = out if out is not None else torch.empty((rows, cols), dtype=dt, device=dev)
    _launch(dev, lib.moe_mxfp8_dequant, rows, cols, _at(codes), _at(scales), _at(o), DT[dt])
    return o


# ------------------------------------------------------------------ block-128 FP8 products

def _fits(dev, t, dtype, shape):
    """Whether an optional operand is as _operands wants it."""
    return t is None or (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == dev)


def _blocks(n):
    return (n + 127) // 128


_FP8_GRADIENTS = "moe_fp8_linear on the transposed codes (FP8Linear.backward)"


def _fp8_pairs(out, wanted, shapes, types, dev):
    """The code and scale tensors of a quantiser: `out`'s (checked), new ones, or None where not wanted."""
    names = ("codes", "scales", "codes_t", "scales_t")
    o = out if out is not None else (None,) * 4
    _operands(dev, *((t, dt, nm, sh) for t, dt, nm, sh in zip(o, types, names, shapes)))
    return [None if not on else (t if t is not None else torch.empty(sh, dtype=dt, device=dev))
            for t, dt, sh, on in zip(o, types, shapes, wanted)]


def moe_fp8_quantize(x, rows=True, cols=False, out=None):
    """x (bf16 or float32 [T][d], d a multiple of 8) as E4M3 codes with an E8M0 scale per 128 values.  Returns (codes [T][d],
    scales [T][ceil(d/128)], codes_t [d][ld], scales_t [d][ceil(T/128)]), uint8: the first two (blocks along the row) with
    `rows`, the last two (the transpose, blocks along the column, ld = T rounded up to 16) with `cols`, else None.  out: the
    four tensors.  Autograd does not see the call (it warns of an x that requires grad)."""
    T, d = _matrix(x, "x")
    _int32(T, d)
    if not (rows or cols):
        raise ValueError("moe_fp8_quantize: neither rows nor cols is asked for")
    dev, u8 = x.device, torch.uint8
    ld = (T + 15) // 16 * 16
    _operands(dev, (x, _one_of(x, DT), "x", None))
    if x.requires_grad and torch.is_grad_enabled():
        _outside_graph("moe_fp8_quantize", _FP8_GRADIENTS)
    c, s, ct, st = _fp8_pairs(out, (rows, rows, cols, cols), ((T, d), (T, _blocks(d)), (d, ld), (d, _blocks(T))), (u8,) * 4, dev)
    _launch(dev, lib.moe_fp8_quantize, T, d, _at(x), DT[x.dtype], _at(c), _at(s), _at(ct), _at(st))
    return c, s, ct, st


def moe_fp8_quantize_weight(w, scale_dtype=torch.float32, codes=True, transpose=False, out=None):
    """A weight (bf16 or float32 [n][kdim], kdim a multiple of 16) as E4M3 codes with a scale (a power of two; float32, or uint8:
    E8M0) per 128 x 128 block.  Returns (codes [n][kdim], scales [ceil(n/128)][ceil(kdim/128)], codes_t [kdim][ld], scales_t
    [ceil(kdim/128)][ceil(n/128)]); the last two, the same codes transposed (ld = n rounded up to 16), with `transpose`, the
    first two with `codes`, else None.  out: the four tensors.  Autograd does not see the call (it warns of a w that requires grad)."""
    n, k = _matrix(w, "w")
    _int32(n, k)
    if not (codes or transpose):
        raise ValueError("moe_fp8_quantize_weight: neither codes nor transpose is asked for")
    if scale_dtype not in (torch.float32, torch.uint8):
        raise TypeError(f"scale_dtype must be float32 or uint8 (got {scale_dtype})")
    dev, u8, sd = w.device, torch.uint8, scale_dtype
    ld = (n + 15) // 16 * 16
    _operands(dev, (w, _one_of(w, DT), "w", None))
    if w.requires_grad and torch.is_grad_enabled():
        _outside_graph("moe_fp8_quantize_weight", _FP8_GRADIENTS)
    c, s, ct, st = _fp8_pairs(out, (codes, codes, transpose, transpose),
                              ((n, k), (_blocks(n), _blocks(k)), (k, ld), (_blocks(k), _blocks(n))), (u8, sd, u8, sd), dev)
    _launch(dev, lib.moe_fp8_quantize_weight, n, k, _at(w), DT[w.dtype], FP8_SCALE_F32 if sd is torch.float32 else FP8_SCALE_E8M0,
            _at(c), _at(s), _at(ct), _at(st))
    return c, s, ct, st


def moe_fp8_dequant(codes, scales, out=None, out_dtype=torch.bfloat16):
    """The values of moe_fp8_quantize's codes and scales (either form: [rows][cols], [rows][ceil(cols/128)]), bf16 or float32."""
    rows, cols = _matrix(codes, "codes")
    dev = codes.device
    dt = out.dtype if out is not None else out_dtype
    if dt not in DT:
        raise TypeError(f"values must be bfloat16 or float32 (got {dt})")
    sshape = (rows, (cols + 127) // 128)
    if not (codes.is_cuda and codes.dtype is torch.uint8 and codes.is_contiguous() and scales is not None
            and _fits(dev, scales, torch.uint8, sshape) and _fits(dev, out, dt, (rows, cols))):
        _operands(dev, (codes, torch.uint8, "codes", None), (scales, torch.uint8, "scales", sshape), (out, dt, "out", (rows, cols)))
    _int32(rows, cols)
    o = out if out is not None else torch.empty((rows, cols), dtype=dt, device=dev)
    _launch(dev, lib.moe_fp8_dequant, rows, cols, _at(codes), _at(scales), _at(o), DT[dt])
    return o


@functools.lru_cache(maxsize=4096)
def _fp8_plan(*sizes):
    """(descriptor, workspace bytes) of moe_fp8_linear: a function of its sizes and types alone."""
    _int32(*sizes)
    d = ctypes.byref(Fp8LinearDesc(*sizes))
    return d, lib.moe_fp8_linear_workspace(d)


def _x_dtype(x_dtype):
    return DT_FP8 if x_dtype is torch.uint8 else DT[x_dtype]


def moe_fp8_linear_workspace(T, n, kdim, x_dtype=torch.bfloat16, out_dtype=torch.bfloat16, w_scale=FP8_SCALE_F32):
    return _fp8_plan(T, n, kdim, _x_dtype(x_dtype), DT[out_dtype], w_scale)[1]


def moe_fp8_linear(x, w, w_scales, x_scales=None, residual=None, out=None, out_dtype=None, ws=None):
    """y = x w^T + residual of block-128 FP8 operands.  x [T][kdim]: bf16 or float32 (quantised by the call), or uint8 codes with
    x_scales uint8 [T][ceil(kdim/128)] (moe_fp8_quantize).  w uint8 codes [n][kdim]; w_scales: float32 or uint8 (E8M0)
    [ceil(n/128)][ceil(kdim/128)], or uint8 [n][ceil(kdim/128)] (a row's own).  residual [T][n] of y's type (may be `out`);
    y [T][n] of out_dtype (bf16 when None), bf16 or float32.  Autograd does not see the call (it warns of operands that require grad)."""
    T, kdim = _matrix(x, "x")
    n = _matrix(w, "w")[0]
    dt = out.dtype if out is not None else (out_dtype or torch.bfloat16)
    if dt not in DT:
        raise TypeError(f"y must be bfloat16 or float32 (got {dt})")
    dev, u8 = x.device, torch.uint8
    kb = (kdim + 127) // 128
    _matrix(w_scales, "w_scales")
    kind = FP8_SCALE_F32 if w_scales.dtype == torch.float32 else (
        FP8_SCALE_E8M0_ROW if w_scales.shape[0] == n and n > 1 else FP8_SCALE_E8M0)
    if (x_scales is not None) != (x.dtype == u8):
        raise TypeError("x_scales belong to uint8 codes, and to them only")
    sshape = (n if kind == FP8_SCALE_E8M0_ROW else (n + 127) // 128, kb)
    if not (x.is_cuda and (x.dtype is u8 or x.dtype in DT) and x.is_contiguous() and _fits(dev, w, u8, (n, kdim))
            and _fits(dev, w_scales, torch.float32 if kind == FP8_SCALE_F32 else u8, sshape) and _fits(dev, x_scales, u8, (T, kb))
            and _fits(dev, residual, dt, (T, n)) and _fits(dev, out, dt, (T, n))):
        _operands(dev, (x, _one_of(x, (*DT, u8)), "x", None), (w, u8, "w", (n, kdim)),
                  (w_scales, _one_of(w_scales, (torch.float32, u8)), "w_scales", sshape), (x_scales, u8, "x_scales", (T, kb)),
                  (residual, dt, "residual", (T, n)), (out, dt, "out", (T, n)))
    if torch.is_grad_enabled() and (x.requires_grad or (residual is not None and residual.requires_grad)):
        _outside_graph("moe_fp8_linear", _FP8_GRADIENTS)
    d, need = _fp8_plan(T, n, kdim, _x_dtype(x.dtype), DT[dt], kind)
    y = out if out is not None else torch.empty((T, n), dtype=dt, device=dev)
    ws, nws = _ws_for(ws, need, dev)
    _launch(dev, lib.moe_fp8_linear, d, _at(x), _at(x_scales), _at(w), _at(w_scales), _at(residual), _at(y), _at(ws), nws)
    return y


# ------------------------------------------------------------------ norms around a block

_RNG = (torch.int64, torch.uint64)


def _gate_kind(gate, T, d):
    """MOE_GATE_* of a gate float32 [T][1] (one a token) or [d] / [1][d] (one a channel)."""
    if gate is None:
        return GATE_NONE
    if not isinstance(gate, torch.Tensor):
        raise TypeError("gate must be a torch.Tensor")
    if tuple(gate.shape) == (T, 1):
        return GATE_TOKEN
    if tuple(gate.shape) in ((d,), (1, d)):
        return GATE_CHANNEL
    raise ValueError(f"gate has shape {tuple(gate.shape)}, expected {(T, 1)} (a token's) or {(1, d)} (a channel's)")


def _constant(v):
    """A number, or what holds one (such as a tensor of one element), as the C side's float: its value at this call."""
    return _f32(v).value


def _norm_desc(T, d, zt, yt, kind, eps, residual_scale, dropout):
    # (values, not objects: a tensor is the same key after its value has changed; -0 as 0, which is the same key)
    if not type(eps) is type(residual_scale) is type(dropout) is float:
        eps, residual_scale, dropout = _constant(eps), _constant(residual_scale), _constant(dropout)
    return _norm_plan(T, d, zt, yt, kind, eps, residual_scale + 0.0, dropout)


@functools.lru_cache(maxsize=4096)
def _norm_plan(T, d, zt, yt, kind, eps, residual_scale, dropout):
    """(descriptor, workspace bytes of the backward call): a function of sizes, types and constants alone."""
    _int32(T, d)
    n = ctypes.byref(BlockNormDesc(T, d, zt, yt, kind, eps, residual_scale, dropout))
    return n, lib.moe_block_norm_backward_workspace(n)


def moe_block_norm_backward_workspace(T, d):
    return _norm_desc(T, d, 0, 0, 0, 1.0, 1.0, 0.0)[1]


def moe_block_norm(z, w_after=None, gate=None, residual=None, w_before=None, residual_scale=1.0, dropout=0.0, rng=None, eps=1e-6,
                   want_y=True, want_u=None, want_codes=False, y_dtype=None, out=None):
    """y = residual_scale * residual + gate * dropout(rmsnorm(z) w_after) and u = rmsnorm(y) w_before, in one pass.
    z [T][d] bf16 or float32; w_after, w_before float32 [d] or None (no norm there); gate float32 [T][1] (one a token) or [1][d]
    (one a channel); residual [T][d] of y's type; rng: int64 or uint64 [2] device tensor (seed, offset), needed with dropout and read when
    the call runs.  Returns (y, u, u_codes, u_scales): y of y_dtype (residual's type, or bf16); u bf16, and its FP8 form
    (moe_fp8_quantize's rows) with want_codes, when w_before is given; None for what is not wanted.  want_u: None means yes.  out: the
    four results' tensors (y may be the residual).  The norm before a block alone: z, w_before, want_y=False.
    residual_scale, dropout and eps are numbers; a tensor of one element counts with its value at the call, and a captured graph keeps
    that value."""
    T, d = _matrix(z, "z")
    yt = residual.dtype if isinstance(residual, torch.Tensor) else (
        out[0].dtype if out is not None and out[0] is not None else (y_dtype or torch.bfloat16))
    if yt not in DT or (y_dtype is not None and y_dtype != yt):
        raise TypeError(f"y must be bfloat16 or float32, and residual of its type (got {yt}, y_dtype {y_dtype})")
    before = w_before is not None
    if not before and (want_u or want_codes):
        raise ValueError("moe_block_norm: u and its codes need w_before")
    u_on = before and want_u is not False
    codes_on = before and want_codes
    dev, f32, u8, bf = z.device, torch.float32, torch.uint8, torch.bfloat16
    kind = GATE_NONE if gate is None else _gate_kind(gate, T, d)
    oy, ou, oc, os_ = out if out is not None else (None,) * 4
    sshape = (T, (d + 127) // 128)
    if not (z.is_cuda and z.dtype in DT and z.is_contiguous() and _fits(dev, w_after, f32, (d,)) and _fits(dev, w_before, f32, (d,))
            and _fits(dev, residual, yt, (T, d)) and (gate is None or _fits(dev, gate, f32, gate.shape))
            and _fits(dev, rng, _one_of(rng, _RNG), (2,))
            and (out is None or (_fits(dev, oy, yt, (T, d)) and _fits(dev, ou, bf, (T, d)) and _fits(dev, oc, u8, (T, d)) and _fits(dev, os_, u8, sshape)))):
        _operands(dev, (z, _one_of(z, DT), "z", None), (w_after, f32, "w_after", (d,)), (w_before, f32, "w_before", (d,)),
                  (gate, f32, "gate", None), (residual, yt, "residual", (T, d)), (rng, _one_of(rng, _RNG), "rng", (2,)),
                  (oy, yt, "y", (T, d)), (ou, bf, "u", (T, d)), (oc, u8, "u_codes", (T, d)), (os_, u8, "u_scales", sshape))
    if torch.is_grad_enabled() and (z.requires_grad or any(t is not None and t.requires_grad for t in (w_after, w_before, gate, residual))):
        _outside_graph("moe_block_norm")
    if oy is None and want_y:
        oy = torch.empty((T, d), dtype=yt, device=dev)
    if ou is None and u_on:
        ou = torch.empty((T, d), dtype=bf, device=dev)
    if oc is None and codes_on:
        oc = torch.empty((T, d), dtype=u8, device=dev)
    if os_ is None and codes_on:
        os_ = torch.empty(sshape, dtype=u8, device=dev)
    oy, ou, oc, os_ = (oy if want_y else None, ou if u_on else None, oc if codes_on else None, os_ if codes_on else None)
    n = _norm_desc(T, d, DT[z.dtype], DT[yt], kind, eps, residual_scale, dropout)[0]
    _launch(dev, lib.moe_block_norm, n, z.data_ptr(), _at(w_after), _at(gate), _at(rng), _at(residual), _at(w_before), _at(oy),
            _at(ou), _at(oc), _at(os_))
    return oy, ou, oc, os_


def moe_block_norm_backward(z, w_after=None, gate=None, y=None, w_before=None, du=None, dy=None, residual_scale=1.0, dropout=0.0,
                            rng=None, eps=1e-6, y_dtype=None, z_dtype=None, want=("dz", "dresidual", "dw_after", "dgate", "dw_before"),
                            out=None, ws=None):
    """Gradients of moe_block_norm at du (bf16, of u) and dy (of y's type, or None: zero): (dz of z's type, dresidual of y's type,
    dw_after, dgate of gate's shape, dw_before, float32), None for what `want` does not name or there is no tensor for.  z, w_after, gate, rng
    and w_before as in the forward call, y its result (with w_before).  z may be None where none of dz through a norm, dw_after and
    dgate is wanted (z_dtype: the type of dz then).  out: the five results' tensors."""
    ref = next((t for t in (z, dy, du, y) if isinstance(t, torch.Tensor)), None)
    T, d = _matrix(ref if z is None else z, "z")
    on = _wanted(want, ("dz", "dresidual", "dw_after", "dgate", "dw_before"))
    on = [on[0], on[1], on[2] and w_after is not None, on[3] and gate is not None, on[4] and w_before is not None]
    o = out if out is not None else (None,) * 5
    yt = next((t.dtype for t in (dy, y, o[1]) if isinstance(t, torch.Tensor)), y_dtype or torch.bfloat16)
    zt = z.dtype if isinstance(z, torch.Tensor) else (o[0].dtype if o[0] is not None else (z_dtype or torch.bfloat16))
    if yt not in DT or zt not in DT or (y_dtype is not None and y_dtype != yt):
        raise TypeError(f"y and z must be bfloat16 or float32 (got y {yt}, y_dtype {y_dtype}, z {zt})")
    dev, f32 = ref.device, torch.float32
    kind = _gate_kind(gate, T, d)
    shapes = ((T, d), (T, d), (d,), tuple(gate.shape) if gate is not None else None, (d,))
    types = (zt, yt, f32, f32, f32)
    bf = torch.bfloat16
    if not (ref.is_cuda and _fits(dev, z, zt, (T, d)) and _fits(dev, w_after, f32, (d,)) and _fits(dev, w_before, f32, (d,))
            and (gate is None or _fits(dev, gate, f32, gate.shape)) and _fits(dev, y, yt, (T, d)) and _fits(dev, du, bf, (T, d))
            and _fits(dev, dy, yt, (T, d)) and _fits(dev, rng, _one_of(rng, _RNG), (2,))
            and (out is None or all(_fits(dev, t, dt, sh) for t, dt, sh in zip(o, types, shapes)))):
        _operands(dev, (ref, _one_of(ref, DT), "z", (T, d)), (z, zt, "z", (T, d)), (w_after, f32, "w_after", (d,)),
                  (w_before, f32, "w_before", (d,)), (gate, f32, "gate", None), (y, yt, "y", (T, d)), (du, bf, "du", (T, d)),
                  (dy, yt, "dy", (T, d)), (rng, _one_of(rng, _RNG), "rng", (2,)),
                  *((t, dt, nm, sh) for t, dt, nm, sh in zip(o, types, ("dz", "dresidual", "dw_after", "dgate", "dw_before"), shapes)))
    r = [None if not w else (t if t is not None else torch.empty(sh, dtype=dt, device=dev))
         for t, dt, sh, w in zip(o, types, shapes, on)]
    n, need = _norm_desc(T, d, DT[zt], DT[yt], kind, eps, residual_scale, dropout)
    ws, nws = _ws_for(ws, need if on[2] or on[4] or (on[3] and kind == GATE_CHANNEL) else 0, dev)
    _launch(dev, lib.moe_block_norm_backward, n, _at(z), _at(w_after), _at(gate), _at(rng), _at(y), _at(w_before), _at(du), _at(dy),
            *map(_at, r), _at(ws), nws)
    return tuple(r)

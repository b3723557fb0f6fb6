"""ctypes binding of libmoe.so (include/moe.h): argument marshalling only.

Every step of the layer runs in the library's CUDA kernels. PyTorch supplies device
memory and the current stream; nothing here computes any part of the layer, and
there is no fallback: if the library is missing or a tensor is not on a CUDA device,
the call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from functools import lru_cache
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# MOE_LIB_PATH selects another build of the same library (it must exist)
LIB_PATH = os.environ.get("MOE_LIB_PATH") or os.path.join(_HERE, "libmoe.so")
ROW_PAD = 128

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT"}

EXPORTS = ("moe_workspace_size", "moe_workspace_size_host", "moe_max_padded_rows",
           "moe_router_topk", "moe_permute", "moe_grouped_swiglu", "moe_expert_gate_up",
           "moe_expert_down", "moe_combine", "moe_forward",
           "moe_forward_host", "moe_device_status", "moe_last_error", "moe_permute_static",
           "moe_selftest_wait_timeout", "moe_forward_rmsnorm", "moe_pack_weights",
           "moe_quantize_int8", "moe_grouped_swiglu_w8", "moe_forward_w8", "moe_gather_rows",
           "moe_forward_host_async", "moe_quantize_int4", "moe_grouped_swiglu_w4", "moe_forward_w4",
           "moe_ipc_alloc", "moe_ipc_open", "moe_ipc_close", "moe_ipc_free",
           "moe_scatter_rows_peer", "moe_combine_peer", "moe_route", "moe_router_losses",
           "moe_router_losses_workspace", "moe_route_backward", "moe_combine_backward",
           "moe_lora_workspace", "moe_lora_add", "moe_lora_rows", "moe_swiglu_rows", "moe_forward_routing")


@dataclass
class Int8Experts:
    """Weight-only int8 experts as written by quantize_int8: codes q1, q3 [E, I, H] and
    q2 [E, H, I] (uint8, offset-binary q + 128, in the library's tiled code layout of
    include/moe.h; same number of elements), per-row scales s1, s3 [E, I] and s2 [E, H]
    fp32."""
    q1: torch.Tensor
    q3: torch.Tensor
    q2: torch.Tensor
    s1: torch.Tensor
    s3: torch.Tensor
    s2: torch.Tensor

    def pointers(self):
        return [_dev(self.q1, "q1", torch.uint8), _dev(self.q3, "q3", torch.uint8),
                _dev(self.q2, "q2", torch.uint8), _dev(self.s1, "s1", torch.float32),
                _dev(self.s3, "s3", torch.float32), _dev(self.s2, "s2", torch.float32)]


@dataclass
class Int4Experts:
    """Weight-only 4-bit experts as written by quantize_int4: codes q1, q3 [E, I, H/2] and
    q2 [E, H, I/2] (uint8, two offset-binary codes q + 8 to a byte, in the library's
    tiled 4-bit layout of include/moe.h) and float16 scales, one per row and 64-column
    group in tile order: s1, s3 [E, I/128, H/64, 128] and s2 [E, H/128, I/64, 128]."""
    q1: torch.Tensor
    q3: torch.Tensor
    q2: torch.Tensor
    s1: torch.Tensor
    s3: torch.Tensor
    s2: torch.Tensor

    def pointers(self):
        return [_dev(self.q1, "q1", torch.uint8), _dev(self.q3, "q3", torch.uint8),
                _dev(self.q2, "q2", torch.uint8), _dev(self.s1, "s1", torch.float16),
                _dev(self.s3, "s3", torch.float16), _dev(self.s2, "s2", torch.float16)]


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


ROW_MAJOR, BLOCKED = 0, 1  # MOE_WEIGHTS_* layouts of the expert weights


class Shape(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int64), ("hidden_size", ctypes.c_int32),
                ("intermediate_size", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("num_experts_per_tok", ctypes.c_int32), ("weight_layout", ctypes.c_int32),
                ("router_bf16_logits", ctypes.c_int32)]


class _RoutingArgs(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int64), ("logits_stride", ctypes.c_int64),
                ("num_experts", ctypes.c_int32), ("num_experts_per_tok", ctypes.c_int32),
                ("scoring", ctypes.c_int32), ("num_groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("logits_bf16", ctypes.c_int32),
                ("weight_scale", ctypes.c_float)]


class _LoraArgs(ctypes.Structure):
    _fields_ = [("num_rows", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("base_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
                ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("num_adapters", ctypes.c_int32),
                ("out_fp32", ctypes.c_int32)]


_lib = None
_P = ctypes.c_void_p
_SZ = ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m sparse_mixture_experts_09_b200.build_lib`")
        L = ctypes.CDLL(LIB_PATH)
        sp = ctypes.POINTER(Shape)
        st = ctypes.c_int
        L.moe_workspace_size.argtypes = [sp]
        L.moe_workspace_size.restype = _SZ
        L.moe_workspace_size_host.argtypes = [sp]
        L.moe_workspace_size_host.restype = _SZ
        L.moe_max_padded_rows.argtypes = [sp]
        L.moe_max_padded_rows.restype = ctypes.c_int64
        L.moe_router_topk.argtypes = [sp, _P, _P, _P, _P, _P, _P, _P]
        L.moe_router_topk.restype = st
        L.moe_permute.argtypes = [sp, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_permute.restype = st
        L.moe_grouped_swiglu.argtypes = [sp, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_grouped_swiglu.restype = st
        L.moe_expert_gate_up.argtypes = [sp, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_expert_gate_up.restype = st
        L.moe_expert_down.argtypes = [sp, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_expert_down.restype = st
        L.moe_combine.argtypes = [sp, _P, _P, _P, _P, _P, _P]
        L.moe_combine.restype = st
        L.moe_forward.argtypes = [sp, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_forward.restype = st
        L.moe_forward_rmsnorm.argtypes = [sp, _P, _P, ctypes.c_float, _P, _P, _P, _P, _P, _P, _P,
                                          _SZ, _P]
        L.moe_forward_rmsnorm.restype = st
        L.moe_pack_weights.argtypes = [sp, _P, _P, _P, _P, _P, _P, _P]
        L.moe_pack_weights.restype = st
        L.moe_forward_host.argtypes = [sp, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_forward_host_async.argtypes = [sp, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_forward_host_async.restype = st
        L.moe_forward_host.restype = st
        L.moe_device_status.argtypes = [_P, _SZ, _P]
        L.moe_device_status.restype = st
        L.moe_permute_static.argtypes = [sp, _P, _P, _P, _P, _P, _P, _P, _P]
        L.moe_permute_static.restype = st
        L.moe_selftest_wait_timeout.argtypes = [_P, _SZ, ctypes.c_uint64, _P]
        L.moe_selftest_wait_timeout.restype = st
        L.moe_quantize_int8.argtypes = [sp] + [_P] * 10
        L.moe_quantize_int8.restype = st
        L.moe_grouped_swiglu_w8.argtypes = [sp] + [_P] * 10 + [_SZ, _P]
        L.moe_grouped_swiglu_w8.restype = st
        L.moe_forward_w8.argtypes = [sp] + [_P] * 12 + [_SZ, _P]
        L.moe_forward_w8.restype = st
        L.moe_quantize_int4.argtypes = [sp] + [_P] * 10
        L.moe_quantize_int4.restype = st
        L.moe_grouped_swiglu_w4.argtypes = [sp] + [_P] * 10 + [_SZ, _P]
        L.moe_grouped_swiglu_w4.restype = st
        L.moe_forward_w4.argtypes = [sp] + [_P] * 12 + [_SZ, _P]
        L.moe_forward_w4.restype = st
        L.moe_gather_rows.argtypes = [_P, ctypes.c_int64, _P, ctypes.c_int64, ctypes.c_int64, _P, _P]
        L.moe_gather_rows.restype = st
        L.moe_ipc_alloc.argtypes = [_SZ, ctypes.POINTER(_P), _P]
        L.moe_ipc_alloc.restype = st
        L.moe_ipc_open.argtypes = [_P, ctypes.POINTER(_P)]
        L.moe_ipc_open.restype = st
        L.moe_ipc_close.argtypes = [_P]
        L.moe_ipc_close.restype = st
        L.moe_ipc_free.argtypes = [_P]
        L.moe_ipc_free.restype = st
        L.moe_scatter_rows_peer.argtypes = [_P, ctypes.c_int64, _P, _P, _P, ctypes.c_int64, _P,
                                            ctypes.c_int, ctypes.c_int64, ctypes.c_int64, _P, _P]
        L.moe_scatter_rows_peer.restype = st
        L.moe_combine_peer.argtypes = [_P, ctypes.c_int, ctypes.c_int64, _P, _P, _P, _P, _P,
                                       ctypes.c_int64, ctypes.c_int, ctypes.c_int, _P, _P]
        L.moe_combine_peer.restype = st
        rp = ctypes.POINTER(_RoutingArgs)
        L.moe_route.argtypes = [rp, _P, _P, _P, _P, _P]
        L.moe_route.restype = st
        L.moe_router_losses_workspace.argtypes = [rp]
        L.moe_router_losses_workspace.restype = _SZ
        L.moe_router_losses.argtypes = [rp, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_router_losses.restype = st
        L.moe_route_backward.argtypes = [rp, _P, _P, _P, _P, _P, _P, _P, _P]
        L.moe_route_backward.restype = st
        L.moe_combine_backward.argtypes = [_P] * 8 + [ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                                      ctypes.c_int, ctypes.c_int64, _P]
        L.moe_combine_backward.restype = st
        lp = ctypes.POINTER(_LoraArgs)
        L.moe_lora_workspace.argtypes = [lp]
        L.moe_lora_workspace.restype = _SZ
        L.moe_lora_add.argtypes = [lp] + [_P] * 8 + [_SZ, _P]
        L.moe_lora_add.restype = st
        L.moe_lora_rows.argtypes = [_P, _P, _P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                    ctypes.c_int, _P, _P]
        L.moe_lora_rows.restype = st
        L.moe_swiglu_rows.argtypes = [_P, _P, _P, ctypes.c_int, ctypes.c_int64, ctypes.c_int, _P, _P]
        L.moe_swiglu_rows.restype = st
        L.moe_forward_routing.argtypes = [sp, rp] + [_P] * 10 + [_SZ, _P]
        L.moe_forward_routing.restype = st
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != 0:
        raise MoeError(status, lib().moe_last_error().decode(errors="replace"))


def make_shape(num_tokens: int, hidden_size: int, intermediate_size: int, num_experts: int,
               num_experts_per_tok: int, weight_layout: int = ROW_MAJOR,
               router_bf16_logits: bool = False) -> Shape:
    return Shape(int(num_tokens), int(hidden_size), int(intermediate_size), int(num_experts),
                 int(num_experts_per_tok), int(weight_layout), int(bool(router_bf16_logits)))


def _dev(t: Optional[torch.Tensor], name: str, dtype=None, nullable=False) -> Optional[int]:
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _sized(name: str, t: Optional[torch.Tensor], n: int, at_least: bool = False) -> None:
    """The kernels index a buffer by the layer's shape alone (the C ABI takes bare
    pointers), so one of the wrong size would be read or written out of bounds: refuse
    it here, before any pointer is taken."""
    if t is None:
        return
    if t.numel() < n or (t.numel() != n and not at_least):
        need = f"at least {n}" if at_least else f"{n}"
        raise ValueError(f"{name} has {t.numel()} elements; the layer's shape needs {need}")


def _layer_sizes(t: int, h: int, e: int, i: int, w_router=None, logit_bias=None, residual=None,
                 out=None, **weights) -> None:
    """Element counts of the tensors of a whole-layer call: w_router [E, H], logit_bias
    [E], residual and out [T, H], and each keyword ``name=(tensor, count)``."""
    _sized("w_router", w_router, e * h)
    _sized("logit_bias", logit_bias, e)
    _sized("residual", residual, t * h)
    _sized("out", out, t * h)
    for name, (tensor, n) in weights.items():
        # x_perm may be a larger buffer: the kernels read its first R_max rows
        _sized(name, tensor, n, at_least=name == "x_perm")


def _bf16_weights(e: int, i: int, h: int, w1, w3, w2) -> dict:
    return {"w1": (w1, e * i * h), "w3": (w3, e * i * h), "w2": (w2, e * h * i)}


def _quant_weights(e: int, i: int, h: int, ex, bits: int) -> dict:
    """Codes and scales of Int8Experts (bits 8) or Int4Experts (bits 4)."""
    per = (lambda n: n) if bits == 8 else (lambda n: n // 2)
    sc = (lambda rows, k: rows) if bits == 8 else (lambda rows, k: rows * k // 64)
    return {"q1": (ex.q1, per(e * i * h)), "q3": (ex.q3, per(e * i * h)),
            "q2": (ex.q2, per(e * h * i)), "s1": (ex.s1, sc(e * i, h)),
            "s3": (ex.s3, sc(e * i, h)), "s2": (ex.s2, sc(e * h, i))}


def _stream(stream) -> Optional[int]:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def workspace_size(shape: Shape) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(shape)))


def workspace_size_host(shape: Shape) -> int:
    return int(lib().moe_workspace_size_host(ctypes.byref(shape)))


def max_padded_rows(shape: Shape) -> int:
    return int(lib().moe_max_padded_rows(ctypes.byref(shape)))


def make_workspace(shape: Shape, device="cuda", host: bool = False) -> torch.Tensor:
    """A zeroed device workspace (zero status word) big enough for ``shape``."""
    n = workspace_size_host(shape) if host else workspace_size(shape)
    if n == 0:
        raise MoeError(2, lib().moe_last_error().decode(errors="replace"))
    return torch.zeros(n, dtype=torch.uint8, device=device)


def router_topk(x, w_router, k: int, logit_bias=None, return_logits=False, stream=None,
                router_bf16_logits: bool = False):
    """(topk_idx [T,k] int32, topk_w [T,k] fp32[, logits [T,E] fp32])."""
    t, h = x.shape
    e = w_router.shape[0]
    shape = make_shape(t, h, ROW_PAD, e, k, router_bf16_logits=router_bf16_logits)
    _layer_sizes(t, h, e, ROW_PAD, w_router, logit_bias)
    idx = torch.empty((t, k), dtype=torch.int32, device=x.device)
    w = torch.empty((t, k), dtype=torch.float32, device=x.device)
    logits = torch.empty((t, e), dtype=torch.float32, device=x.device) if return_logits else None
    _check(lib().moe_router_topk(ctypes.byref(shape), _dev(x, "x", torch.bfloat16),
                                 _dev(w_router, "w_router", torch.bfloat16),
                                 _dev(logit_bias, "logit_bias", torch.float32, True),
                                 _dev(idx, "idx"), _dev(w, "w"), _dev(logits, "logits", None, True),
                                 _stream(stream)))
    return (idx, w, logits) if return_logits else (idx, w)


def permute(topk_idx, x, num_experts: int, intermediate_size: int, ws, stream=None) -> dict:
    """Expert-contiguous permutation of the routed rows (see moe_permute)."""
    t, k = topk_idx.shape
    h = x.shape[1]
    shape = make_shape(t, h, intermediate_size, num_experts, k)
    _sized("x", x, t * h, at_least=True)      # the gather reads rows 0 .. T-1
    rmax = max_padded_rows(shape)
    dev = x.device
    out = {
        "counts": torch.empty(num_experts, dtype=torch.int32, device=dev),
        "offsets": torch.empty(num_experts + 1, dtype=torch.int32, device=dev),
        "row_of": torch.empty((t, k), dtype=torch.int32, device=dev),
        "token_of_row": torch.full((rmax,), -2, dtype=torch.int32, device=dev),
        "x_perm": torch.zeros((rmax, h), dtype=torch.bfloat16, device=dev),
    }
    _check(lib().moe_permute(ctypes.byref(shape), _dev(topk_idx, "topk_idx", torch.int32),
                             _dev(x, "x", torch.bfloat16), _dev(out["counts"], "counts"),
                             _dev(out["offsets"], "offsets"), _dev(out["row_of"], "row_of"),
                             _dev(out["token_of_row"], "token_of_row"), _dev(out["x_perm"], "x_perm"),
                             _dev(ws, "ws"), ws.numel(), _stream(stream)))
    return out


def permute_static(topk_idx, x, num_experts: int, intermediate_size: int, stream=None) -> dict:
    """moe_permute_static: the permutation without a workspace, for callers that cannot
    allocate device memory (its scratch is a static array in the library; calls that
    overlap on the GPU race on it). Same results as ``permute``."""
    t, k = topk_idx.shape
    h = x.shape[1]
    shape = make_shape(t, h, intermediate_size, num_experts, k)
    _sized("x", x, t * h, at_least=True)      # the gather reads rows 0 .. T-1
    rmax = max_padded_rows(shape)
    dev = x.device
    out = {
        "counts": torch.empty(num_experts, dtype=torch.int32, device=dev),
        "offsets": torch.empty(num_experts + 1, dtype=torch.int32, device=dev),
        "row_of": torch.empty((t, k), dtype=torch.int32, device=dev),
        "token_of_row": torch.full((rmax,), -2, dtype=torch.int32, device=dev),
        "x_perm": torch.zeros((rmax, h), dtype=torch.bfloat16, device=dev),
    }
    _check(lib().moe_permute_static(ctypes.byref(shape), _dev(topk_idx, "topk_idx", torch.int32),
                                    _dev(x, "x", torch.bfloat16), _dev(out["counts"], "counts"),
                                    _dev(out["offsets"], "offsets"), _dev(out["row_of"], "row_of"),
                                    _dev(out["token_of_row"], "token_of_row"),
                                    _dev(out["x_perm"], "x_perm"), _stream(stream)))
    return out


def _out_rows(y, rows: int, h: int, device):
    """The experts' fp32 output: y itself (its first rows x h elements are written; it
    must hold at least that many), or a new zeroed [rows, h] tensor."""
    if y is None:
        return torch.zeros((rows, h), dtype=torch.float32, device=device)
    _sized("y_perm", y, rows * h, at_least=True)
    return y


def grouped_swiglu(x_perm, offsets, w1, w3, w2, num_tokens: int, k: int, ws, stream=None,
                   weight_layout: int = ROW_MAJOR, y=None):
    """y_perm [R_max, H] fp32 = w2[e] (silu(w1[e] x) * w3[e] x) per routed row (into
    `y` when given: an fp32 CUDA tensor of at least R_max x H elements)."""
    e, i, h = w1.shape
    shape = make_shape(num_tokens, h, i, e, k, weight_layout)
    _layer_sizes(0, h, e, i, x_perm=(x_perm, max_padded_rows(shape) * h),
                 offsets=(offsets, e + 1), **_bf16_weights(e, i, h, w1, w3, w2))
    y = _out_rows(y, max_padded_rows(shape), h, x_perm.device)
    _check(lib().moe_grouped_swiglu(ctypes.byref(shape), _dev(x_perm, "x_perm", torch.bfloat16),
                                    _dev(offsets, "offsets", torch.int32),
                                    _dev(w1, "w1", torch.bfloat16), _dev(w3, "w3", torch.bfloat16),
                                    _dev(w2, "w2", torch.bfloat16), _dev(y, "y_perm"),
                                    _dev(ws, "ws"), ws.numel(), _stream(stream)))
    return y


def expert_gate_up(x_perm, offsets, w1, w3, num_tokens: int, k: int, ws, h=None, stream=None,
                   weight_layout: int = ROW_MAJOR):
    """h [R_max, I] bf16 = bf16(silu(x_perm w1[e]^T) * (x_perm w3[e]^T)) (GEMM1 alone)."""
    e, i, hd = w1.shape
    shape = make_shape(num_tokens, hd, i, e, k, weight_layout)
    if h is None:
        h = torch.zeros((max_padded_rows(shape), i), dtype=torch.bfloat16, device=x_perm.device)
    _check(lib().moe_expert_gate_up(ctypes.byref(shape), _dev(x_perm, "x_perm", torch.bfloat16),
                                    _dev(offsets, "offsets", torch.int32),
                                    _dev(w1, "w1", torch.bfloat16), _dev(w3, "w3", torch.bfloat16),
                                    _dev(h, "h", torch.bfloat16), _dev(ws, "ws"), ws.numel(),
                                    _stream(stream)))
    return h


def expert_down(h, offsets, w2, num_tokens: int, k: int, ws, y=None, stream=None,
                weight_layout: int = ROW_MAJOR):
    """y_perm [R_max, H] fp32 = h w2[e]^T (GEMM2 alone)."""
    e, hd, i = w2.shape
    shape = make_shape(num_tokens, hd, i, e, k, weight_layout)
    if y is None:
        y = torch.zeros((max_padded_rows(shape), hd), dtype=torch.float32, device=h.device)
    _check(lib().moe_expert_down(ctypes.byref(shape), _dev(h, "h", torch.bfloat16),
                                 _dev(offsets, "offsets", torch.int32), _dev(w2, "w2", torch.bfloat16),
                                 _dev(y, "y_perm", torch.float32), _dev(ws, "ws"), ws.numel(),
                                 _stream(stream)))
    return y


def combine(y_perm, row_of, topk_w, residual=None, num_experts: int = 8, intermediate_size: int = ROW_PAD,
            stream=None):
    """out [T,H] bf16 = residual + sum_j topk_w[:,j] * y_perm[row_of[:,j]]."""
    t, k = row_of.shape
    h = y_perm.shape[1]
    shape = make_shape(t, h, intermediate_size, max(num_experts, k), k)
    _sized("topk_w", topk_w, t * k)
    _sized("residual", residual, t * h)
    out = torch.empty((t, h), dtype=torch.bfloat16, device=y_perm.device)
    _check(lib().moe_combine(ctypes.byref(shape), _dev(y_perm, "y_perm", torch.float32),
                             _dev(row_of, "row_of", torch.int32), _dev(topk_w, "topk_w", torch.float32),
                             _dev(residual, "residual", torch.bfloat16, True), _dev(out, "out"),
                             _stream(stream)))
    return out


def forward(x, w_router, w1, w3, w2, k: int, residual=None, logit_bias=None, ws=None, out=None,
            stream=None, weight_layout: int = ROW_MAJOR, router_bf16_logits: bool = False):
    """The whole layer on device tensors; returns out [T,H] bf16."""
    t, h = x.shape
    e, i, _ = w1.shape
    shape = make_shape(t, h, i, e, k, weight_layout, router_bf16_logits)
    _layer_sizes(t, h, e, i, w_router, logit_bias, residual, out,
                 **_bf16_weights(e, i, h, w1, w3, w2))
    if ws is None:
        ws = make_workspace(shape, x.device)
    if out is None:
        out = torch.empty((t, h), dtype=torch.bfloat16, device=x.device)
    _check(lib().moe_forward(ctypes.byref(shape), _dev(x, "x", torch.bfloat16),
                             _dev(w_router, "w_router", torch.bfloat16),
                             _dev(logit_bias, "logit_bias", torch.float32, True),
                             _dev(w1, "w1", torch.bfloat16), _dev(w3, "w3", torch.bfloat16),
                             _dev(w2, "w2", torch.bfloat16),
                             _dev(residual, "residual", torch.bfloat16, True), _dev(out, "out"),
                             _dev(ws, "ws"), ws.numel(), _stream(stream)))
    return out


def forward_rmsnorm(h, norm_weight, eps: float, w_router, w1, w3, w2, k: int, logit_bias=None,
                    ws=None, out=None, stream=None, weight_layout: int = ROW_MAJOR):
    """out = h + moe(rms_norm(h)) on device tensors (the mixture half of the block)."""
    t, hd = h.shape
    e, i, _ = w1.shape
    shape = make_shape(t, hd, i, e, k, weight_layout)
    _layer_sizes(t, hd, e, i, w_router, logit_bias, None, out, norm_weight=(norm_weight, hd),
                 **_bf16_weights(e, i, hd, w1, w3, w2))
    if ws is None:
        ws = make_workspace(shape, h.device)
    if out is None:
        out = torch.empty((t, hd), dtype=torch.bfloat16, device=h.device)
    _check(lib().moe_forward_rmsnorm(ctypes.byref(shape), _dev(h, "h", torch.bfloat16),
                                     _dev(norm_weight, "norm_weight", torch.bfloat16), float(eps),
                                     _dev(w_router, "w_router", torch.bfloat16),
                                     _dev(logit_bias, "logit_bias", torch.float32, True),
                                     _dev(w1, "w1", torch.bfloat16), _dev(w3, "w3", torch.bfloat16),
                                     _dev(w2, "w2", torch.bfloat16), _dev(out, "out"),
                                     _dev(ws, "ws"), ws.numel(), _stream(stream)))
    return out


def forward_host(x_host, w_router, w1, w3, w2, k: int, residual_host=None, logit_bias=None,
                 ws=None, out_host=None, stream=None, weight_layout: int = ROW_MAJOR,
                 wait: bool = True):
    """The layer with host (ideally pinned) activations; returns out_host. With
    wait=False the call only enqueues (moe_forward_host_async): out_host is ready once
    the stream has been synchronised."""
    t, h = x_host.shape
    e, i, _ = w1.shape
    shape = make_shape(t, h, i, e, k, weight_layout)
    _layer_sizes(t, h, e, i, w_router, logit_bias, residual_host=(residual_host, t * h),
                 out_host=(out_host, t * h), **_bf16_weights(e, i, h, w1, w3, w2))
    for name, a in (("x_host", x_host), ("residual_host", residual_host), ("out_host", out_host)):
        if a is not None and (a.is_cuda or a.dtype != torch.bfloat16 or not a.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous bf16 host tensor")
    if ws is None:
        ws = make_workspace(shape, w1.device, host=True)
    if out_host is None:
        out_host = torch.empty((t, h), dtype=torch.bfloat16, pin_memory=True)
    fn = lib().moe_forward_host if wait else lib().moe_forward_host_async
    _check(fn(ctypes.byref(shape), x_host.data_ptr(),
                                  _dev(w_router, "w_router", torch.bfloat16),
                                  _dev(logit_bias, "logit_bias", torch.float32, True),
                                  _dev(w1, "w1", torch.bfloat16), _dev(w3, "w3", torch.bfloat16),
                                  _dev(w2, "w2", torch.bfloat16),
                                  None if residual_host is None else residual_host.data_ptr(),
                                  out_host.data_ptr(), _dev(ws, "ws"), ws.numel(), _stream(stream)))
    return out_host


def selftest_wait_timeout(ws, timeout_ns: int, stream=None) -> None:
    """Launch the bounded-wait check: a wait that nothing completes gives up after
    ``timeout_ns`` and records MOE_ERR_TIMEOUT in ``ws``'s status word."""
    _check(lib().moe_selftest_wait_timeout(_dev(ws, "ws"), ws.numel(), int(timeout_ns), _stream(stream)))


def pack_weights(w1, w3, w2, stream=None):
    """Row-major expert weights -> the blocked layout (new tensors of the same shapes);
    pass weight_layout=BLOCKED with them."""
    e, i, h = w1.shape
    shape = make_shape(1, h, i, e, 1)
    out = [torch.empty_like(t) for t in (w1, w3, w2)]
    _check(lib().moe_pack_weights(ctypes.byref(shape), _dev(w1, "w1", torch.bfloat16),
                                  _dev(w3, "w3", torch.bfloat16), _dev(w2, "w2", torch.bfloat16),
                                  _dev(out[0], "w1_blocked"), _dev(out[1], "w3_blocked"),
                                  _dev(out[2], "w2_blocked"), _stream(stream)))
    return tuple(out)


def device_status(ws, stream=None) -> None:
    """Raise MoeError(MOE_ERR_TIMEOUT) if a kernel gave up a bounded wait since last checked."""
    _check(lib().moe_device_status(_dev(ws, "ws"), ws.numel(), _stream(stream)))


def quantize_int8(w1, w3, w2, stream=None) -> Int8Experts:
    """Row-major bf16 expert weights -> Int8Experts (per-row symmetric int8)."""
    e, i, h = w1.shape
    shape = make_shape(1, h, i, e, 1)
    dev = w1.device
    q = [torch.empty(t.shape, dtype=torch.uint8, device=dev) for t in (w1, w3, w2)]
    sc = [torch.empty((e, i), dtype=torch.float32, device=dev),
          torch.empty((e, i), dtype=torch.float32, device=dev),
          torch.empty((e, h), dtype=torch.float32, device=dev)]
    out = Int8Experts(q[0], q[1], q[2], sc[0], sc[1], sc[2])
    _check(lib().moe_quantize_int8(ctypes.byref(shape), _dev(w1, "w1", torch.bfloat16),
                                   _dev(w3, "w3", torch.bfloat16), _dev(w2, "w2", torch.bfloat16),
                                   *out.pointers(), _stream(stream)))
    return out


def grouped_swiglu_w8(x_perm, offsets, experts: Int8Experts, num_tokens: int, k: int, ws,
                      stream=None, y=None):
    """grouped_swiglu with int8 expert weights: y_perm [R_max, H] fp32 (into `y` when
    given)."""
    e, i, h = experts.q1.shape
    shape = make_shape(num_tokens, h, i, e, k)
    _layer_sizes(0, h, e, i, x_perm=(x_perm, max_padded_rows(shape) * h),
                 offsets=(offsets, e + 1), **_quant_weights(e, i, h, experts, 8))
    y = _out_rows(y, max_padded_rows(shape), h, x_perm.device)
    _check(lib().moe_grouped_swiglu_w8(ctypes.byref(shape), _dev(x_perm, "x_perm", torch.bfloat16),
                                       _dev(offsets, "offsets", torch.int32), *experts.pointers(),
                                       _dev(y, "y_perm"), _dev(ws, "ws"), ws.numel(),
                                       _stream(stream)))
    return y


def forward_w8(x, w_router, experts: Int8Experts, k: int, residual=None, logit_bias=None,
               ws=None, out=None, stream=None, router_bf16_logits: bool = False):
    """The whole layer with int8 expert weights; returns out [T,H] bf16."""
    t, h = x.shape
    e, i, _ = experts.q1.shape
    shape = make_shape(t, h, i, e, k, ROW_MAJOR, router_bf16_logits)
    _layer_sizes(t, h, e, i, w_router, logit_bias, residual, out,
                 **_quant_weights(e, i, h, experts, 8))
    if ws is None:
        ws = make_workspace(shape, x.device)
    if out is None:
        out = torch.empty((t, h), dtype=torch.bfloat16, device=x.device)
    _check(lib().moe_forward_w8(ctypes.byref(shape), _dev(x, "x", torch.bfloat16),
                                _dev(w_router, "w_router", torch.bfloat16),
                                _dev(logit_bias, "logit_bias", torch.float32, True),
                                *experts.pointers(),
                                _dev(residual, "residual", torch.bfloat16, True), _dev(out, "out"),
                                _dev(ws, "ws"), ws.numel(), _stream(stream)))
    return out


def quantize_int4(w1, w3, w2, stream=None) -> Int4Experts:
    """Row-major bf16 expert weights -> Int4Experts (symmetric 4-bit, a half scale per
    64-column group of a row)."""
    e, i, h = w1.shape
    shape = make_shape(1, h, i, e, 1)
    dev = w1.device
    q = [torch.empty((e, i, h // 2), dtype=torch.uint8, device=dev),
         torch.empty((e, i, h // 2), dtype=torch.uint8, device=dev),
         torch.empty((e, h, i // 2), dtype=torch.uint8, device=dev)]
    sc = [torch.empty((e, i // 128, h // 64, 128), dtype=torch.float16, device=dev),
          torch.empty((e, i // 128, h // 64, 128), dtype=torch.float16, device=dev),
          torch.empty((e, h // 128, i // 64, 128), dtype=torch.float16, device=dev)]
    out = Int4Experts(q[0], q[1], q[2], sc[0], sc[1], sc[2])
    _check(lib().moe_quantize_int4(ctypes.byref(shape), _dev(w1, "w1", torch.bfloat16),
                                   _dev(w3, "w3", torch.bfloat16), _dev(w2, "w2", torch.bfloat16),
                                   *out.pointers(), _stream(stream)))
    return out


def grouped_swiglu_w4(x_perm, offsets, experts: Int4Experts, num_tokens: int, k: int, ws,
                      stream=None, y=None):
    """grouped_swiglu with 4-bit expert weights: y_perm [R_max, H] fp32 (into `y` when
    given)."""
    e, i, h2 = experts.q1.shape
    shape = make_shape(num_tokens, 2 * h2, i, e, k)
    _layer_sizes(0, 2 * h2, e, i, x_perm=(x_perm, max_padded_rows(shape) * 2 * h2),
                 offsets=(offsets, e + 1), **_quant_weights(e, i, 2 * h2, experts, 4))
    y = _out_rows(y, max_padded_rows(shape), 2 * h2, x_perm.device)
    _check(lib().moe_grouped_swiglu_w4(ctypes.byref(shape), _dev(x_perm, "x_perm", torch.bfloat16),
                                       _dev(offsets, "offsets", torch.int32), *experts.pointers(),
                                       _dev(y, "y_perm"), _dev(ws, "ws"), ws.numel(),
                                       _stream(stream)))
    return y


def forward_w4(x, w_router, experts: Int4Experts, k: int, residual=None, logit_bias=None,
               ws=None, out=None, stream=None, router_bf16_logits: bool = False):
    """The whole layer with 4-bit expert weights; returns out [T,H] bf16."""
    t, h = x.shape
    e, i, _ = experts.q1.shape
    shape = make_shape(t, h, i, e, k, ROW_MAJOR, router_bf16_logits)
    _layer_sizes(t, h, e, i, w_router, logit_bias, residual, out,
                 **_quant_weights(e, i, h, experts, 4))
    if ws is None:
        ws = make_workspace(shape, x.device)
    if out is None:
        out = torch.empty((t, h), dtype=torch.bfloat16, device=x.device)
    _check(lib().moe_forward_w4(ctypes.byref(shape), _dev(x, "x", torch.bfloat16),
                                _dev(w_router, "w_router", torch.bfloat16),
                                _dev(logit_bias, "logit_bias", torch.float32, True),
                                *experts.pointers(),
                                _dev(residual, "residual", torch.bfloat16, True), _dev(out, "out"),
                                _dev(ws, "ws"), ws.numel(), _stream(stream)))
    return out


def gather_rows(src, index, stream=None):
    """out[i] = src[index[i]] (a zero row where index[i] is outside [0, len(src))); src is
    a 2-D CUDA tensor whose rows are a multiple of 16 bytes, index an int64 CUDA tensor."""
    if src.dim() != 2:
        raise ValueError("src must be 2-D")
    n = index.numel()
    out = torch.empty((n, src.shape[1]), dtype=src.dtype, device=src.device)
    row_bytes = src.shape[1] * src.element_size()
    _check(lib().moe_gather_rows(_dev(src, "src") if src.shape[0] else None, src.shape[0],
                                 _dev(index, "index", torch.int64) if n else None, n, row_bytes,
                                 _dev(out, "dst") if n else None, _stream(stream)))
    return out


# ---- expert parallelism over peer memory ----

IPC_HANDLE_BYTES = 64


def ipc_alloc(nbytes: int):
    """A device buffer other processes can map: (device address, IPC handle bytes). The
    caller frees it with ipc_free once every other process has unmapped it."""
    ptr = _P()
    handle = ctypes.create_string_buffer(IPC_HANDLE_BYTES)
    _check(lib().moe_ipc_alloc(int(nbytes), ctypes.byref(ptr), ctypes.cast(handle, _P)))
    return int(ptr.value), handle.raw


def ipc_open(handle: bytes) -> int:
    """Address in this process of another process's ipc_alloc buffer."""
    if len(handle) != IPC_HANDLE_BYTES:
        raise ValueError(f"an IPC handle has {IPC_HANDLE_BYTES} bytes, got {len(handle)}")
    buf = ctypes.create_string_buffer(bytes(handle), IPC_HANDLE_BYTES)
    ptr = _P()
    _check(lib().moe_ipc_open(ctypes.cast(buf, _P), ctypes.byref(ptr)))
    return int(ptr.value)


def ipc_close(ptr: int) -> None:
    _check(lib().moe_ipc_close(ptr))


def ipc_free(ptr: int) -> None:
    _check(lib().moe_ipc_free(ptr))


class _DeviceArray:
    """A contiguous device array described to torch by its address
    (__cuda_array_interface__); torch.as_tensor then wraps it without copying."""

    def __init__(self, ptr: int, shape, typestr: str):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr,
                                         "data": (int(ptr), False), "version": 2, "strides": None}


_TYPESTR = {torch.bfloat16: ("<i2", torch.int16), torch.float32: ("<f4", torch.float32),
            torch.int32: ("<i4", torch.int32), torch.int64: ("<i8", torch.int64)}


def tensor_at(ptr: int, shape, dtype, device) -> torch.Tensor:
    """A tensor over device memory this library allocated (it does not own the memory:
    keep the buffer alive while the tensor is used)."""
    typestr, base = _TYPESTR[dtype]
    t = torch.as_tensor(_DeviceArray(ptr, shape, typestr), device=device)
    return t.view(dtype) if base != dtype else t


def scatter_rows_peer(src, src_index, dst_rank, dst_row, dst_bases, dst_rows: int, bad=None,
                      stream=None) -> None:
    """Row dst_row[i] of buffer dst_bases[dst_rank[i]] = src[src_index[i]] for every i.
    src: 2-D CUDA tensor (rows a multiple of 16 bytes); src_index, dst_row int64 and
    dst_rank int32 CUDA tensors of one length; dst_bases: int64 CUDA tensor of device
    addresses (this GPU's buffers or ipc_open mappings), each buffer dst_rows rows of
    src's row size. Out-of-range rows are skipped and counted into `bad` (int32 CUDA
    tensor of one element) when given."""
    if src.dim() != 2:
        raise ValueError("src must be 2-D")
    n = src_index.numel()
    if dst_rank.numel() != n or dst_row.numel() != n:
        raise ValueError("src_index, dst_rank and dst_row must have the same length")
    if n == 0:
        return
    _check(lib().moe_scatter_rows_peer(
        _dev(src, "src") if src.shape[0] else None, src.shape[0],
        _dev(src_index, "src_index", torch.int64), _dev(dst_rank, "dst_rank", torch.int32),
        _dev(dst_row, "dst_row", torch.int64), n, _dev(dst_bases, "dst_bases", torch.int64),
        dst_bases.numel(), int(dst_rows), src.shape[1] * src.element_size(),
        _dev(bad, "bad", torch.int32, True), _stream(stream)))


def combine_peer(y_bases, y_rows: int, slot_rank, slot_row, topk_w, hidden: int, residual=None,
                 bad=None, stream=None):
    """out [T, hidden] bf16 = residual + sum_j topk_w[:, j] * (row slot_row[t k + j] of
    the fp32 buffer y_bases[slot_rank[t k + j]]), moe_combine's arithmetic. y_bases:
    int64 CUDA tensor of device addresses, each buffer y_rows x hidden fp32; slot_rank
    int32 and slot_row int64 CUDA tensors [T, k]; topk_w fp32 [T, k]."""
    t, k = topk_w.shape
    _sized("slot_rank", slot_rank, t * k)
    _sized("slot_row", slot_row, t * k)
    _sized("residual", residual, t * hidden)
    out = torch.empty((t, hidden), dtype=torch.bfloat16, device=topk_w.device)
    if t == 0:
        return out
    _check(lib().moe_combine_peer(
        _dev(y_bases, "y_bases", torch.int64), y_bases.numel(), int(y_rows),
        _dev(slot_rank, "slot_rank", torch.int32), _dev(slot_row, "slot_row", torch.int64),
        _dev(topk_w, "topk_w", torch.float32), _dev(residual, "residual", torch.bfloat16, True),
        _dev(out, "out"), t, k, hidden, _dev(bad, "bad", torch.int32, True), _stream(stream)))
    return out


# ---- general routing, router losses and their gradients ----

_SCORING = {"softmax": 0, "sigmoid": 1}


class Routing(NamedTuple):
    """A routing rule (include/moe.h): k experts per token by softmax or sigmoid scores;
    with num_groups > 1 only the topk_groups groups whose group_top best experts sum
    highest are open; the weights are renormalised to sum to 1 (or not), times scale."""
    k: int
    scoring: str = "softmax"
    num_groups: int = 1
    topk_groups: int = 1
    group_top: int = 1
    renormalize: bool = True
    scale: float = 1.0


class RouterLosses(NamedTuple):
    """losses [2] fp32 (load balancing, z-loss); counts [E + 1] int32 (slots per expert,
    then the tokens that count); prob_mean [E] fp32 (mean probability per expert)."""
    losses: torch.Tensor
    counts: torch.Tensor
    prob_mean: torch.Tensor


def _on(device: torch.device, stream, call):
    """call(raw stream) with the tensors' device and the stream current, so that the outputs and
    scratch it allocates belong to the stream that its kernels run on."""
    if stream is None:
        if device.index == torch.cuda.current_device():
            # the raw handle alone: building a Stream object costs 3 us a call
            return call(torch._C._cuda_getCurrentRawStream(device.index))
        with torch.cuda.device(device):
            return call(torch._C._cuda_getCurrentRawStream(device.index))
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _arg(t, name: str, dtypes, shape, device=None) -> int:
    """The address of a contiguous CUDA tensor of one of `dtypes`, of exactly `shape`, on
    `device` (None: any)."""
    if (t.is_cuda and t.shape == shape and t.dtype in dtypes and t.is_contiguous()
            and (device is None or t.device == device)):
        return t.data_ptr()
    return _rows(t, name, dtypes, shape, device, contiguous=True)


def _rows(t, name: str, dtypes, shape, device=None, contiguous: bool = False) -> int:
    """As _arg for a tensor whose rows are contiguous and may be strided (its row stride is
    a matter for the caller); names what is wrong."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its rows")
    return t.data_ptr()


_F32, _I32, _BF16 = (torch.float32,), (torch.int32,), (torch.bfloat16,)
_LOGITS = (torch.float32, torch.bfloat16)


@lru_cache(maxsize=256)
def _routing_struct(routing: Routing, t: int, stride: int, e: int, bf16: bool) -> _RoutingArgs:
    if routing.scoring not in _SCORING:
        raise ValueError(f"scoring must be 'softmax' or 'sigmoid', got {routing.scoring!r}")
    return _RoutingArgs(t, stride, e, routing.k, _SCORING[routing.scoring], routing.num_groups,
                        routing.topk_groups, routing.group_top, int(routing.renormalize), int(bf16),
                        routing.scale)


def _routing_args(logits, routing: Routing) -> _RoutingArgs:
    if logits.dim() != 2:
        raise ValueError(f"logits must be [tokens, experts], got {tuple(logits.shape)}")
    t, e = logits.shape
    if logits.dtype not in _LOGITS:
        raise ValueError(f"logits must be torch.float32 or torch.bfloat16, got {logits.dtype}")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    if e > 1 and logits.stride(1) != 1:
        raise ValueError("logits must be contiguous along the experts")
    return _routing_struct(routing, t, logits.stride(0) if t > 1 else e, e, logits.dtype is torch.bfloat16)


def route(logits, routing: Routing, bias=None, stream=None):
    """(topk_idx [T, k] int32, topk_w [T, k] fp32) of router logits [T, E] (fp32 or bf16,
    rows may be strided) under `routing`; bias [E] fp32 is added to the scores for the
    selection only (see moe_route)."""
    args = _routing_args(logits, routing)
    t, e = logits.shape
    dev = logits.device
    b = None if bias is None else _arg(bias, "bias", _F32, (e,), dev)

    def call(st):
        idx = torch.empty(t, routing.k, dtype=torch.int32, device=dev)
        w = torch.empty(t, routing.k, dtype=torch.float32, device=dev)
        _check(lib().moe_route(args, logits.data_ptr(), b, idx.data_ptr(), w.data_ptr(), st))
        return idx, w

    return _on(dev, stream, call)


def forward_routing(x, w_router, w1, w3, w2, routing: Routing, bias=None, residual=None,
                    logit_bias=None, ws=None, out=None, stream=None, weight_layout: int = ROW_MAJOR,
                    router_bf16_logits: bool = False):
    """forward with `routing` (and its selection bias [E] fp32) in place of Mixtral's rule;
    returns out [T,H] bf16."""
    t, h = x.shape
    e, i, _ = w1.shape
    shape = make_shape(t, h, i, e, routing.k, weight_layout, router_bf16_logits)
    args = _routing_struct(routing, t, e, e, False)
    _layer_sizes(t, h, e, i, w_router, logit_bias, residual, out, bias=(bias, e),
                 **_bf16_weights(e, i, h, w1, w3, w2))
    xp = _dev(x, "x", torch.bfloat16)

    def call(st):
        work = make_workspace(shape, x.device) if ws is None else ws
        dst = torch.empty(t, h, dtype=torch.bfloat16, device=x.device) if out is None else out
        _check(lib().moe_forward_routing(
            shape, args, xp, _dev(w_router, "w_router", torch.bfloat16),
            _dev(logit_bias, "logit_bias", torch.float32, True), _dev(bias, "bias", torch.float32, True),
            _dev(w1, "w1", torch.bfloat16), _dev(w3, "w3", torch.bfloat16),
            _dev(w2, "w2", torch.bfloat16), _dev(residual, "residual", torch.bfloat16, True),
            _dev(dst, "out", torch.bfloat16), _dev(work, "ws"), work.numel(), st))
        return dst

    return _on(x.device, stream, call)


def _token_mask(mask, t: int, dev) -> Optional[int]:
    return None if mask is None else _arg(mask, "token_mask", (torch.bool, torch.uint8), (t,), dev)


def router_losses(logits, topk_idx, routing: Routing, token_mask=None, stream=None) -> RouterLosses:
    """Load-balancing loss and z-loss over the tokens whose token_mask (bool or uint8 [T];
    None: all) is true (see moe_router_losses). topk_idx [T, k] int32 as routed. A tuple
    (losses [2], counts [E + 1], prob_mean [E])."""
    args = _routing_args(logits, routing)
    t, e = logits.shape
    dev = logits.device
    idx = _arg(topk_idx, "topk_idx", _I32, (t, routing.k), dev)
    mask = _token_mask(token_mask, t, dev)

    def call(st):
        n = lib().moe_router_losses_workspace(args)    # 0: few tokens need none
        ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        losses = torch.empty(2, dtype=torch.float32, device=dev)
        counts = torch.empty(e + 1, dtype=torch.int32, device=dev)
        prob = torch.empty(e, dtype=torch.float32, device=dev)
        _check(lib().moe_router_losses(args, logits.data_ptr(), idx, mask, losses.data_ptr(),
                                       counts.data_ptr(), prob.data_ptr(),
                                       None if ws is None else ws.data_ptr(), n, st))
        return RouterLosses(losses, counts, prob)

    return _on(dev, stream, call)


def route_backward(logits, topk_idx, routing: Routing, d_topk_w=None, counts=None, d_losses=None,
                   token_mask=None, stream=None):
    """Gradient in the logits [T, E] (their type) of sum(d_topk_w * topk_w) plus
    sum(d_losses * losses), the selection held fixed: d_topk_w [T, k] fp32 or None; counts
    as router_losses returned them, with d_losses [2] fp32, or both None (see
    moe_route_backward)."""
    args = _routing_args(logits, routing)
    t, e = logits.shape
    dev = logits.device
    idx = _arg(topk_idx, "topk_idx", _I32, (t, routing.k), dev)
    dw = None if d_topk_w is None else _arg(d_topk_w, "d_topk_w", _F32, (t, routing.k), dev)
    c = None if counts is None else _arg(counts, "counts", _I32, (e + 1,), dev)
    dl = None if d_losses is None else _arg(d_losses, "d_losses", _F32, (2,), dev)
    mask = _token_mask(token_mask, t, dev)

    def call(st):
        out = torch.empty(t, e, dtype=logits.dtype, device=dev)
        _check(lib().moe_route_backward(args, logits.data_ptr(), idx, dw, c, dl, mask,
                                        out.data_ptr(), st))
        return out

    return _on(dev, stream, call)


def combine_backward(d_out, y_perm, row_of, topk_w, counts=None, offsets=None, need_dy: bool = True,
                     need_dw: bool = True, stream=None):
    """(dy_perm, d_topk_w): gradient of combine for d_out [T, H] bf16 (see
    moe_combine_backward). dy_perm is fp32 like y_perm [rows, H], zero in the rows no slot
    names; counts [E] and offsets [E + 1] are permute's. need_dy=False or need_dw=False
    leaves that one out (None); counts and offsets are needed for dy_perm only."""
    if d_out.dim() != 2 or row_of.dim() != 2 or y_perm.dim() != 2:
        raise ValueError("d_out, y_perm and row_of must be 2-D")
    t, h = d_out.shape
    k, rows = row_of.shape[1], y_perm.shape[0]
    dev = d_out.device
    d = _arg(d_out, "d_out", (torch.bfloat16,), (t, h))
    y = _arg(y_perm, "y_perm", _F32, (rows, h), dev)
    r = _arg(row_of, "row_of", _I32, (t, k), dev)
    w = _arg(topk_w, "topk_w", _F32, (t, k), dev)
    e, c, o = 1, None, None
    if need_dy:
        if counts is None or offsets is None:
            raise ValueError("counts and offsets are required for dy_perm")
        e = counts.numel()
        c = _arg(counts, "counts", _I32, (e,), dev)
        o = _arg(offsets, "offsets", _I32, (e + 1,), dev)

    def call(st):
        dy = torch.empty(rows, h, dtype=torch.float32, device=dev) if need_dy else None
        dw = torch.empty(t, k, dtype=torch.float32, device=dev) if need_dw else None
        _check(lib().moe_combine_backward(d, y, r, w, c, o, dy.data_ptr() if need_dy else None,
                                          dw.data_ptr() if need_dw else None, t, k, h, e, rows, st))
        return dy, dw

    return _on(dev, stream, call)


# ---- low-rank adapters of many requests beside a shared projection ----

def lora_add(base, x, a, b, adapter, scale=None, out=None, stream=None):
    """base + scale[g] * (x a[g]^T) b[g]^T per row, g = adapter[row] (int32; a value outside
    [0, G) is a row without an adapter): base [R, N] bf16 or fp32, x [R, H] bf16, a [G, rank, H]
    and b [G, N, rank] bf16, scale [G] fp32 or None. Rows of base, x and out may be strided.
    Writes `out` when given (base itself: in place), else a new tensor (see moe_lora_add)."""
    if x.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("x must be [rows, in], a [adapters, rank, in], b [adapters, out, rank]")
    r, h = x.shape
    ad, rank, _ = a.shape
    n = b.shape[1]
    dev = x.device
    xp = _rows(x, "x", _BF16, (r, h))
    ap = _arg(a, "a", _BF16, (ad, rank, h), dev)
    bp = _arg(b, "b", _BF16, (ad, n, rank), dev)
    ip = _arg(adapter, "adapter", _I32, (r,), dev)
    sp = None if scale is None else _arg(scale, "scale", _F32, (ad,), dev)
    base_p = _rows(base, "base", _LOGITS, (r, n), dev)

    def call(st):
        dst = torch.empty(r, n, dtype=base.dtype, device=dev) if out is None else out
        out_p = dst.data_ptr() if out is None else _rows(out, "out", (base.dtype,), (r, n), dev)
        # one row has no stride to speak of
        args = _LoraArgs(r, x.stride(0) if r > 1 else h, base.stride(0) if r > 1 else n,
                         dst.stride(0) if r > 1 else n, h, n, rank, ad, int(base.dtype == torch.float32))
        size = lib().moe_lora_workspace(args)      # 0: few rows need none
        ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        _check(lib().moe_lora_add(args, base_p, xp, ap, bp, ip, sp, out_p,
                                  None if ws is None else ws.data_ptr(), size, st))
        return dst

    return _on(dev, stream, call)


@dataclass
class LoraExperts:
    """Low-rank adapters of every request beside every expert's projections: a1, a3
    [L, E, rank, H], b1, b3 [L, E, I, rank] (gate and up), a2 [L, E, rank, I], b2
    [L, E, H, rank] (down), bf16, L adapters; scale [L] fp32 or None. A pair may be None: that
    projection has no adapters. Ranks may differ between the pairs."""
    a1: Optional[torch.Tensor] = None
    b1: Optional[torch.Tensor] = None
    a3: Optional[torch.Tensor] = None
    b3: Optional[torch.Tensor] = None
    a2: Optional[torch.Tensor] = None
    b2: Optional[torch.Tensor] = None
    scale: Optional[torch.Tensor] = None


def lora_rows(token_of_row, offsets, adapter, num_adapters: int, stream=None):
    """Adapter of every routed row (see moe_lora_rows): adapter[token] * E + expert, or -1.
    token_of_row and offsets are permute's; adapter [T] int32 per token."""
    if token_of_row.dim() != 1 or offsets.dim() != 1 or adapter.dim() != 1:
        raise ValueError("token_of_row, offsets and adapter must be 1-D")
    rows, e, dev = token_of_row.numel(), offsets.numel() - 1, token_of_row.device
    tp = _arg(token_of_row, "token_of_row", _I32, (rows,))
    op = _arg(offsets, "offsets", _I32, (e + 1,), dev)
    ap = _arg(adapter, "adapter", _I32, (adapter.numel(),), dev)

    def call(st):
        ids = torch.empty(rows, dtype=torch.int32, device=dev)
        _check(lib().moe_lora_rows(tp, op, ap, adapter.numel(), rows, e, num_adapters, ids.data_ptr(), st))
        return ids

    return _on(dev, stream, call)


def swiglu_rows(gate, up, offsets, h=None, stream=None):
    """h [R, I] bf16 = bf16(silu(gate) * up) of fp32 gate and up [R, I], for the rows below
    offsets[E] (the others of `h` are untouched)."""
    if gate.dim() != 2:
        raise ValueError("gate must be [rows, intermediate]")
    rows, i = gate.shape
    dev = gate.device
    gp, up_p = _arg(gate, "gate", _F32, (rows, i)), _arg(up, "up", _F32, (rows, i), dev)
    op = _arg(offsets, "offsets", _I32, (offsets.numel(),), dev)
    hp = None if h is None else _arg(h, "h", _BF16, (rows, i), dev)

    def call(st):
        dst = torch.empty(rows, i, dtype=torch.bfloat16, device=dev) if h is None else h
        _check(lib().moe_swiglu_rows(gp, up_p, op, offsets.numel() - 1, rows, i,
                                     dst.data_ptr() if hp is None else hp, st))
        return dst

    return _on(dev, stream, call)


def forward_lora(x, w_router, w1, w3, w2, k: int, adapters: LoraExperts, adapter, residual=None,
                 logit_bias=None, stream=None, weight_layout: int = ROW_MAJOR,
                 router_bf16_logits: bool = False, routing: Optional[Routing] = None, bias=None):
    """The whole layer with adapter[t] (int32 [T], outside [0, L): none) beside every expert
    projection of token t:
        gate = w1 x + s B1 A1 x,  up = w3 x + s B3 A3 x,  h = bf16(silu(gate) * up),
        y = w2 h + s B2 A2 h      (fp32 but h)
    `routing` (with its selection bias) replaces Mixtral's rule when given (its k is used).
    Returns out [T,H] bf16. The gate and up projections run as plain grouped GEMMs into
    fp32, since the adapters come between them and the activation."""
    t, h = x.shape
    e, i, _ = w1.shape
    if routing is not None:
        k = routing.k
    _layer_sizes(t, h, e, i, w_router, logit_bias, residual, None, adapter=(adapter, t), bias=(bias, e),
                 **_bf16_weights(e, i, h, w1, w3, w2))
    pairs, count = {}, 0
    for name, a, b, n_in, n_out in (("1", adapters.a1, adapters.b1, h, i),
                                    ("3", adapters.a3, adapters.b3, h, i),
                                    ("2", adapters.a2, adapters.b2, i, h)):
        if (a is None) != (b is None):
            raise ValueError(f"a{name} and b{name} go together")
        if a is None:
            continue
        if a.dim() != 4 or a.shape[1] != e or a.shape[3] != n_in:
            raise ValueError(f"a{name} must be [L, {e}, rank, {n_in}], got {tuple(a.shape)}")
        count = count or a.shape[0]
        if a.shape[0] != count or tuple(b.shape) != (count, e, n_out, a.shape[2]):
            raise ValueError(f"b{name} must be [{count}, {e}, {n_out}, {a.shape[2]}], got {tuple(b.shape)}")
        pairs[name] = (a, b)
    if not pairs:
        raise ValueError("adapters holds no pair")
    _sized("scale", adapters.scale, count)

    def call(st):
        wide = make_shape(t, i, h, e, k, weight_layout)   # the gate and up GEMMs: H in, I out
        shape = make_shape(t, h, i, e, k, weight_layout)
        ws = make_workspace(shape if workspace_size(shape) >= workspace_size(wide) else wide, x.device)
        rows = max_padded_rows(shape)
        if routing is None:
            idx, w = router_topk(x, w_router, k, logit_bias, router_bf16_logits=router_bf16_logits)
        else:
            logits = router_topk(x, w_router, 1, logit_bias, True, router_bf16_logits=router_bf16_logits)[2]
            idx, w = route(logits, routing, bias)
        perm = permute(idx, x, e, i, ws)
        ids = lora_rows(perm["token_of_row"], perm["offsets"], adapter, count)
        scale = None if adapters.scale is None else adapters.scale.repeat_interleave(e)

        def project(rows_in, weights, n_out, name):
            y = torch.empty(rows, n_out, dtype=torch.float32, device=x.device)
            expert_down(rows_in, perm["offsets"], weights, t, k, ws, y=y, weight_layout=weight_layout)
            if name in pairs:
                # where adapters and experts cannot be merged (a shard's experts) this copies: on the call's stream
                a, b = (p.reshape(count * e, *p.shape[2:]) for p in pairs[name])
                lora_add(y, rows_in[:rows], a, b, ids, scale, out=y)
            return y

        gate, up = project(perm["x_perm"], w1, i, "1"), project(perm["x_perm"], w3, i, "3")
        act = swiglu_rows(gate, up, perm["offsets"])
        y = project(act, w2, h, "2")
        return combine(y, perm["row_of"], w, residual, e, i)

    return _on(x.device, stream, call)

"""Routed-expert MoE layer on MI355X -- Python binding of libmoe_gfx950.so.

Thin ctypes marshalling over the C ABI in ``include/moe.h``: the functions
here have the C names without the ``moe_`` prefix, take torch tensors (or raw
device addresses) and a HIP stream, and raise ``MoeError`` on a negative
status.  Every step of the layer runs in the library's HIP kernels; this
module computes nothing.  Importing it does not need a GPU; calling the
compute entry points does.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libmoe_gfx950.so")

OK, EINVAL, EUNSUPPORTED, EWORKSPACE, EHIP = 0, -1, -2, -3, -4
ACT_SITU, ACT_SWIGLU = 0, 1
OUT_BF16, OUT_F32, OUT_BOTH = 0, 1, 2
PATH_AUTO, PATH_GEMV, PATH_MFMA = 0, 1, 2
OUT_HALF = OUT_BF16  # moe_linear: the 16-bit output, in the descriptor's type
BF16, F16, F32, MXFP4 = 0, 1, 2, 3
MX_FLOOR, MX_FIT = 0, 1
SCORE_SIGMOID, SCORE_SOFTMAX = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
(LINEAR_NONE, LINEAR_RELU, LINEAR_SILU, LINEAR_GELU, LINEAR_GELU_TANH, LINEAR_SITU_GLU,
 LINEAR_SWIGLU) = range(7)
(LINEAR_ROWS16X8, LINEAR_ROWS16X16, LINEAR_ROWS16X32, LINEAR_TILE64X32, LINEAR_TILE64X64, LINEAR_TILE128X64,
 LINEAR_TILE128X128, LINEAR_ANY64X32, LINEAR_ANY64X64, LINEAR_ANY128X128, LINEAR_TILE256X256,
 LINEAR_TILE256X128) = range(12)

EXPORTS = ("moe_workspace_bytes", "moe_path_for", "moe_route", "moe_expert_forward",
           "moe_layer", "moe_layer_noalloc", "moe_layer_timed", "moe_set_one_token_router_wait",
           "moe_latent_workspace_bytes", "moe_latent_path_for", "moe_latent_layer",
           "moe_latent_layer_timed", "moe_gate", "moe_route_gated", "moe_linear_workspace_bytes",
           "moe_linear_path_for", "moe_linear", "moe_mx_quantize", "moe_mx_dequantize",
           "moe_mx_linear_workspace_bytes", "moe_mx_linear_path_for", "moe_mx_linear", "moe_group_workspace_bytes",
           "moe_group", "moe_grouped_path_for", "moe_grouped_linear", "moe_combine", "moe_status_str")
TIMED_EVENTS = 6
NOALLOC_WS_BYTES = 128 << 20  # MOE_NOALLOC_WS_BYTES: the static workspace of moe_layer_noalloc


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_str(status)} ({status})")
        self.status = status


class LayerDesc(ctypes.Structure):
    """Mirror of moe_layer_desc."""
    _fields_ = [
        ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("d_model", ctypes.c_int32),
        ("d_ffn", ctypes.c_int32), ("n_shared", ctypes.c_int32),
        ("renorm", ctypes.c_int32), ("routed_scale", ctypes.c_float),
        ("act", ctypes.c_int32), ("situ_b1", ctypes.c_float), ("situ_b2", ctypes.c_float),
        ("path", ctypes.c_int32),
        ("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
        ("w1_q", ctypes.c_void_p), ("w1_s", ctypes.c_void_p),
        ("w3_q", ctypes.c_void_p), ("w3_s", ctypes.c_void_p),
        ("w2_q", ctypes.c_void_p), ("w2_s", ctypes.c_void_p),
        ("sh_w1", ctypes.c_void_p), ("sh_w3", ctypes.c_void_p), ("sh_w2", ctypes.c_void_p),
    ]


class LatentDesc(ctypes.Structure):
    """Mirror of moe_latent_desc."""
    _fields_ = [
        ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("hidden", ctypes.c_int32),
        ("latent", ctypes.c_int32), ("d_ffn", ctypes.c_int32), ("n_shared", ctypes.c_int32),
        ("renorm", ctypes.c_int32), ("routed_scale", ctypes.c_float),
        ("act", ctypes.c_int32), ("situ_b1", ctypes.c_float), ("situ_b2", ctypes.c_float),
        ("latent_norm", ctypes.c_int32), ("rms_eps", ctypes.c_float),
        ("path", ctypes.c_int32),
        ("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
        ("down", ctypes.c_void_p),
        ("w1_q", ctypes.c_void_p), ("w1_s", ctypes.c_void_p),
        ("w3_q", ctypes.c_void_p), ("w3_s", ctypes.c_void_p),
        ("w2_q", ctypes.c_void_p), ("w2_s", ctypes.c_void_p),
        ("norm_w", ctypes.c_void_p), ("up", ctypes.c_void_p),
        ("sh_w1", ctypes.c_void_p), ("sh_w3", ctypes.c_void_p), ("sh_w2", ctypes.c_void_p),
    ]


class GateDesc(ctypes.Structure):
    """Mirror of moe_gate_desc."""
    _fields_ = [
        ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("score", ctypes.c_int32),
        ("n_groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
        ("group_score", ctypes.c_int32), ("renorm", ctypes.c_int32),
        ("routed_scale", ctypes.c_float), ("bias", ctypes.c_void_p),
    ]
    device = None  # of the tensors that make_gate_desc was given


class LinearDesc(ctypes.Structure):
    """Mirror of moe_linear_desc."""
    _fields_ = [
        ("n_in", ctypes.c_int32), ("n_out", ctypes.c_int32), ("type", ctypes.c_int32),
        ("act", ctypes.c_int32), ("situ_b1", ctypes.c_float), ("situ_b2", ctypes.c_float),
        ("bias_type", ctypes.c_int32), ("residual_type", ctypes.c_int32), ("ldw", ctypes.c_int64),
        ("w", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
        ("bias", ctypes.c_void_p), ("bias_up", ctypes.c_void_p),
    ]
    device = None  # of the tensors that make_linear_desc was given


class MxLinearDesc(ctypes.Structure):
    """Mirror of moe_mx_linear_desc."""
    _fields_ = [
        ("n_in", ctypes.c_int32), ("n_out", ctypes.c_int32), ("type", ctypes.c_int32),
        ("act", ctypes.c_int32), ("situ_b1", ctypes.c_float), ("situ_b2", ctypes.c_float),
        ("bias_type", ctypes.c_int32), ("residual_type", ctypes.c_int32),
        ("ldw", ctypes.c_int64), ("ldw_s", ctypes.c_int64),
        ("w", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_s", ctypes.c_void_p), ("w_up_s", ctypes.c_void_p),
        ("bias", ctypes.c_void_p), ("bias_up", ctypes.c_void_p),
    ]
    device = None  # of the tensors that make_mx_linear_desc was given


class GroupedDesc(ctypes.Structure):
    """Mirror of moe_grouped_desc."""
    _fields_ = [
        ("n_groups", ctypes.c_int32), ("n_in", ctypes.c_int32), ("n_out", ctypes.c_int32), ("type", ctypes.c_int32),
        ("operands", ctypes.c_int32), ("act", ctypes.c_int32), ("situ_b1", ctypes.c_float), ("situ_b2", ctypes.c_float),
        ("bias_type", ctypes.c_int32), ("ldw", ctypes.c_int64), ("group_w", ctypes.c_int64), ("ldw_s", ctypes.c_int64),
        ("group_w_s", ctypes.c_int64), ("w", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_s", ctypes.c_void_p),
        ("w_up_s", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("bias_up", ctypes.c_void_p),
    ]
    device = None  # of the tensors that make_grouped_desc was given


_lib = None


def lib() -> ctypes.CDLL:
    """Load the built HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m "
                               "quantized_expert_gemv_sigmoid_amd.build` (or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        P = ctypes.POINTER(LayerDesc)
        L.moe_workspace_bytes.restype = sz
        L.moe_workspace_bytes.argtypes = [P, i32]
        L.moe_path_for.restype = i32
        L.moe_path_for.argtypes = [P, i32]
        L.moe_route.restype = i32
        L.moe_route.argtypes = [P, vp, i32, vp, vp, vp, vp, sz, vp]
        L.moe_expert_forward.restype = i32
        L.moe_expert_forward.argtypes = [P, vp, i32, vp, vp, i32, vp, vp, i32, vp, sz, vp]
        L.moe_layer.restype = i32
        L.moe_layer.argtypes = [P, vp, i32, vp, vp, i32, vp, vp, vp, vp, sz, vp]
        L.moe_layer_noalloc.restype = i32
        L.moe_layer_noalloc.argtypes = [P, vp, i32, vp, vp, i32, vp, vp, vp, vp]
        L.moe_layer_timed.restype = i32
        L.moe_layer_timed.argtypes = [P, vp, i32, vp, vp, i32, vp, sz, vp, ctypes.POINTER(vp)]
        PL = ctypes.POINTER(LatentDesc)
        L.moe_latent_workspace_bytes.restype = sz
        L.moe_latent_workspace_bytes.argtypes = [PL, i32]
        L.moe_latent_path_for.restype = i32
        L.moe_latent_path_for.argtypes = [PL, i32]
        L.moe_latent_layer.restype = i32
        L.moe_latent_layer.argtypes = [PL, vp, i32, vp, vp, i32, vp, vp, vp, vp, sz, vp]
        L.moe_latent_layer_timed.restype = i32
        L.moe_latent_layer_timed.argtypes = [PL, vp, i32, vp, vp, i32, vp, sz, vp, ctypes.POINTER(vp)]
        L.moe_set_one_token_router_wait.restype = i32
        L.moe_set_one_token_router_wait.argtypes = [i32]
        i64 = ctypes.c_int64
        L.moe_gate.restype = i32
        L.moe_gate.argtypes = [ctypes.POINTER(GateDesc), vp, i32, i64, i32, vp, vp, vp, vp]
        L.moe_route_gated.restype = i32
        L.moe_route_gated.argtypes = [P, ctypes.POINTER(GateDesc), vp, i32, vp, vp, vp, vp, sz, vp]
        L.moe_linear_workspace_bytes.restype = sz
        L.moe_linear_workspace_bytes.argtypes = [ctypes.POINTER(LinearDesc), i32]
        L.moe_linear_path_for.restype = i32
        L.moe_linear_path_for.argtypes = [ctypes.POINTER(LinearDesc), vp, i64, i32]
        L.moe_linear.restype = i32
        L.moe_linear.argtypes = [ctypes.POINTER(LinearDesc), vp, i64, i32, vp, i64, vp, vp, i64, i32,
                                 vp, sz, vp]
        L.moe_mx_quantize.restype = i32
        L.moe_mx_quantize.argtypes = [vp, i32, i64, i32, i32, i32, vp, i64, vp, i64, vp]
        L.moe_mx_dequantize.restype = i32
        L.moe_mx_dequantize.argtypes = [vp, i64, vp, i64, i32, i32, vp, i32, i64, vp]
        PM, PG = ctypes.POINTER(MxLinearDesc), ctypes.POINTER(GroupedDesc)
        L.moe_mx_linear_workspace_bytes.restype = sz
        L.moe_mx_linear_workspace_bytes.argtypes = [PM, i32]
        L.moe_mx_linear_path_for.restype = i32
        L.moe_mx_linear_path_for.argtypes = [PM, i32]
        L.moe_mx_linear.restype = i32
        L.moe_mx_linear.argtypes = [PM, vp, i64, vp, i64, i32, vp, i64, vp, vp, i64, i32, vp, sz, vp]
        L.moe_group_workspace_bytes.restype = sz
        L.moe_group_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_group.restype = i32
        L.moe_group.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]
        L.moe_grouped_path_for.restype = i32
        L.moe_grouped_path_for.argtypes = [PG, vp, i64, i32]
        L.moe_grouped_linear.restype = i32
        L.moe_grouped_linear.argtypes = [PG, vp, i64, vp, i64, i32, vp, vp, i32, vp, vp, i64, i32, vp]
        L.moe_combine.restype = i32
        L.moe_combine.argtypes = [vp, i32, i64, i32, vp, vp, i32, i32, i32, vp, i32, i64, vp, i32, i64, vp]
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_status_str.argtypes = [i32]
        _lib = L
    return _lib


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


def _ws(ws):
    """Workspace as (device address, bytes): a torch tensor or an (addr, bytes) pair."""
    if ws is None:
        return None, 0
    if isinstance(ws, tuple):
        return int(ws[0]), int(ws[1])
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _check(status: int, what: str) -> None:
    if status != OK:
        raise MoeError(status, what)


def status_str(status: int) -> str:
    return lib().moe_status_str(status).decode()


def workspace_bytes(desc: LayerDesc, max_tokens: int) -> int:
    """Bytes of workspace a call with up to max_tokens tokens needs (its
    contents need no initialisation)."""
    return int(lib().moe_workspace_bytes(ctypes.byref(desc), max_tokens))


def workspace(desc: LayerDesc, max_tokens: int, device="cuda"):
    """An uninitialised workspace (uint8 tensor) for calls of up to max_tokens tokens."""
    import torch
    n = workspace_bytes(desc, max_tokens)
    if n == 0:
        raise MoeError(EINVAL, "moe_workspace_bytes: invalid or unsupported descriptor")
    return torch.empty(n, dtype=torch.uint8, device=device)


def set_one_token_router_wait(microseconds: int) -> None:
    _check(lib().moe_set_one_token_router_wait(int(microseconds)), "moe_set_one_token_router_wait")


def path_for(desc: LayerDesc, T: int) -> int:
    r = int(lib().moe_path_for(ctypes.byref(desc), T))
    if r < 0:
        raise MoeError(r, "moe_path_for")
    return r


def route(desc: LayerDesc, x, T: int, ids, weights, counts, ws, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_route(ctypes.byref(desc), _ptr(x), T, _ptr(ids), _ptr(weights), _ptr(counts),
                           wp, wn, _stream(stream)), "moe_route")


def expert_forward(desc: LayerDesc, x, T: int, ids, weights, include_shared: int, out_bf16,
                   out_f32, out_mode: int, ws, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_expert_forward(ctypes.byref(desc), _ptr(x), T, _ptr(ids), _ptr(weights),
                                    include_shared, _ptr(out_bf16), _ptr(out_f32), out_mode,
                                    wp, wn, _stream(stream)), "moe_expert_forward")


def layer(desc: LayerDesc, x, T: int, out_bf16, out_f32, out_mode: int, ws, ids=None,
          weights=None, counts=None, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_layer(ctypes.byref(desc), _ptr(x), T, _ptr(out_bf16), _ptr(out_f32),
                           out_mode, _ptr(ids), _ptr(weights), _ptr(counts), wp, wn,
                           _stream(stream)), "moe_layer")


def layer_noalloc(desc: LayerDesc, x, T: int, out_bf16, out_f32, out_mode: int, ids=None,
                  weights=None, counts=None, stream=None) -> None:
    """moe_layer on the library's static per-GPU workspace (no allocation)."""
    _check(lib().moe_layer_noalloc(ctypes.byref(desc), _ptr(x), T, _ptr(out_bf16), _ptr(out_f32),
                                   out_mode, _ptr(ids), _ptr(weights), _ptr(counts), _stream(stream)),
           "moe_layer_noalloc")


def _event_array(events, stream):
    assert len(events) == TIMED_EVENTS
    for e in events:
        if not e.cuda_event:  # torch creates the HIP event at its first record
            e.record(stream)
    return (ctypes.c_void_p * TIMED_EVENTS)(*[e.cuda_event for e in events])


def layer_timed(desc: LayerDesc, x, T: int, out_bf16, out_f32, out_mode: int, ws, events,
                stream=None) -> None:
    """moe_layer recording the 6 phase-boundary events (torch.cuda.Event with
    enable_timing) on the stream."""
    arr = _event_array(events, stream)
    wp, wn = _ws(ws)
    _check(lib().moe_layer_timed(ctypes.byref(desc), _ptr(x), T, _ptr(out_bf16), _ptr(out_f32),
                                 out_mode, wp, wn, _stream(stream), arr), "moe_layer_timed")


@dataclass
class DeviceLayer:
    """Device tensors of one layer and the descriptor that points at them."""
    tensors: dict
    desc: LayerDesc


def make_desc(n_experts: int, top_k: int, d_model: int, d_ffn: int, n_shared: int,
              tensors: dict, act: int = ACT_SITU, situ_b1: float = 4.0, situ_b2: float = 25.0,
              renorm: int = 1, routed_scale: float = 1.0, path: int = PATH_AUTO) -> LayerDesc:
    """Fill a descriptor from device tensors keyed router_w, router_bias,
    w1_q, w1_s, w3_q, w3_s, w2_q, w2_s, sh_w1, sh_w3, sh_w2."""
    d = LayerDesc()
    d.n_experts, d.top_k, d.d_model, d.d_ffn, d.n_shared = n_experts, top_k, d_model, d_ffn, n_shared
    d.renorm, d.routed_scale, d.act = renorm, routed_scale, act
    d.situ_b1, d.situ_b2, d.path = situ_b1, situ_b2, path
    for name in ("router_w", "router_bias", "w1_q", "w1_s", "w3_q", "w3_s", "w2_q", "w2_s",
                 "sh_w1", "sh_w3", "sh_w2"):
        setattr(d, name, _ptr(tensors.get(name)))
    return d


# ------------------------------------------------------------------ latent layer

def latent_workspace_bytes(desc: LatentDesc, max_tokens: int) -> int:
    return int(lib().moe_latent_workspace_bytes(ctypes.byref(desc), max_tokens))


def latent_workspace(desc: LatentDesc, max_tokens: int, device="cuda"):
    """An uninitialised workspace (uint8 tensor) for latent-layer calls of up to max_tokens tokens."""
    import torch
    n = latent_workspace_bytes(desc, max_tokens)
    if n == 0:
        raise MoeError(EINVAL, "moe_latent_workspace_bytes: invalid or unsupported descriptor")
    return torch.empty(n, dtype=torch.uint8, device=device)


def latent_path_for(desc: LatentDesc, T: int) -> int:
    r = int(lib().moe_latent_path_for(ctypes.byref(desc), T))
    if r < 0:
        raise MoeError(r, "moe_latent_path_for")
    return r


def latent_layer(desc: LatentDesc, x, T: int, out_bf16, out_f32, out_mode: int, ws, ids=None,
                 weights=None, counts=None, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_latent_layer(ctypes.byref(desc), _ptr(x), T, _ptr(out_bf16), _ptr(out_f32),
                                  out_mode, _ptr(ids), _ptr(weights), _ptr(counts), wp, wn,
                                  _stream(stream)), "moe_latent_layer")


def latent_layer_timed(desc: LatentDesc, x, T: int, out_bf16, out_f32, out_mode: int, ws, events,
                       stream=None) -> None:
    """moe_latent_layer recording the 6 phase-boundary events on the stream."""
    arr = _event_array(events, stream)
    wp, wn = _ws(ws)
    _check(lib().moe_latent_layer_timed(ctypes.byref(desc), _ptr(x), T, _ptr(out_bf16),
                                        _ptr(out_f32), out_mode, wp, wn, _stream(stream), arr),
           "moe_latent_layer_timed")


def make_latent_desc(n_experts: int, top_k: int, hidden: int, latent: int, d_ffn: int,
                     n_shared: int, tensors: dict, act: int = ACT_SITU, situ_b1: float = 4.0,
                     situ_b2: float = 25.0, renorm: int = 1, routed_scale: float = 1.0,
                     latent_norm: int = 1, rms_eps: float = 1e-5,
                     path: int = PATH_AUTO) -> LatentDesc:
    """Fill a latent-layer descriptor from device tensors keyed router_w,
    router_bias, down, w1_q, w1_s, w3_q, w3_s, w2_q, w2_s, norm_w, up, sh_w1,
    sh_w3, sh_w2."""
    d = LatentDesc()
    d.n_experts, d.top_k, d.hidden, d.latent = n_experts, top_k, hidden, latent
    d.d_ffn, d.n_shared = d_ffn, n_shared
    d.renorm, d.routed_scale, d.act = renorm, routed_scale, act
    d.situ_b1, d.situ_b2 = situ_b1, situ_b2
    d.latent_norm, d.rms_eps, d.path = latent_norm, rms_eps, path
    for name in ("router_w", "router_bias", "down", "w1_q", "w1_s", "w3_q", "w3_s", "w2_q",
                 "w2_s", "norm_w", "up", "sh_w1", "sh_w3", "sh_w2"):
        setattr(d, name, _ptr(tensors.get(name)))
    return d


# -------------------------------------------- routing from logits, dense product

_torch = None  # torch, and what a call looks up in it
_types = {}    # dtype -> moe_type
_raw_stream = _current = None


def _setup() -> None:
    global _torch, _raw_stream, _current
    import torch
    _types.update({torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32})
    # (the current stream's address without a Stream object around it, where torch has it)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
    # (and the current device's number, where torch has it by itself: of a tensor there, so CUDA is initialised)
    _current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch


def _type_of(t) -> int:
    """moe_type of a tensor's dtype."""
    if _torch is None:
        _setup()
    r = _types.get(t.dtype)
    if r is None:
        raise MoeError(EINVAL, f"dtype {t.dtype}")
    return r


def _rows(t, rows: int, cols: int, what: str) -> int:
    """Elements between the rows of a tensor of at least `rows` rows of `cols` contiguous values (one row has none: cols)."""
    shape = t.shape
    if len(shape) == 2 and shape[0] >= rows and shape[1] == cols and t.is_contiguous():
        return cols
    stride = t.stride()
    if len(shape) != 2 or shape[0] < rows or shape[1] != cols or (stride[1] != 1 and cols > 1):
        raise MoeError(EINVAL, f"{what}: {rows} rows of {cols} contiguous values wanted, got {tuple(shape)}, strides {tuple(stride)}")
    return stride[0] if rows > 1 else cols


def _flat(t, n: int, dtype, what: str):
    """The address of n contiguous values of that dtype, or None."""
    if t is None:
        return None
    if t.dtype != dtype or t.numel() < n or not t.is_contiguous():
        raise MoeError(EINVAL, f"{what}: {n} contiguous {dtype} values wanted, got {tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def _choices(t, T: int, k: int, dtype, what: str):
    """_flat of T rows of k choices: a table of several rows is of that width."""
    if t is not None and T > 1 and len(t.shape) == 2 and t.shape[1] != k:
        raise MoeError(EINVAL, f"{what}: {T} rows of {k} values wanted, got {tuple(t.shape)}")
    return _flat(t, T * k, dtype, what)


def _same_device(desc, first, *others) -> None:
    """The tensors of a call lie on one device, and those of the descriptor (desc.device, where known) too."""
    i = first.get_device()
    known = None if desc is None else desc.device
    if i >= 0 and (known is None or known.index == i):
        for t in others:
            if t is not None and t.get_device() != i:
                break
        else:
            return
    d = first.device
    if known is not None and known != d:
        raise MoeError(EINVAL, f"tensors on {known} and {d}")
    for t in others:
        if t is not None and t.device != d:
            raise MoeError(EINVAL, f"tensors on {d} and {t.device}")


def _ws_tensor(ws) -> tuple:
    return () if ws is None or isinstance(ws, tuple) else (ws,)


def _call(x, stream, f, *args) -> int:
    """f(*args, stream) on x's device: that device's current stream where none is given."""
    i = x.get_device()
    if i < 0:  # (not a GPU's: the arguments that were refused first aside, there is nothing to launch on)
        raise MoeError(EINVAL, f"tensors on {x.device}")
    s = _raw_stream(i) if stream is None else _stream(stream)
    if i != _current():
        with _torch.cuda.device(i):
            return f(*args, s)
    return f(*args, s)


def make_gate_desc(n_experts: int, top_k: int, score: int = SCORE_SIGMOID, bias=None,
                   n_groups: int = 1, top_groups: int = 1, group_score: int = GROUP_MAX,
                   renorm: int = 1, routed_scale: float = 1.0) -> GateDesc:
    """Fill a gate descriptor; bias: a float32 tensor of n_experts values, or None.  The
    descriptor holds its address only: keep the tensor."""
    d = GateDesc()
    d.n_experts, d.top_k, d.score = n_experts, top_k, score
    d.n_groups, d.top_groups, d.group_score = n_groups, top_groups, group_score
    d.renorm, d.routed_scale = renorm, routed_scale
    if bias is not None and _type_of(bias) != F32:
        raise MoeError(EINVAL, f"bias: {bias.dtype}")
    if bias is not None:
        d.bias, d.device = _flat(bias, n_experts, bias.dtype, "bias"), bias.device
    return d


def gate(desc: GateDesc, logits, T: int, ids, weights, counts=None, stream=None) -> None:
    """moe_gate on the first T rows of logits ([.., n_experts], float32, bfloat16 or float16;
    rows may be apart)."""
    E, n = desc.n_experts, T * desc.top_k
    ty = _type_of(logits)
    _same_device(desc, logits, ids, weights, counts)
    i32 = _torch.int32
    _check(_call(logits, stream, lib().moe_gate, desc, logits.data_ptr(), ty, _rows(logits, T, E, "logits"), T,
                 _flat(ids, n, i32, "ids"), _flat(weights, n, _torch.float32, "weights"), _flat(counts, E, i32, "counts")),
           "moe_gate")


def route_gated(desc: LayerDesc, gate_desc: GateDesc, x, T: int, ids, weights, counts, ws,
                stream=None) -> None:
    """moe_route_gated on the first T rows of x ([.., d_model], contiguous bfloat16 or their bits)."""
    if _torch is None:
        _setup()
    E, n = desc.n_experts, T * desc.top_k
    if x.dtype not in (_torch.bfloat16, _torch.int16):
        raise MoeError(EINVAL, f"x: {x.dtype}")
    _same_device(gate_desc, x, ids, weights, counts, *_ws_tensor(ws))
    wp, wn = _ws(ws)
    i32 = _torch.int32
    _check(_call(x, stream, lib().moe_route_gated, desc, gate_desc, _flat(x, T * desc.d_model, x.dtype, "x"), T,
                 _flat(ids, n, i32, "ids"), _flat(weights, n, _torch.float32, "weights"), _flat(counts, E, i32, "counts"),
                 wp, wn), "moe_route_gated")


def make_linear_desc(w, w_up=None, bias=None, bias_up=None, act: int = LINEAR_NONE,
                     situ_b1: float = 4.0, situ_b2: float = 25.0,
                     residual_type: Optional[int] = None) -> LinearDesc:
    """Fill a product's descriptor from w [n_out][n_in] (bfloat16 or float16; rows may be apart),
    w_up like it for a gated act, biases [n_out] of w's dtype or float32; residual_type: F32, or
    None for w's.  The descriptor holds addresses only: keep the tensors."""
    d = LinearDesc()
    n, k = w.shape
    d.n_in, d.n_out, d.type, d.act = k, n, _type_of(w), act
    d.situ_b1, d.situ_b2 = situ_b1, situ_b2
    if d.type == F32:
        raise MoeError(EINVAL, f"w: {w.dtype}")
    d.ldw = _rows(w, n, k, "w")
    _same_device(None, w, w_up, bias, bias_up)
    if w_up is not None and (w_up.dtype != w.dtype or _rows(w_up, n, k, "w_up") != d.ldw or w_up.shape != w.shape):
        raise MoeError(EINVAL, "w_up: not laid out as w")
    b = bias if bias is not None else bias_up
    d.bias_type = d.type if b is None else _type_of(b)
    d.residual_type = d.type if residual_type is None else residual_type
    d.w, d.w_up, d.device = w.data_ptr(), None if w_up is None else w_up.data_ptr(), w.device
    d.bias = None if bias is None else _flat(bias, n, b.dtype, "bias")
    d.bias_up = None if bias_up is None else _flat(bias_up, n, b.dtype, "bias_up")
    return d


def linear_workspace_bytes(desc: LinearDesc, max_tokens: int) -> int:
    return int(lib().moe_linear_workspace_bytes(ctypes.byref(desc), max_tokens))


def linear_workspace(desc: LinearDesc, max_tokens: int, device="cuda"):
    """An uninitialised workspace (uint8 tensor) for products of up to max_tokens tokens."""
    import torch
    n = linear_workspace_bytes(desc, max_tokens)
    if n == 0:
        raise MoeError(EINVAL, "moe_linear_workspace_bytes: invalid or unsupported descriptor")
    return torch.empty(n, dtype=torch.uint8, device=device)


def linear_path_for(desc: LinearDesc, x, T: int) -> tuple:
    """(kernel, parts of n_in) that `linear` takes for the first T rows of x: one of LINEAR_ROWS16X8 .. TILE256X256."""
    r = int(lib().moe_linear_path_for(ctypes.byref(desc), x.data_ptr(), _rows(x, T, desc.n_in, "x"), T))
    if r < 0:
        raise MoeError(r, "moe_linear_path_for")
    return r % 256, r // 256


def linear(desc: LinearDesc, x, T: int, out_half, out_f32, out_mode: int, ws, residual=None,
           stream=None) -> None:
    """moe_linear on the first T rows of x; residual: [.., n_out] of the descriptor's residual
    type (one expanded row: the same for every token).  Two outputs have the same row distance."""
    n, half = desc.n_out, desc.type
    if _type_of(x) != half:
        raise MoeError(EINVAL, f"x: {x.dtype}")
    _same_device(desc, x, out_half, out_f32, residual, *_ws_tensor(ws))
    op, fp, ldo = _outputs(out_half, out_f32, out_mode, T, n, half)
    rp, ldr = _residual(residual, T, n, desc.residual_type)
    wp, wn = _ws(ws)
    _check(_call(x, stream, lib().moe_linear, desc, x.data_ptr(), _rows(x, T, desc.n_in, "x"), T,
                 rp, ldr, op, fp, ldo, out_mode, wp, wn), "moe_linear")


# ------------------------------------- MXFP4 rows and their product, products of groups

def _bytes(t, rows: int, cols: int, what: str) -> int:
    """_rows of a uint8 tensor."""
    if _torch is None:
        _setup()
    if t.dtype != _torch.uint8:
        raise MoeError(EINVAL, f"{what}: {t.dtype}")
    return _rows(t, rows, cols, what)


def mx_quantize(x, T: int, codes, scales, rule: int = MX_FLOOR, stream=None) -> None:
    """moe_mx_quantize on the first T rows of x ([.., n], bfloat16, float16 or float32; rows may be
    apart): codes [.., 16 ceil(n / 32)] and scales [.., ceil(n / 32)], uint8."""
    if len(x.shape) != 2:
        raise MoeError(EINVAL, f"x: {tuple(x.shape)}")
    n = x.shape[1]
    b = (n + 31) // 32
    ty = _type_of(x)
    _same_device(None, x, codes, scales)
    _check(_call(x, stream, lib().moe_mx_quantize, x.data_ptr(), ty, _rows(x, T, n, "x"), T, n, rule, codes.data_ptr(),
                 _bytes(codes, T, 16 * b, "codes"), scales.data_ptr(), _bytes(scales, T, b, "scales")), "moe_mx_quantize")


def mx_dequantize(codes, scales, T: int, out, stream=None) -> None:
    """moe_mx_dequantize of the first T rows into out [.., n], bfloat16, float16 or float32."""
    if len(out.shape) != 2:
        raise MoeError(EINVAL, f"out: {tuple(out.shape)}")
    n = out.shape[1]
    b = (n + 31) // 32
    ty = _type_of(out)
    _same_device(None, out, codes, scales)
    _check(_call(out, stream, lib().moe_mx_dequantize, codes.data_ptr(), _bytes(codes, T, 16 * b, "codes"), scales.data_ptr(),
                 _bytes(scales, T, b, "scales"), T, n, out.data_ptr(), ty, _rows(out, T, n, "out")), "moe_mx_dequantize")


def _outputs(out_half, out_f32, out_mode: int, T: int, n: int, half: int) -> tuple:
    """(address of out_half, of out_f32, their row distance) as out_mode asks."""
    ldo = op = fp = None
    if out_mode != OUT_F32 and out_half is not None:
        if _type_of(out_half) != half:
            raise MoeError(EINVAL, f"out_half: {out_half.dtype}")
        ldo, op = _rows(out_half, T, n, "out_half"), out_half.data_ptr()
    if out_mode != OUT_HALF and out_f32 is not None:
        if _type_of(out_f32) != F32:
            raise MoeError(EINVAL, f"out_f32: {out_f32.dtype}")
        ld, fp = _rows(out_f32, T, n, "out_f32"), out_f32.data_ptr()
        if ldo is not None and ld != ldo:
            raise MoeError(EINVAL, "outputs with different row distances")
        ldo = ld
    return op, fp, n if ldo is None else ldo


def _residual(residual, T: int, n: int, ty: int) -> tuple:
    if residual is None:
        return None, 0
    if _type_of(residual) != ty:
        raise MoeError(EINVAL, f"residual: {residual.dtype}")
    return residual.data_ptr(), _rows(residual, T, n, "residual")


def make_mx_linear_desc(w, w_s, w_up=None, w_up_s=None, bias=None, bias_up=None, type: int = BF16, act: int = LINEAR_NONE,
                        situ_b1: float = 4.0, situ_b2: float = 25.0, residual_type: Optional[int] = None) -> MxLinearDesc:
    """Fill an MXFP4 product's descriptor from codes w [n_out][n_in / 2] and scales w_s
    [n_out][n_in / 32] (uint8; rows may be apart), w_up and w_up_s like them for a gated act, biases
    [n_out] of the 16-bit `type` or float32; residual_type: F32, or None for `type`.  The
    descriptor holds addresses only: keep the tensors."""
    d = MxLinearDesc()
    n, k = w.shape[0], w.shape[1] * 2
    d.n_in, d.n_out, d.type, d.act = k, n, type, act
    d.situ_b1, d.situ_b2 = situ_b1, situ_b2
    d.ldw, d.ldw_s = _bytes(w, n, k // 2, "w"), _bytes(w_s, n, k // 32, "w_s")
    _same_device(None, w, w_s, w_up, w_up_s, bias, bias_up)
    if (w_up is None) != (w_up_s is None):
        raise MoeError(EINVAL, "w_up and w_up_s come together")
    if w_up is not None and (_bytes(w_up, n, k // 2, "w_up") != d.ldw or _bytes(w_up_s, n, k // 32, "w_up_s") != d.ldw_s):
        raise MoeError(EINVAL, "w_up: not laid out as w")
    b = bias if bias is not None else bias_up
    d.bias_type = type if b is None else _type_of(b)
    d.residual_type = type if residual_type is None else residual_type
    d.w, d.w_s, d.device = w.data_ptr(), w_s.data_ptr(), w.device
    d.w_up, d.w_up_s = _ptr(w_up), _ptr(w_up_s)
    d.bias = None if bias is None else _flat(bias, n, b.dtype, "bias")
    d.bias_up = None if bias_up is None else _flat(bias_up, n, b.dtype, "bias_up")
    return d


def mx_linear_workspace_bytes(desc: MxLinearDesc, max_tokens: int) -> int:
    return int(lib().moe_mx_linear_workspace_bytes(ctypes.byref(desc), max_tokens))


def mx_linear_workspace(desc: MxLinearDesc, max_tokens: int, device="cuda"):
    """An uninitialised workspace (uint8 tensor) for MXFP4 products of up to max_tokens tokens."""
    import torch
    n = mx_linear_workspace_bytes(desc, max_tokens)
    if n == 0:
        raise MoeError(EINVAL, "moe_mx_linear_workspace_bytes: invalid or unsupported descriptor")
    return torch.empty(n, dtype=torch.uint8, device=device)


def mx_linear_path_for(desc: MxLinearDesc, T: int) -> tuple:
    """(kernel, parts of n_in) that `mx_linear` takes for T tokens: one of LINEAR_ROWS16X8 .. TILE256X128."""
    r = int(lib().moe_mx_linear_path_for(ctypes.byref(desc), T))
    if r < 0:
        raise MoeError(r, "moe_mx_linear_path_for")
    return r % 256, r // 256


def mx_linear(desc: MxLinearDesc, x, x_s, T: int, out_half, out_f32, out_mode: int, ws, residual=None, stream=None) -> None:
    """moe_mx_linear on the first T rows of codes x [.., n_in / 2] and scales x_s [.., n_in / 32]
    (uint8); residual: [.., n_out] of the descriptor's residual type (one expanded row: the same for
    every token).  Two outputs have the same row distance."""
    n, k = desc.n_out, desc.n_in
    ldx, ldxs = _bytes(x, T, k // 2, "x"), _bytes(x_s, T, k // 32, "x_s")
    _same_device(desc, x, x_s, out_half, out_f32, residual, *_ws_tensor(ws))
    op, fp, ldo = _outputs(out_half, out_f32, out_mode, T, n, desc.type)
    rp, ldr = _residual(residual, T, n, desc.residual_type)
    wp, wn = _ws(ws)
    _check(_call(x, stream, lib().moe_mx_linear, desc, x.data_ptr(), ldx, x_s.data_ptr(), ldxs, T, rp, ldr, op, fp, ldo,
                 out_mode, wp, wn), "moe_mx_linear")


def _matrices(t, dtype, what: str) -> tuple:
    """(elements between rows, between matrices) of a tensor [groups][n][k] of rows of contiguous values."""
    if t.dtype != dtype or len(t.shape) != 3 or (t.stride(2) != 1 and t.shape[2] > 1):
        raise MoeError(EINVAL, f"{what}: matrices of rows of contiguous {dtype} values wanted, got {tuple(t.shape)} {t.dtype}")
    return (t.stride(1) if t.shape[1] > 1 else t.shape[2]), t.stride(0) if t.shape[0] > 1 else 0


def make_grouped_desc(w, w_up=None, bias=None, bias_up=None, act: int = LINEAR_NONE, situ_b1: float = 4.0,
                      situ_b2: float = 25.0, w_s=None, w_up_s=None, type: Optional[int] = None) -> GroupedDesc:
    """Fill a descriptor of products by group from w [n_groups][n_out][n_in] (bfloat16 or float16;
    rows and matrices may be apart), w_up like it for a gated act, biases [n_groups][n_out] of w's
    dtype or float32.  MXFP4: codes w [..][n_in / 2] and scales w_s [..][n_in / 32], uint8 (w_up_s
    for w_up), and the 16-bit `type` of outputs and biases (BF16 where it is None).  The descriptor
    holds addresses only: keep the tensors."""
    d = GroupedDesc()
    if _torch is None:
        _setup()
    mx = w_s is not None
    ld, group = _matrices(w, _torch.uint8 if mx else w.dtype, "w")
    g, n, k = w.shape
    d.n_groups, d.n_out, d.n_in, d.act = g, n, 2 * k if mx else k, act
    d.situ_b1, d.situ_b2 = situ_b1, situ_b2
    d.type = (BF16 if type is None else type) if mx else _type_of(w)
    d.operands = MXFP4 if mx else d.type
    if d.type not in (BF16, F16) or (not mx and type not in (None, d.type)):
        raise MoeError(EINVAL, f"type {type} with w of {w.dtype}")
    d.ldw, d.group_w = ld, group
    _same_device(None, w, w_up, w_s, w_up_s, bias, bias_up)
    if w_up is not None and (w_up.shape != w.shape or _matrices(w_up, w.dtype, "w_up") != (ld, group)):
        raise MoeError(EINVAL, "w_up: not laid out as w")
    if w_up_s is not None and (w_up is None or not mx) or mx and (w_up is None) != (w_up_s is None):
        raise MoeError(EINVAL, "w_up and w_up_s come together")
    if mx:
        if w_s.shape != (g, n, d.n_in // 32):
            raise MoeError(EINVAL, f"w_s: {tuple(w_s.shape)} for codes {tuple(w.shape)}")
        d.ldw_s, d.group_w_s = _matrices(w_s, _torch.uint8, "w_s")
        if w_up_s is not None and (w_up_s.shape != w_s.shape or _matrices(w_up_s, _torch.uint8, "w_up_s") != (d.ldw_s, d.group_w_s)):
            raise MoeError(EINVAL, "w_up_s: not laid out as w_s")
        d.w_s, d.w_up_s = w_s.data_ptr(), _ptr(w_up_s)
    b = bias if bias is not None else bias_up
    d.bias_type = d.type if b is None else _type_of(b)
    d.w, d.w_up, d.device = w.data_ptr(), _ptr(w_up), w.device
    for v, what in ((bias, "bias"), (bias_up, "bias_up")):
        if v is not None and tuple(v.shape) != (g, n):
            raise MoeError(EINVAL, f"{what}: {tuple(v.shape)}")
    d.bias = None if bias is None else _flat(bias, g * n, b.dtype, "bias")
    d.bias_up = None if bias_up is None else _flat(bias_up, g * n, b.dtype, "bias_up")
    return d


def _grouped_x(desc: GroupedDesc, x, rows: int, what: str = "x") -> int:
    """Row distance of x, of which `rows` rows are read."""
    if desc.operands == MXFP4:
        return _bytes(x, rows, desc.n_in // 2, what)
    if _type_of(x) != desc.operands:
        raise MoeError(EINVAL, f"{what}: {x.dtype}")
    return _rows(x, rows, desc.n_in, what)


def grouped_path_for(desc: GroupedDesc, x, R: int, rows=None) -> int:
    """The kernel that `grouped_linear` takes for R rows of x, gathered by `rows` where that is given: one of
    LINEAR_TILE64X32 .. TILE256X128."""
    ldx = _grouped_x(desc, x, x.shape[0] if rows is not None else min(R, x.shape[0]))
    r = int(lib().moe_grouped_path_for(ctypes.byref(desc), x.data_ptr(), ldx, R))
    if r < 0:
        raise MoeError(r, "moe_grouped_path_for")
    return r % 256


def grouped_linear(desc: GroupedDesc, x, offsets, R: int, out_half, out_f32, out_mode: int, rows=None, x_s=None,
                   stream=None) -> None:
    """moe_grouped_linear: rows offsets[g] .. offsets[g + 1] - 1 of the R rows with group g's
    weights.  x: [.., n_in] of w's dtype, row r behind row r, or behind it row rows[r] (int32);
    MXFP4: codes [.., n_in / 2] and scales x_s [.., n_in / 32].  offsets: int32 [n_groups + 1].
    Outputs [.., n_out]; two have the same row distance."""
    n = desc.n_out
    x_rows = x.shape[0]
    ldx = _grouped_x(desc, x, x_rows if rows is not None else R)
    if (x_s is None) != (desc.operands != MXFP4):
        raise MoeError(EINVAL, "x_s: the scales of MXFP4 rows")
    ldxs = 0 if x_s is None else _bytes(x_s, x_rows if rows is not None else R, desc.n_in // 32, "x_s")
    _same_device(desc, x, x_s, offsets, rows, out_half, out_f32)
    op, fp, ldo = _outputs(out_half, out_f32, out_mode, R, n, desc.type)
    i32 = _torch.int32
    _check(_call(x, stream, lib().moe_grouped_linear, desc, x.data_ptr(), ldx, _ptr(x_s), ldxs, x_rows, _flat(rows, R, i32, "rows"),
                 _flat(offsets, desc.n_groups + 1, i32, "offsets"), R, op, fp, ldo, out_mode), "moe_grouped_linear")


def group_workspace_bytes(max_tokens: int, top_k: int, n_experts: int) -> int:
    return int(lib().moe_group_workspace_bytes(max_tokens, top_k, n_experts))


def group_workspace(max_tokens: int, top_k: int, n_experts: int, device="cuda"):
    """An uninitialised workspace (uint8 tensor) for `group` of up to max_tokens tokens."""
    import torch
    n = group_workspace_bytes(max_tokens, top_k, n_experts)
    if n == 0:
        raise MoeError(EINVAL, "moe_group_workspace_bytes: invalid or unsupported sizes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def group(ids, T: int, n_experts: int, offsets, tokens, places, ws, stream=None) -> None:
    """moe_group on the first T rows of ids [.., k]: offsets [n_experts + 1], tokens [T k], places
    [T][k], all contiguous int32."""
    if len(ids.shape) != 2 or ids.shape[0] < T:
        raise MoeError(EINVAL, f"ids: {tuple(ids.shape)}")
    if _torch is None:
        _setup()
    k, i32 = ids.shape[1], _torch.int32
    _same_device(None, ids, offsets, tokens, places, *_ws_tensor(ws))
    wp, wn = _ws(ws)
    _check(_call(ids, stream, lib().moe_group, _flat(ids, T * k, i32, "ids"), T, k, n_experts,
                 _flat(offsets, n_experts + 1, i32, "offsets"), _flat(tokens, T * k, i32, "tokens"),
                 _choices(places, T, k, i32, "places"), wp, wn), "moe_group")


def combine(y, R: int, places, weights, T: int, out, residual=None, stream=None) -> None:
    """moe_combine: out [.., n] = the rows places[t][j] (int32 [.., k]) of the first R of y [.., n],
    each times weights[t][j] (float32, or None), added up, plus residual [.., n].  y, out and
    residual: bfloat16, float16 or float32 each."""
    if len(places.shape) != 2 or places.shape[0] < T or len(y.shape) != 2:
        raise MoeError(EINVAL, f"places: {tuple(places.shape)}, y: {tuple(y.shape)}")
    k, n = places.shape[1], y.shape[1]
    yt, ot = _type_of(y), _type_of(out)
    _same_device(None, y, places, weights, out, residual)
    rt = F32 if residual is None else _type_of(residual)
    rp, ldr = _residual(residual, T, n, rt)
    _check(_call(y, stream, lib().moe_combine, y.data_ptr(), yt, _rows(y, R, n, "y"), R, _flat(places, T * k, _torch.int32, "places"),
                 _choices(weights, T, k, _torch.float32, "weights"), T, k, n, rp, rt, ldr, out.data_ptr(), ot,
                 _rows(out, T, n, "out")), "moe_combine")

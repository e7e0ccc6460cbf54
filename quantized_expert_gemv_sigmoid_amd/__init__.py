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
BF16, F16, F32 = 0, 1, 2
SCORE_SIGMOID, SCORE_SOFTMAX = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
(LINEAR_NONE, LINEAR_RELU, LINEAR_SILU, LINEAR_GELU, LINEAR_GELU_TANH, LINEAR_SITU_GLU,
 LINEAR_SWIGLU) = range(7)
(LINEAR_ROWS16X8, LINEAR_ROWS16X16, LINEAR_ROWS16X32, LINEAR_TILE64X32, LINEAR_TILE64X64, LINEAR_TILE128X64,
 LINEAR_TILE128X128, LINEAR_ANY64X32, LINEAR_ANY64X64, LINEAR_ANY128X128, LINEAR_TILE256X256) = range(11)

EXPORTS = ("moe_workspace_bytes", "moe_path_for", "moe_route", "moe_expert_forward",
           "moe_layer", "moe_layer_noalloc", "moe_layer_timed", "moe_set_one_token_router_wait",
           "moe_latent_workspace_bytes", "moe_latent_path_for", "moe_latent_layer",
           "moe_latent_layer_timed", "moe_gate", "moe_route_gated", "moe_linear_workspace_bytes",
           "moe_linear_path_for", "moe_linear", "moe_status_str")
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
_raw_stream = None


def _setup() -> None:
    global _torch, _raw_stream
    import torch
    _types.update({torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32})
    # (the current stream's address without a Stream object around it, where torch has it)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
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
    shape, stride = t.shape, t.stride()
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


def _same_device(desc, first, *others) -> None:
    """The tensors of a call lie on one device, and those of the descriptor (desc.device, where known) too."""
    d = first.device
    if desc is not None and desc.device is not None and desc.device != d:
        raise MoeError(EINVAL, f"tensors on {desc.device} and {d}")
    for t in others:
        if t is not None and t.device != d:
            raise MoeError(EINVAL, f"tensors on {d} and {t.device}")


def _ws_tensor(ws) -> tuple:
    return () if ws is None or isinstance(ws, tuple) else (ws,)


def _call(x, stream, f, *args) -> int:
    """f(*args, stream) on x's device: that device's current stream where none is given."""
    i = x.device.index
    if i is None:  # (not a GPU's: the arguments that were refused first aside, there is nothing to launch on)
        raise MoeError(EINVAL, f"tensors on {x.device}")
    s = _raw_stream(i) if stream is None else _stream(stream)
    if i != _torch.cuda.current_device():
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
    ldo = ldr = op = fp = rp = None
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
    if residual is not None:
        if _type_of(residual) != desc.residual_type:
            raise MoeError(EINVAL, f"residual: {residual.dtype}")
        ldr, rp = _rows(residual, T, n, "residual"), residual.data_ptr()
    wp, wn = _ws(ws)
    _check(_call(x, stream, lib().moe_linear, desc, x.data_ptr(), _rows(x, T, desc.n_in, "x"), T,
                 rp, ldr or 0, op, fp, n if ldo is None else ldo, out_mode, wp, wn), "moe_linear")

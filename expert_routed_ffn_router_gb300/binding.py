"""Thin ctypes binding of the C ABI in include/moe.h.

Argument marshalling only: torch tensors supply device pointers (``data_ptr()``) and the
current CUDA stream; every step of the layer runs in the library's CUDA kernels.  The
functions carry the C names.  A missing or unbuildable library raises -- there is no
fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _build

MOE_OK = 0
MOE_ERR_DEVICE_TIMEOUT = -6

_lib = None


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status} ({moe_error_string(status)})")
        self.status = status


class MoeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "E", "K", "I", "I_shared")]


class MoeWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("W_gate", "bias", "W1", "W3", "W2", "W1s",
                                               "W3s", "W2s")]


class MoeWorkspaceLayout(ctypes.Structure):
    """moe_workspace_layout_t: byte offsets of the layer's intermediates in the workspace."""
    _fields_ = [(n, ctypes.c_size_t) for n in ("offsets", "perm", "slot_pos", "Xp", "h", "Yp",
                                               "Ysh", "bytes")]


class MoeRouting(ctypes.Structure):
    """moe_routing_t: scoring (0 sigmoid, 1 softmax), n_group, topk_group, group_top,
    renorm.  The defaults are the plain router."""
    _fields_ = [(n, ctypes.c_int32) for n in ("scoring", "n_group", "topk_group",
                                              "group_top", "renorm")]

    @classmethod
    def make(cls, scoring: str = "sigmoid", n_group: int = 1, topk_group: int = 1,
             group_top: int = 1, renorm: bool = True) -> "MoeRouting":
        return cls({"sigmoid": 0, "softmax": 1}[scoring], int(n_group), int(topk_group),
                   int(group_top), int(bool(renorm)))


class MoeWeightsFp8(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("W_gate", "bias", "W1", "W3", "W2", "S1", "S3",
                                               "S2", "W1s", "W3s", "W2s", "S1s", "S3s", "S2s")]


class MoeResidual(ctypes.Structure):
    """moe_residual_t."""
    _fields_ = [("post", ctypes.c_int32), ("pre", ctypes.c_int32), ("alpha", ctypes.c_float),
                ("eps_post", ctypes.c_float), ("eps_pre", ctypes.c_float)] + [
                    (n, ctypes.c_void_p) for n in ("gamma_post", "beta_post", "gate", "gate_token", "gamma_pre",
                                                   "beta_pre")]


class MoeResidualGrads(ctypes.Structure):
    """moe_residual_grads_t."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("gamma_post", "beta_post", "gate", "gate_token", "gamma_pre",
                                               "beta_pre")]


class MoeGraceReplication(ctypes.Structure):
    _fields_ = [("heaviest", ctypes.c_int32), ("n_replica", ctypes.c_int32),
                ("n_hot", ctypes.c_int32), ("rho", ctypes.c_double), ("W_mean", ctypes.c_double),
                ("W_max", ctypes.c_longlong), ("W_r", ctypes.c_longlong)]


def _routing(routing):
    if routing is None:
        return None
    if isinstance(routing, dict):
        routing = MoeRouting.make(**routing)
    return ctypes.byref(routing)


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load libmoe_gb300.so (building it first when it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.build() if build_if_missing else _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library {path} is missing; run the package build first")
    lib = ctypes.CDLL(path)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sig = {
        "moe_workspace_bytes": ([ctypes.POINTER(MoeShape)], Z),
        "moe_workspace_layout": ([ctypes.POINTER(MoeShape), ctypes.POINTER(MoeWorkspaceLayout)], I),
        "moe_error_string": ([I], ctypes.c_char_p),
        "moe_read_status": ([P, P], I),
        "moe_debug_set_wait_limit": ([ctypes.c_ulonglong, I], None),
        "moe_debug_set_stage_events": ([P, I], None),
        "moe_debug_set_ffn_variant": ([I], None),
        "moe_debug_set_shared_side": ([I], None),
        "moe_debug_set_sync_status": ([I], None),
        "moe_router_topk": ([P, P, P, I, I, I, I, P, P, P, Z, P], I),
        "moe_router_topk_ex": ([P, P, P, I, I, I, I, ctypes.POINTER(MoeRouting), P, P, P, Z,
                                P], I),
        "moe_router_topk_noalloc": ([P, P, P, I, I, I, I, P, P, P], I),
        "moe_router_topk_noalloc_status": ([P], I),
        "moe_dispatch": ([P, P, I, I, I, I, P, P, P, P, P, P, P, Z, P], I),
        "moe_expert_ffn": ([P, P, I, I, I, I, P, P, P, P, I, P, Z, P], I),
        "moe_expert_ffn_workspace_bytes": ([I, I, I], Z),
        "moe_combine": ([P, P, P, P, I, I, I, P, P], I),
        "moe_layer_forward": ([ctypes.POINTER(MoeShape), ctypes.POINTER(MoeWeights), P, P, P,
                               P, P, P, P, Z, P], I),
        "moe_layer_forward_ex": ([ctypes.POINTER(MoeShape), ctypes.POINTER(MoeWeights),
                                  ctypes.POINTER(MoeRouting), P, P, P, P, P, P, P, Z, P], I),
        "moe_quantize_weight_fp8": ([P, I, I, I, P, P, P], I),
        "moe_quantize_rows_fp8": ([P, ctypes.c_longlong, I, P, P], I),
        "moe_layer_forward_fp8": ([ctypes.POINTER(MoeShape), ctypes.POINTER(MoeWeightsFp8),
                                   ctypes.POINTER(MoeRouting), P, P, P, P, P, P, P, Z, P], I),
        "moe_layer_norm": ([P, I, P, P, I, I, ctypes.c_float, P, P, P, P], I),
        "moe_layer_norm_backward_workspace_bytes": ([I, I], Z),
        "moe_layer_norm_backward": ([P, P, I, P, P, P, P, I, I, P, P, P, P, Z, P], I),
        "moe_route_logits": ([P, I, P, I, I, I, ctypes.POINTER(MoeRouting), P, P, P], I),
        "moe_route_logits_backward": ([P, I, I, I, I, ctypes.POINTER(MoeRouting), P, P, P, P], I),
        "moe_checkpoint_pack": ([P, ctypes.c_longlong, I, P, P, P], I),
        "moe_checkpoint_unpack": ([P, P, ctypes.c_longlong, I, P, P], I),
        "moe_expert_ffn_backward_workspace_bytes": ([I, I, I, I, I], Z),
        "moe_expert_ffn_backward": ([P, P, P, P, P, P, I, I, I, I, I, P, P, P, P, P, P, P, P, P, Z, P], I),
        "moe_combine_backward": ([P, I, P, P, P, I, I, I, P, P, P], I),
        "moe_dispatch_backward": ([P, P, P, I, I, I, P, I, P], I),
        "moe_residual_norm": ([P, I, P, I, ctypes.POINTER(MoeResidual), I, I, P, P, P, P], I),
        "moe_residual_norm_backward_workspace_bytes": ([I, I], Z),
        "moe_residual_norm_backward": ([P, P, P, I, P, I, P, ctypes.POINTER(MoeResidual), I, I, P, P,
                                        ctypes.POINTER(MoeResidualGrads), P, Z, P], I),
        "moe_orthogonalize_workspace_bytes": ([I, I, I], Z),
        "moe_orthogonalize": ([P, I, P, ctypes.c_float, I, I, I, I, I, P, ctypes.c_float, P, P, Z, P], I),
        "moe_grace_metrics": ([P, I, P, I, P, P], I),
        "moe_grace_group": ([P, I, I, ctypes.c_double, P], I),
        "moe_grace_choose_r": ([P, I, I, P, I, P, P, P, P], I),
        "moe_grace_replicate": ([P, I, P, I, P, P, P, ctypes.POINTER(MoeGraceReplication)], I),
        "moe_grace_route_table": ([P, I, ctypes.POINTER(MoeGraceReplication), P, I, P, P], I),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
I8 = torch.int8


def _chk(t, dtype=None, numel=None, name="tensor"):
    """The C ABI takes bare pointers: a tensor of another element type, or smaller than the
    sizes passed beside it, would be misread (or read past its end) by the kernels."""
    if t is None:
        return
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name}: {t.numel()} elements, expected {numel}")


def _ptr(t, dtype=None, numel=None, name="tensor"):
    """Device pointer of a contiguous CUDA tensor (None stays NULL), after _chk."""
    if t is None:
        return None
    _chk(t, dtype, numel, name)
    if not t.is_cuda:
        raise ValueError(f"{name}: device tensors are required")
    if not t.is_contiguous():
        raise ValueError(f"{name}: contiguous tensors are required")
    return ctypes.c_void_p(t.data_ptr())


def _ptrs(*specs):
    """Pointers of (tensor, dtype, numel, name) arguments: every element type and size is
    checked before any device check."""
    out = []
    for t, dtype, numel, name in specs:
        if t is None:
            out.append(None)
        elif t.dtype is dtype and t.is_cuda and t.numel() == numel and t.is_contiguous():
            out.append(t.data_ptr())
        else:
            break
    else:
        return out
    # some argument does not fit: say which, in the order above
    for spec in specs:
        _chk(*spec)
    return [_ptr(*spec) for spec in specs]


def _ptrs_here(ref, *specs):
    """As _ptrs, for tensors that have to lie on the current device (ref is one of them)."""
    dev, out = ref.get_device(), []
    for t, dtype, numel, name in specs:
        if t is None:
            out.append(None)
        elif t.dtype is dtype and t.get_device() == dev and t.numel() == numel and t.is_contiguous():
            out.append(t.data_ptr())
        else:
            break
    else:
        if dev >= 0 and dev == _current_device():    # (-1: host memory)
            return out
    out = _ptrs(*specs)
    for t, _, _, name in specs:
        if t is not None:
            _here(t, name)
    return out


def _here(t, name):
    if t.get_device() != _current_device():
        raise ValueError(f"{name}: on device {t.get_device()}, the current one is {_current_device()}")


def _wstruct(cls, weights: dict, specs, io_specs):
    """A weights structure from (name, dtype, numel) specs (a missing name stays NULL), with
    the layer's input / output tensors (io_specs): every type and size is checked first."""
    ws = [(weights.get(n), dt, k, n) for n, dt, k in specs]
    for spec in ws + list(io_specs):
        _chk(*spec)
    return cls(*[None if t is None else _ptr(t, dt, k, n).value for t, dt, k, n in ws])


def _ws(ws):
    """Pointer and bytes of a workspace."""
    if ws.is_cuda and ws.is_contiguous():
        return ws.data_ptr(), ws.nbytes
    return _ptr(ws), ws.nbytes


# The current stream's handle without a Stream object around it (2.7 us a call saved, a fifth
# of a small operator's call); the documented way where a torch release lacks it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


_current_device = _raw_device or torch.cuda.current_device


def _ws_here(ws):
    if ws.get_device() == _current_device() and ws.is_contiguous():
        return ws.data_ptr(), ws.nbytes
    out = _ws(ws)
    _here(ws, "ws")
    return out


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and _raw_device is not None and torch.cuda.is_initialized():
        return _raw_stream(_raw_device())
    return torch.cuda.current_stream().cuda_stream


def _stream_here(stream):
    """As _stream, behind _ptrs_here (CUDA is initialised)."""
    if stream is None and _raw_stream is not None and _raw_device is not None:
        return _raw_stream(_raw_device())
    return _stream(stream)


def _check(fn, rc):
    if rc != MOE_OK:
        raise MoeError(fn, rc)


# ------------------------------------------------------------------------- C entry points
def moe_error_string(status: int) -> str:
    return load().moe_error_string(int(status)).decode()


def moe_workspace_bytes(T, H, E, K, I, I_shared) -> int:
    s = MoeShape(T, H, E, K, I, I_shared)
    return int(load().moe_workspace_bytes(ctypes.byref(s)))


def moe_workspace_layout(T, H, E, K, I, I_shared) -> dict:
    """Byte offsets of offsets, perm, slot_pos, Xp, h, Yp and Ysh inside the layer's
    workspace, and its size ("bytes")."""
    s = MoeShape(T, H, E, K, I, I_shared)
    lay = MoeWorkspaceLayout()
    _check("moe_workspace_layout", load().moe_workspace_layout(ctypes.byref(s), ctypes.byref(lay)))
    return {n: int(getattr(lay, n)) for n, _ in MoeWorkspaceLayout._fields_}


def moe_read_status(ws, stream=None) -> int:
    return int(load().moe_read_status(_ptr(ws), _stream(stream)))


def moe_debug_set_wait_limit(limit_ns: int, inject_stall: int = 0) -> None:
    load().moe_debug_set_wait_limit(int(limit_ns), int(inject_stall))


def moe_debug_set_ffn_variant(variant: int) -> None:
    """0: automatic; 1: single-CTA FFN kernel; 2: CTA-pair (2-SM MMA) FFN kernel."""
    load().moe_debug_set_ffn_variant(int(variant))


def moe_debug_set_sync_status(on: bool) -> None:
    """Debug mode: calls synchronise and return their workspace's status word (a device-side
    error then raises MoeError from the call itself)."""
    load().moe_debug_set_sync_status(1 if on else 0)


def moe_debug_set_shared_side(mode: int) -> None:
    """-1: by batch size (default); 0: shared expert in the routed launch; 1: side stream."""
    load().moe_debug_set_shared_side(int(mode))


def moe_debug_set_stage_events(events) -> None:
    """events: list of >= 6 recorded torch.cuda.Event (timing enabled), or None."""
    if events is None:
        load().moe_debug_set_stage_events(None, 0)
        return
    arr = (ctypes.c_void_p * len(events))(*[ev.cuda_event for ev in events])
    load().moe_debug_set_stage_events(ctypes.cast(arr, ctypes.c_void_p), len(events))


def _router_args(X, W_gate, bias, K, topk_idx, topk_w):
    T, H = X.shape
    E, K = W_gate.shape[0], int(K)
    x, wg, b, i, w = _ptrs((X, BF16, T * H, "X"), (W_gate, BF16, E * H, "W_gate"),
                           (bias, F32, E, "bias"), (topk_idx, I32, T * K, "topk_idx"),
                           (topk_w, F32, T * K, "topk_w"))
    return (x, wg, b, T, H, E, K), (i, w)


def moe_router_topk(X, W_gate, bias, K, topk_idx, topk_w, ws, stream=None):
    a, o = _router_args(X, W_gate, bias, K, topk_idx, topk_w)
    _check("moe_router_topk", load().moe_router_topk(
        *a, *o, _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_router_topk_ex(X, W_gate, bias, K, routing, topk_idx, topk_w, ws, stream=None):
    """routing: MoeRouting, a dict of MoeRouting.make keywords, or None (defaults)."""
    a, o = _router_args(X, W_gate, bias, K, topk_idx, topk_w)
    _check("moe_router_topk_ex", load().moe_router_topk_ex(
        *a, _routing(routing), *o, _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_router_topk_noalloc(X, W_gate, bias, K, topk_idx, topk_w, stream=None):
    """The router without a workspace (its scratch is a fixed array of the library)."""
    a, o = _router_args(X, W_gate, bias, K, topk_idx, topk_w)
    _check("moe_router_topk_noalloc", load().moe_router_topk_noalloc(*a, *o, _stream(stream)))


def moe_router_topk_noalloc_status(stream=None) -> int:
    return int(load().moe_router_topk_noalloc_status(_stream(stream)))


def moe_dispatch(X, topk_idx, E, counts, offsets, perm, slot_pos, Xp, affinity, ws,
                 stream=None):
    T, H = X.shape
    K, E = topk_idx.shape[1], int(E)
    x, i, c, o, pm, sp, xp, af = _ptrs(
        (X, BF16, T * H, "X"), (topk_idx, I32, T * K, "topk_idx"), (counts, I32, E, "counts"),
        (offsets, I32, E + 1, "offsets"), (perm, I32, T * K, "perm"),
        (slot_pos, I32, T * K, "slot_pos"), (Xp, BF16, T * K * H, "Xp"),
        (affinity, I32, E * E, "affinity"))
    _check("moe_dispatch", load().moe_dispatch(
        x, i, T, H, E, K, c, o, pm, sp, xp, af, _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_expert_ffn_workspace_bytes(rows: int, n_groups: int, I: int) -> int:
    return int(load().moe_expert_ffn_workspace_bytes(int(rows), int(n_groups), int(I)))


def moe_expert_ffn(Xp, offsets, n_groups, W1, W3, W2, Yp, ws, stream=None):
    rows, H = Xp.shape
    I, G = W1.shape[-1], int(n_groups)
    out_fp32 = 1 if Yp.dtype == torch.float32 else 0
    xp, o, w1, w3, w2, yp = _ptrs(
        (Xp, BF16, rows * H, "Xp"), (offsets, I32, G + 1, "offsets"),
        (W1, BF16, G * H * I, "W1"), (W3, BF16, G * H * I, "W3"), (W2, BF16, G * I * H, "W2"),
        (Yp, F32 if out_fp32 else BF16, rows * H, "Yp"))
    _check("moe_expert_ffn", load().moe_expert_ffn(
        xp, o, G, rows, H, I, w1, w3, w2, yp, out_fp32, _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def moe_combine(Yp, slot_pos, topk_w, Ysh, Y, stream=None):
    T, K = slot_pos.shape
    H = Y.shape[1]
    yp, sp, w, ysh, y = _ptrs((Yp, BF16, T * K * H, "Yp"), (slot_pos, I32, T * K, "slot_pos"),
                              (topk_w, F32, T * K, "topk_w"), (Ysh, F32, T * H, "Ysh"),
                              (Y, F32, T * H, "Y"))
    _check("moe_combine", load().moe_combine(yp, sp, w, ysh, T, H, K, y, _stream(stream)))


def _io_specs(shape: MoeShape, X, Y, topk_idx, topk_w, counts, affinity):
    T, H, E, K = shape.T, shape.H, shape.E, shape.K
    return [(X, BF16, T * H, "X"), (Y, F32, T * H, "Y"), (topk_idx, I32, T * K, "topk_idx"),
            (topk_w, F32, T * K, "topk_w"), (counts, I32, E, "counts"),
            (affinity, I32, E * E, "affinity")]


def _layer_args(shape: MoeShape, weights: dict, io):
    H, E, I, Is = shape.H, shape.E, shape.I, shape.I_shared
    w = _wstruct(MoeWeights, weights,
                 (("W_gate", BF16, E * H), ("bias", F32, E), ("W1", BF16, E * H * I),
                  ("W3", BF16, E * H * I), ("W2", BF16, E * I * H), ("W1s", BF16, H * Is),
                  ("W3s", BF16, H * Is), ("W2s", BF16, Is * H)), io)
    return w, _ptrs(*io)


def moe_layer_forward(shape: MoeShape, weights: dict, X, Y, topk_idx, topk_w, counts,
                      affinity, ws, stream=None):
    w, io = _layer_args(shape, weights, _io_specs(shape, X, Y, topk_idx, topk_w, counts, affinity))
    _check("moe_layer_forward", load().moe_layer_forward(
        ctypes.byref(shape), ctypes.byref(w), *io, _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_layer_forward_ex(shape: MoeShape, weights: dict, routing, X, Y, topk_idx, topk_w,
                         counts, affinity, ws, stream=None):
    w, io = _layer_args(shape, weights, _io_specs(shape, X, Y, topk_idx, topk_w, counts, affinity))
    _check("moe_layer_forward_ex", load().moe_layer_forward_ex(
        ctypes.byref(shape), ctypes.byref(w), _routing(routing), *io, _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def moe_quantize_weight_fp8(W, stream=None):
    """W bf16 [G, R, C] or [R, C] (device; R the reduction dimension) -> (E4M3 bytes uint8,
    transposed: [G, C, R] or [C, R]; int32 scale exponents [G, R/128, C/128] or
    [R/128, C/128])."""
    shape = W.shape
    G, R, C = (1,) + tuple(shape) if W.dim() == 2 else tuple(shape)
    Wq = torch.empty(shape[:-2] + (C, R), dtype=torch.uint8, device=W.device)
    S = torch.empty(shape[:-2] + (R // 128, C // 128), dtype=torch.int32, device=W.device)
    _check("moe_quantize_weight_fp8", load().moe_quantize_weight_fp8(
        _ptr(W, BF16, name="W"), G, R, C, _ptr(Wq), _ptr(S), _stream(stream)))
    return Wq, S


def moe_quantize_rows_fp8(x, out=None, stream=None):
    rows, n = x.shape
    if out is None:
        out = torch.empty_like(x)
    _check("moe_quantize_rows_fp8", load().moe_quantize_rows_fp8(
        _ptr(x), rows, n, _ptr(out), _stream(stream)))
    return out


def quantize_expert_weights_fp8(weights: dict, stream=None) -> dict:
    """bf16 layer weights (W_gate, bias, W1, W3, W2[, W1s, W3s, W2s]) -> the FP8 layer's
    weights (E4M3 bytes and tile scale exponents); W_gate and bias are kept."""
    out = {"W_gate": weights["W_gate"], "bias": weights["bias"]}
    for w, sc in (("W1", "S1"), ("W3", "S3"), ("W2", "S2"), ("W1s", "S1s"), ("W3s", "S3s"),
                  ("W2s", "S2s")):
        if weights.get(w) is None:
            out[w] = out[sc] = None
            continue
        out[w], out[sc] = moe_quantize_weight_fp8(weights[w], stream)
    return out


def moe_layer_forward_fp8(shape: MoeShape, weights8: dict, routing, X, Y, topk_idx, topk_w,
                          counts, affinity, ws, stream=None):
    H, E, I, Is = shape.H, shape.E, shape.I, shape.I_shared
    tiles, tiles_s = (H // 128) * (I // 128), (H // 128) * (Is // 128)
    io = _io_specs(shape, X, Y, topk_idx, topk_w, counts, affinity)
    w = _wstruct(MoeWeightsFp8, weights8,
                 (("W_gate", BF16, E * H), ("bias", F32, E), ("W1", U8, E * H * I),
                  ("W3", U8, E * H * I), ("W2", U8, E * I * H), ("S1", I32, E * tiles),
                  ("S3", I32, E * tiles), ("S2", I32, E * tiles), ("W1s", U8, H * Is),
                  ("W3s", U8, H * Is), ("W2s", U8, Is * H), ("S1s", I32, tiles_s),
                  ("S3s", I32, tiles_s), ("S2s", I32, tiles_s)), io)
    _check("moe_layer_forward_fp8", load().moe_layer_forward_fp8(
        ctypes.byref(shape), ctypes.byref(w), _routing(routing), *_ptrs(*io), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


# -------------------------------------------------------------- training around the layer
def _fp32_flag(t, name):
    if t.dtype not in (BF16, F32):
        raise ValueError(f"{name}: dtype {t.dtype}, expected {BF16} or {F32}")
    return 1 if t.dtype == F32 else 0


def moe_layer_norm(x, gamma, beta, eps, y, mean=None, rstd=None, stream=None):
    """x bf16 or fp32 [T, H] -> y bf16; beta, mean and rstd may be None."""
    T, H = x.shape
    f = _fp32_flag(x, "x")
    xp, g, b, yp, m, r = _ptrs((x, x.dtype, T * H, "x"), (gamma, F32, H, "gamma"), (beta, F32, H, "beta"),
                               (y, BF16, T * H, "y"), (mean, F32, T, "mean"), (rstd, F32, T, "rstd"))
    _check("moe_layer_norm", load().moe_layer_norm(xp, f, g, b, T, H, float(eps), yp, m, r,
                                                   _stream(stream)))


def moe_layer_norm_backward_workspace_bytes(T: int, H: int) -> int:
    return int(load().moe_layer_norm_backward_workspace_bytes(int(T), int(H)))


def moe_layer_norm_backward(dy, x, gamma, mean, rstd, dres, dx, dgamma, dbeta, ws, stream=None):
    """dres: a gradient of x's type to add to dx, or None."""
    T, H = x.shape
    f = _fp32_flag(x, "x")
    d, xp, g, m, r, e, o, dg, db = _ptrs(
        (dy, BF16, T * H, "dy"), (x, x.dtype, T * H, "x"), (gamma, F32, H, "gamma"), (mean, F32, T, "mean"),
        (rstd, F32, T, "rstd"), (dres, x.dtype, T * H, "dres"), (dx, x.dtype, T * H, "dx"),
        (dgamma, F32, H, "dgamma"), (dbeta, F32, H, "dbeta"))
    _check("moe_layer_norm_backward", load().moe_layer_norm_backward(
        d, xp, f, g, m, r, e, T, H, o, dg, db, *_ws(ws), _stream(stream)))


def moe_route_logits(logits, bias, K, routing, topk_idx, topk_w, stream=None):
    """logits bf16 or fp32 [T, E]; bias may be None; routing as in moe_router_topk_ex."""
    T, E = logits.shape
    K, f = int(K), _fp32_flag(logits, "logits")
    l, b, i, w = _ptrs((logits, logits.dtype, T * E, "logits"), (bias, F32, E, "bias"),
                       (topk_idx, I32, T * K, "topk_idx"), (topk_w, F32, T * K, "topk_w"))
    _check("moe_route_logits", load().moe_route_logits(l, f, b, T, E, K, _routing(routing), i, w,
                                                       _stream(stream)))


def moe_route_logits_backward(logits, routing, topk_idx, d_topk_w, d_logits, stream=None):
    T, E = logits.shape
    K, f = topk_idx.shape[1], _fp32_flag(logits, "logits")
    l, i, w, d = _ptrs((logits, logits.dtype, T * E, "logits"), (topk_idx, I32, T * K, "topk_idx"),
                       (d_topk_w, F32, T * K, "d_topk_w"), (d_logits, logits.dtype, T * E, "d_logits"))
    _check("moe_route_logits_backward", load().moe_route_logits_backward(
        l, f, T, E, K, _routing(routing), i, w, d, _stream(stream)))


def moe_checkpoint_pack(x, q=None, scale=None, stream=None):
    """x bf16 [rows, n] -> (E4M3 bytes uint8 [rows, n], scale exponents int8
    [rows, ceil(n / 128)]), into q and scale where given."""
    rows, n = x.shape
    nb = (n + 127) // 128
    q = torch.empty(rows, n, dtype=U8, device=x.device) if q is None else q
    scale = torch.empty(rows, nb, dtype=I8, device=x.device) if scale is None else scale
    xp, qp, sp = _ptrs((x, BF16, rows * n, "x"), (q, U8, rows * n, "q"), (scale, I8, rows * nb, "scale"))
    _check("moe_checkpoint_pack", load().moe_checkpoint_pack(xp, rows, n, qp, sp, _stream(stream)))
    return q, scale


def moe_checkpoint_unpack(q, scale, out=None, stream=None):
    rows, n = q.shape
    out = torch.empty(rows, n, dtype=BF16, device=q.device) if out is None else out
    qp, sp, o = _ptrs((q, U8, rows * n, "q"), (scale, I8, rows * ((n + 127) // 128), "scale"),
                      (out, BF16, rows * n, "out"))
    _check("moe_checkpoint_unpack", load().moe_checkpoint_unpack(qp, sp, rows, n, o, _stream(stream)))
    return out


def moe_expert_ffn_backward_workspace_bytes(T, H, E, K, I) -> int:
    return int(load().moe_expert_ffn_backward_workspace_bytes(T, H, E, K, I))


def moe_expert_ffn_backward(x, x_scale, dY, offsets, slot_pos, topk_w, W1, W3, W2, dX, d_topk_w,
                            dW1, dW3, dW2, ws, stream=None):
    """x bf16 with x_scale None, or a checkpoint's (q, scale); topk_w (all 1) and d_topk_w (not
    wanted) may be None."""
    T, H = x.shape
    E, _, I = W1.shape
    K, n = slot_pos.shape[1], E * H * I
    xp, xs, dy, o, sp, w, w1, w3, w2, dx, dw, d1, d3, d2 = _ptrs(
        (x, BF16 if x_scale is None else U8, T * H, "x"), (x_scale, I8, T * ((H + 127) // 128), "x_scale"),
        (dY, BF16, T * H, "dY"), (offsets, I32, E + 1, "offsets"), (slot_pos, I32, T * K, "slot_pos"),
        (topk_w, F32, T * K, "topk_w"), (W1, BF16, n, "W1"), (W3, BF16, n, "W3"), (W2, BF16, n, "W2"),
        (dX, BF16, T * H, "dX"), (d_topk_w, F32, T * K, "d_topk_w"), (dW1, BF16, n, "dW1"),
        (dW3, BF16, n, "dW3"), (dW2, BF16, n, "dW2"))
    _check("moe_expert_ffn_backward", load().moe_expert_ffn_backward(
        xp, xs, dy, o, sp, w, T, H, E, K, I, w1, w3, w2, dx, dw, d1, d3, d2, *_ws(ws), _stream(stream)))


def moe_combine_backward(dY, Yp, slot_pos, topk_w, dYp, d_topk_w=None, stream=None):
    """dY bf16 or fp32 [T, H]; topk_w (all 1), d_topk_w (not wanted) and with it Yp may be None."""
    T, K = slot_pos.shape
    H, f = dY.shape[1], _fp32_flag(dY, "dY")
    d, y, s, w, o, dw = _ptrs_here(
        dY, (dY, dY.dtype, T * H, "dY"), (Yp, BF16, T * K * H, "Yp"), (slot_pos, I32, T * K, "slot_pos"),
        (topk_w, F32, T * K, "topk_w"), (dYp, BF16, T * K * H, "dYp"), (d_topk_w, F32, T * K, "d_topk_w"))
    _check("moe_combine_backward", load().moe_combine_backward(d, f, y, s, w, T, H, K, o, dw, _stream_here(stream)))


def moe_dispatch_backward(dXp, slot_pos, dres, dX, stream=None):
    """dX bf16 or fp32 [T, H]; dres of its type, or None."""
    T, K = slot_pos.shape
    H, f = dX.shape[1], _fp32_flag(dX, "dX")
    p, s, r, o = _ptrs_here(
        dX, (dXp, BF16, T * K * H, "dXp"), (slot_pos, I32, T * K, "slot_pos"), (dres, dX.dtype, T * H, "dres"),
        (dX, dX.dtype, T * H, "dX"))
    _check("moe_dispatch_backward", load().moe_dispatch_backward(p, s, r, T, H, K, o, f, _stream_here(stream)))


_NORMS = {"none": 0, "layer": 1, "rms": 2}
_COLUMN_KEYS = frozenset(("gamma_post", "beta_post", "gate", "gate_token", "gamma_pre", "beta_pre"))
_RESIDUAL_KEYS = _COLUMN_KEYS | {"post", "pre", "alpha", "eps_post", "eps_pre"}


def _param_specs(p, T, H):
    """Specs of a joined residual's parameters for _ptrs."""
    if not _RESIDUAL_KEYS.issuperset(p):
        raise ValueError(f"{next(n for n in p if n not in _RESIDUAL_KEYS)}: unknown, expected some of {sorted(_RESIDUAL_KEYS)}")
    get = p.get
    return ((get("gamma_post"), F32, H, "gamma_post"), (get("beta_post"), F32, H, "beta_post"), (get("gate"), F32, H, "gate"),
            (get("gate_token"), F32, T, "gate_token"), (get("gamma_pre"), F32, H, "gamma_pre"),
            (get("beta_pre"), F32, H, "beta_pre"))


def _grad_specs(g, T, H):
    if not _COLUMN_KEYS.issuperset(g):
        raise ValueError(f"{next(n for n in g if n not in _COLUMN_KEYS)}: unknown gradient, expected some of {sorted(_COLUMN_KEYS)}")
    get = g.get
    return ((get("gamma_post"), F32, H, "gradient of gamma_post"), (get("beta_post"), F32, H, "gradient of beta_post"),
            (get("gate"), F32, H, "gradient of gate"), (get("gate_token"), F32, T, "gradient of gate_token"),
            (get("gamma_pre"), F32, H, "gradient of gamma_pre"), (get("beta_pre"), F32, H, "gradient of beta_pre"))


def _norm_kind(p, name):
    kind = _NORMS.get(p.get(name, "none"))
    if kind is None:
        raise ValueError(f"{name}: {p[name]}, expected one of {tuple(_NORMS)}")
    return kind


def _residual(p, post, pre, columns):
    get = p.get
    return ctypes.byref(MoeResidual(post, pre, get("alpha", 1.0), get("eps_post", 1e-5), get("eps_pre", 1e-5), *columns))


def moe_residual_norm(x, y, p, r, n=None, stats=None, stream=None):
    """p: dict with post and pre ("none", "layer" or "rms"; default "none"), alpha (default 1),
    eps_post, eps_pre (default 1e-5) and the fp32 parameters gamma_post, beta_post, gate, gamma_pre,
    beta_pre [H] and gate_token [T], each of which may be missing or None."""
    T, H = x.shape
    fx, fy, post, pre, k = _fp32_flag(x, "x"), _fp32_flag(y, "y"), _norm_kind(p, "post"), _norm_kind(p, "pre"), T * H
    xp, yp, rp, np_, sp, *cols = _ptrs_here(
        x, (x, x.dtype, k, "x"), (y, y.dtype, k, "y"), (r, x.dtype, k, "r"), (n, BF16, k, "n"),
        (stats, F32, 4 * T, "stats"), *_param_specs(p, T, H))
    _check("moe_residual_norm", load().moe_residual_norm(xp, fx, yp, fy, _residual(p, post, pre, cols), T, H, rp, np_, sp,
                                                         _stream_here(stream)))


def moe_residual_norm_backward_workspace_bytes(T: int, H: int) -> int:
    return int(load().moe_residual_norm_backward_workspace_bytes(int(T), int(H)))


def moe_residual_norm_backward(dn, dr, y, r, stats, p, dx, dy, grads, ws, stream=None):
    """p as in the forward call; grads: dict of the wanted parameters' gradients by the
    parameters' names.  dn (without pre), dr, y and r (see the header) may be None."""
    T, H = dx.shape
    fx, fy, post, pre = _fp32_flag(dx, "dx"), 0 if y is None else _fp32_flag(y, "y"), _norm_kind(p, "post"), _norm_kind(p, "pre")
    k, xt = T * H, dx.dtype
    d, e, yp, rp, sp, dxp, dyp, *cols = _ptrs_here(
        dx, (dn, BF16, k, "dn"), (dr, xt, k, "dr"), (y, F32 if fy else BF16, k, "y"), (r, xt, k, "r"),
        (stats, F32, 4 * T, "stats"), (dx, xt, k, "dx"), (dy, BF16, k, "dy"), *_param_specs(p, T, H),
        *_grad_specs(grads, T, H))
    _check("moe_residual_norm_backward", load().moe_residual_norm_backward(
        d, e, yp, fy, rp, fx, sp, _residual(p, post, pre, cols[:6]), T, H, dxp, dyp,
        ctypes.byref(MoeResidualGrads(*cols[6:])), *_ws_here(ws), _stream_here(stream)))


def moe_orthogonalize_workspace_bytes(B: int, R: int, C: int) -> int:
    return int(load().moe_orthogonalize_workspace_bytes(int(B), int(R), int(C)))


def moe_orthogonalize(g, out, ws, momentum=None, mu=0.95, nesterov=False, steps=5, coeffs=None, scale=1.0,
                      stream=None):
    """g bf16 or fp32 [B, R, C] or [R, C] -> out bf16; momentum fp32, updated, or None; coeffs: a
    sequence of `steps` triples (a, b, c), or None (the default in every step)."""
    b, R, C = ((1,) + tuple(g.shape))[-3:]
    n, f = b * R * C, _fp32_flag(g, "g")
    arr = None
    if coeffs is not None:
        flat = [float(v) for step in coeffs for v in step]
        if len(flat) != 3 * int(steps):
            raise ValueError(f"coeffs: {len(flat)} values, expected {3 * int(steps)}")
        arr = (ctypes.c_float * len(flat))(*flat)
    gp, m, o = _ptrs_here(g, (g, g.dtype, n, "g"), (momentum, F32, n, "momentum"), (out, BF16, n, "out"))
    _check("moe_orthogonalize", load().moe_orthogonalize(
        gp, f, m, float(mu), 1 if nesterov else 0, b, R, C, int(steps), arr, float(scale), o, *_ws_here(ws),
        _stream_here(stream)))


# ------------------------------------------------------------------- convenience wrapper
class MoELayer:
    """Holds a layer's weights, outputs and workspace (torch allocations) and runs
    moe_layer_forward.  weights: dict of device tensors W_gate, bias, W1, W3, W2 and
    (optionally) W1s, W3s, W2s."""

    def __init__(self, weights: dict, T: int, K: int, with_affinity: bool = True,
                 routing=None, fp8: bool = False, weights8: dict | None = None):
        self.w = weights
        self.routing = routing
        # FP8 experts: the weights are quantised once here (static, 128 x 128 tiles), unless
        # another layer's quantised weights are passed in
        self.w8 = (weights8 if weights8 is not None else quantize_expert_weights_fp8(weights)) if fp8 else None
        E, H = weights["W_gate"].shape
        I = weights["W1"].shape[-1]
        Is = 0 if weights.get("W1s") is None else weights["W1s"].shape[-1]
        self.shape = MoeShape(T, H, E, K, I, Is)
        dev = weights["W_gate"].device
        self.Y = torch.empty(T, H, dtype=torch.float32, device=dev)
        self.topk_idx = torch.empty(T, K, dtype=torch.int32, device=dev)
        self.topk_w = torch.empty(T, K, dtype=torch.float32, device=dev)
        self.counts = torch.empty(E, dtype=torch.int32, device=dev)
        self.affinity = (torch.empty(E, E, dtype=torch.int32, device=dev)
                         if with_affinity else None)
        nbytes = moe_workspace_bytes(T, H, E, K, I, Is)
        if nbytes == 0:
            raise MoeError("moe_workspace_bytes", -2)
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)

    def forward(self, X, stream=None):
        if self.w8 is not None:
            moe_layer_forward_fp8(self.shape, self.w8, self.routing, X, self.Y, self.topk_idx,
                                  self.topk_w, self.counts, self.affinity, self.ws, stream)
        elif self.routing is None:
            moe_layer_forward(self.shape, self.w, X, self.Y, self.topk_idx, self.topk_w,
                              self.counts, self.affinity, self.ws, stream)
        else:
            moe_layer_forward_ex(self.shape, self.w, self.routing, X, self.Y, self.topk_idx,
                                 self.topk_w, self.counts, self.affinity, self.ws, stream)
        return self.Y

    def status(self, stream=None) -> int:
        return moe_read_status(self.ws, stream)

    def intermediates(self) -> dict:
        """Views (no copies) of the last forward's offsets [E+1], perm [T*K], slot_pos
        [T,K] and Xp [T*K,H] inside the workspace (moe_workspace_layout)."""
        s = self.shape
        lay = moe_workspace_layout(s.T, s.H, s.E, s.K, s.I, s.I_shared)
        TK = s.T * s.K

        def view(off, n, dtype, shape):
            nbytes = n * torch.empty((), dtype=dtype).element_size()
            return self.ws[off:off + nbytes].view(dtype).view(*shape)
        return dict(offsets=view(lay["offsets"], s.E + 1, torch.int32, (s.E + 1,)),
                    perm=view(lay["perm"], TK, torch.int32, (TK,)),
                    slot_pos=view(lay["slot_pos"], TK, torch.int32, (s.T, s.K)),
                    Xp=view(lay["Xp"], TK * s.H, torch.bfloat16, (TK, s.H)))


# ------------------------------------------------------ GRACE-MoE placement (host arrays)
def _np(a, dtype):
    import numpy as np
    return np.ascontiguousarray(a, dtype=dtype)


def _hp(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def moe_grace_metrics(affinity, group_of, D: int):
    import numpy as np
    A = _np(affinity, np.int32)
    g = _np(group_of, np.int32)
    U, S = ctypes.c_double(), ctypes.c_double()
    _check("moe_grace_metrics", load().moe_grace_metrics(_hp(A), A.shape[0], _hp(g), int(D),
                                                         ctypes.byref(U), ctypes.byref(S)))
    return U.value, S.value


def moe_grace_group(affinity, D: int, r: float):
    import numpy as np
    A = _np(affinity, np.int32)
    g = np.zeros(A.shape[0], np.int32)
    _check("moe_grace_group", load().moe_grace_group(_hp(A), A.shape[0], int(D), float(r), _hp(g)))
    return g


def moe_grace_choose_r(affinity, D: int, r_grid):
    import numpy as np
    A = _np(affinity, np.int32)
    r = _np(r_grid, np.float64)
    U, S = np.zeros(len(r)), np.zeros(len(r))
    g = np.zeros(A.shape[0], np.int32)
    k = ctypes.c_int()
    _check("moe_grace_choose_r", load().moe_grace_choose_r(
        _hp(A), A.shape[0], int(D), _hp(r), len(r), _hp(U), _hp(S), ctypes.byref(k), _hp(g)))
    return dict(U=U, S=S, knee=k.value, r=float(r[k.value]), group_of=g)


def moe_grace_replicate(counts, group_of, D: int):
    import numpy as np
    c = _np(counts, np.int32)
    g = _np(group_of, np.int32)
    W = np.zeros(D, np.int64)
    hot = np.zeros(len(c), np.int32)
    rg = np.zeros(max(D - 1, 1), np.int32)
    rep = MoeGraceReplication()
    _check("moe_grace_replicate", load().moe_grace_replicate(
        _hp(c), len(c), _hp(g), int(D), _hp(W), _hp(hot), _hp(rg), ctypes.byref(rep)))
    return dict(W=W.tolist(), W_mean=rep.W_mean, W_max=rep.W_max, heaviest=rep.heaviest,
                rho=rep.rho, n_replica=rep.n_replica, hot=hot[:rep.n_hot].tolist(),
                W_r=rep.W_r, replica_gpus=rg[:rep.n_replica].tolist(), _struct=rep)


def moe_grace_route_table(rep: dict, gpus_per_node: int):
    import numpy as np
    W = _np(rep["W"], np.int64)
    D = len(W)
    st = rep["_struct"]
    rg = _np(rep["replica_gpus"] or [0], np.int32)
    n = 1 + st.n_replica
    pred = np.zeros(n)
    table = np.zeros((D, n))
    _check("moe_grace_route_table", load().moe_grace_route_table(
        _hp(W), D, ctypes.byref(st), _hp(rg), int(gpus_per_node), _hp(pred), _hp(table)))
    return dict(instances=[st.heaviest] + list(rep["replica_gpus"]), predicted=pred, table=table)

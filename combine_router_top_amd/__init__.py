"""Python binding of libmoe (MI355X / gfx950 MoE-layer hot path).

A thin ctypes layer over the C ABI in ``include/moe.h``: it checks tensor
shapes and dtypes, passes ``data_ptr()`` and the current HIP stream, and turns
status codes into exceptions.  Every step of the layer runs in the library's
HIP kernels; there is no fallback.  If ``libmoe.so`` has not been built, every
call raises.

Functions (same names as the C calls, which spell 4bit as fourbit):
    route(p, x, w_gate, bias=None, want_logits=False) -> (topk_idx, topk_w[, logits])
    dispatch(p, topk_idx, x) -> dict(counts_all, offsets, perm, inv, x_packed)
    dispatch_noalloc(p, topk_idx, x) -> the same, with no workspace (static scratch)
    expert_gemm(p, x_packed, offsets, w1, w3, w2) -> (h, y_packed)
    combine(p, y_packed, inv, topk_w) -> y
    layer(p, x, w_gate, bias, w1, w3, w2, routing=False, overlap=False, fold_weight=False, ...)
        -> y or (y, dict)
    layer_ws_offset(p, MOE_WS_H | MOE_WS_Y_PACKED) -> byte offset in the layer workspace
    dispatch_padded(p, capacity, topk_idx, x) -> dict(counts_all, offsets, perm, inv, x_packed)
    expert_gemm_padded(p, capacity, x_packed, offsets, w1, w3, w2) -> (h, y_packed)
    expert_gemm_train(p, x_packed, offsets, w1, w3, w2) -> (g, u, h, y_packed)
    expert_gemm_backward(p, x_packed, offsets, w1, w3, w2, g, u, h, dy_packed)
        -> (dx_packed, dw1, dw3, dw2)
    combine_backward(p, dy, y_packed, inv, topk_w) -> (dy_packed, dtopk_w)
    quantize_rows(x) -> (q, scale)
    pack_weights(w) -> packed;  quantize_weights(w) -> (packed, scale)   (w [n,K,N] or [K,N])
    gemm_quantized(a, a_scale, packed, b_scale) -> C
    expert_gemm_quantized(p, x_packed, offsets, w1, s1, w3, s3, w2, s2) -> (h, y_packed)
    select(p, gate, logits, balance=None) -> (topk_idx, topk_w)      (gate: a Gate)
    route_scored(p, gate, x, w_gate, bias=None, balance=None, want_logits=False)
        -> (topk_idx, topk_w[, logits])
    route_backward(p, gate, x, w_gate, logits, topk_idx, dtopk_w, dx_add=None)
        -> (dlogits, dx, dw_gate, dbias)
    pack_weights_4bit(q) -> packed;  quantize_weights_4bit(w, group=128, zero=False)
        -> (packed, scale, zero or None)                             (w [n,K,N] or [K,N])
    gemm_4bit(a, packed, scale, zero=None, group=128) -> C
    expert_gemm_4bit(p, x_packed, offsets, w1, s1, z1, w3, s3, z3, w2, s2, z2, group=128)
        -> (h, y_packed)
    gemm_signal(A, B, flags, epoch) -> C          (C = rnd(A B), a flag per 256 x 256 tile)
    tile_forward(C, dst, flags, epoch, spin_limit, timeouts, workgroups)

The training, scored-routing, 8-bit and 4-bit calls take tensors and streams of the current device only.
With ``stream=`` they order nothing against the current stream, and what they allocate
belongs to the given one: wait for it before reading the outputs elsewhere, and
``record_stream`` outputs that outlive such a use.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass
from typing import Dict, Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 0, 1, 2, 3, 4
MOE_DTYPE_F32, MOE_DTYPE_BF16 = 0, 1
MOE_F_WRITE_LOGITS, MOE_F_OVERLAP, MOE_F_FOLD_WEIGHT = 1, 2, 4
MOE_WS_H, MOE_WS_Y_PACKED = 0, 1
MOE_CALL_ROUTE, MOE_CALL_DISPATCH, MOE_CALL_EXPERT_GEMM, MOE_CALL_COMBINE, MOE_CALL_LAYER = range(5)
MOE_CALL_DISPATCH_PADDED, MOE_CALL_EXPERT_GEMM_PADDED = 5, 6
MOE_CALL_EXPERT_GEMM_BACKWARD, MOE_CALL_EXPERT_GEMM_QUANTIZED = 7, 8
MOE_CALL_ROUTE_SCORED, MOE_CALL_ROUTE_BACKWARD, MOE_CALL_EXPERT_GEMM_FOURBIT = 9, 10, 11
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_SCOPE_AGENT, MOE_SCOPE_SYSTEM = 0, 1

EXPORTED = ["moe_last_error", "moe_version", "moe_workspace_bytes", "moe_route", "moe_dispatch",
            "moe_expert_gemm", "moe_combine", "moe_layer", "moe_dispatch_padded",
            "moe_expert_gemm_padded", "moe_gemm_signal_tiles", "moe_gemm_signal", "moe_tile_forward",
            "moe_dispatch_noalloc", "moe_layer_ws_offset", "moe_layer_set_gemm_events",
            "moe_expert_gemm_train", "moe_expert_gemm_backward", "moe_combine_backward",
            "moe_quantize_rows", "moe_packed_weights_bytes", "moe_pack_weights",
            "moe_quantize_weights", "moe_gemm_quantized", "moe_expert_gemm_quantized",
            "moe_select", "moe_route_scored", "moe_route_backward", "moe_packed_weights_fourbit_bytes",
            "moe_pack_weights_fourbit", "moe_quantize_weights_fourbit", "moe_gemm_fourbit",
            "moe_gemm_fourbit_workspace_bytes", "moe_expert_gemm_fourbit"]


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libmoe status {status}: {msg}")
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("f", ctypes.c_int32), ("expert_lo", ctypes.c_int32),
                ("n_local", ctypes.c_int32), ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class RoutingOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("topk_idx", "topk_w", "logits", "counts_all", "offsets", "perm", "inv")]


class GateRule(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("score", "groups", "topk_groups", "group_top", "renorm")] + [
        ("scale", ctypes.c_float)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} not built; run python -m combine_router_top_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
        P = ctypes.POINTER(Problem)
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_version.restype = ctypes.c_char_p
        L.moe_workspace_bytes.argtypes = [P, i32]
        L.moe_workspace_bytes.restype = sz
        L.moe_layer_ws_offset.argtypes = [P, i32]
        L.moe_layer_ws_offset.restype = sz
        L.moe_layer_set_gemm_events.argtypes = [vp, vp]
        L.moe_route.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_dispatch.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_dispatch_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_expert_gemm.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_combine.argtypes = [P, vp, vp, vp, vp, vp]
        L.moe_layer.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(RoutingOut), vp, sz,
                                vp, vp]
        L.moe_dispatch_padded.argtypes = [P, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_expert_gemm_padded.argtypes = [P, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_gemm_signal_tiles.argtypes = [i32, i32]
        L.moe_gemm_signal_tiles.restype = ctypes.c_int64
        u32 = ctypes.c_uint32
        L.moe_gemm_signal.argtypes = [i32, i32, i32, vp, vp, vp, vp, u32, i32, vp]
        L.moe_tile_forward.argtypes = [i32, i32, vp, vp, vp, u32, u32, i32, vp, i32, vp]
        i64 = ctypes.c_int64
        L.moe_expert_gemm_train.argtypes = [P] + [vp] * 10
        L.moe_expert_gemm_backward.argtypes = [P] + [vp] * 14 + [sz, vp]
        L.moe_combine_backward.argtypes = [P] + [vp] * 7
        L.moe_quantize_rows.argtypes = [i64, i32, i32, vp, vp, vp, vp]
        L.moe_packed_weights_bytes.argtypes = [i32, i32, i32]
        L.moe_packed_weights_bytes.restype = sz
        L.moe_pack_weights.argtypes = [i32, i32, i32, vp, vp, vp]
        L.moe_quantize_weights.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp]
        L.moe_gemm_quantized.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, i32, vp]
        L.moe_expert_gemm_quantized.argtypes = [P] + [vp] * 11 + [sz, vp]
        G = ctypes.POINTER(GateRule)
        L.moe_select.argtypes = [P, G] + [vp] * 5
        L.moe_route_scored.argtypes = [P, G] + [vp] * 8 + [sz, vp]
        L.moe_route_backward.argtypes = [P, G] + [vp] * 11 + [sz, vp]
        L.moe_packed_weights_fourbit_bytes.argtypes = [i32, i32, i32]
        L.moe_packed_weights_fourbit_bytes.restype = sz
        L.moe_pack_weights_fourbit.argtypes = [i32, i32, i32, vp, vp, vp]
        L.moe_quantize_weights_fourbit.argtypes = [i32] * 5 + [vp] * 5
        L.moe_gemm_fourbit_workspace_bytes.argtypes = [i32] * 3
        L.moe_gemm_fourbit_workspace_bytes.restype = sz
        L.moe_gemm_fourbit.argtypes = [i32] * 4 + [vp] * 5 + [i32, vp, sz, vp]
        L.moe_expert_gemm_fourbit.argtypes = [P, i32] + [vp] * 14 + [sz, vp]
        for n in ("moe_select", "moe_route_scored", "moe_route_backward", "moe_pack_weights_fourbit",
                  "moe_quantize_weights_fourbit", "moe_gemm_fourbit", "moe_expert_gemm_fourbit"):
            getattr(L, n).restype = i32
        for n in ("moe_expert_gemm_train", "moe_expert_gemm_backward", "moe_combine_backward",
                  "moe_quantize_rows", "moe_pack_weights", "moe_quantize_weights",
                  "moe_gemm_quantized", "moe_expert_gemm_quantized"):
            getattr(L, n).restype = i32
        for n in ("moe_route", "moe_dispatch", "moe_expert_gemm", "moe_combine", "moe_layer",
                  "moe_dispatch_padded", "moe_expert_gemm_padded", "moe_gemm_signal",
                  "moe_tile_forward", "moe_dispatch_noalloc"):
            getattr(L, n).restype = i32
        _lib = L
    return _lib


def _check(st: int):
    if st != MOE_OK:
        raise MoeError(st, lib().moe_last_error().decode())


def _fits(bits: int, what: str) -> None:
    """``bits``: sizes or-ed together.  ctypes would pass them modulo 2^32; small
    negative ones are the library's to refuse."""
    if not -(1 << 31) <= bits < 1 << 31:
        raise ValueError(f"{what} does not fit 32 bits")


@dataclass(frozen=True)
class Spec:
    """Problem description (mirrors moe_problem_t)."""
    T: int
    d: int
    E: int
    k: int
    f: int
    expert_lo: int
    n_local: int
    dtype: str  # "bf16" or "f32"
    flags: int = 0

    @property
    def rows_max(self) -> int:
        return self.T * min(self.k, self.n_local)

    def c(self) -> Problem:
        T, d, E, k, f, lo, n = self.T, self.d, self.E, self.k, self.f, self.expert_lo, self.n_local
        if (T | d | E | k | f | lo | n) >> 31:
            _fits(T | d | E | k | f | lo | n, "a size of the problem")
        return Problem(T, d, E, k, f, lo, n, MOE_DTYPE_BF16 if self.dtype == "bf16" else MOE_DTYPE_F32, self.flags)

    def ref(self):
        """The C structure by reference, made once: the fields of a Spec do not change."""
        r = self.__dict__.get("_ref")
        if r is None:
            r = ctypes.byref(self.c())
            object.__setattr__(self, "_ref", r)
        return r

    def __reduce__(self):   # copies and pickles without the reference
        return Spec, (self.T, self.d, self.E, self.k, self.f, self.expert_lo, self.n_local, self.dtype, self.flags)

    @staticmethod
    def of(w, flags: int = 0) -> "Spec":
        """From any object with T, d, E, k, f, expert_lo, n_local, dtype fields."""
        return Spec(w.T, w.d, w.E, w.k, w.f, w.expert_lo, w.n_local, w.dtype, flags)


@dataclass(frozen=True)
class Gate:
    """How tokens choose experts from their logits (mirrors moe_gate_t): ``score``
    "softmax" or "sigmoid"; of ``groups`` groups of neighbouring experts the
    ``topk_groups`` best stay, a group's value being the sum of its ``group_top`` (1 or
    2) best experts'; ``renorm``: a token's weights sum to ``scale``."""
    score: str = "softmax"
    groups: int = 1
    topk_groups: int = 1
    group_top: int = 1
    renorm: bool = True
    scale: float = 1.0

    def c(self) -> GateRule:
        if self.score not in ("softmax", "sigmoid"):
            raise ValueError(f"score: expected 'softmax' or 'sigmoid', got {self.score!r}")
        for v in (self.groups, self.topk_groups, self.group_top):
            _fits(v, "a size of the gate")
        return GateRule(MOE_SCORE_SIGMOID if self.score == "sigmoid" else MOE_SCORE_SOFTMAX, self.groups,
                        self.topk_groups, self.group_top, int(bool(self.renorm)), self.scale)

    def ref(self):
        """The C structure by reference, made once: the fields of a Gate do not change."""
        r = self.__dict__.get("_ref")
        if r is None:
            r = ctypes.byref(self.c())
            object.__setattr__(self, "_ref", r)
        return r

    def __reduce__(self):   # copies and pickles without the reference
        return Gate, (self.score, self.groups, self.topk_groups, self.group_top, self.renorm, self.scale)


def workspace_bytes(p: Spec, call: int = MOE_CALL_LAYER) -> int:
    n = lib().moe_workspace_bytes(p.ref(), call)
    if n == 0 and lib().moe_last_error():
        raise MoeError(MOE_ERR_INVALID_ARG, lib().moe_last_error().decode())
    return int(n)


# ---------------------------------------------------------------------------
# torch helpers (device memory and streams only)
# ---------------------------------------------------------------------------
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dt(p: Spec):
    t = _torch()
    return t.bfloat16 if p.dtype == "bf16" else t.float32


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    t = _torch()
    # what torch.cuda.current_stream().cuda_stream gives, without the Stream object
    return t._C._cuda_getCurrentRawStream(t._C._cuda_getDevice())


def _need(t, shape, dtype, name):
    torch = _torch()
    if t is None:
        raise ValueError(f"{name} is required")
    if t.shape != shape and tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device tensor")
    return t


def _current() -> int:
    """The current device; without any, a number that no tensor has."""
    try:
        return _torch()._C._cuda_getDevice()
    except RuntimeError:
        return -2


def _at(cur, t, shape, dtype, name) -> int:
    """Address of a tensor that ``_need`` accepts and that lies on the current
    device ``cur``, on whose stream the call runs."""
    if t is not None and t.get_device() == cur and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _need(t, shape, dtype, name)
    raise ValueError(f"{name} is on device {t.get_device()}, the current device is {cur}")


def _stream_at(cur, stream) -> int:
    if stream is None:
        # what torch.cuda.current_stream().cuda_stream gives, without the Stream object
        return _torch()._C._cuda_getCurrentRawStream(cur)
    if stream.device_index != cur:
        raise ValueError(f"the stream is on device {stream.device_index}, the current device is {cur}")
    return stream.cuda_stream


def _workspace_at(cur, p, call, workspace, stream):
    """(tensor, address, bytes) of the given workspace or of a new one."""
    if workspace is None:
        with _alloc_on(stream):
            workspace = alloc_workspace(p, call, f"cuda:{cur}")
        if workspace is None:
            return None, None, 0
    if workspace.get_device() != cur:
        raise ValueError(f"workspace is on device {workspace.get_device()}, the current device is {cur}")
    return workspace, workspace.data_ptr(), workspace.numel()


_here_and_now = contextlib.nullcontext()


def _alloc_on(stream):
    """Context for what a call with ``stream=`` allocates: on that stream, so that
    fills come before the call's kernels there and memory given back meets only
    later work there."""
    return _here_and_now if stream is None else _torch().cuda.stream(stream)


def alloc_workspace(p: Spec, call: int = MOE_CALL_LAYER, device="cuda"):
    torch = _torch()
    n = workspace_bytes(p, call)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device) if n else None


# ---------------------------------------------------------------------------
# the five calls
# ---------------------------------------------------------------------------
def route(p: Spec, x, w_gate, bias=None, want_logits: bool = False, workspace=None, stream=None,
          out=None):
    torch = _torch()
    dt = _dt(p)
    _need(x, (p.T, p.d), dt, "x")
    _need(w_gate, (p.d, p.E), dt, "w_gate")
    if bias is not None:
        _need(bias, (p.E,), torch.float32, "bias")
    dev = x.device
    idx = torch.empty((p.T, p.k), dtype=torch.int32, device=dev) if out is None else out[0]
    w = torch.empty((p.T, p.k), dtype=torch.float32, device=dev) if out is None else out[1]
    logits = torch.empty((p.T, p.E), dtype=torch.float32, device=dev) if want_logits else None
    ws = workspace if workspace is not None else alloc_workspace(p, MOE_CALL_ROUTE, dev)
    pc = p.c()
    _check(lib().moe_route(ctypes.byref(pc), _ptr(x), _ptr(w_gate), _ptr(bias), _ptr(logits),
                           _ptr(idx), _ptr(w), _ptr(ws), 0 if ws is None else ws.numel(),
                           _stream(stream)))
    return (idx, w, logits) if want_logits else (idx, w)


def _dispatch_out(p: Spec, topk_idx, x, out):
    torch = _torch()
    dt = _dt(p)
    _need(topk_idx, (p.T, p.k), torch.int32, "topk_idx")
    _need(x, (p.T, p.d), dt, "x")
    dev = x.device
    o = out if out is not None else {
        "counts_all": torch.empty(p.E, dtype=torch.int32, device=dev),
        "offsets": torch.empty(p.n_local + 1, dtype=torch.int32, device=dev),
        "perm": torch.full((p.rows_max,), -7, dtype=torch.int32, device=dev),
        "inv": torch.empty(p.T * p.k, dtype=torch.int32, device=dev),
        "x_packed": torch.zeros((p.rows_max, p.d), dtype=dt, device=dev),
    }
    _need(o["counts_all"], (p.E,), torch.int32, "counts_all")
    _need(o["offsets"], (p.n_local + 1,), torch.int32, "offsets")
    _need(o["perm"], (p.rows_max,), torch.int32, "perm")
    _need(o["inv"], (p.T * p.k,), torch.int32, "inv")
    _need(o["x_packed"], (p.rows_max, p.d), dt, "x_packed")
    return o


def dispatch(p: Spec, topk_idx, x, workspace=None, stream=None, out=None) -> Dict[str, object]:
    """Returns counts_all, offsets, perm, inv, x_packed.  Fresh outputs are
    pre-filled (perm with -7, x_packed with 0) so that untouched rows are
    visible; ``out`` (a dict of the same tensors) is written in place."""
    o = _dispatch_out(p, topk_idx, x, out)
    ws = workspace if workspace is not None else alloc_workspace(p, MOE_CALL_DISPATCH, x.device)
    pc = p.c()
    _check(lib().moe_dispatch(ctypes.byref(pc), _ptr(topk_idx), _ptr(x), _ptr(o["counts_all"]),
                              _ptr(o["offsets"]), _ptr(o["perm"]), _ptr(o["inv"]),
                              _ptr(o["x_packed"]), _ptr(ws), 0 if ws is None else ws.numel(),
                              _stream(stream)))
    return o


def dispatch_noalloc(p: Spec, topk_idx, x, stream=None, out=None) -> Dict[str, object]:
    """moe_dispatch_noalloc: the same outputs as ``dispatch`` with no
    workspace (the library's static per-device scratch; calls that overlap on
    one device race)."""
    o = _dispatch_out(p, topk_idx, x, out)
    pc = p.c()
    _check(lib().moe_dispatch_noalloc(ctypes.byref(pc), _ptr(topk_idx), _ptr(x),
                                      _ptr(o["counts_all"]), _ptr(o["offsets"]), _ptr(o["perm"]),
                                      _ptr(o["inv"]), _ptr(o["x_packed"]), _stream(stream)))
    return o


def expert_gemm(p: Spec, x_packed, offsets, w1, w3, w2, workspace=None, stream=None, out=None):
    torch = _torch()
    dt = _dt(p)
    _need(x_packed, (p.rows_max, p.d), dt, "x_packed")
    _need(offsets, (p.n_local + 1,), torch.int32, "offsets")
    _need(w1, (p.n_local, p.d, p.f), dt, "w1")
    _need(w3, (p.n_local, p.d, p.f), dt, "w3")
    _need(w2, (p.n_local, p.f, p.d), dt, "w2")
    dev = x_packed.device
    if out is None:
        h = torch.zeros((p.rows_max, p.f), dtype=dt, device=dev)
        yp = torch.zeros((p.rows_max, p.d), dtype=dt, device=dev)
    else:
        h, yp = out
    ws = workspace if workspace is not None else alloc_workspace(p, MOE_CALL_EXPERT_GEMM, dev)
    pc = p.c()
    _check(lib().moe_expert_gemm(ctypes.byref(pc), _ptr(x_packed), _ptr(offsets), _ptr(w1),
                                 _ptr(w3), _ptr(w2), _ptr(h), _ptr(yp), _ptr(ws),
                                 0 if ws is None else ws.numel(), _stream(stream)))
    return h, yp


def combine(p: Spec, y_packed, inv, topk_w, stream=None, out=None, rows: Optional[int] = None):
    """``rows``: rows of y_packed (default rows_max; n_local * capacity for
    the padded layout).  ``topk_w=None`` sums the rows unweighted."""
    torch = _torch()
    dt = _dt(p)
    _need(y_packed, (p.rows_max if rows is None else rows, p.d), dt, "y_packed")
    _need(inv, (p.T * p.k,), torch.int32, "inv")
    if topk_w is not None:
        _need(topk_w, (p.T, p.k), torch.float32, "topk_w")
    y = torch.empty((p.T, p.d), dtype=dt, device=y_packed.device) if out is None else out
    pc = p.c()
    _check(lib().moe_combine(ctypes.byref(pc), _ptr(y_packed), _ptr(inv), _ptr(topk_w), _ptr(y),
                             _stream(stream)))
    return y


def dispatch_padded(p: Spec, capacity: int, topk_idx, x, workspace=None, stream=None,
                    out=None) -> Dict[str, object]:
    """Padded fixed-capacity dispatch: n_local * capacity rows.  Fresh
    outputs are pre-filled (perm with -7, x_packed with ones) so that
    rows the call fails to write are visible."""
    torch = _torch()
    dt = _dt(p)
    _need(topk_idx, (p.T, p.k), torch.int32, "topk_idx")
    _need(x, (p.T, p.d), dt, "x")
    rows = p.n_local * int(capacity)
    dev = x.device
    o = out if out is not None else {
        "counts_all": torch.empty(p.E, dtype=torch.int32, device=dev),
        "offsets": torch.empty(p.n_local + 1, dtype=torch.int32, device=dev),
        "perm": torch.full((rows,), -7, dtype=torch.int32, device=dev),
        "inv": torch.empty(p.T * p.k, dtype=torch.int32, device=dev),
        "x_packed": torch.ones((rows, p.d), dtype=dt, device=dev),
    }
    _need(o["counts_all"], (p.E,), torch.int32, "counts_all")
    _need(o["offsets"], (p.n_local + 1,), torch.int32, "offsets")
    _need(o["perm"], (rows,), torch.int32, "perm")
    _need(o["inv"], (p.T * p.k,), torch.int32, "inv")
    _need(o["x_packed"], (rows, p.d), dt, "x_packed")
    ws = workspace if workspace is not None else alloc_workspace(p, MOE_CALL_DISPATCH_PADDED, dev)
    pc = p.c()
    _check(lib().moe_dispatch_padded(ctypes.byref(pc), int(capacity), _ptr(topk_idx), _ptr(x),
                                     _ptr(o["counts_all"]), _ptr(o["offsets"]), _ptr(o["perm"]),
                                     _ptr(o["inv"]), _ptr(o["x_packed"]), _ptr(ws),
                                     0 if ws is None else ws.numel(), _stream(stream)))
    return o


def expert_gemm_padded(p: Spec, capacity: int, x_packed, offsets, w1, w3, w2, workspace=None,
                       stream=None, out=None):
    torch = _torch()
    dt = _dt(p)
    rows = p.n_local * int(capacity)
    _need(x_packed, (rows, p.d), dt, "x_packed")
    _need(offsets, (p.n_local + 1,), torch.int32, "offsets")
    _need(w1, (p.n_local, p.d, p.f), dt, "w1")
    _need(w3, (p.n_local, p.d, p.f), dt, "w3")
    _need(w2, (p.n_local, p.f, p.d), dt, "w2")
    dev = x_packed.device
    if out is None:
        h = torch.ones((rows, p.f), dtype=dt, device=dev)
        yp = torch.ones((rows, p.d), dtype=dt, device=dev)
    else:
        h, yp = out
    ws = workspace if workspace is not None else alloc_workspace(p, MOE_CALL_EXPERT_GEMM_PADDED, dev)
    pc = p.c()
    _check(lib().moe_expert_gemm_padded(ctypes.byref(pc), int(capacity), _ptr(x_packed),
                                        _ptr(offsets), _ptr(w1), _ptr(w3), _ptr(w2), _ptr(h),
                                        _ptr(yp), _ptr(ws), 0 if ws is None else ws.numel(),
                                        _stream(stream)))
    return h, yp


# ---------------------------------------------------------------------------
# training
# ---------------------------------------------------------------------------
def expert_gemm_train(p: Spec, x_packed, offsets, w1, w3, w2, stream=None, out=None):
    """``expert_gemm`` that also returns the unactivated products the backward
    pass reads: (g, u, h, y_packed).  ``out``: these four, written in place."""
    torch = _torch()
    dt, cur, rows = _dt(p), _current(), p.rows_max
    wide, tall, up = (rows, p.d), (rows, p.f), (p.n_local, p.d, p.f)
    ins = (_at(cur, x_packed, wide, dt, "x_packed"), _at(cur, offsets, (p.n_local + 1,), torch.int32, "offsets"),
           _at(cur, w1, up, dt, "w1"), _at(cur, w3, up, dt, "w3"), _at(cur, w2, (p.n_local, p.f, p.d), dt, "w2"))
    if out is None:
        with _alloc_on(stream):
            out = tuple(torch.zeros(n, dtype=dt, device=x_packed.device) for n in (tall, tall, tall, wide))
    g, u, h, yp = out
    _check(lib().moe_expert_gemm_train(p.ref(), *ins, _at(cur, g, tall, dt, "g"), _at(cur, u, tall, dt, "u"),
                                       _at(cur, h, tall, dt, "h"), _at(cur, yp, wide, dt, "y_packed"),
                                       _stream_at(cur, stream)))
    return g, u, h, yp


def expert_gemm_backward(p: Spec, x_packed, offsets, w1, w3, w2, g, u, h, dy_packed, workspace=None,
                         stream=None, out=None):
    """Gradients (dx_packed, dw1, dw3, dw2) of ``expert_gemm_train``.  ``out``:
    these four, written in place; a None among them is not computed."""
    torch = _torch()
    dt, cur, rows = _dt(p), _current(), p.rows_max
    wide, tall, up, down = (rows, p.d), (rows, p.f), (p.n_local, p.d, p.f), (p.n_local, p.f, p.d)
    ins = (_at(cur, x_packed, wide, dt, "x_packed"), _at(cur, offsets, (p.n_local + 1,), torch.int32, "offsets"),
           _at(cur, w1, up, dt, "w1"), _at(cur, w3, up, dt, "w3"), _at(cur, w2, down, dt, "w2"),
           _at(cur, g, tall, dt, "g"), _at(cur, u, tall, dt, "u"), _at(cur, h, tall, dt, "h"),
           _at(cur, dy_packed, wide, dt, "dy_packed"))
    if out is None:
        with _alloc_on(stream):
            out = (torch.zeros(wide, dtype=dt, device=x_packed.device), torch.empty_like(w1),
                   torch.empty_like(w3), torch.empty_like(w2))
    dx, dw1, dw3, dw2 = out
    outs = (None if dx is None else _at(cur, dx, wide, dt, "dx_packed"),
            None if dw1 is None else _at(cur, dw1, up, dt, "dw1"),
            None if dw3 is None else _at(cur, dw3, up, dt, "dw3"),
            None if dw2 is None else _at(cur, dw2, down, dt, "dw2"))
    ws, at, size = _workspace_at(cur, p, MOE_CALL_EXPERT_GEMM_BACKWARD, workspace, stream)
    _check(lib().moe_expert_gemm_backward(p.ref(), *ins, *outs, at, size, _stream_at(cur, stream)))
    return dx, dw1, dw3, dw2


def combine_backward(p: Spec, dy, y_packed, inv, topk_w, stream=None, out=None,
                     rows: Optional[int] = None):
    """Gradients (dy_packed, dtopk_w) of ``combine``.  ``rows`` as there;
    ``topk_w=None``: unit weights.  ``out``: the two, written in place; with
    dtopk_w None it is not computed and ``y_packed`` may be None."""
    torch = _torch()
    dt, cur = _dt(p), _current()
    packed, slots = (p.rows_max if rows is None else rows, p.d), (p.T, p.k)
    pdy = _at(cur, dy, (p.T, p.d), dt, "dy")
    if out is None:
        with _alloc_on(stream):
            out = (torch.zeros(packed, dtype=dt, device=dy.device),
                   torch.empty(slots, dtype=torch.float32, device=dy.device))
    dyp, dw = out
    _check(lib().moe_combine_backward(
        p.ref(), pdy, None if dw is None and y_packed is None else _at(cur, y_packed, packed, dt, "y_packed"),
        _at(cur, inv, (p.T * p.k,), torch.int32, "inv"),
        None if topk_w is None else _at(cur, topk_w, slots, torch.float32, "topk_w"),
        _at(cur, dyp, packed, dt, "dy_packed"),
        None if dw is None else _at(cur, dw, slots, torch.float32, "dtopk_w"), _stream_at(cur, stream)))
    return dyp, dw


# ---------------------------------------------------------------------------
# 8-bit weights and activations
# ---------------------------------------------------------------------------
def _dtype_code(t, name):
    torch = _torch()
    if t.dtype is torch.bfloat16:
        return MOE_DTYPE_BF16
    if t.dtype is torch.float32:
        return MOE_DTYPE_F32
    raise ValueError(f"{name}: expected torch.bfloat16 or torch.float32, got {t.dtype}")


def quantize_rows(x, stream=None, out=None):
    """(q int8, scale fp32) of the rows of x [rows, K] (bf16 or fp32):
    scale = max|x| / 127, q = rint(x * (127 * (1 / max|x|)))."""
    torch = _torch()
    code, cur = _dtype_code(x, "x"), _current()
    rows, K = x.shape
    _fits(K, "a row of x")
    px = _at(cur, x, (rows, K), x.dtype, "x")
    if out is None:
        with _alloc_on(stream):
            out = (torch.empty((rows, K), dtype=torch.int8, device=x.device),
                   torch.empty((rows,), dtype=torch.float32, device=x.device))
    q, s = out
    _check(lib().moe_quantize_rows(rows, K, code, px, _at(cur, q, (rows, K), torch.int8, "q"),
                                   _at(cur, s, (rows,), torch.float32, "scale"), _stream_at(cur, stream)))
    return q, s


def packed_weights_shape(K: int, N: int):
    """Shape of one packed [K, N] matrix: (N/16, K/64, 4, 16, 16), rounded up."""
    return (-(-N // 16), -(-K // 64), 4, 16, 16)


def packed_weights_bytes(n: int, K: int, N: int) -> int:
    _fits(int(n) | int(K) | int(N), "a size of the weights")
    b = int(lib().moe_packed_weights_bytes(int(n), int(K), int(N)))
    if b == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, lib().moe_last_error().decode())
    return b


def _packed_out(w, out, stream):
    torch = _torch()
    lead, K, N = tuple(w.shape[:-2]), w.shape[-2], w.shape[-1]
    if len(lead) > 1:
        raise ValueError(f"w: expected [n, K, N] or [K, N], got {tuple(w.shape)}")
    n = lead[0] if lead else 1
    packed_weights_bytes(n, K, N)
    if out is None:
        with _alloc_on(stream):
            out = torch.empty(lead + packed_weights_shape(K, N), dtype=torch.int8, device=w.device)
    return n, K, N, lead, out


def pack_weights(w, stream=None, out=None):
    """int8 weights [n, K, N] or [K, N] in the order the 8-bit products read."""
    torch = _torch()
    cur = _current()
    n, K, N, lead, packed = _packed_out(w, out, stream)
    _check(lib().moe_pack_weights(n, K, N, _at(cur, w, w.shape, torch.int8, "w"),
                                  _at(cur, packed, lead + packed_weights_shape(K, N), torch.int8, "packed"),
                                  _stream_at(cur, stream)))
    return packed


def quantize_weights(w, stream=None, out=None):
    """(packed, scale) of bf16 or fp32 weights [n, K, N] or [K, N], one scale
    per output channel."""
    torch = _torch()
    code, cur = _dtype_code(w, "w"), _current()
    n, K, N, lead, packed = _packed_out(w, None if out is None else out[0], stream)
    pw = _at(cur, w, w.shape, w.dtype, "w")
    with _alloc_on(stream):
        s = torch.empty(lead + (N,), dtype=torch.float32, device=w.device) if out is None else out[1]
    _check(lib().moe_quantize_weights(
        n, K, N, code, pw, _at(cur, packed, lead + packed_weights_shape(K, N), torch.int8, "packed"),
        _at(cur, s, lead + (N,), torch.float32, "scale"), _stream_at(cur, stream)))
    return packed, s


def gemm_quantized(a, a_scale, packed, b_scale, dtype=None, stream=None, out=None):
    """C = rnd((a b) a_scale b_scale): int8 a [M, K], packed weights of one
    [K, N] matrix, a scale per row and per output channel; ``dtype`` (default
    torch.bfloat16, or that of ``out``) is C's."""
    torch = _torch()
    cur = _current()
    M, K = a.shape
    N = b_scale.shape[0]
    _fits(M | N | K, "a size of the product")
    pa = _at(cur, a, (M, K), torch.int8, "a")
    if out is None:
        with _alloc_on(stream):
            out = torch.empty((M, N), dtype=dtype or torch.bfloat16, device=a.device)
    _check(lib().moe_gemm_quantized(
        M, N, K, pa, _at(cur, a_scale, (M,), torch.float32, "a_scale"),
        _at(cur, packed, packed_weights_shape(K, N), torch.int8, "packed"),
        _at(cur, b_scale, (N,), torch.float32, "b_scale"), _at(cur, out, (M, N), dtype or out.dtype, "out"),
        _dtype_code(out, "out"), _stream_at(cur, stream)))
    return out


def expert_gemm_quantized(p: Spec, x_packed, offsets, w1, s1, w3, s3, w2, s2, workspace=None,
                          stream=None, out=None):
    """``expert_gemm`` with packed 8-bit weights [n_local, ...] and their channel
    scales, and rows quantised on the way: (h, y_packed)."""
    torch = _torch()
    dt, cur, n = _dt(p), _current(), (p.n_local,)
    wide, tall = (p.rows_max, p.d), (p.rows_max, p.f)
    up, down = n + packed_weights_shape(p.d, p.f), n + packed_weights_shape(p.f, p.d)
    f32, i8 = torch.float32, torch.int8
    ins = (_at(cur, x_packed, wide, dt, "x_packed"), _at(cur, offsets, (p.n_local + 1,), torch.int32, "offsets"),
           _at(cur, w1, up, i8, "w1"), _at(cur, s1, n + (p.f,), f32, "s1"),
           _at(cur, w3, up, i8, "w3"), _at(cur, s3, n + (p.f,), f32, "s3"),
           _at(cur, w2, down, i8, "w2"), _at(cur, s2, n + (p.d,), f32, "s2"))
    if out is None:
        with _alloc_on(stream):
            out = tuple(torch.zeros(v, dtype=dt, device=x_packed.device) for v in (tall, wide))
    h, yp = out
    outs = (_at(cur, h, tall, dt, "h"), _at(cur, yp, wide, dt, "y_packed"))
    ws, at, size = _workspace_at(cur, p, MOE_CALL_EXPERT_GEMM_QUANTIZED, workspace, stream)
    _check(lib().moe_expert_gemm_quantized(p.ref(), *ins, *outs, at, size, _stream_at(cur, stream)))
    return h, yp


# ---------------------------------------------------------------------------
# scored routing
# ---------------------------------------------------------------------------
def _choice_out(cur, p, like, out, stream):
    """(topk_idx, topk_w) of ``out``, or new ones beside ``like``, and their addresses."""
    torch, slots = _torch(), (p.T, p.k)
    if out is None:
        with _alloc_on(stream):
            idx, w = like.new_empty(slots, dtype=torch.int32), like.new_empty(slots, dtype=torch.float32)
        return idx, w, idx.data_ptr(), w.data_ptr()
    idx, w = out
    return idx, w, _at(cur, idx, slots, torch.int32, "topk_idx"), _at(cur, w, slots, torch.float32, "topk_w")


def select(p: Spec, gate: Gate, logits, balance=None, stream=None, out=None):
    """(topk_idx, topk_w) from fp32 logits [T, E] by the rule of ``gate``; ``balance`` [E]
    is added to the scores for the choice alone.  ``out``: the two, written in place."""
    torch = _torch()
    cur, slots, f32 = _current(), (p.T, p.k), torch.float32
    pl = _at(cur, logits, (p.T, p.E), f32, "logits")
    pb = None if balance is None else _at(cur, balance, (p.E,), f32, "balance")
    idx, w, pi, pw = _choice_out(cur, p, logits, out, stream)
    _check(lib().moe_select(p.ref(), gate.ref(), pl, pb, pi, pw, _stream_at(cur, stream)))
    return idx, w


def route_scored(p: Spec, gate: Gate, x, w_gate, bias=None, balance=None, want_logits: bool = False,
                 workspace=None, stream=None, out=None):
    """``route`` by the rule of ``gate``: (topk_idx, topk_w[, logits]).  ``bias`` is part
    of the logits, ``balance`` of the choice alone."""
    torch = _torch()
    dt, cur, slots, f32 = _dt(p), _current(), (p.T, p.k), torch.float32
    px, pw = _at(cur, x, (p.T, p.d), dt, "x"), _at(cur, w_gate, (p.d, p.E), dt, "w_gate")
    pb = None if bias is None else _at(cur, bias, (p.E,), f32, "bias")
    pc = None if balance is None else _at(cur, balance, (p.E,), f32, "balance")
    idx, w, pi, pv = _choice_out(cur, p, x, out, stream)
    with _alloc_on(stream):
        logits = torch.empty((p.T, p.E), dtype=f32, device=x.device) if want_logits else None
    ws, at, size = _workspace_at(cur, p, MOE_CALL_ROUTE_SCORED, workspace, stream)
    _check(lib().moe_route_scored(p.ref(), gate.ref(), px, pw, pb, pc, _ptr(logits),
                                  pi, pv, at, size, _stream_at(cur, stream)))
    return (idx, w, logits) if want_logits else (idx, w)


def route_backward(p: Spec, gate: Gate, x, w_gate, logits, topk_idx, dtopk_w, dx_add=None, workspace=None,
                   stream=None, out=None):
    """Gradients (dlogits, dx, dw_gate, dbias) of ``route_scored`` and ``select``;
    ``dx_add`` is added to dx.  ``out``: these four, written in place; a None among them
    is not computed (without dx, ``w_gate`` may be None; without dw_gate, ``x``)."""
    torch = _torch()
    dt, cur, slots, f32 = _dt(p), _current(), (p.T, p.k), torch.float32
    wide, gates, all_e = (p.T, p.d), (p.d, p.E), (p.T, p.E)
    pl = _at(cur, logits, all_e, f32, "logits")
    ins = (_at(cur, topk_idx, slots, torch.int32, "topk_idx"), _at(cur, dtopk_w, slots, f32, "dtopk_w"),
           None if dx_add is None else _at(cur, dx_add, wide, dt, "dx_add"))
    if out is None:
        px, pw = _at(cur, x, wide, dt, "x"), _at(cur, w_gate, gates, dt, "w_gate")
        with _alloc_on(stream):   # of the inputs' sizes, which were checked
            dl, dx, dwg, db = torch.empty_like(logits), torch.empty_like(x), torch.empty_like(w_gate), logits.new_empty((p.E,))
        outs = (dl.data_ptr(), dx.data_ptr(), dwg.data_ptr(), db.data_ptr())
    else:
        dl, dx, dwg, db = out
        px = None if x is None and dwg is None else _at(cur, x, wide, dt, "x")
        pw = None if w_gate is None and dx is None else _at(cur, w_gate, gates, dt, "w_gate")
        outs = (None if dl is None else _at(cur, dl, all_e, f32, "dlogits"),
                None if dx is None else _at(cur, dx, wide, dt, "dx"),
                None if dwg is None else _at(cur, dwg, gates, dt, "dw_gate"),
                None if db is None else _at(cur, db, (p.E,), f32, "dbias"))
    ws, at, size = _workspace_at(cur, p, MOE_CALL_ROUTE_BACKWARD, workspace, stream)
    _check(lib().moe_route_backward(p.ref(), gate.ref(), px, pw, pl, *ins, *outs, at, size, _stream_at(cur, stream)))
    return dl, dx, dwg, db


# ---------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------
def packed_weights_4bit_shape(K: int, N: int):
    """Shape of one packed [K, N] matrix of int32 words: (N/16, K/128, 64, 4), rounded up."""
    return (-(-N // 16), -(-K // 128), 64, 4)


def packed_weights_4bit_bytes(n: int, K: int, N: int) -> int:
    _fits(int(n) | int(K) | int(N), "a size of the weights")
    b = int(lib().moe_packed_weights_fourbit_bytes(int(n), int(K), int(N)))
    if b == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, lib().moe_last_error().decode())
    return b


def _groups(K: int, group: int) -> int:
    if group not in (32, 64, 128):
        raise ValueError(f"group: expected 32, 64 or 128, got {group}")
    return -(-K // group)


def _matrices(w):
    lead, K, N = tuple(w.shape[:-2]), w.shape[-2], w.shape[-1]
    if len(lead) > 1:
        raise ValueError(f"w: expected [n, K, N] or [K, N], got {tuple(w.shape)}")
    n = lead[0] if lead else 1
    packed_weights_4bit_bytes(n, K, N)
    return n, K, N, lead


def pack_weights_4bit(q, stream=None, out=None):
    """uint8 values 0 .. 15 [n, K, N] or [K, N] in the order the 4-bit products read."""
    torch = _torch()
    cur = _current()
    n, K, N, lead = _matrices(q)
    shape = lead + packed_weights_4bit_shape(K, N)
    pq = _at(cur, q, q.shape, torch.uint8, "q")
    if out is None:
        with _alloc_on(stream):
            out = torch.empty(shape, dtype=torch.int32, device=q.device)
    _check(lib().moe_pack_weights_fourbit(n, K, N, pq, _at(cur, out, shape, torch.int32, "packed"),
                                       _stream_at(cur, stream)))
    return out


def quantize_weights_4bit(w, group: int = 128, zero: bool = False, stream=None, out=None):
    """(packed, scale, zero) of bf16 or fp32 weights [n, K, N] or [K, N]: a bf16 scale, and
    with ``zero`` a zero point (else None: 8), for each group of K in each column.  ``out``:
    the three, written in place; zero points among them only with ``zero``."""
    torch = _torch()
    if out is not None and out[2] is not None and not zero:
        raise ValueError("out has zero points, which are not made without zero=True")
    code, cur = _dtype_code(w, "w"), _current()
    n, K, N, lead = _matrices(w)
    shape, rows = lead + packed_weights_4bit_shape(K, N), lead + (_groups(K, group), N)
    pw = _at(cur, w, w.shape, w.dtype, "w")
    if out is None:
        with _alloc_on(stream):
            out = (torch.empty(shape, dtype=torch.int32, device=w.device),
                   torch.empty(rows, dtype=torch.bfloat16, device=w.device),
                   torch.empty(rows, dtype=torch.uint8, device=w.device) if zero else None)
    packed, s, z = out
    _check(lib().moe_quantize_weights_fourbit(
        n, K, N, group, code, pw, _at(cur, packed, shape, torch.int32, "packed"), _at(cur, s, rows, torch.bfloat16, "scale"),
        _at(cur, z, rows, torch.uint8, "zero") if zero else None, _stream_at(cur, stream)))
    return packed, s, z if zero else None


def gemm_4bit_workspace_bytes(M: int, N: int, K: int) -> int:
    """Bytes of scratch of ``gemm_4bit`` (0 for few rows)."""
    _fits(M | N | K, "a size of the product")
    n = int(lib().moe_gemm_fourbit_workspace_bytes(M, N, K))
    if n == 0 and lib().moe_last_error():
        raise MoeError(MOE_ERR_INVALID_ARG, lib().moe_last_error().decode())
    return n


def gemm_4bit(a, packed, scale, zero=None, group: int = 128, dtype=None, workspace=None, stream=None, out=None):
    """C = rnd(a W): bf16 a [M, K], packed 4-bit weights of one [K, N] matrix with their
    scales and zero points (None: 8); ``dtype`` (default torch.bfloat16, or that of
    ``out``) is C's."""
    torch = _torch()
    cur = _current()
    M, K = a.shape
    N = scale.shape[-1]
    _fits(M | N | K, "a size of the product")
    rows = (_groups(K, group), N)
    pa = _at(cur, a, (M, K), torch.bfloat16, "a")
    if out is None:
        with _alloc_on(stream):
            out = a.new_empty((M, N), dtype=dtype or torch.bfloat16)
        po = out.data_ptr()
    else:
        po = _at(cur, out, (M, N), dtype or out.dtype, "out")
    ins = (_at(cur, packed, packed_weights_4bit_shape(K, N), torch.int32, "packed"),
           _at(cur, scale, rows, torch.bfloat16, "scale"),
           None if zero is None else _at(cur, zero, rows, torch.uint8, "zero"),
           po, _dtype_code(out, "out"))
    if workspace is None:
        need = gemm_4bit_workspace_bytes(M, N, K)
        if need:
            with _alloc_on(stream):
                workspace = a.new_empty(need, dtype=torch.uint8)
    elif workspace.get_device() != cur:
        raise ValueError(f"workspace is on device {workspace.get_device()}, the current device is {cur}")
    _check(lib().moe_gemm_fourbit(M, N, K, group, pa, *ins, _ptr(workspace),
                                  0 if workspace is None else workspace.numel(), _stream_at(cur, stream)))
    return out


def expert_gemm_4bit(p: Spec, x_packed, offsets, w1, s1, z1, w3, s3, z3, w2, s2, z2, group: int = 128,
                     workspace=None, stream=None, out=None):
    """``expert_gemm`` with packed 4-bit weights [n_local, ...], their scales and zero
    points (each None or not): (h, y_packed).  Without ``out`` both are made, and zeroed at
    their full size, by each call."""
    torch = _torch()
    dt, cur, n = _dt(p), _current(), (p.n_local,)
    wide, tall, i32, bf, u8 = (p.rows_max, p.d), (p.rows_max, p.f), torch.int32, torch.bfloat16, torch.uint8
    up, down = n + packed_weights_4bit_shape(p.d, p.f), n + packed_weights_4bit_shape(p.f, p.d)
    gu, gd = n + (_groups(p.d, group), p.f), n + (_groups(p.f, group), p.d)
    ins = (_at(cur, x_packed, wide, dt, "x_packed"), _at(cur, offsets, (p.n_local + 1,), i32, "offsets"),
           _at(cur, w1, up, i32, "w1"), _at(cur, s1, gu, bf, "s1"), None if z1 is None else _at(cur, z1, gu, u8, "z1"),
           _at(cur, w3, up, i32, "w3"), _at(cur, s3, gu, bf, "s3"), None if z3 is None else _at(cur, z3, gu, u8, "z3"),
           _at(cur, w2, down, i32, "w2"), _at(cur, s2, gd, bf, "s2"), None if z2 is None else _at(cur, z2, gd, u8, "z2"))
    if out is None:
        with _alloc_on(stream):
            out = tuple(torch.zeros(v, dtype=dt, device=x_packed.device) for v in (tall, wide))
    h, yp = out
    outs = (_at(cur, h, tall, dt, "h"), _at(cur, yp, wide, dt, "y_packed"))
    ws, at, size = _workspace_at(cur, p, MOE_CALL_EXPERT_GEMM_FOURBIT, workspace, stream)
    _check(lib().moe_expert_gemm_fourbit(p.ref(), group, *ins, *outs, at, size, _stream_at(cur, stream)))
    return h, yp


def gemm_signal_tiles(M: int, N: int) -> int:
    n = int(lib().moe_gemm_signal_tiles(int(M), int(N)))
    if n <= 0:
        raise MoeError(MOE_ERR_INVALID_ARG, lib().moe_last_error().decode())
    return n


def gemm_signal(A, B, flags, epoch: int, scope: int = MOE_SCOPE_AGENT, stream=None, out=None):
    """C = rnd(A B) (bf16 [M,K] x [K,N]); flags (int32 or uint32 device
    tensor of gemm_signal_tiles(M, N) entries) receive `epoch` per finished
    256 x 256 tile."""
    torch = _torch()
    M, K = A.shape
    N = B.shape[1]
    _need(A, (M, K), torch.bfloat16, "A")
    _need(B, (K, N), torch.bfloat16, "B")
    _need(flags, (gemm_signal_tiles(M, N),), flags.dtype, "flags")
    C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device) if out is None else out
    _need(C, (M, N), torch.bfloat16, "C")
    _check(lib().moe_gemm_signal(M, N, K, _ptr(A), _ptr(B), _ptr(C), _ptr(flags), int(epoch),
                                 int(scope), _stream(stream)))
    return C


def tile_forward(C, dst, flags, epoch: int, spin_limit: int, timeouts, workgroups: int = 4,
                 scope: int = MOE_SCOPE_AGENT, stream=None):
    """Copies each 256 x 256 tile of C to dst once flags[tile] == epoch;
    adds 1 to timeouts[0] per tile whose flag did not arrive in spin_limit polls."""
    torch = _torch()
    M, N = C.shape
    _need(C, (M, N), torch.bfloat16, "C")
    _need(dst, (M, N), torch.bfloat16, "dst")
    _need(flags, (gemm_signal_tiles(M, N),), flags.dtype, "flags")
    _need(timeouts, (1,), timeouts.dtype, "timeouts")
    _check(lib().moe_tile_forward(M, N, _ptr(C), _ptr(dst), _ptr(flags), int(epoch),
                                  int(spin_limit), int(scope), _ptr(timeouts), int(workgroups),
                                  _stream(stream)))
    return dst


def layer_set_gemm_events(before: int, after: int) -> None:
    """The next layer() call on this thread records the two HIP events (raw
    hipEvent_t handles, timing enabled) on its launch stream around its expert
    GEMM."""
    _check(lib().moe_layer_set_gemm_events(ctypes.c_void_p(before or 0), ctypes.c_void_p(after or 0)))


def layer_ws_offset(p: Spec, what: int) -> int:
    """Byte offset of h (MOE_WS_H) or y_packed (MOE_WS_Y_PACKED) inside a
    moe_layer workspace of problem p."""
    pc = p.c()
    n = int(lib().moe_layer_ws_offset(ctypes.byref(pc), int(what)))
    if n == ctypes.c_size_t(-1).value:
        raise MoeError(MOE_ERR_INVALID_ARG, lib().moe_last_error().decode())
    return n


def layer(p: Spec, x, w_gate, bias, w1, w3, w2, routing: bool = False, want_logits: bool = False,
          overlap: bool = False, workspace=None, stream=None, stream2=None, out=None,
          fold_weight: bool = False):
    """The whole layer.  With ``routing`` also returns the routing/dispatch
    tensors; with ``overlap`` runs the two-stream dispatch overlap (needs
    ``stream2``, a torch.cuda.Stream, or creates none and runs one stream);
    with ``fold_weight`` the routing weights scale the expert output rows in
    the down projection and combine sums them unweighted."""
    torch = _torch()
    dt = _dt(p)
    _need(x, (p.T, p.d), dt, "x")
    _need(w_gate, (p.d, p.E), dt, "w_gate")
    if bias is not None:
        _need(bias, (p.E,), torch.float32, "bias")
    _need(w1, (p.n_local, p.d, p.f), dt, "w1")
    _need(w3, (p.n_local, p.d, p.f), dt, "w3")
    _need(w2, (p.n_local, p.f, p.d), dt, "w2")
    dev = x.device
    flags = (p.flags | (MOE_F_WRITE_LOGITS if want_logits else 0) | (MOE_F_OVERLAP if overlap else 0)
             | (MOE_F_FOLD_WEIGHT if fold_weight else 0))
    q = Spec(p.T, p.d, p.E, p.k, p.f, p.expert_lo, p.n_local, p.dtype, flags)
    y = torch.empty((p.T, p.d), dtype=dt, device=dev) if out is None else out
    r = None
    ro = None
    if routing or want_logits:
        r = {
            "topk_idx": torch.empty((p.T, p.k), dtype=torch.int32, device=dev),
            "topk_w": torch.empty((p.T, p.k), dtype=torch.float32, device=dev),
            "counts_all": torch.empty(p.E, dtype=torch.int32, device=dev),
            "offsets": torch.empty(p.n_local + 1, dtype=torch.int32, device=dev),
            "perm": torch.full((p.rows_max,), -7, dtype=torch.int32, device=dev),
            "inv": torch.empty(p.T * p.k, dtype=torch.int32, device=dev),
        }
        if want_logits:
            r["logits"] = torch.empty((p.T, p.E), dtype=torch.float32, device=dev)
        ro = RoutingOut(*[_ptr(r.get(n)) for n in
                          ("topk_idx", "topk_w", "logits", "counts_all", "offsets", "perm", "inv")])
    ws = workspace if workspace is not None else alloc_workspace(q, MOE_CALL_LAYER, dev)
    pc = q.c()
    s2 = _stream(stream2) if (overlap and stream2 is not None) else None
    _check(lib().moe_layer(ctypes.byref(pc), _ptr(x), _ptr(w_gate), _ptr(bias), _ptr(w1), _ptr(w3),
                           _ptr(w2), _ptr(y), ctypes.byref(ro) if ro is not None else None,
                           _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream), s2))
    return (y, r) if r is not None else y

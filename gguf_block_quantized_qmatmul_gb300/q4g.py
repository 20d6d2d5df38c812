"""4-bit weights with group scales, and mixture-of-experts layers: the Python
side of qmm_q4g_* and qmm_moe_* (``include/qmm.h`` states what each computes,
its types, limits and errors).

  q4g_pack(codes, scales, zeros)    lay checkpoint tensors out, once    -> Q4GWeights
  q4g_pack_q4_0(wq, K)              the same from GGUF Q4_0 blocks
  q4g_dequantize(w)                 f32 [experts, N, K]
  q4g_matmul(w, x)                  y = x . W^T
  moe_route(logits, top_k, ...)     experts, weights and sorted slots   -> Route
  moe_gate_up(w, x, route)          silu(x . Wg^T) * (x . Wu^T) of each token's experts
  moe_down(w, h, route)             weighted sum of the experts' second products

Tensors are CUDA tensors; activations are f32, f16 or bf16 with their last
dimension contiguous (rows may be further apart).  Work goes to the current
stream, or to `stream` (temporaries and outputs are then allocated on it).
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from . import _check, _lib

FLOATS = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"max": 0, "top2": 1}


class _Desc(ctypes.Structure):
    """qmm_q4g"""
    _fields_ = [("data", ctypes.c_void_p), ("experts", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("group", ctypes.c_int32), ("paired", ctypes.c_int32)]


class _RouteConfig(ctypes.Structure):
    """qmm_route_config"""
    _fields_ = [("score", ctypes.c_int32), ("top_k", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


class _Routing(ctypes.Structure):
    """qmm_routing"""
    _fields_ = [("ids", ctypes.c_void_p), ("weights", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("order", ctypes.c_void_p),
                ("T", ctypes.c_int64), ("top_k", ctypes.c_int64)]


def declare(lib) -> None:
    """Argument types of this module's entry points."""
    i64, sz, p, i32 = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int
    for name, args, res in (
            ("qmm_q4g_bytes", [i64, i64, i64, i32, i32], sz),
            ("qmm_q4g_pack", [p, p, i32, p, i64, i64, i64, i32, i32, p, p], i32),
            ("qmm_q4g_pack_q4_0", [p, i64, i64, i64, i32, p, p], i32),
            ("qmm_q4g_dequantize", [p, p, p], i32),
            ("qmm_q4g_matmul_workspace", [p, i32, i64], sz),
            ("qmm_q4g_matmul", [p, i32, p, i64, i64, p, p, sz, p], i32),
            ("qmm_moe_route_workspace", [i64, i64, i64], sz),
            ("qmm_moe_route", [p, i32, p, i64, i64, i64, p, p, p, p, p, p, sz, p], i32),
            ("qmm_moe_gate_up_workspace", [p, i32, i64, i64], sz),
            ("qmm_moe_gate_up", [p, i32, p, i64, p, p, p, sz, p], i32),
            ("qmm_moe_down_workspace", [p, i32, i64, i64], sz),
            ("qmm_moe_down", [p, i32, p, i64, p, p, p, sz, p], i32)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _on(stream):
    """The context in which a call with stream=... allocates and launches."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


def _need(ok: bool, text: str) -> None:
    if not ok:
        raise ValueError(text)


class Q4GWeights:
    """Laid-out weights: `data` (uint8) and what they are.  Made by q4g_pack or q4g_pack_q4_0."""

    def __init__(self, data: torch.Tensor, experts: int, N: int, K: int, group: int, gate_up: bool):
        self.data, self.experts, self.N, self.K, self.group, self.gate_up = data, experts, N, K, group, gate_up
        self.device = data.get_device()
        self._desc = _Desc(data.data_ptr(), experts, N, K, group, int(gate_up))
        self._ptr = ctypes.addressof(self._desc)
        self._workspace = {}  # bytes by (call, type, rows, top_k)

    def _workspace_bytes(self, name: str, *args) -> int:
        key = (name,) + args
        n = self._workspace.get(key)
        if n is None:
            if len(self._workspace) > 4096:
                self._workspace.clear()
            n = self._workspace[key] = int(getattr(_lib(), name + "_workspace")(self._ptr, *args))
        return n


class Route(NamedTuple):
    """A routing: ids and weights [T, top_k]; offsets [experts + 1]; order [T top_k], the slots t top_k + j by expert."""
    ids: torch.Tensor
    weights: torch.Tensor
    offsets: Optional[torch.Tensor] = None
    order: Optional[torch.Tensor] = None


def _laid_out(experts, N, K, group, gate_up, device):
    n = int(_lib().qmm_q4g_bytes(experts, N, K, group, int(gate_up)))
    return torch.empty(n, dtype=torch.uint8, device=device)


def q4g_pack(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None, gate_up: bool = False,
             stream=None) -> Q4GWeights:
    """Lay weights out.  codes uint8 [experts, N, K / 2] (even k in the low
    nibble) or [N, K / 2]; scales f16 or bf16 [.., N, K / group]; zeros uint8 of
    that shape or None (8).  gate_up: the first N / 2 rows of an expert are its
    gate rows, the others its up rows (for moe_gate_up)."""
    if codes.dim() == 2:
        codes, scales = codes.unsqueeze(0), scales.unsqueeze(0)
        zeros = None if zeros is None else zeros.unsqueeze(0)
    _need(codes.dim() == 3 and scales.dim() == 3 and codes.shape[:2] == scales.shape[:2], "codes [.., N, K / 2] and scales [.., N, K / group]")
    _need(codes.dtype == torch.uint8 and scales.dtype in (torch.float16, torch.bfloat16), "codes are uint8, scales f16 or bf16")
    _need(zeros is None or (zeros.dtype == torch.uint8 and zeros.shape == scales.shape), "zeros are uint8, shaped as scales")
    E, N, half = codes.shape
    K, groups = 2 * half, scales.shape[2]
    _need(groups > 0 and K % groups == 0, "K is a multiple of the number of groups")
    _need(codes.is_cuda and scales.get_device() == codes.get_device() and (zeros is None or zeros.get_device() == codes.get_device()),
          "tensors are on one CUDA device")
    group = K // groups
    with _on(stream):
        codes, scales = codes.contiguous(), scales.contiguous()
        zeros = None if zeros is None else zeros.contiguous()
        out = _laid_out(E, N, K, group, gate_up, codes.device)
        _check(_lib().qmm_q4g_pack(codes.data_ptr(), scales.data_ptr(), FLOATS[scales.dtype], 0 if zeros is None else zeros.data_ptr(), E, N,
                                   K, group, int(gate_up), out.data_ptr(), _raw_stream(codes.get_device())), "qmm_q4g_pack")
    return Q4GWeights(out, E, N, K, group, gate_up)


def q4g_pack_q4_0(wq: torch.Tensor, K: int, gate_up: bool = False, stream=None) -> Q4GWeights:
    """Lay GGUF Q4_0 blocks out: wq uint8 [experts, N, row bytes] or [N, row bytes], as quantize_weights makes them."""
    if wq.dim() == 2:
        wq = wq.unsqueeze(0)
    _need(wq.dim() == 3 and wq.dtype == torch.uint8 and wq.is_cuda and wq.is_contiguous() and K % 32 == 0 and wq.shape[2] == K // 32 * 18,
          "wq is contiguous uint8 [.., N, K / 32 * 18]")
    E, N = wq.shape[:2]
    with _on(stream):
        out = _laid_out(E, N, K, 32, gate_up, wq.device)
        _check(_lib().qmm_q4g_pack_q4_0(wq.data_ptr(), E, N, K, int(gate_up), out.data_ptr(), _raw_stream(wq.get_device())), "qmm_q4g_pack_q4_0")
    return Q4GWeights(out, E, N, K, 32, gate_up)


def q4g_dequantize(w: Q4GWeights, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    with _on(stream):
        if out is None:
            out = torch.empty((w.experts, w.N, w.K), dtype=torch.float32, device=w.data.device)
        _need(out.dtype == torch.float32 and out.is_contiguous() and out.numel() == w.experts * w.N * w.K and out.get_device() == w.device,
              "out is contiguous f32 [experts, N, K] on the weights' device")
        _check(_lib().qmm_q4g_dequantize(w._ptr, out.data_ptr(), _raw_stream(w.device)), "qmm_q4g_dequantize")
    return out


def _activations(w: Q4GWeights, x: torch.Tensor, dims: int) -> tuple[int, int]:
    """(type, elements from a row to the next) of activations [.., K]."""
    xt = FLOATS.get(x.dtype)
    if xt is None or x.dim() != dims or x.shape[-1] != w.K or x.get_device() != w.device:
        raise ValueError(f"activations are f32, f16 or bf16, {dims}-dimensional, {w.K} wide, on the weights' device")
    if x.is_contiguous():
        return xt, w.K
    _need(x.stride(-1) == 1 and (dims == 2 or x.shape[1] == 1 or x.shape[0] == 1 or x.stride(0) == x.shape[1] * x.stride(1)),
          "rows of activations are contiguous and evenly apart")
    return xt, x.stride(0) if dims == 2 or x.shape[1] == 1 else x.stride(1)


def _output(out, shape, x):
    if out is None:
        return torch.empty(shape, dtype=x.dtype, device=x.device)
    _need(tuple(out.shape) == tuple(shape) and out.dtype == x.dtype and out.is_contiguous() and out.get_device() == x.get_device(),
          f"out is contiguous {tuple(shape)}, of the activations' type and device")
    return out


def _buffer(workspace, need, x):
    """(pointer, bytes, tensor): a caller's workspace as it is (the library checks its size), else a new one."""
    if workspace is not None:
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if not need:
        return 0, 0, None
    t = torch.empty(need, dtype=torch.uint8, device=x.device)
    return t.data_ptr(), need, t


def q4g_matmul(w: Q4GWeights, x: torch.Tensor, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """y [M, N] = x [M, K] . W^T (one weight matrix)."""
    if stream is not None:
        with _on(stream):
            return q4g_matmul(w, x, out, workspace)
    xt, ld = _activations(w, x, 2)
    M = x.shape[0]
    out = _output(out, (M, w.N), x)
    ptr, size, keep = _buffer(workspace, w._workspace_bytes("qmm_q4g_matmul", xt, M), x)
    status = _lib().qmm_q4g_matmul(w._ptr, xt, x.data_ptr(), ld, M, out.data_ptr(), ptr, size, _raw_stream(w.device))
    if status:
        _check(status, "qmm_q4g_matmul")
    return out


def q4g_matmul_workspace(w: Q4GWeights, dtype: torch.dtype, M: int) -> int:
    return w._workspace_bytes("qmm_q4g_matmul", FLOATS[dtype], M)


def moe_route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: torch.Tensor | None = None, groups: int = 1,
              top_groups: int = 1, group_score: str = "max", renorm: bool = True, scale: float = 1.0, order: bool = True,
              workspace: torch.Tensor | None = None, stream=None) -> Route:
    """Route logits [T, experts] to top_k experts each.  bias f32 [experts] is
    added to the scores that are compared, not to the weights.  order=False
    leaves the sorted slots (offsets, order) out."""
    if stream is not None:
        with _on(stream):
            return moe_route(logits, top_k, score, bias, groups, top_groups, group_score, renorm, scale, order, workspace)
    xt = FLOATS.get(logits.dtype)
    _need(xt is not None and logits.dim() == 2 and logits.is_cuda and logits.stride(1) == 1, "logits are CUDA f32, f16 or bf16 [T, experts]")
    T, E = logits.shape
    device = logits.get_device()
    _need(bias is None or (bias.dtype == torch.float32 and bias.shape == (E,) and bias.is_contiguous() and bias.get_device() == device),
          "bias is f32 [experts]")
    cfg = _RouteConfig(SCORES[score], top_k, groups, top_groups, GROUP_SCORES[group_score], renorm, scale)
    dev, k = logits.device, max(top_k, 0)
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    weights = torch.empty((T, k), dtype=torch.float32, device=dev)
    offsets = slots = None
    need = 0
    if order:
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        slots = torch.empty(T * k, dtype=torch.int32, device=dev)
        if T > 32:
            need = _lib().qmm_moe_route_workspace(T, E, top_k)
    ptr, size, keep = _buffer(workspace, need, logits)
    status = _lib().qmm_moe_route(ctypes.addressof(cfg), xt, logits.data_ptr(), logits.stride(0) if T > 1 else E, T, E,
                                  0 if bias is None else bias.data_ptr(), ids.data_ptr(), weights.data_ptr(),
                                  0 if offsets is None else offsets.data_ptr(), 0 if slots is None else slots.data_ptr(), ptr, size,
                                  _raw_stream(device))
    if status:
        _check(status, "qmm_moe_route")
    return Route(ids, weights, offsets, slots)


def _routing(w: Q4GWeights, r: Route, weights: bool) -> _Routing:
    T, k = r.ids.shape
    ok = r.offsets is not None and r.order is not None
    for t in r:
        ok = ok and (t.dtype == torch.float32 if t is r.weights else t.dtype == torch.int32) and t.is_contiguous() and t.get_device() == w.device
    _need(ok and r.offsets.numel() == w.experts + 1 and r.order.numel() == T * k and r.weights.shape == r.ids.shape,
          "a Route has int32 ids [T, top_k], f32 weights, int32 offsets [experts + 1] and order [T top_k], contiguous, on the weights' device")
    return _Routing(r.ids.data_ptr(), r.weights.data_ptr(), r.offsets.data_ptr(), r.order.data_ptr(), T, k)


def moe_gate_up(w: Q4GWeights, x: torch.Tensor, route: Route, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h [T, top_k, F] of x [T, K]; w packed with gate_up=True, N = 2 F."""
    if stream is not None:
        with _on(stream):
            return moe_gate_up(w, x, route, out, workspace)
    xt, ld = _activations(w, x, 2)
    r = _routing(w, route, False)
    _need(r.T == x.shape[0], "route and x have the same tokens")
    out = _output(out, (r.T, r.top_k, w.N // 2), x)
    ptr, size, keep = _buffer(workspace, w._workspace_bytes("qmm_moe_gate_up", xt, r.T, r.top_k), x)
    status = _lib().qmm_moe_gate_up(w._ptr, xt, x.data_ptr(), ld, ctypes.addressof(r), out.data_ptr(), ptr, size, _raw_stream(w.device))
    if status:
        _check(status, "qmm_moe_gate_up")
    return out


def moe_down(w: Q4GWeights, h: torch.Tensor, route: Route, out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [T, N] of h [T, top_k, K] and the route's weights."""
    if stream is not None:
        with _on(stream):
            return moe_down(w, h, route, out, workspace)
    xt, ld = _activations(w, h, 3)
    r = _routing(w, route, True)
    _need((r.T, r.top_k) == tuple(h.shape[:2]), "route and h have the same slots")
    out = _output(out, (r.T, w.N), h)
    ptr, size, keep = _buffer(workspace, w._workspace_bytes("qmm_moe_down", xt, r.T, r.top_k), h)
    status = _lib().qmm_moe_down(w._ptr, xt, h.data_ptr(), ld, ctypes.addressof(r), out.data_ptr(), ptr, size, _raw_stream(w.device))
    if status:
        _check(status, "qmm_moe_down")
    return out

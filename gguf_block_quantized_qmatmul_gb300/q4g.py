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
stream, or to `stream` (temporaries and outputs are then allocated on it).  The
products and the routing are called through ``_build/_qmm_torch.so`` (a CPython
extension over the same C ABI), which costs a call less than ctypes.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.util
import os
from typing import NamedTuple, Optional

import torch

from . import _build, _check, _lib

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


def _load_binding():
    path = _build.BINDING
    if not os.path.exists(path):
        raise ImportError(f"{os.path.basename(path)} is not built ({path}); run __graft_entry__.build() or "
                          f"python -m gguf_block_quantized_qmatmul_gb300.build")
    _lib()
    spec = importlib.util.spec_from_file_location("_qmm_torch", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


class _Binding:
    """The extension's functions, loaded at the first call."""

    def __getattr__(self, name):
        module = _load_binding()
        for f in ("matmul", "route", "gate_up", "down"):
            setattr(self, f, getattr(module, f))
        return getattr(module, name)


_binding = _Binding()


def _raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


@contextlib.contextmanager
def _on(device: int, stream):
    """Where a call allocates and launches: the device of its tensors, and there `stream` (a torch stream or a raw
    handle of that device) or the current one."""
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)
        _need(stream.device.index == device, "stream is one of the tensors' device")
        with torch.cuda.stream(stream):
            yield


def _need(ok: bool, text: str) -> None:
    if not ok:
        raise ValueError(text)


class Q4GWeights:
    """Laid-out weights: `data` (uint8, qmm_q4g_bytes bytes) and what they are.  Made by q4g_pack or q4g_pack_q4_0, or
    from such data that a program kept.  Can be copied, pickled and saved; `data` may be set anew (moved, reloaded), on
    the CPU too, where it only waits to be moved.  What the weights are does not change."""

    def __init__(self, data: torch.Tensor, experts: int, N: int, K: int, group: int, gate_up: bool):
        self._desc = _Desc(0, experts, N, K, group, int(bool(gate_up)))
        self._ptr = ctypes.addressof(self._desc)
        n = int(_lib().qmm_q4g_bytes(experts, N, K, group, int(bool(gate_up))))
        _need(n > 0 or N == 0, "experts, N, K and group are a shape that q4g_pack takes")
        self._bytes = n
        self.data = data

    experts = property(lambda self: self._desc.experts)
    N = property(lambda self: self._desc.N)
    K = property(lambda self: self._desc.K)
    group = property(lambda self: self._desc.group)
    gate_up = property(lambda self: bool(self._desc.paired))
    device = property(lambda self: self._data.get_device(), doc="index of the CUDA device, -1 on the CPU")

    @property
    def data(self) -> torch.Tensor:
        return self._data

    @data.setter
    def data(self, t: torch.Tensor) -> None:
        _need(t.dtype == torch.uint8 and t.is_contiguous() and t.numel() == self._bytes and t.data_ptr() % 16 == 0,
              "laid-out weights are qmm_q4g_bytes contiguous bytes (uint8) from a 16-byte boundary on")
        self._data = t

    def _descriptor(self) -> int:
        """Address of the qmm_q4g, at where the data is now."""
        _need(self._data.is_cuda and self._data.numel() == self._bytes, "the weights are on a CUDA device")
        self._desc.data = self._data.data_ptr()
        return self._ptr

    def __reduce__(self):
        return Q4GWeights, (self._data, self.experts, self.N, self.K, self.group, self.gate_up)


class Route(NamedTuple):
    """A routing: ids and weights [T, top_k]; offsets [experts + 1]; order [T top_k], the slots t top_k + j by expert."""
    ids: torch.Tensor
    weights: torch.Tensor
    offsets: Optional[torch.Tensor] = None
    order: Optional[torch.Tensor] = None


_tuple_new = tuple.__new__


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
    with _on(codes.get_device(), stream):
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
    with _on(wq.get_device(), stream):
        out = _laid_out(E, N, K, 32, gate_up, wq.device)
        _check(_lib().qmm_q4g_pack_q4_0(wq.data_ptr(), E, N, K, int(gate_up), out.data_ptr(), _raw_stream(wq.get_device())), "qmm_q4g_pack_q4_0")
    return Q4GWeights(out, E, N, K, 32, gate_up)


def q4g_dequantize(w: Q4GWeights, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    with _on(w.device, stream):
        if out is None:
            out = torch.empty((w.experts, w.N, w.K), dtype=torch.float32, device=w.data.device)
        _need(out.dtype == torch.float32 and out.is_contiguous() and out.numel() == w.experts * w.N * w.K and out.get_device() == w.device,
              "out is contiguous f32 [experts, N, K] on the weights' device")
        _check(_lib().qmm_q4g_dequantize(w._descriptor(), out.data_ptr(), _raw_stream(w.device)), "qmm_q4g_dequantize")
    return out


def q4g_matmul(w: Q4GWeights, x: torch.Tensor, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """y [M, N] = x [M, K] . W^T (one weight matrix)."""
    if stream is not None:
        with _on(w.device, stream):
            return q4g_matmul(w, x, out, workspace)
    y = _binding.matmul(w._ptr, w._data, x, out, workspace)
    if type(y) is int:
        _check(y, "qmm_q4g_matmul")
    return y


def q4g_matmul_workspace(w: Q4GWeights, dtype: torch.dtype, M: int) -> int:
    with torch.cuda.device(w.device):  # a plan depends on its device
        return int(_lib().qmm_q4g_matmul_workspace(w._descriptor(), FLOATS[dtype], M))


def moe_route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: torch.Tensor | None = None, groups: int = 1,
              top_groups: int = 1, group_score: str = "max", renorm: bool = True, scale: float = 1.0, order: bool = True,
              workspace: torch.Tensor | None = None, stream=None) -> Route:
    """Route logits [T, experts] to top_k experts each.  bias f32 [experts] is
    added to the scores that are compared, not to the weights.  order=False
    leaves the sorted slots (offsets, order) out.  ids, offsets and order share
    one allocation."""
    if stream is not None:
        with _on(logits.get_device(), stream):
            return moe_route(logits, top_k, score, bias, groups, top_groups, group_score, renorm, scale, order, workspace)
    r = _binding.route(logits, bias, top_k, SCORES[score], groups, top_groups, GROUP_SCORES[group_score], renorm, scale, order, workspace)
    if type(r) is int:
        _check(r, "qmm_moe_route")
    return _tuple_new(Route, r)  # a third of the time of Route(*r)


def moe_gate_up(w: Q4GWeights, x: torch.Tensor, route: Route, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h [T, top_k, F] of x [T, K]; w packed with gate_up=True, N = 2 F."""
    if stream is not None:
        with _on(w.device, stream):
            return moe_gate_up(w, x, route, out, workspace)
    h = _binding.gate_up(w._ptr, w._data, x, *route, out, workspace)
    if type(h) is int:
        _check(h, "qmm_moe_gate_up")
    return h


def moe_down(w: Q4GWeights, h: torch.Tensor, route: Route, out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [T, N] of h [T, top_k, K] and the route's weights."""
    if stream is not None:
        with _on(w.device, stream):
            return moe_down(w, h, route, out, workspace)
    y = _binding.down(w._ptr, w._data, h, *route, out, workspace)
    if type(y) is int:
        _check(y, "qmm_moe_down")
    return y

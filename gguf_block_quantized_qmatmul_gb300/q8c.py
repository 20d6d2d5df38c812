"""8-bit products with a scale per output channel and per token, and the norms
around a block: the Python side of qmm_q8c_* and qmm_block_norm
(``include/qmm.h`` states what each computes, its types, limits and errors).

  q8c_quantize(x)                   int8 codes and f32 scales of rows        -> Rows8
  q8c_pack(codes, scales)           lay a weight matrix out, once            -> Q8CWeights
  q8c_dequantize(w)                 f32 [N, K]
  q8c_matmul(w, x)                  y = x . W^T; x floats or Rows8
  block_norm(y, weight, ...)        (r', h): norm, gate, residual and the next norm; h floats or Rows8

Tensors are CUDA tensors; activations are f32, f16 or bf16 with their last
dimension contiguous (rows may be further apart).  Work goes to the current
stream, or to `stream` (temporaries and outputs are then allocated on it).
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _check, _lib
from .q4g import FLOATS, _binding, _need, _on, _raw_stream


class _Desc(ctypes.Structure):
    """qmm_q8c"""
    _fields_ = [("data", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class _Norm(ctypes.Structure):
    """qmm_norm"""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("y", "residual", "gate", "post_weight", "weight", "residual_out", "h", "codes", "scales")]
                + [(n, ctypes.c_int64) for n in ("ldy", "ldr", "ldg", "ldro", "ldh")]
                + [("type", ctypes.c_int), ("weight_type", ctypes.c_int)] + [(n, ctypes.c_float) for n in ("scale", "eps", "weight_offset")])


def declare(lib) -> None:
    """Argument types of this module's entry points."""
    i64, sz, p, i32 = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int
    for name, args, res in (
            ("qmm_q8c_bytes", [i64, i64], sz),
            ("qmm_q8c_pack", [p, i64, p, i64, i64, p, p], i32),
            ("qmm_q8c_dequantize", [p, p, p], i32),
            ("qmm_q8c_quantize", [i32, p, i64, i64, i64, p, i64, p, p], i32),
            ("qmm_q8c_matmul_workspace", [p, i32, i64], sz),
            ("qmm_q8c_matmul", [p, i32, p, i64, p, i64, p, i32, p, p, sz, p], i32),
            ("qmm_block_norm", [p, i64, i64, p], i32)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


class Rows8(NamedTuple):
    """Rows as 8-bit codes: codes int8 [rows, K] (rows may be further apart), scales f32 [rows]."""
    codes: torch.Tensor
    scales: torch.Tensor


class Q8CWeights:
    """A laid-out weight matrix: `data` (uint8, qmm_q8c_bytes bytes) and its shape.  Made by q8c_pack, or from such data
    that a program kept.  Can be copied, pickled and saved; `data` may be set anew (moved, reloaded), on the CPU too,
    where it only waits to be moved.  The shape does not change."""

    def __init__(self, data: torch.Tensor, N: int, K: int):
        self._desc = _Desc(0, N, K)
        self._ptr = ctypes.addressof(self._desc)
        n = int(_lib().qmm_q8c_bytes(N, K))
        _need(n > 0 or (N == 0 and K > 0), "N and K are a shape that q8c_pack takes")
        self._bytes = n
        self.data = data

    N = property(lambda self: self._desc.N)
    K = property(lambda self: self._desc.K)
    device = property(lambda self: self._data.get_device(), doc="index of the CUDA device, -1 on the CPU")

    @property
    def data(self) -> torch.Tensor:
        return self._data

    @data.setter
    def data(self, t: torch.Tensor) -> None:
        _need(t.dtype == torch.uint8 and t.is_contiguous() and t.numel() == self._bytes and t.data_ptr() % 16 == 0,
              "laid-out weights are qmm_q8c_bytes contiguous bytes (uint8) from a 16-byte boundary on")
        self._data = t

    def _descriptor(self) -> int:
        """Address of the qmm_q8c, at where the data is now."""
        _need(self._data.is_cuda and self._data.numel() == self._bytes, "the weights are on a CUDA device")
        self._desc.data = self._data.data_ptr()
        return self._ptr

    def __reduce__(self):
        return Q8CWeights, (self._data, self.N, self.K)


def _rows(t: torch.Tensor, what: str) -> int:
    """Elements from a row of t [rows, K] to the next."""
    _need(t.dim() == 2 and (t.shape[1] <= 1 or t.stride(1) == 1), f"{what} is [rows, K], rows contiguous")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    _need(ld >= t.shape[1], f"rows of {what} do not overlap")
    return ld


def _codes(rows: int, K: int, device) -> torch.Tensor:
    """int8 [rows, K] whose rows start on 16-byte boundaries"""
    return torch.empty((rows, (K + 15) // 16 * 16), dtype=torch.int8, device=device)[:, :K]


def q8c_quantize(x: torch.Tensor, stream=None) -> Rows8:
    """8-bit codes and one scale per row of x [rows, K] (activations, or a weight matrix by output channel):
    scale = max|x| / 127, code = round(x (1 / scale)) in f32, halves away from zero."""
    _need(x.is_cuda and x.dtype in FLOATS, "x is CUDA f32, f16 or bf16")
    ld, (M, K), device = _rows(x, "x"), x.shape, x.get_device()
    with _on(device, stream):
        codes, scales = _codes(M, K, x.device), torch.empty(M, dtype=torch.float32, device=x.device)
        _check(_lib().qmm_q8c_quantize(FLOATS[x.dtype], x.data_ptr(), ld, M, K, codes.data_ptr(), max(codes.stride(0), K), scales.data_ptr(),
                                       _raw_stream(device)), "qmm_q8c_quantize")
    return Rows8(codes, scales)


def q8c_pack(codes: torch.Tensor, scales: torch.Tensor, stream=None) -> Q8CWeights:
    """Lay a weight matrix out: codes int8 [N, K]; scales f32, f16 or bf16 [N] or [N, 1], one per output channel."""
    _need(codes.is_cuda and codes.dtype == torch.int8, "codes are CUDA int8 [N, K]")
    ld, (N, K), device = _rows(codes, "codes"), codes.shape, codes.get_device()
    _need(scales.dtype in FLOATS and scales.numel() == N and scales.shape[0] == N and scales.get_device() == device,
          "scales are f32, f16 or bf16 [N] on the codes' device")
    with _on(device, stream):
        scales = scales.reshape(N).float().contiguous()
        out = torch.empty(int(_lib().qmm_q8c_bytes(N, K)), dtype=torch.uint8, device=codes.device)
        _check(_lib().qmm_q8c_pack(codes.data_ptr(), ld, scales.data_ptr(), N, K, out.data_ptr(), _raw_stream(device)), "qmm_q8c_pack")
    return Q8CWeights(out, N, K)


def q8c_dequantize(w: Q8CWeights, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    with _on(w.device, stream):
        if out is None:
            out = torch.empty((w.N, w.K), dtype=torch.float32, device=w.data.device)
        _need(out.dtype == torch.float32 and out.is_contiguous() and out.numel() == w.N * w.K and out.get_device() == w.device,
              "out is contiguous f32 [N, K] on the weights' device")
        _check(_lib().qmm_q8c_dequantize(w._descriptor(), out.data_ptr(), _raw_stream(w.device)), "qmm_q8c_dequantize")
    return out


def q8c_matmul(w: Q8CWeights, x, bias: torch.Tensor | None = None, dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [M, N] = x [M, K] . W^T (+ bias f32 [N]).  x: floats, quantized row by row in the call, or Rows8.  y is of
    `dtype`, by default that of x (of Rows8: f32)."""
    if stream is not None:
        with _on(w.device, stream):
            return q8c_matmul(w, x, bias, dtype, out, workspace)
    if type(x) is Rows8:
        y = _binding.matmul8(w._ptr, w._data, x.codes, x.scales, bias, dtype, out, workspace)
    else:
        y = _binding.matmul8(w._ptr, w._data, x, None, bias, dtype, out, workspace)
    if type(y) is int:
        _check(y, "qmm_q8c_matmul")
    return y


def q8c_matmul_workspace(w: Q8CWeights, M: int, quantized: bool = False) -> int:
    with torch.cuda.device(w.device):  # a plan depends on its device
        return int(_lib().qmm_q8c_matmul_workspace(w._descriptor(), int(quantized), M))


_tuple_new = tuple.__new__


def block_norm(y: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, post_weight: torch.Tensor | None = None,
               gate: torch.Tensor | None = None, scale: float = 1.0, eps: float = 1e-6, weight_offset: float = 0.0, quantize: bool = False,
               out: torch.Tensor | None = None, residual_out: torch.Tensor | None = None, stream=None):
    """(r', h) of a block's output y [T, K], in one pass:
    v = y / sqrt(mean(y^2) + eps) (weight_offset + post_weight), or y; r' = residual + scale gate v;
    h = r' / sqrt(mean(r'^2) + eps) (weight_offset + weight), as floats or, with quantize, as Rows8.
    gate: [K] or [T, K] of y's type.  weights: [K], both of one type.  out and residual_out may be y or residual, with its
    strides, not both the same.
    Small float results (256 KB) share one allocation, which lives as long as either does."""
    if stream is not None:
        with _on(y.get_device(), stream):
            return block_norm(y, weight, residual, post_weight, gate, scale, eps, weight_offset, quantize, out, residual_out)
    r = _binding.norm(y, weight, residual, post_weight, gate, scale, eps, weight_offset, quantize, out, residual_out)
    if type(r) is int:
        _check(r, "qmm_block_norm")
    return (r[0], _tuple_new(Rows8, r[1:])) if quantize else r

"""Microscaled 4-bit floating point: quantized rows, and products with weights of that format.  As in the
package's other calls, only arguments are marshalled here; every step runs in the library's HIP kernels.

    t = MXTensor.quantize(x)                    # x [rows, K] fp16/bf16/fp32
    up = MXLinear(MXTensor(codes, scales))      # weights [N, K], laid out once
    y = up.gemm(x)                              # x [M, K] fp16/bf16 as it is
    y = up.gemm(t, dtype=torch.bfloat16)        # both sides in 4 bits
    h = MXGatedLinear(gate, up, activation="silu").gemm(x)      # act(x Wg^T) * (x Wu^T)

Blocks of 32 consecutive inputs share a scale 2 ** (byte - 127); include/gptq_mi355x.h states the format.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import BF16, F16, F32, GPTQError, load_library
from .serving import _CODES, _Queue, _here

__all__ = ["MXTensor", "MXLinear", "MXGatedLinear"]

ACTIVATIONS = {"silu": 1, "gelu_tanh": 2}

# The C structures of include/gptq_mi355x.h, packed by call (see serving.py).
_TENSOR = struct.Struct("PPqqii")          # gptq_mx_tensor
_WEIGHT = struct.Struct("Piiii")           # gptq_mx_weight

_ALL = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}


def _raise(st, where):
    raise GPTQError(st, where, load_library())


def _rows16(x):
    """(x, elements between its rows) with rows 16 bytes aligned and dense; copied if they are not so."""
    width, size = x.shape[1], x.element_size()
    if x.data_ptr() & 15 == 0:
        if x.is_contiguous():
            return x, width
        row, one = x.stride()
        if one == 1 and width <= row <= 1 << 21 and row * size % 16 == 0 and x.shape[0] > 1:
            return x, row
    return x.clone(memory_format=torch.contiguous_format), width


class MXTensor:
    """Rows in the format: codes uint8 [rows, K / 2] (the even input in the low four bits) and scales uint8
    [rows, K / 32].  Keeps the tensors it is given, or copies of those that the library cannot read in
    place (codes contiguous and 16-byte aligned; rows of scales 4-byte aligned)."""

    def __init__(self, codes, scales):
        if codes.dim() != 2 or codes.shape[1] < 16 or codes.shape[1] % 16:
            raise ValueError("codes must be [rows, K / 2] with K a multiple of 32")
        rows, K = codes.shape[0], codes.shape[1] * 2
        if tuple(scales.shape) != (rows, K // 32):
            raise ValueError(f"scales must be [{rows}, {K // 32}]")
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if scales.device != codes.device:
            raise ValueError("codes and scales must be on one device")
        if not codes.is_contiguous() or codes.data_ptr() & 15:
            codes = codes.clone(memory_format=torch.contiguous_format)
        if not _scales_fit(scales):
            room = _new_scales(rows, K, scales.device)
            room.copy_(scales)
            scales = room
        self._set(codes, scales, rows, K)

    def _set(self, codes, scales, rows, K):
        self.codes, self.scales, self.rows, self.K = codes, scales, rows, K
        self.device = codes.device
        self._index = codes.get_device()
        self._stride = scales.stride(0) if rows > 1 else (K // 32 + 3) // 4 * 4
        self._c = _TENSOR.pack(codes.data_ptr(), scales.data_ptr(), self._stride, rows, K, 0)

    @classmethod
    def _empty(cls, rows, K, device):
        t = cls.__new__(cls)
        t._set(torch.empty((rows, K // 2), dtype=torch.uint8, device=device), _new_scales(rows, K, device), rows, K)
        return t

    @classmethod
    def quantize(cls, x, stream=None):
        """x [rows, K] (fp16/bf16/fp32, K a multiple of 32) in the format: each block's scale is
        2 ** (floor(log2 max|x|) - 2), values rounded to nearest, ties to even, past 6 to 6; a block with an
        infinity or NaN is NaN (gptq_mx_quantize)."""
        code = _ALL.get(x.dtype)
        if code is None:
            raise TypeError("x must be float16, bfloat16 or float32")
        if x.dim() != 2 or x.shape[1] < 32 or x.shape[1] % 32:
            raise ValueError("x must be [rows, K] with K a multiple of 32")
        index = x.get_device()
        ptr = _here(stream, index)
        if ptr is not None:
            return cls._quantize(ptr, x, code)
        with _Queue(stream, index, x) as ptr:
            return cls._quantize(ptr, x, code)

    @classmethod
    def _quantize(cls, ptr, x, code):
        x, stride = _rows16(x)
        t = cls._empty(x.shape[0], x.shape[1], x.device)
        st = load_library().gptq_mx_quantize(x.data_ptr(), stride, code, t._c, ptr)
        if st:
            _raise(st, "gptq_mx_quantize")
        return t

    def dequantize(self, dtype=torch.bfloat16, stream=None):
        """The values as [rows, K] of dtype (fp16/bf16/fp32), each rounded once (gptq_mx_dequantize)."""
        code = _ALL.get(dtype)
        if code is None:
            raise TypeError("dtype must be float16, bfloat16 or float32")
        ptr = _here(stream, self._index)
        if ptr is not None:
            return self._dequantize(ptr, dtype, code)
        with _Queue(stream, self._index, self.codes, self.scales) as ptr:
            return self._dequantize(ptr, dtype, code)

    def _dequantize(self, ptr, dtype, code):
        out = torch.empty((self.rows, self.K), dtype=dtype, device=self.device)
        st = load_library().gptq_mx_dequantize(self._c, out.data_ptr(), code, ptr)
        if st:
            _raise(st, "gptq_mx_dequantize")
        return out


def _new_scales(rows, K, device):
    """uint8 [rows, K / 32] whose rows are whole 32-bit words."""
    return torch.empty((rows, (K // 32 + 3) // 4 * 4), dtype=torch.uint8, device=device)[:, :K // 32]


def _scales_fit(s):
    """Whether the library reads s in place: the words of its rows, the last one's included, are s's own."""
    width = s.shape[1]
    if s.data_ptr() & 3 or (width > 1 and s.stride(1) != 1):
        return False
    row = s.stride(0) if s.shape[0] > 1 else (width + 3) // 4 * 4
    if row < width or row % 4 or row > 1 << 20:
        return False
    end = s.data_ptr() + s.shape[0] * row
    return end <= s.untyped_storage().data_ptr() + s.untyped_storage().nbytes()


class _MXProduct:
    """Weights laid out for the products (gptq_mx_pack)."""

    def _load(self, weight, up, activation, stream):
        for name, t in (("weight", weight),) if up is None else (("gate", weight), ("up", up)):
            if not isinstance(t, MXTensor):
                raise TypeError(f"{name} must be an MXTensor")
        if up is not None and (up.rows != weight.rows or up.K != weight.K or up.device != weight.device):
            raise ValueError("gate and up must have one shape and device")
        self._lib = load_library()
        self.N, self.K, self.device = weight.rows, weight.K, weight.device
        self._index = weight._index
        size = ctypes.c_size_t(0)
        st = self._lib.gptq_mx_weight_bytes(self.N, self.K, 0 if up is None else 1, ctypes.byref(size))
        if st:
            _raise(st, "gptq_mx_weight_bytes")
        ptr = _here(stream, self._index)
        if ptr is not None:
            self._pack(ptr, weight, up, size.value)
        else:
            parts = [t for w in (weight, up) if w is not None for t in (w.codes, w.scales)]
            with _Queue(stream, self._index, *parts) as ptr:
                self._pack(ptr, weight, up, size.value)
        self._c = _WEIGHT.pack(self.packed.data_ptr(), self.N, self.K, activation, 0)

    def _pack(self, ptr, weight, up, size):
        self.packed = torch.empty(size, dtype=torch.uint8, device=self.device)
        st = self._lib.gptq_mx_pack(weight._c, None if up is None else up._c, self.packed.data_ptr(), ptr)
        if st:
            _raise(st, "gptq_mx_pack")

    def gemm(self, x, out=None, dtype=None, stream=None):
        """The product with x: a [M, K] fp16/bf16 tensor as it is (the result has its type), or an MXTensor
        (the result is of `dtype`, bfloat16 by default).  out, when given, is a contiguous [M, N] tensor of
        that type (gptq_mx_gemm, gptq_mx_gemm_mx)."""
        if isinstance(x, MXTensor):
            M, index = x.rows, x._index
            if x.K != self.K:
                raise ValueError(f"x must have {self.K} inputs")
            if dtype is None:
                dtype = torch.bfloat16 if out is None else out.dtype
            parts = (x.codes, x.scales)
        else:
            if x.dim() != 2 or x.shape[1] != self.K:
                raise ValueError(f"x must be [M, {self.K}]")
            if dtype is not None and dtype is not x.dtype:
                raise TypeError("the result has x's dtype")
            M, index, dtype, parts = x.shape[0], x.get_device(), x.dtype, (x,)
        if dtype not in _CODES:
            raise TypeError("x, or dtype, must be float16 or bfloat16")
        if index != self._index:
            raise ValueError(f"x must be on {self.device}")
        if out is not None and (tuple(out.shape) != (M, self.N) or out.dtype is not dtype or out.get_device() != index
                                or not out.is_contiguous()):
            raise ValueError(f"out must be a contiguous [M, {self.N}] tensor of {dtype} on {self.device}")
        ptr = _here(stream, index)
        if ptr is not None:
            return self._gemm(ptr, x, M, out, dtype)
        with _Queue(stream, index, out, self.packed, *parts) as ptr:
            return self._gemm(ptr, x, M, out, dtype)

    def _gemm(self, ptr, x, M, out, dtype):
        if out is None:
            out = torch.empty((M, self.N), dtype=dtype, device=self.device)
        if isinstance(x, MXTensor):
            st, where = self._lib.gptq_mx_gemm_mx(self._c, x._c, out.data_ptr(), _CODES[dtype], ptr), "gptq_mx_gemm_mx"
        else:
            x, stride = _rows16(x)
            st = self._lib.gptq_mx_gemm(self._c, x.data_ptr(), stride, _CODES[dtype], M, out.data_ptr(), ptr)
            where = "gptq_mx_gemm"
        if st:
            _raise(st, where)
        return out


class MXLinear(_MXProduct):
    """y = x W^T for weights W [N, K] in the format.  The source tensors may be freed afterwards."""

    def __init__(self, weight, stream=None):
        self._load(weight, None, 0, stream)


class MXGatedLinear(_MXProduct):
    """act(x Wg^T) * (x Wu^T) in one kernel for the two projections [N, K] of a gated feed-forward block;
    activation "silu" or "gelu_tanh"."""

    def __init__(self, gate, up, activation="silu", stream=None):
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
        self.activation = activation
        self._load(gate, up, ACTIVATIONS[activation], stream)

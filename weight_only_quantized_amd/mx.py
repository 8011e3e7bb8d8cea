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

_E_SHAPE = 2                               # GPTQ_E_SHAPE
_ALL = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}


def _raise(st, where):
    raise GPTQError(st, where, load_library())


def _rows16(x):
    """(x, elements between its rows) with rows 16 bytes aligned and dense; copied if they are not so."""
    if x.is_contiguous():
        if not x.data_ptr() & 15:
            return x, x.shape[1]
    elif not x.data_ptr() & 15:
        row, one = x.stride()
        if one == 1 and x.shape[1] <= row <= 1 << 21 and row * x.element_size() % 16 == 0 and x.shape[0] > 1:
            return x, row
    return x.clone(memory_format=torch.contiguous_format), x.shape[1]


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
        stride = _words(K)
        if _scales_fit(scales):
            stride = scales.stride(0) if rows > 1 else stride
        else:
            room = torch.empty((rows, stride), dtype=torch.uint8, device=scales.device)[:, :K // 32]
            room.copy_(scales)
            scales = room
        self._codes, self._scales = self._keep = codes, scales
        self._set(rows, K, codes.get_device(), codes.data_ptr(), scales.data_ptr(), stride)

    def _set(self, rows, K, index, codes, scales, stride):
        if K > 0x7fffffff:
            _raise(_E_SHAPE, "MXTensor")       # as the library says of rows past 2^20 inputs that its structure can name
        self.rows, self.K, self._index, self._stride = rows, K, index, stride
        self._c = _TENSOR.pack(codes, scales, stride, rows, K, 0)

    def __reduce__(self):
        # a copy or an unpickled tensor packs the addresses of its own memory
        return type(self), (self.codes, self.scales)

    # quantize makes one buffer, whose views a call that only passes the tensor on does not need
    @property
    def codes(self):
        if self._codes is None:
            self._codes = self._keep[0].as_strided((self.rows, self.K // 2), (self.K // 2, 1))
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._scales = self._keep[0].as_strided((self.rows, self.K // 32), (self._stride, 1),
                                                    _codes_room(self.rows, self.K))
        return self._scales

    @property
    def device(self):
        return self._keep[0].device

    @classmethod
    def quantize(cls, x, stream=None):
        """x [rows, K] (fp16/bf16/fp32, K a multiple of 32) in the format: each block's scale is
        2 ** (floor(log2 max|x|) - 2), values rounded to nearest, ties to even, past 6 to 6; a block with an
        infinity or NaN is NaN (gptq_mx_quantize)."""
        code, shape = _ALL.get(x.dtype), x.shape
        if code is None:
            raise TypeError("x must be float16, bfloat16 or float32")
        if len(shape) != 2 or shape[1] < 32 or shape[1] % 32:
            raise ValueError("x must be [rows, K] with K a multiple of 32")
        index = x.get_device()
        ptr = _here(stream, index)
        if ptr is not None:
            return cls._quantize(ptr, x, code, index)
        with _Queue(stream, index, x) as ptr:
            return cls._quantize(ptr, x, code, index)

    @classmethod
    def _quantize(cls, ptr, x, code, index):
        x, x_stride = _rows16(x)
        rows, K = x.shape
        at, stride = _codes_room(rows, K), _words(K)
        room = x.new_empty(at + rows * stride, dtype=torch.uint8)
        t = cls.__new__(cls)
        t._keep, t._codes, t._scales = (room,), None, None
        base = room.data_ptr()
        t._set(rows, K, index, base, base + at, stride)
        st = load_library().gptq_mx_quantize(x.data_ptr(), x_stride, code, t._c, ptr)
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
        with _Queue(stream, self._index, *self._keep) as ptr:
            return self._dequantize(ptr, dtype, code)

    def _dequantize(self, ptr, dtype, code):
        out = self._keep[0].new_empty((self.rows, self.K), dtype=dtype)
        st = load_library().gptq_mx_dequantize(self._c, out.data_ptr(), code, ptr)
        if st:
            _raise(st, "gptq_mx_dequantize")
        return out


def _words(K):
    """Bytes between rows of scales that are whole 32-bit words."""
    return (K // 32 + 3) // 4 * 4


def _codes_room(rows, K):
    """Bytes from a quantized tensor's codes to its scales (K / 2 is a multiple of 16)."""
    return rows * K // 2


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

    def _load(self, weight, up, activation):
        for name, t in (("gate", weight), ("up", up)) if activation else (("weight", weight),):
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
        ptr = _here(None, self._index)
        if ptr is not None:
            self._pack(ptr, weight, up, size.value)
        else:
            with _Queue(None, self._index) as ptr:
                self._pack(ptr, weight, up, size.value)
        self._c = _WEIGHT.pack(self.packed.data_ptr(), self.N, self.K, activation, 0)

    def _pack(self, ptr, weight, up, size):
        self.packed = torch.empty(size, dtype=torch.uint8, device=self.device)
        st = self._lib.gptq_mx_pack(weight._c, None if up is None else up._c, self.packed.data_ptr(), ptr)
        if st:
            _raise(st, "gptq_mx_pack")
        # the sources may be freed at once: memory of another stream stays theirs until this one has read it
        stream = torch.cuda.current_stream(self._index)
        for t in (weight,) if up is None else (weight, up):
            for part in t._keep:
                part.record_stream(stream)

    def gemm(self, x, out=None, dtype=None, stream=None):
        """The product with x: a [M, K] fp16/bf16 tensor as it is (the result has its type), or an MXTensor
        (the result is of `dtype`, bfloat16 by default).  out, when given, is a contiguous [M, N] tensor of
        that type (gptq_mx_gemm, gptq_mx_gemm_mx)."""
        if isinstance(x, MXTensor):
            M, index, parts = x.rows, x._index, x._keep
            if x.K != self.K:
                raise ValueError(f"x must have {self.K} inputs")
            if dtype is None:
                dtype = torch.bfloat16 if out is None else out.dtype
        else:
            shape = x.shape
            if len(shape) != 2 or shape[1] != self.K:
                raise ValueError(f"x must be [M, {self.K}]")
            M, index, parts = shape[0], x.get_device(), (x,)
            if dtype is not None and dtype is not x.dtype:
                raise TypeError("the result has x's dtype")
            dtype = x.dtype
        code = _CODES.get(dtype)
        if code is None:
            raise TypeError("x, or dtype, must be float16 or bfloat16")
        if index != self._index:
            raise ValueError(f"x must be on {self.device}")
        if out is not None and (out.shape != (M, self.N) or out.dtype is not dtype or out.get_device() != index
                                or not out.is_contiguous()):
            raise ValueError(f"out must be a contiguous [M, {self.N}] tensor of {dtype} on {self.device}")
        ptr = _here(stream, index)
        if ptr is not None:
            return self._gemm(ptr, x, M, out, dtype, code)
        with _Queue(stream, index, out, self.packed, *parts) as ptr:
            return self._gemm(ptr, x, M, out, dtype, code)

    def _gemm(self, ptr, x, M, out, dtype, code):
        if out is None:
            out = self.packed.new_empty((M, self.N), dtype=dtype)
        if isinstance(x, MXTensor):
            st, where = self._lib.gptq_mx_gemm_mx(self._c, x._c, out.data_ptr(), code, ptr), "gptq_mx_gemm_mx"
        else:
            x, stride = _rows16(x)
            st = self._lib.gptq_mx_gemm(self._c, x.data_ptr(), stride, code, M, out.data_ptr(), ptr)
            where = "gptq_mx_gemm"
        if st:
            _raise(st, where)
        return out


class MXLinear(_MXProduct):
    """y = x W^T for weights W [N, K] in the format.  The source tensors may be freed afterwards."""

    def __init__(self, weight):
        self._load(weight, None, 0)


class MXGatedLinear(_MXProduct):
    """act(x Wg^T) * (x Wu^T) in one kernel for the two projections [N, K] of a gated feed-forward block;
    activation "silu" or "gelu_tanh"."""

    def __init__(self, gate, up, activation="silu"):
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
        self.activation = activation
        self._load(gate, up, ACTIVATIONS[activation])

"""Refusals of the entry points on microscaled 4-bit floating point (host checks: no GPU, no launch), and
pins of their oracle."""
import copy
import ctypes
import pickle
import struct
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle.mx_oracle as mo
import weight_only_quantized_amd as wq

A = 1 << 20          # a well-aligned address: the checks only compare addresses, nothing is read
P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class Tensor(ctypes.Structure):
    _fields_ = [("codes", P), ("scales", P), ("scale_stride", I64), ("rows", I64), ("K", I32), ("reserved", I32)]


class Weight(ctypes.Structure):
    _fields_ = [("packed", P), ("N", I32), ("K", I32), ("activation", I32), ("reserved", I32)]


def tensor(**kw):
    t = Tensor(A, A + (64 << 20), 8, 4, 256, 0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def weight(**kw):
    w = Weight(A + (128 << 20), 48, 256, 0, 0)
    for k, v in kw.items():
        setattr(w, k, v)
    return w


FREE = A + (512 << 20)
ref = lambda s: ctypes.byref(s) if s is not None else None  # noqa: E731


def quantize(x=FREE, stride=256, dtype=1, t=None):
    return wq.STATUS[wq.load_library().gptq_mx_quantize(x, stride, dtype, ref(tensor() if t is None else t), None)]


def dequantize(t=None, out=FREE, dtype=1):
    return wq.STATUS[wq.load_library().gptq_mx_dequantize(ref(tensor() if t is None else t), out, dtype, None)]


def pack(t=None, up=None, out=FREE):
    return wq.STATUS[wq.load_library().gptq_mx_pack(ref(tensor() if t is None else t), ref(up), out, None)]


def gemm(w=None, x=FREE, stride=256, dtype=1, M=3, y=FREE + (64 << 20)):
    return wq.STATUS[wq.load_library().gptq_mx_gemm(ref(weight() if w is None else w), x, stride, dtype, M, y, None)]


def gemm_mx(w=None, t=None, y=FREE, dtype=1):
    return wq.STATUS[wq.load_library().gptq_mx_gemm_mx(ref(weight() if w is None else w), ref(tensor() if t is None else t), y,
                                                       dtype, None)]


def test_the_binding_packs_the_header_structures():
    from weight_only_quantized_amd import mx
    for packed, structure, n in ((mx._TENSOR, Tensor, 7), (mx._WEIGHT, Weight, 6)):
        assert packed.size == ctypes.sizeof(structure)
        assert packed.pack(*range(1, n)) == bytes(structure(*range(1, n))), structure


TENSOR_REFUSALS = [("E_INVALID_ARG", dict(codes=None)), ("E_INVALID_ARG", dict(scales=None)),
                   ("E_INVALID_ARG", dict(codes=A + 8)), ("E_INVALID_ARG", dict(scales=A + (64 << 20) + 2)),
                   ("E_INVALID_ARG", dict(scale_stride=7)), ("E_INVALID_ARG", dict(scale_stride=4)),
                   ("E_INVALID_ARG", dict(scale_stride=10)), ("E_INVALID_ARG", dict(scale_stride=(1 << 20) + 4)),
                   ("E_INVALID_ARG", dict(reserved=1)), ("E_SHAPE", dict(rows=-1)), ("E_SHAPE", dict(rows=(1 << 24) + 1)),
                   ("E_SHAPE", dict(K=0)), ("E_SHAPE", dict(K=-32)), ("E_SHAPE", dict(K=48)), ("E_SHAPE", dict(K=(1 << 20) + 32))]


@pytest.mark.parametrize("want,kw", TENSOR_REFUSALS)
def test_tensor_refusals(want, kw):
    t = tensor(**kw)
    assert quantize(t=t) == want
    assert dequantize(t=t) == want
    assert pack(t=t) == want
    assert pack(t=tensor(), up=t) == want
    if "K" not in kw:
        assert gemm_mx(t=t) == want
    else:
        assert gemm_mx(t=t) in ("E_SHAPE", "E_INVALID_ARG")


def test_quantize_and_dequantize_refusals():
    lib = wq.load_library()
    assert lib.gptq_mx_quantize(FREE, 256, 1, None, None) == 1 and lib.gptq_mx_dequantize(None, FREE, 1, None) == 1
    for kw in (dict(x=None), dict(x=FREE + 2), dict(stride=255), dict(stride=128), dict(stride=260), dict(stride=(1 << 32) + 8),
               dict(dtype=3), dict(dtype=-1), dict(x=A), dict(x=A + (64 << 20)), dict(t=tensor(scales=A))):
        assert quantize(**kw) == "E_INVALID_ARG", kw
    assert quantize(dtype=2, stride=258) == "E_INVALID_ARG"          # fp32 rows 16 bytes apart
    for kw in (dict(out=None), dict(out=FREE + 8), dict(dtype=3), dict(out=A), dict(out=A + (64 << 20) - 16)):
        assert dequantize(**kw) == "E_INVALID_ARG", kw
    assert quantize(t=tensor(rows=0, codes=None, scales=None), x=None) == "OK"
    assert dequantize(t=tensor(rows=0, codes=None, scales=None), out=None) == "OK"


def test_pack_refusals():
    lib = wq.load_library()
    n = ctypes.c_size_t(0)
    assert lib.gptq_mx_weight_bytes(48, 256, 0, None) == 1 and lib.gptq_mx_weight_bytes(48, 256, 2, ctypes.byref(n)) == 1
    for N, K in ((0, 256), (-1, 256), ((1 << 20) + 1, 256), (48, 0), (48, 40), (48, (1 << 20) + 32)):
        assert lib.gptq_mx_weight_bytes(N, K, 0, ctypes.byref(n)) == 2
    # whole tiles of 16 outputs and 256 inputs: codes, scales, a byte a row
    for N, K, sides in ((1, 32, 1), (48, 256, 1), (49, 288, 2), (1 << 20, 1 << 20, 2)):
        assert lib.gptq_mx_weight_bytes(N, K, sides - 1, ctypes.byref(n)) == 0
        tiles, stages = sides * -(-N // 16), -(-K // 256)
        assert n.value == -(-(tiles * stages * (2048 + 128) + tiles * 16) // 256) * 256
    assert pack(t=tensor(rows=0)) == "E_SHAPE" and pack(t=tensor(rows=(1 << 20) + 1)) == "E_SHAPE"
    for kw in (dict(out=None), dict(out=FREE + 128), dict(out=A), dict(out=A + (64 << 20)), dict(up=tensor(rows=5)),
               dict(up=tensor(K=288, scale_stride=12))):
        assert pack(**kw) == "E_INVALID_ARG", kw
    assert pack(out=A + (200 << 20), up=tensor(codes=A + (200 << 20))) == "E_INVALID_ARG"


def test_gemm_refusals():
    lib = wq.load_library()
    assert lib.gptq_mx_gemm(None, FREE, 256, 1, 3, FREE, None) == 1 and lib.gptq_mx_gemm_mx(None, None, FREE, 1, None) == 1
    assert lib.gptq_mx_gemm_mx(ctypes.byref(weight()), None, FREE, 1, None) == 1
    for want, kw in (("E_INVALID_ARG", dict(packed=None)), ("E_INVALID_ARG", dict(packed=A + 16)), ("E_INVALID_ARG", dict(reserved=1)),
                     ("E_INVALID_ARG", dict(activation=3)), ("E_INVALID_ARG", dict(activation=-1)), ("E_SHAPE", dict(N=0)),
                     ("E_SHAPE", dict(N=(1 << 20) + 1)), ("E_SHAPE", dict(K=0)), ("E_SHAPE", dict(K=33))):
        assert gemm(weight(**kw)) == want, kw
        assert gemm_mx(weight(**kw)) == want, kw
    for kw in (dict(x=None), dict(x=FREE + 8), dict(y=None), dict(y=FREE + 8), dict(stride=248), dict(stride=260), dict(dtype=2),
               dict(stride=(1 << 21) + 8), dict(dtype=3), dict(y=FREE + 256), dict(y=A + (128 << 20)), dict(x=FREE, y=FREE)):
        assert gemm(**kw) == "E_INVALID_ARG", kw
    assert gemm(M=-1) == "E_SHAPE" and gemm(M=(1 << 24) + 1) == "E_SHAPE"
    assert gemm(weight(N=1 << 20), M=1 << 24, y=1 << 46) == "E_SHAPE"          # more threads than a launch has
    assert gemm(M=0, x=None, y=None) == "OK"
    for kw in (dict(y=None), dict(y=FREE + 8), dict(dtype=2), dict(dtype=5), dict(t=tensor(K=288, scale_stride=12)), dict(y=A),
               dict(y=A + (64 << 20)), dict(y=A + (128 << 20))):
        assert gemm_mx(**kw) == "E_INVALID_ARG", kw
    assert gemm_mx(t=tensor(rows=0, codes=None, scales=None), y=None) == "OK"


def test_binding_refusals():
    import torch
    u8 = torch.uint8
    z = lambda *s, dtype=u8: torch.zeros(s, dtype=dtype)  # noqa: E731
    ok = wq.MXTensor(z(4, 48), z(4, 3))
    assert (ok.rows, ok.K) == (4, 96) and ok.codes.shape == (4, 48) and ok.scales.shape == (4, 3)
    for codes, scales, error in ((z(4, 40), z(4, 3), ValueError), (z(4, 48), z(4, 4), ValueError), (z(48), z(3), ValueError),
                                 (z(4, 48, dtype=torch.int8), z(4, 3), TypeError), (z(4, 48), z(4, 3, dtype=torch.float32), TypeError),
                                 (z(4, 0), z(4, 0), ValueError)):
        with pytest.raises(error):
            wq.MXTensor(codes, scales)
    with pytest.raises(ValueError):
        wq.MXTensor.quantize(torch.zeros(4, 96))                               # not on a GPU
    with pytest.raises(ValueError):
        wq.MXTensor.quantize(torch.zeros(4, 90))
    with pytest.raises(ValueError):
        wq.MXTensor.quantize(torch.zeros(96))
    with pytest.raises(TypeError):
        wq.MXTensor.quantize(torch.zeros(4, 96, dtype=torch.float64))
    with pytest.raises(TypeError):
        ok.dequantize(torch.float64)
    with pytest.raises(ValueError):
        ok.dequantize()                                                         # not on a GPU
    with pytest.raises(ValueError):
        wq.MXLinear(ok)
    with pytest.raises(TypeError):
        wq.MXLinear(z(4, 48))
    with pytest.raises(TypeError):
        wq.MXGatedLinear(ok, None)
    with pytest.raises(ValueError):
        wq.MXGatedLinear(ok, wq.MXTensor(z(5, 48), z(5, 3)))
    with pytest.raises(ValueError):
        wq.MXGatedLinear(ok, ok, activation="relu")


def test_scales_are_kept_or_copied():
    import torch
    from weight_only_quantized_amd.mx import _scales_fit
    codes = torch.zeros((5, 48), dtype=torch.uint8)
    wide = torch.arange(60, dtype=torch.uint8).view(5, 12)
    kept = wide[:, :3]
    t = wq.MXTensor(codes, kept)
    assert t.scales.data_ptr() == kept.data_ptr()
    # rows of 3 bytes, rows that start between words, a last row whose word is not in its storage: copied
    for s in (torch.arange(15, dtype=torch.uint8).view(5, 3), wide[:, 1:4], wide[:, 4:7], wide.t()[:5, :3]):
        assert not _scales_fit(s)
        t = wq.MXTensor(codes, s)
        assert t.scales.data_ptr() != s.data_ptr() and t.scales.stride(0) == 4 and torch.equal(t.scales, s)
    short = torch.zeros(5 * 8 - 5, dtype=torch.uint8).as_strided((5, 3), (8, 1))
    assert not _scales_fit(short)


# ---- the oracle ----------------------------------------------------------------------------------

def test_oracle_values_and_packing():
    codes = np.array([[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * 2], dtype=np.uint8)
    want = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6] * 2)
    assert np.array_equal(mo.values(codes, np.array([[127]]))[0], want)
    assert np.array_equal(mo.values(codes, np.array([[129]]))[0], 4 * want)
    assert np.array_equal(mo.values(codes, np.array([[0]]))[0], want * 2.0 ** -127)
    assert np.isnan(mo.values(codes, np.array([[255]]))).all()
    assert np.array_equal(mo.pack(mo.unpack(codes)), codes)


def test_oracle_quantizes_by_the_definition():
    """Against exact rationals: the scale by counting binades, the code by trying all."""
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((40, 32)) * np.exp2(rng.integers(-20, 20, (40, 1)))).astype(np.float32).astype(np.float64)
    x[0] = 0
    x[1, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9]           # ties, and past 6
    x[1, 8:] = 0
    x[2, 0], x[3, 0] = np.inf, np.nan
    codes, scales = mo.quantize(x)
    nib = mo.unpack(codes)
    for i in range(40):
        if i in (2, 3):
            assert scales[i, 0] == 255 and not nib[i].any()
            continue
        most, e = max(abs(Fraction(v)) for v in x[i]), -127
        if most:
            while Fraction(2) ** (e + 1) * 4 <= most:
                e += 1
        assert scales[i, 0] == e + 127
        for v, n in zip(x[i], nib[i]):
            t = abs(Fraction(v)) / Fraction(2) ** e
            off = [abs(t - Fraction(float(g))) for g in mo.VALUES]
            near = [k for k in range(8) if off[k] == min(off)]
            assert n & 7 == (near[0] if len(near) == 1 else [k for k in near if k % 2 == 0][0])
            assert bool(n & 8) == (v < 0)
    assert [int(n) for n in nib[1, :8]] == [0, 2, 2, 4, 4, 6, 6, 7]


def test_oracle_activations():
    g = np.array([-30.0, -1.0, 0.0, 0.5, 20.0])
    assert np.allclose(mo.silu(g), g * 0.5 * (1 + np.tanh(g / 2)), rtol=1e-9, atol=1e-12)
    t = np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    assert np.allclose(mo.gelu_tanh(g), 0.5 * g * (1 + np.tanh(t)), rtol=1e-12, atol=1e-12)


def test_planted_mistakes_fail():
    """A scale rounded up, ties away from zero, nibbles swapped: each changes what the pins fix."""
    x = np.zeros((1, 32))
    x[0, :4] = [7.0, 0.25, 2.5, -5.0]
    codes, scales = mo.quantize(x)
    assert scales[0, 0] == 127 and [int(n) for n in mo.unpack(codes)[0, :4]] == [7, 0, 4, 14]
    up = int(np.ceil(np.log2(7.0 / 6))) + 127
    assert up != scales[0, 0]
    away = [int(np.argmin(np.abs(abs(v) - mo.VALUES[::-1]))) for v in x[0, :4]]
    assert [7 - a for a in away] != [7, 0, 4, 6]
    assert not np.array_equal((codes & 15) << 4 | codes >> 4, codes)


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle"])
@pytest.mark.parametrize("rows,inputs", [(0, 32), (1, 96), (5, 96), (3, 128)])
def test_copies_of_a_tensor_describe_their_own_memory(how, rows, inputs):
    codes = torch.arange(rows * inputs // 2).reshape(rows, inputs // 2).to(torch.uint8)
    scales = torch.arange(rows * inputs // 32).reshape(rows, inputs // 32).to(torch.uint8)
    t = wq.MXTensor(codes, scales)
    u = {"copy": copy.copy, "deepcopy": copy.deepcopy, "pickle": lambda v: pickle.loads(pickle.dumps(v))}[how](t)
    assert (u.rows, u.K) == (rows, inputs) and torch.equal(u.codes, codes) and torch.equal(u.scales, scales)
    at, scales_at, stride, n, k, _ = struct.unpack("PPqqii", u._c)
    assert (at, scales_at, n, k) == (u.codes.data_ptr(), u.scales.data_ptr(), rows, inputs)
    assert stride >= inputs // 32 and stride % 4 == 0
    if rows:
        assert scales_at + rows * stride <= u.scales.untyped_storage().data_ptr() + u.scales.untyped_storage().nbytes()
        if how != "copy":
            assert at != t.codes.data_ptr() and scales_at != t.scales.data_ptr()

"""Checks of results on microscaled 4-bit floating point that the GPU tests make, and the values they make
them on: here, so that a test on the CPU can hand them wrong results and see them refused."""
from fractions import Fraction

import numpy as np

import oracle.mx_oracle as mo


# ---- quantizing ----------------------------------------------------------------------------------

def quantized(x, codes, scales):
    """Asserts that codes and scales are x quantized by the definition, in exact rationals: the scale by counting
    binades, each code by trying all."""
    nib = mo.unpack(codes)
    for i in range(x.shape[0]):
        for b in range(x.shape[1] // 32):
            v, n = x[i, 32 * b:32 * b + 32], nib[i, 32 * b:32 * b + 32]
            if not np.isfinite(v).all():
                assert scales[i, b] == 255 and not n.any()
                continue
            most, e = max(abs(Fraction(t)) for t in v), -127
            while e < 127 and Fraction(2) ** (e + 1) * 4 <= most:
                e += 1
            assert scales[i, b] == e + 127
            for t, c in zip(v, n):
                off = [abs(abs(Fraction(t)) / Fraction(2) ** e - Fraction(float(g))) for g in mo.VALUES]
                near = [k for k in range(8) if off[k] == min(off)]
                assert c & 7 == (near[0] if len(near) == 1 else [k for k in near if k % 2 == 0][0])
                assert bool(c & 8) == bool(np.signbit(t))


# ---- float16 activations: weights relative to their output's largest scale --------------------------

def live(codes):
    """Which blocks hold more than zeros, [rows, K / 32]."""
    return ((np.asarray(codes) & 0x77) != 0).reshape(codes.shape[0], -1, 16).any(-1)


def float16_weights(codes, scales):
    """The weights that float16 activations meet, as float64: rounded to nearest even to multiples of 2^-37 of the
    largest scale of their row's blocks that hold more than zeros, but to no more than float16's 11 bits."""
    top = np.where(live(codes), scales, 0).max(1).astype(np.int64)[:, None]
    n = mo.unpack(codes)
    v = np.where(n & 8, -mo.VALUES[n & 7], mo.VALUES[n & 7])
    lifted = v * np.ldexp(1.0, scales.astype(np.int64) - top + 13).repeat(32, 1)
    return lifted.astype(np.float16).astype(np.float64) * np.ldexp(1.0, top - 140)


def deep_weights(rng, N, K, low, high, unit):
    """Rows whose first block has the largest scale and whose others lie 2^-low .. 2^-high below it; what these add up to
    with deep_inputs(unit) is near one.  Rows are of different size."""
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    codes[:, 0] = 0x77
    top = 120 + low - unit + rng.integers(-2, 3, (N, 1))
    scales = top - rng.integers(low, high + 1, (N, K // 32))
    scales[:, :1] = top
    assert 0 <= scales.min() and scales.max() < 255
    return codes, scales.astype(np.uint8)


def deep_inputs(rng, M, K, unit):
    """Multiples of 2^unit / 4 up to 4 2^unit, zero where the weights' first block would drown the others."""
    x = rng.integers(-16, 17, (M, K)) / 4 * 2.0 ** unit
    x[:, :32] = 0
    return x


# Scales below the largest: one octave of exactness after the other; the last ones are float16's subnormals.
DEPTHS = [(8, 11), (20, 23), (27, 30), (33, 36)]
UNITS = [13, -12]


def product(got, x, weights, tag):
    """Asserts that got is x W^T rounded once.  Sums of the values above are exact in float32 in any order: in units of half
    the smallest scale (or of 2^-37 of the largest, what smaller weights are rounded to) weights are whole numbers up to 96, in units
    of 2^unit / 4 activations up to 16, so 256 products add up to less than 2^19 units."""
    import torch
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[tag]
    want = torch.from_numpy(np.asarray(x, dtype=np.float32)).to(got.device) @ \
        torch.from_numpy(weights.astype(np.float32)).to(got.device).t()
    assert torch.equal(got, want.to(dt))

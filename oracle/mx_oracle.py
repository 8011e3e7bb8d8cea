"""Float64 oracle of the operators on microscaled 4-bit floating point: rows quantized to blocks of 32
e2m1 values with one e8m0 scale, products with such rows, and the gated feed-forward projection.  Plain
numpy, test infrastructure only."""
import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def unpack(codes):
    """uint8 [rows, K / 2] -> [rows, K] of 0..15, the even element in the low four bits."""
    codes = np.asarray(codes, dtype=np.uint8)
    return np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)


def pack(nibbles):
    n = np.asarray(nibbles, dtype=np.uint8)
    return (n[:, 0::2] | n[:, 1::2] << 4).astype(np.uint8)


def scale_values(scales):
    s = np.asarray(scales).astype(np.int64)
    return np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))


def values(codes, scales):
    """float64 [rows, K]."""
    n = unpack(codes)
    v = np.where(n & 8, -VALUES[n & 7], VALUES[n & 7])
    return v * np.repeat(scale_values(scales), 32, axis=1)


def quantize(x):
    """(codes, scales) of x [rows, K]: for each block the largest power of two 2^e, |e| <= 127, with
    4 * 2^e <= max |x| (2^-127 if there is none); each value goes to the nearest of the format's times 2^e,
    and of two as near the one with the even code."""
    x = np.asarray(x, dtype=np.float64)
    rows, K = x.shape
    b = x.reshape(rows, K // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    most = np.abs(b).max(-1)
    _, e = np.frexp(most)                                   # most = f 2^e, f in [1/2, 1)
    e = np.where(most > 0, np.clip(e - 3, -127, 127), -127)
    t = np.abs(b) / np.ldexp(1.0, e)[..., None]
    near = np.abs(t[..., None] - VALUES)                    # exact: both sides hold few bits
    best = near.min(-1, keepdims=True)
    code = np.argmax(near == best, -1)                      # the lower of two as near
    tie = np.take_along_axis(near, np.minimum(code + 1, 7)[..., None], -1)[..., 0] == best[..., 0]
    code = np.where(tie & (code < 7) & (code % 2 == 1), code + 1, code)
    code = code | np.where(np.signbit(x.reshape(b.shape)), 8, 0)
    code = np.where(bad[..., None], 0, code)
    return pack(code.reshape(rows, K)), np.where(bad, 255, e + 127).astype(np.uint8)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def gelu_tanh(g):
    # 0.5 g (1 + tanh t) = g / (1 + exp(-2 t))
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-2.0 * np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3)))


ACTIVATIONS = {"silu": silu, "gelu_tanh": gelu_tanh}


def gemm(x, w):
    """x [M, K] and w [N, K] as values."""
    return np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T


def gated(x, gate, up, activation):
    return ACTIVATIONS[activation](gemm(x, gate)) * gemm(x, up)

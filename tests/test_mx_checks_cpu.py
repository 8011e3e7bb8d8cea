"""The checks of tests/mx_checks.py refuse wrong results (planted here, on the CPU) and take right ones."""
import numpy as np
import pytest
import torch

import mx_checks as mc
import oracle.mx_oracle as mo


def _inputs():
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((40, 64)) * np.exp2(rng.integers(-20, 20, (40, 1)))).astype(np.float32).astype(np.float64)
    x[1, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9]           # ties, and past 6
    x[1, 8:32] = 0
    x[2, 0], x[3, 40] = np.inf, np.nan
    x[4, 32:] = 0
    x[5, :32] = 2.0 ** -140
    x[6, 3] = -0.0
    return x


def _requantized(x, exponents, codes_of=None):
    """x quantized under other scales, or with other codes for its magnitudes in units."""
    rows, K = x.shape
    good, scales = mo.quantize(x)
    bad = scales == 255
    with np.errstate(invalid="ignore"):
        size = np.abs(x.reshape(rows, -1, 32)) / np.ldexp(1.0, exponents.astype(np.int64))[..., None]
        code = codes_of(size) if codes_of else np.abs(size[..., None] - mo.VALUES).argmin(-1)
    code = np.where(bad[..., None], 0, code | np.where(np.signbit(x.reshape(size.shape)), 8, 0))
    return mo.pack(code.reshape(rows, K)), np.where(bad, 255, exponents + 127).astype(np.uint8)


def test_the_definition_is_taken():
    x = _inputs()
    codes, scales = mo.quantize(x)
    mc.quantized(x, codes, scales)


PLANTED = ["scale up", "scale down", "ties away", "ties down", "nibbles swapped", "sign of zero lost", "nan kept", "cut"]


@pytest.mark.parametrize("mistake", PLANTED)
def test_wrong_quantizers_are_refused(mistake):
    x = _inputs()
    codes, scales = mo.quantize(x)
    e = scales.astype(np.int64) - 127
    if mistake == "scale up":
        codes, scales = _requantized(x, np.where(scales == 255, 0, e + 1))
    elif mistake == "scale down":
        codes, scales = _requantized(x, np.where(scales == 255, 0, np.maximum(e - 1, -127)))
    elif mistake == "ties away":
        codes, scales = _requantized(x, e, lambda s: 7 - np.abs(s[..., None] - mo.VALUES[::-1]).argmin(-1))
    elif mistake == "ties down":
        codes, scales = _requantized(x, e)
    elif mistake == "nibbles swapped":
        codes = (codes << 4 | codes >> 4).astype(np.uint8)
    elif mistake == "sign of zero lost":
        n = mo.unpack(codes)
        codes = mo.pack(np.where(n == 8, 0, n))
    elif mistake == "nan kept":
        scales = np.where(scales == 255, 254, scales).astype(np.uint8)
    else:
        codes, scales = _requantized(x, e, lambda s: (s[..., None] >= mo.VALUES).sum(-1).clip(1) - 1)
    with pytest.raises(AssertionError):
        mc.quantized(x, codes, scales)


def _rounded(x, w):
    return (torch.from_numpy(x.astype(np.float32)) @ torch.from_numpy(w.astype(np.float32)).t()).half()


@pytest.mark.parametrize("unit", mc.UNITS)
@pytest.mark.parametrize("low,high", mc.DEPTHS + [(33, 48)])
def test_products_of_wrong_weights_are_refused(low, high, unit):
    rng = np.random.default_rng(low)
    N, K, M = 90, 288, 3
    codes, scales = mc.deep_weights(rng, N, K, low, high, unit)
    x = mc.deep_inputs(rng, M, K, unit)
    right, plain = mc.float16_weights(codes, scales), mo.values(codes, scales)
    # all sums are exact in float32: float64 gives the same
    assert np.array_equal(x @ right.T, (x.astype(np.float32) @ right.astype(np.float32).T).astype(np.float64))
    mc.product(_rounded(x, right), x, right, "f16")
    top = scales.max(1).astype(np.int64)[:, None]
    lifted = right * np.ldexp(1.0, 140 - top)
    refused = [np.zeros_like(right), np.where(np.abs(plain) < np.ldexp(1.0, top - 127 - low), 0, plain),
               np.ldexp(right, 1)]
    if low >= 27:
        refused.append(np.where(np.abs(lifted) < 2.0 ** -14, 0, right))                  # subnormal operands as zeros
    if high > 36:
        unit_of = np.ldexp(1.0, top - 127 - 37)
        refused += [plain, np.trunc(plain / unit_of) * unit_of,                           # not rounded; cut
                    np.sign(plain) * np.floor(np.abs(plain) / unit_of + 0.5) * unit_of]    # ties away from zero
    for w in refused:
        with pytest.raises(AssertionError):
            mc.product(_rounded(x, w), x, right, "f16")


def test_blocks_of_zeros_do_not_count():
    codes, scales = np.zeros((2, 48), np.uint8), np.full((2, 3), 254, np.uint8)
    codes[0, 16:32], scales[0, 1] = 0x21, 127
    codes[1, :16] = 0x88
    assert mc.live(codes).tolist() == [[False, True, False], [False] * 3]
    assert np.array_equal(mc.float16_weights(codes, scales), mo.values(codes, scales))

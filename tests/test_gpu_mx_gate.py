"""The gate of the microscaled gated projection where 1 + exp(-a) passes 2^126 (a = g, or gelu's 2 t): its reciprocal lies
below float32's normal range, g times it within, and a large up side brings the result near one.

Bound: the header's formula in float32.  exp's argument, below 90, is rounded seven times at most: 7 2^-24 90 of the result; a
subnormal reciprocal of at least 2^-128 has steps of 2^-149, so is off by 2^-22 of itself; three products, a sum and a reciprocal
2^-21; and the result's own rounding."""
import numpy as np
import pytest

import oracle.mx_oracle as mo

pytestmark = pytest.mark.gpu
K = 96
# g as the sum of inputs 0, 1 and 32; in the format each block's must be so many halves of one power of two
PARTS = {"silu": [(-64.0, -24.0, 0.0), (-80.0, -7.5, 0.0), (-64.0, -23.5, 0.0), (-88.0, -0.625, 0.0)],
         "gelu_tanh": [(-10.0, -0.03125, 0.0), (-10.0, -0.015625, 0.0)]}
MX_PARTS = {"silu": [(-64.0, -24.0, 0.0), (-64.0, -24.0, 0.5), (-64.0, -24.0, -0.5)],
            "gelu_tanh": [(-8.0, -2.0, -0.03125), (-8.0, -2.0, -0.015625)]}


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("x_kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gates_past_2_126(act, x_kind, M):
    import torch
    import weight_only_quantized_amd as wq
    N = 2050
    one = np.zeros((N, K), np.uint8)
    gate, up = one.copy(), one.copy()
    gate[:, [0, 1, 32]], up[:, 64] = 2, 2                    # ones: g = x0 + x1 + x32, u = 2^120 x64
    scales = np.full((N, 3), 127, np.uint8)
    high = scales.copy()
    high[:, 2] = 247
    mx = lambda n, s: wq.MXTensor(torch.from_numpy(mo.pack(n)).cuda(), torch.from_numpy(s).cuda())  # noqa: E731
    layer = wq.MXGatedLinear(mx(gate, scales), mx(up, high), activation=act)
    for parts in (MX_PARTS if x_kind == "mx" else PARTS)[act]:
        x = np.zeros((M, K))
        x[:, [0, 1, 32]], x[:, 64] = parts, 1.0
        if x_kind == "mx":
            codes, s = mo.quantize(x)
            assert np.array_equal(mo.values(codes, s), x)
            given, tag = wq.MXTensor(torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda()), "bf16"
        else:
            given, tag = torch.from_numpy(x).to(torch.float16 if x_kind == "f16" else torch.bfloat16).cuda(), x_kind
            assert np.array_equal(given.cpu().double().numpy(), x)
        got = layer.gemm(given, dtype=torch.float16 if tag == "f16" else torch.bfloat16).cpu().double().numpy()
        g = sum(parts)
        a = g if act == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
        assert 2.0 ** 126 < np.exp(-a) < 2.0 ** 128
        want = mo.ACTIVATIONS[act](np.array([g]))[0] * 2.0 ** 120
        assert 0.01 < abs(want) < 10
        half = 2.0 ** -11 if tag == "f16" else 2.0 ** -8
        assert np.all(np.abs(got - want) <= (half + 2.0 ** -21 + 2.0 ** -22 + 7 * 2.0 ** -24 * 90) * abs(want)), (g, got[0, 0], want)

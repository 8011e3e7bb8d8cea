"""Float16 activations with microscaled weights far below their output's largest scale, on the GPU: exact down to 2^-36 of it,
and below that rounded as the header states, to multiples of 2^-37 of it.  The activations are zero where the
largest scale stands, so the small weights alone make the results, which are compared bit by bit."""
import numpy as np
import pytest

import mx_checks as mc
import oracle.mx_oracle as mo
from test_gpu_mx import _check_gated, _dev, _exact_on_gpu, _f64, _mx

pytestmark = pytest.mark.gpu

# few rows: one, four and eight tiles of outputs a wave, one to four tiles of rows; many rows by tiles of 64, 128 and
# 256; see the rules in mx_skinny.hip and mx_tiled.hip
SHAPES = [(2, 300), (12, 13000), (30, 500), (40, 25700), (64, 1300), (200, 4100), (1301, 4001), (4000, 4090)]
GATED = [(2, 150), (48, 12805), (200, 2050), (1301, 2001), (4000, 2045)]
K = 288


@pytest.mark.parametrize("unit", mc.UNITS)
@pytest.mark.parametrize("low,high", mc.DEPTHS)
@pytest.mark.parametrize("M,N", SHAPES)
def test_exact_down_to_2_36(low, high, unit, M, N):
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M + N + low)
    w, x = mc.deep_weights(rng, N, K, low, high, unit), mc.deep_inputs(rng, M, K, unit)
    assert np.array_equal(mc.float16_weights(*w), mo.values(*w))
    mc.product(wq.MXLinear(_mx(*w)).gemm(_dev(x, "f16")), x, mo.values(*w), "f16")


@pytest.mark.parametrize("M,N", SHAPES)
def test_rounded_below(M, N):
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M + N)
    w, x = mc.deep_weights(rng, N, K, 33, 48, 13), mc.deep_inputs(rng, M, K, 13)
    assert not np.array_equal(mc.float16_weights(*w), mo.values(*w))
    mc.product(wq.MXLinear(_mx(*w)).gemm(_dev(x, "f16")), x, mc.float16_weights(*w), "f16")


@pytest.mark.parametrize("low,high", [(27, 30), (33, 36), (33, 48)])
@pytest.mark.parametrize("M,N", GATED)
def test_gated(low, high, M, N):
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M + N)
    g, u = (mc.deep_weights(rng, N, K, low, high, 13) for _ in range(2))
    x = mc.deep_inputs(rng, M, K, 13)
    gv, uv = (_f64(v) for v in _exact_on_gpu(x, mc.float16_weights(*g), mc.float16_weights(*u)))
    want = mo.silu(gv) * uv
    _check_gated(_f64(wq.MXGatedLinear(_mx(*g), _mx(*u)).gemm(_dev(x, "f16"))), want, gv, uv, "silu", "f16")
    with pytest.raises(AssertionError):
        _check_gated(np.zeros_like(want), want, gv, uv, "silu", "f16")

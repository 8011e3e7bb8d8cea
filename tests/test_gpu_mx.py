"""Microscaled 4-bit floating point on the GPU against the float64 oracle.

Quantizing is compared bit by bit.  Products are tested in two ways.  With values whose partial sums all
fit float32 (multiples of 2^-4 below 2^20) the sum has no rounding in any order, so a product must be the
correctly rounded result bit by bit.  With other values a sum of K products is off by at most
K 2^-23 sum |x w| (K additions, each rounded or cut to 24 bits), and the result by half a step of its type
more.

A gated result g u / (1 + exp(-a)) (a = g, or gelu's 2 t) has besides: three products, a sum and a reciprocal,
2^-21 of itself; the exponential, whose argument is rounded at most seven times (gelu: g g, g, the fused sum, g,
the constants, log2 e), so off by 7 2^-24 |a|, as is exp(-a) relative to itself; and where 1 + exp(-a)
passes 2^126, its reciprocal is below float32's normal range, off by at most 2^-126."""
import numpy as np
import pytest

import oracle.mx_oracle as mo

pytestmark = pytest.mark.gpu
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SMALLEST = {"f16": 2.0 ** -25, "bf16": 0.0}          # half of the smallest step


def _dt(tag):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[tag]


def _dev(a, tag=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if tag is None else t.to(_dt(tag))).cuda()


def _mx(codes, scales):
    import weight_only_quantized_amd as wq
    return wq.MXTensor(_dev(codes), _dev(scales))


def _f64(t):
    import torch
    torch.cuda.synchronize()
    return t.detach().cpu().double().numpy()


def _rounded(v, tag):
    """float64 -> the nearest of the type, as float64 (through float32, which holds v exactly)."""
    import torch
    assert np.array_equal(v.astype(np.float32).astype(np.float64), v)
    return torch.from_numpy(v.astype(np.float32)).to(_dt(tag)).double().numpy()


def _random(rng, rows, K, lo=124, hi=131):
    """Codes and scales; products of two such rows sum without rounding where K (6 * 16)^2 < 2^24 2^-8."""
    return rng.integers(0, 256, (rows, K // 2), dtype=np.uint8), rng.integers(lo, hi, (rows, K // 32), dtype=np.uint8)


def _exact_pair(rng, rows, K):
    # values are multiples of 1/2 up to 12 in size: products multiples of 1/4 up to 144, K 144 * 4 < 2^24
    assert K <= 16384
    return _random(rng, rows, K, 127, 129)


# ---- quantizing ----------------------------------------------------------------------------------

def _check_quantized(x, tag):
    import weight_only_quantized_amd as wq
    t = wq.MXTensor.quantize(x)
    codes, scales = mo.quantize(_f64(x))
    got_c, got_s = t.codes.cpu().numpy(), t.scales.cpu().numpy()
    assert np.array_equal(got_s, scales)
    assert np.array_equal(got_c, codes)
    want = mo.values(codes, scales)
    for out in ("f32", "bf16"):
        back = _f64(t.dequantize(_dt(out)))
        assert np.array_equal(back, want.astype(np.float32).astype(np.float64), equal_nan=True), out
    import torch
    want16 = torch.from_numpy(want.astype(np.float32)).half().double().numpy()
    assert np.array_equal(_f64(t.dequantize(torch.float16)), want16, equal_nan=True)


@pytest.mark.parametrize("tag", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 4096), (3, 96), (17, 4160), (130, 32), (5, 14336), (513, 544)])
def test_quantize(tag, rows, K):
    rng = np.random.default_rng(rows * 7 + K)
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-9, 9, (rows, K // 32)).repeat(32, 1))
    x[0, :32] = 0
    x[-1, -32:] *= -1
    _check_quantized(_dev(x, tag), tag)


@pytest.mark.parametrize("tag", ["f16", "bf16"])
def test_quantize_every_16_bit_value(tag):
    """Every bit pattern, alone in its block and beside a larger one of every few binades."""
    import torch
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).cuda().view(_dt(tag))
    x = torch.zeros((65536, 32), dtype=_dt(tag), device="cuda")
    x[:, 5] = bits
    _check_quantized(x, tag)
    for top in ([2.0 ** -24, 2.0 ** -14, 0.0625, 1.0, 5.0, 448.0, 65504.0] if tag == "f16"
                else [2.0 ** -133, 2.0 ** -126, 2.0 ** -124, 2.0 ** -60, 1.0, 7.0, 2.0 ** 100, 3.3e38]):
        x[:, 30] = top
        _check_quantized(x, tag)


def test_quantize_float32_ties_and_ends():
    grid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.0, 0.0])
    cols = np.concatenate([grid, np.nextafter(grid.astype(np.float32), np.float32(9)).astype(np.float64),
                           np.nextafter(grid.astype(np.float32), np.float32(-9)).astype(np.float64)])
    x = np.zeros((160, 64))
    for i, e in enumerate(np.linspace(-149, 124, 160).astype(int)):
        x[i, :30] = np.ldexp(cols, e)
        x[i, 31] = np.ldexp(4.0, min(e, 124))
        x[i, 32:62] = -np.ldexp(cols, e)
    x = x.astype(np.float32).astype(np.float64)
    _check_quantized(_dev(x, "f32"), "f32")


def test_quantize_not_finite():
    import torch
    x = torch.ones((4, 96), device="cuda")
    x[0, 3], x[1, 40], x[2, 95] = float("inf"), float("-inf"), float("nan")
    for tag in ("f16", "bf16", "f32"):
        _check_quantized(x.to(_dt(tag)), tag)


def test_quantize_strides_and_padding():
    import torch
    import weight_only_quantized_amd as wq
    wide = torch.randn((37, 512), device="cuda").bfloat16()
    for x in (wide[:, 64:160], wide[:, 4:100], wide.t()[:, :32], wide[::2, :96], wide[:1, 8:40]):
        _check_quantized(x, "bf16")
    # bytes between a row's scales and the next row's are left alone
    lib = wq.load_library()
    x = wide[:, :96].contiguous()
    codes = torch.full((37, 48), 7, dtype=torch.uint8, device="cuda")
    scales = torch.full((37, 8), 201, dtype=torch.uint8, device="cuda")
    from weight_only_quantized_amd.mx import _TENSOR
    c = _TENSOR.pack(codes.data_ptr(), scales.data_ptr(), 8, 37, 96, 0)
    assert lib.gptq_mx_quantize(x.data_ptr(), 96, 1, c, torch.cuda.current_stream().cuda_stream) == 0
    want_c, want_s = mo.quantize(_f64(x))
    assert np.array_equal(codes.cpu().numpy(), want_c) and np.array_equal(scales[:, :3].cpu().numpy(), want_s)
    assert (scales[:, 3:] == 201).all()


# ---- products ------------------------------------------------------------------------------------

def _x16(rng, M, K, tag):
    """Multiples of 1/4 up to 4: with weights that are multiples of 1/2 up to 12, sums stay exact."""
    return rng.integers(-16, 17, (M, K)) / 4.0


SHAPES = [(1, 40, 32), (2, 16, 96), (1, 257, 128), (16, 33, 160), (17, 64, 256), (33, 1, 288), (48, 100, 512),
          (49, 130, 544), (64, 96, 1024), (65, 48, 416), (100, 255, 704), (128, 256, 256), (129, 300, 1120),
          (257, 513, 800), (300, 64, 4160), (520, 770, 1280), (1, 4096, 4096), (16, 1000, 8192)]


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_exact(tag, M, N, K):
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    w = _exact_pair(rng, N, K)
    layer = wq.MXLinear(_mx(*w))
    wv = mo.values(*w)
    x = _x16(rng, M, K, tag)
    assert np.array_equal(_f64(layer.gemm(_dev(x, tag))), _rounded(mo.gemm(x, wv), tag))
    xq = _exact_pair(rng, M, K)
    assert np.array_equal(_f64(layer.gemm(_mx(*xq), dtype=_dt(tag))), _rounded(mo.gemm(mo.values(*xq), wv), tag))


def _check_gated(got, want, g, u, act, tag, sums=0.0):
    a = g if act == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    off = 2.0 ** -21 + 7 * 2.0 ** -24 * np.minimum(np.abs(a), 90.0)
    bound = (HALF_STEP[tag] + off) * np.abs(want) + 2.0 ** -126 * np.abs(g * u) + SMALLEST[tag] + sums
    worst = np.max(np.abs(got - want) - bound)
    assert worst <= 0, worst


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gated(act, tag, M, N, K):
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    g, u = _exact_pair(rng, N, K), _exact_pair(rng, N, K)
    g = (g[0], g[1] - 5)                       # gates of all sizes, not only of the flat ends
    layer = wq.MXGatedLinear(_mx(*g), _mx(*u), activation=act)
    x16, xq = _x16(rng, M, K, tag) / 16, _exact_pair(rng, M, K)
    xq = (xq[0], xq[1] - 4)
    for x, xv in ((_dev(x16, tag), x16), (_mx(*xq), mo.values(*xq))):
        want = mo.gated(xv, mo.values(*g), mo.values(*u), act)
        got = _f64(layer.gemm(x, dtype=_dt(tag)))
        _check_gated(got, want, mo.gemm(xv, mo.values(*g)), mo.gemm(xv, mo.values(*u)), act, tag)


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 512, 14336), (7, 300, 4096), (40, 200, 2048), (200, 384, 4096), (700, 520, 1056)])
def test_product_any_values(tag, M, N, K):
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M + N + K)
    w = mo.quantize(rng.standard_normal((N, K)) * np.exp(rng.standard_normal((N, 1))))
    x = _f64(_dev(rng.standard_normal((M, K)) * np.exp(rng.standard_normal((1, K))), tag))
    xq = mo.quantize(x)
    layer = wq.MXLinear(_mx(*w))
    wv = mo.values(*w)
    for given, xv in ((_dev(x, tag), x), (_mx(*xq), mo.values(*xq))):
        want, most = mo.gemm(xv, wv), mo.gemm(np.abs(xv), np.abs(wv))
        got = _f64(layer.gemm(given, dtype=_dt(tag)))
        assert np.all(np.abs(got - want) <= HALF_STEP[tag] * np.abs(want) + K * 2.0 ** -23 * most + SMALLEST[tag])
        # the sums' own error is far below the results' rounding, taken over all of them
        assert np.linalg.norm(got - want) <= (HALF_STEP[tag] * 1.01) * np.linalg.norm(want)


@pytest.mark.parametrize("M", [1, 30, 64, 70, 200, 700])
@pytest.mark.parametrize("K", [32, 96, 160, 288, 416, 1056])
def test_product_reads_nothing_beside(M, K):
    """Rows whose neighbours in memory are NaN: inputs past K, bytes past a row's scales, rows past the last."""
    import torch
    import weight_only_quantized_amd as wq
    from weight_only_quantized_amd.mx import _scales_fit
    rng = np.random.default_rng(M + K)
    w = _exact_pair(rng, 200, K)
    layer, wv = wq.MXLinear(_mx(*w)), mo.values(*w)
    x = _x16(rng, M, K, "bf16")
    wide = torch.full((M + 300, K + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:M, :K] = _dev(x, "bf16")
    assert np.array_equal(_f64(layer.gemm(wide[:M, :K])), _rounded(mo.gemm(x, wv), "bf16"))
    c, s = _exact_pair(rng, M, K)
    codes = torch.full((M + 300, K // 2), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((M + 300, K // 32 // 4 * 4 + 8), 255, dtype=torch.uint8, device="cuda")
    codes[:M], scales[:M, :K // 32] = _dev(c), _dev(s)
    assert _scales_fit(scales[:M, :K // 32])
    t = wq.MXTensor(codes[:M], scales[:M, :K // 32])
    assert t.scales.data_ptr() == scales.data_ptr()
    assert np.array_equal(_f64(layer.gemm(t)), _rounded(mo.gemm(mo.values(c, s), wv), "bf16"))


@pytest.mark.parametrize("x_kind", ["16", "mx"])
@pytest.mark.parametrize("M,N,K", [(4400, 4104, 96), (4097, 4360, 1056), (2049, 8200, 1312), (5000, 4096, 2048)])
def test_product_of_many_tiles(x_kind, M, N, K):
    """More tiles than the card has compute units: a workgroup takes several, one after the other."""
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M + N + K)
    w = _exact_pair(rng, N, K)
    wv = mo.values(*w)
    if x_kind == "16":
        x = _x16(rng, M, K, "f16")
        given, xv = _dev(x, "f16"), x
    else:
        xq = _exact_pair(rng, M, K)
        given, xv = _mx(*xq), mo.values(*xq)
    import torch
    got = wq.MXLinear(_mx(*w)).gemm(given, dtype=torch.float16)
    # float32 holds these sums exactly in any order, as it does in the product
    want = torch.from_numpy(xv.astype(np.float32)).cuda() @ torch.from_numpy(wv.astype(np.float32)).cuda().t()
    assert torch.equal(got, want.half())

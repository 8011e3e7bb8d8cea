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


# ---- every form of the products ------------------------------------------------------------------

def _exact_on_gpu(x, *sides):
    """x W^T of exactly summable values, in float32 (any order gives the same), as float64 tensors."""
    import torch
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    return [(t @ torch.from_numpy(w.astype(np.float32)).cuda().t()).double() for w in sides]


# rows, outputs, inputs: one and several row tiles, one to nine steps (even, odd, last ones not full), few and many
# tiles a wave, tiles of 64, 128 and 256; see the rules in mx_skinny.hip and mx_tiled.hip
FORMS = ([(m, 12805, k) for m in (1, 8, 9, 16, 17, 33, 64) for k in (288, 1120)]
         + [(200, 4100, k) for k in (32, 64, 96, 256, 288, 512, 544, 768, 1056, 1312, 1568, 2304)]
         + [(m, 6401, k) for m in (5, 16, 30, 48, 60) for k in (416,)] + [(1301, 4001, 416), (1301, 4000, 1312), (300, 130, 2048)])


@pytest.mark.parametrize("x_kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("M,N,K", FORMS)
def test_every_form(x_kind, M, N, K):
    import torch
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M + N + K)
    w = _exact_pair(rng, N, K)
    if x_kind == "mx":
        xq = _exact_pair(rng, M, K)
        given, xv, dt = _mx(*xq), mo.values(*xq), torch.bfloat16
    else:
        xv = _x16(rng, M, K, x_kind)
        given, dt = _dev(xv, x_kind), _dt(x_kind)
    got = wq.MXLinear(_mx(*w)).gemm(given, dtype=dt)
    assert torch.equal(got, _exact_on_gpu(xv, mo.values(*w))[0].to(dt))


@pytest.mark.parametrize("x_kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("M,N,K", [(m, 6404, 416) for m in (1, 16, 30, 48, 60)] + [(200, 2050, k) for k in (96, 544, 1312)]
                         + [(1301, 2001, 416), (4100, 2056, 288), (4100, 2051, 1056)])
def test_every_gated_form(x_kind, M, N, K):
    import torch
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M + N + K)
    g, u = _exact_pair(rng, N, K), _exact_pair(rng, N, K)
    g = (g[0], g[1] - 5)
    if x_kind == "mx":
        xq = _exact_pair(rng, M, K)
        xq = (xq[0], xq[1] - 4)
        given, xv, tag = _mx(*xq), mo.values(*xq), "bf16"
    else:
        xv = _x16(rng, M, K, x_kind) / 16
        given, tag = _dev(xv, x_kind), x_kind
    gv, uv = _exact_on_gpu(xv, mo.values(*g), mo.values(*u))
    got = wq.MXGatedLinear(_mx(*g), _mx(*u), activation="silu").gemm(given, dtype=_dt(tag))
    gv, uv = _f64(gv), _f64(uv)
    _check_gated(_f64(got), mo.silu(gv) * uv, gv, uv, "silu", tag)


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(33, 25605, 288), (48, 25700, 1120), (40, 25664, 32), (47, 25599, 2336)])
def test_eight_tiles_a_wave(tag, M, N, K):
    """33 to 48 rows of 16 bits by many outputs: whole groups of eight tiles, and last ones of one and of seven."""
    import torch
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M + N + K)
    w = _exact_pair(rng, N, K)
    for n, by in ((5, 3), (N - 20, 1), (N - 1, 2)):          # rows of their own largest scale: multiples of 2^-6 below 2^18
        w[1][n] -= by
    xv = _x16(rng, M, K, tag)
    want = _exact_on_gpu(xv, mo.values(*w))[0].to(_dt(tag))
    assert torch.equal(wq.MXLinear(_mx(*w)).gemm(_dev(xv, tag)), want)


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(48, 12805, 416), (33, 12864, 96)])
def test_eight_gated_tiles_a_wave(tag, M, N, K):
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M + N + K)
    g, u = _exact_pair(rng, N, K), _exact_pair(rng, N, K)
    g = (g[0], g[1] - 5)
    xv = _x16(rng, M, K, tag) / 16
    gv, uv = (_f64(v) for v in _exact_on_gpu(xv, mo.values(*g), mo.values(*u)))
    got = wq.MXGatedLinear(_mx(*g), _mx(*u), activation="silu").gemm(_dev(xv, tag))
    _check_gated(_f64(got), mo.silu(gv) * uv, gv, uv, "silu", tag)


# ---- the ends of the format ----------------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 40, 300])
def test_blocks_of_nan(M):
    """A block of NaN makes the outputs it takes part in NaN, and no others."""
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M)
    K, N = 544, 4100
    w, xq = _exact_pair(rng, N, K), _exact_pair(rng, M, K)
    w[1][7, 16], w[1][4099, 0], xq[1][M // 2, 3] = 255, 255, 255
    layer = wq.MXLinear(_mx(*w))
    x = _x16(rng, M, K, "f16")
    x[0, 5] = np.nan
    for given, xv, tag in ((_dev(x, "f16"), x, "f16"), (_dev(x, "bf16"), x, "bf16"), (_mx(*xq), mo.values(*xq), "bf16")):
        got = _f64(layer.gemm(given, dtype=_dt(tag)))
        bad = np.isnan(xv).any(1)[:, None] | np.isnan(mo.values(*w)).any(1)[None]
        assert np.array_equal(np.isnan(got), bad)
        want = _rounded(mo.gemm(np.nan_to_num(xv), np.nan_to_num(mo.values(*w))), tag)
        assert np.array_equal(got[~bad], want[~bad])


@pytest.mark.parametrize("M", [1, 12, 300])
def test_infinite_activations(M):
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M)
    K, N = 288, 4100
    w = (np.full((N, K // 2), 0x22, np.uint8), np.full((N, K // 32), 127, np.uint8))       # all ones
    x = _x16(rng, M, K, "bf16")
    x[0, 7] = np.inf
    x[-1, 200] = -np.inf
    for tag in ("f16", "bf16"):
        got, want = _f64(wq.MXLinear(_mx(*w)).gemm(_dev(x, tag))), x.sum(1)
        for m in range(M):
            if np.isfinite(want[m]):
                assert (got[m] == _rounded(want[m:m + 1], tag)[0]).all()
            else:
                assert np.array_equal(got[m], np.full(N, want[m]), equal_nan=True)


@pytest.mark.parametrize("M", [2, 200])
@pytest.mark.parametrize("x_kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("top", [40, 127, 200])
def test_scales_far_apart(x_kind, M, top):
    """Rows of weights of one size each, 2^-36 and up below the largest of their own; whole rows by the type's range."""
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M + top)
    K, N = 256, 4100
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = rng.integers(top - 36, top + 1, (N, K // 32)).astype(np.uint8)
    scales[:, 3] = top
    wv = mo.values(codes, scales)
    layer = wq.MXLinear(_mx(codes, scales))
    shift = 2.0 ** (127 - top)                               # results near one: the types hold them
    if x_kind == "mx":
        c = rng.integers(0, 256, (M, K // 2), dtype=np.uint8)
        s = np.full((M, K // 32), 254 - top, np.uint8)
        given, xv, tag = _mx(c, s), mo.values(c, s), "bf16"
    elif x_kind == "bf16":
        xv = _x16(rng, M, K, "bf16") * shift
        given, tag = _dev(xv, "bf16"), "bf16"
    else:
        if top != 127:
            pytest.skip("float16 has no activations that bring such results near one")
        xv = _x16(rng, M, K, "f16")
        given, tag = _dev(xv, "f16"), "f16"
    want, most = mo.gemm(xv, wv), mo.gemm(np.abs(xv), np.abs(wv))
    got = _f64(layer.gemm(given, dtype=_dt(tag)))
    assert np.all(np.abs(got - want) <= HALF_STEP[tag] * np.abs(want) + K * 2.0 ** -23 * most + SMALLEST[tag])


@pytest.mark.parametrize("M", [2, 40, 200, 1100])
@pytest.mark.parametrize("case", ["bf16 weights", "bf16 activations", "f16 activations", "mx weights", "mx activations"])
def test_operands_below_the_normal_range(case, M):
    """Subnormal 16-bit operands, and scales at the format's ends, times what brings them near one.  Sums are fewer
    than 2^22 steps of one size: float32 holds them exactly."""
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M)
    K, N = 256, 1300
    # the smallest weight scale, and the activations' unit or smallest scale byte
    low, unit, kind = {"bf16 weights": (0, 120, "bf16"), "bf16 activations": (249, -131, "bf16"), "f16 activations": (144, -22, "f16"),
                       "mx weights": (0, 251, "mx"), "mx activations": (251, 0, "mx")}[case]
    w = rng.integers(0, 256, (N, K // 2), dtype=np.uint8), rng.integers(low, low + 4, (N, K // 32)).astype(np.uint8)
    if kind == "mx":
        xq = rng.integers(0, 256, (M, K // 2), dtype=np.uint8), rng.integers(unit, unit + 4, (M, K // 32)).astype(np.uint8)
        given, xv, tag = _mx(*xq), mo.values(*xq), "bf16"
    else:
        xv = rng.integers(-16, 17, (M, K)) / 4 * 2.0 ** unit
        given, tag = _dev(xv, kind), kind
        assert np.array_equal(_f64(given), xv)
    got = _f64(wq.MXLinear(_mx(*w)).gemm(given, dtype=_dt(tag)))
    assert np.array_equal(got, _rounded(mo.gemm(xv, mo.values(*w)), tag))


def test_float16_weights_below_the_range():
    """Scales more than 2^-36 below their row's largest: rounded to 2^-37 of that, as stated."""
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(0)
    K, N, M = 128, 64, 3
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = rng.integers(127 - 60, 128 - 36, (N, K // 32)).astype(np.uint8)
    scales[:, 0] = 127
    x = _x16(rng, M, K, "f16")
    x[:, :32] = 0                                            # only the small blocks count
    want = mo.gemm(x * 2.0 ** 15, mo.values(codes, scales))
    got = _f64(wq.MXLinear(_mx(codes, scales)).gemm(_dev(x * 2.0 ** 13, "f16"))) * 4
    assert np.all(np.abs(got - want) <= (np.abs(x) * 2.0 ** 15).sum(1)[:, None] * 2.0 ** -37 + 2.0 ** -11 * np.abs(want) + 2.0 ** -23)


# ---- calls ---------------------------------------------------------------------------------------

def test_strides_out_and_equal_bits():
    import torch
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(3)
    K, N = 288, 333
    w = _exact_pair(rng, N, K)
    layer = wq.MXLinear(_mx(*w))
    wide = torch.randn((90, 1024), device="cuda").bfloat16()
    for x in (wide[:, 8:8 + K], wide[:, 3:3 + K], wide[::3, :K], wide.t()[:K].t()[:, :K], wide[5:6, :K], wide[:0, :K]):
        out = torch.empty((x.shape[0], N), dtype=torch.bfloat16, device="cuda")
        assert layer.gemm(x, out=out) is out
        assert torch.equal(out, layer.gemm(x.contiguous()))
    for M in (1, 64, 300):
        x = torch.randn((M, K), device="cuda").half()
        a = layer.gemm(x)
        for _ in range(3):
            assert torch.equal(a, layer.gemm(x))
    q = wq.MXTensor.quantize(wide[:, :K])
    assert layer.gemm(q).dtype == torch.bfloat16 and layer.gemm(q, dtype=torch.float16).dtype == torch.float16
    for kw, error in ((dict(dtype=torch.float32), TypeError), (dict(out=torch.empty((90, N), device="cuda")), TypeError),
                      (dict(out=torch.empty((89, N), device="cuda").half()), ValueError)):
        with pytest.raises(error):
            layer.gemm(q, **kw)
    with pytest.raises(ValueError):
        layer.gemm(wide)
    with pytest.raises(TypeError):
        layer.gemm(wide[:, :K].float())
    with pytest.raises(wq.GPTQError):
        layer.gemm(q, out=layer.packed[:90 * N * 2].view(torch.bfloat16).view(90, N))


def test_other_streams_and_graphs():
    import torch
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(4)
    K, N, M = 1056, 700, 150
    g, u, d = (_mx(*mo.quantize(rng.standard_normal(s) / 30)) for s in ((N, K), (N, K), (K, 704)))
    up, down = wq.MXGatedLinear(g, u), wq.MXLinear(d)
    x = torch.randn((M, K), device="cuda").bfloat16()

    def block(x, stream=None):
        h = torch.zeros((M, 704), dtype=x.dtype, device="cuda")
        h[:, :N] = up.gemm(wq.MXTensor.quantize(x))
        return down.gemm(wq.MXTensor.quantize(h)) + down.gemm(h)

    want = block(x)
    side = torch.cuda.Stream()
    q = wq.MXTensor.quantize(x, stream=side)
    h = up.gemm(q, stream=side)
    back = q.dequantize(torch.float32, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(h, up.gemm(wq.MXTensor.quantize(x)))
    assert torch.equal(back, wq.MXTensor.quantize(x).dequantize(torch.float32))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x)
    torch.cuda.current_stream().wait_stream(side)
    static, graph = x.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(static)
    for i in range(4):
        new = torch.randn((M, K), device="cuda").bfloat16() if i else x
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, block(new) if i else want), i


def test_feed_forward_block_with_adapters():
    """Gate, up and down projections in the format, a request's adapter beside the last: as a layer is served."""
    import torch
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(6)
    D, F, M = 512, 1376, 9
    g, u, d = (mo.quantize(rng.standard_normal(s) / s[1] ** 0.5) for s in ((F, D), (F, D), (D, F)))
    up, down = wq.MXGatedLinear(_mx(*g), _mx(*u), activation="gelu_tanh"), wq.MXLinear(_mx(*d))
    a = torch.randn((3, 16, F), device="cuda").bfloat16() * F ** -0.5
    b = torch.randn((3, D, 16), device="cuda").bfloat16() * 0.25
    bank = wq.LoraBank(a, b, torch.ones(3, device="cuda"))
    ids = torch.tensor([0, 1, 2, -1, 0, 0, 2, 1, -1], dtype=torch.int32, device="cuda")
    x = torch.randn((M, D), device="cuda").bfloat16()
    for mx in (False, True):
        h = up.gemm(wq.MXTensor.quantize(x) if mx else x)
        hv, y = _f64(h), down.gemm(wq.MXTensor.quantize(h) if mx else h)
        got = _f64(bank.add(y, h, ids, out=y))
        if mx:
            xv, hin = mo.values(*mo.quantize(_f64(x))), mo.values(*mo.quantize(hv))
        else:
            xv, hin = _f64(x), hv
        # each step against the step before it as it was, rounded: half a step each, and sums' own error
        want_h = mo.gated(xv, mo.values(*g), mo.values(*u), "gelu_tanh")
        assert np.linalg.norm(hv - want_h) <= 1.02 * HALF_STEP["bf16"] * np.linalg.norm(want_h)
        y0, extra = mo.gemm(hin, mo.values(*d)), np.zeros((M, D))
        av, bv = _f64(a), _f64(b)
        for m, i in enumerate(ids.tolist()):
            if i >= 0:
                extra[m] = bv[i] @ (av[i] @ hv[m])
        bound = HALF_STEP["bf16"] * 1.05 * (np.linalg.norm(y0) + np.linalg.norm(y0 + extra))
        assert np.linalg.norm(got - (y0 + extra)) <= bound


def test_offsets_past_32_bits():
    """Weights of more than 4 GiB of codes, results of more than 2^32 bytes, quantized rows past 2^31 values."""
    import torch
    import weight_only_quantized_amd as wq
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    N, K = (1 << 19) + 5, 16640
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(127, 129, (N, K // 32), dtype=torch.uint8, device="cuda", generator=gen)
    assert codes.numel() > 1 << 32
    layer = wq.MXLinear(wq.MXTensor(codes, scales))
    rng = np.random.default_rng(1)
    at = [0, 1, 262143, 262144, 400001, N - 17, N - 1]
    wv = mo.values(codes[at].cpu().numpy(), scales[at].cpu().numpy())
    x = _x16(rng, 3, K, "f16") / 4
    got = _f64(layer.gemm(_dev(x, "f16"))[:, at])
    assert np.array_equal(got, _rounded(mo.gemm(x, wv), "f16"))
    xq = _random(rng, 70, K, 124, 126)
    got = _f64(layer.gemm(_mx(*xq), dtype=torch.float16)[:, at])
    assert np.array_equal(got, _rounded(mo.gemm(mo.values(*xq), wv), "f16"))
    del codes, scales, layer
    M, N, K = 70001, 33000, 32
    w = _exact_pair(rng, N, K)
    x = (torch.randint(-16, 17, (M, K), device="cuda", generator=gen) / 4).bfloat16()
    y = wq.MXLinear(_mx(*w)).gemm(x)
    assert y.numel() * 2 > 1 << 32
    rows = [0, 1, 32767, 65536, M - 1]
    assert np.array_equal(_f64(y[rows]), _rounded(mo.gemm(_f64(x[rows]), mo.values(*w)), "bf16"))
    del y
    x = torch.randn((1 << 17, 16448), device="cuda", generator=gen).bfloat16()
    assert x.numel() > 1 << 31
    t = wq.MXTensor.quantize(x)
    back = t.dequantize(torch.bfloat16)
    rows = [0, 65535, 65536, 130560, 131071]
    c, s = mo.quantize(_f64(x[rows]))
    assert np.array_equal(t.codes[rows].cpu().numpy(), c) and np.array_equal(t.scales[rows].cpu().numpy(), s)
    assert np.array_equal(_f64(back[rows]), mo.values(c, s))

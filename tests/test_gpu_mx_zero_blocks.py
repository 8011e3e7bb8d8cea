"""Blocks of zeros among microscaled weights, on the GPU.  A block whose codes are all 0 or -0 is worth nothing
whatever its scale below 255, so it must not decide to which unit the other weights of its output are rounded
where they meet float16 activations.  Sums of the values used are exact in float32 in any order: results are
compared bit by bit, those of the gated form under the bound that tests/test_gpu_mx.py derives."""
import numpy as np
import pytest

import oracle.mx_oracle as mo

pytestmark = pytest.mark.gpu
ZEROS = np.array([0x00, 0x08, 0x80, 0x88], np.uint8)


def _dt(tag):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16}[tag]


def _mx(codes, scales):
    import torch
    import weight_only_quantized_amd as wq
    return wq.MXTensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())


def _weights(rng, N, K, lo, byte):
    """Rows of ordinary blocks, scales 2^lo and twice that; in every row some blocks of zeros under scale `byte`."""
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = rng.integers(127 + lo, 129 + lo, (N, K // 32)).astype(np.uint8)
    zero = rng.random((N, K // 32)) < 0.4
    zero[:, 1] = True
    zero[:, 2] = False
    codes[zero.repeat(16, 1)] = rng.choice(ZEROS, int(zero.sum()) * 16)
    scales[zero] = byte
    return codes, scales


def _inputs(rng, M, K, x_kind, lo):
    """(what the call takes, its values, the results' type): multiples of 2^lo / 4 up to 4 2^lo, or codes so scaled."""
    import torch
    if x_kind == "mx":
        codes = rng.integers(0, 256, (M, K // 2), dtype=np.uint8)
        scales = rng.integers(127 + lo, 129 + lo, (M, K // 32)).astype(np.uint8)
        return _mx(codes, scales), mo.values(codes, scales), "bf16"
    x = rng.integers(-16, 17, (M, K)) / 4 * 2.0 ** lo
    return torch.from_numpy(x).to(_dt(x_kind)).cuda(), x, x_kind


# few rows, one and several output tiles a wave; many rows by tiles of 64, 128 and 256
SHAPES = [(1, 70, 96), (12, 13000, 288), (40, 25700, 288), (64, 1300, 544), (200, 4100, 288), (1301, 4001, 288),
          (4000, 4090, 288)]


@pytest.mark.parametrize("byte", [170, 254])
@pytest.mark.parametrize("x_kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(x_kind, byte, M, N, K):
    import torch
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M + N + K)
    w = _weights(rng, N, K, 0, byte)
    given, xv, tag = _inputs(rng, M, K, x_kind, 0)
    got = wq.MXLinear(_mx(*w)).gemm(given, dtype=_dt(tag))
    want = torch.from_numpy(xv.astype(np.float32)).cuda() @ torch.from_numpy(mo.values(*w).astype(np.float32)).cuda().t()
    assert torch.equal(got, want.to(_dt(tag)))


@pytest.mark.parametrize("x_kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("M,N,K", [(1, 70, 96), (48, 12805, 288), (300, 2050, 288)])
def test_gated(x_kind, M, N, K):
    import torch
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M + N + K)
    g, u = _weights(rng, N, K, -5, 254), _weights(rng, N, K, 0, 200)
    given, xv, tag = _inputs(rng, M, K, x_kind, -4)
    got = wq.MXGatedLinear(_mx(*g), _mx(*u)).gemm(given, dtype=_dt(tag)).cpu().double().numpy()
    x32 = torch.from_numpy(xv.astype(np.float32)).cuda()
    gv, uv = ((x32 @ torch.from_numpy(mo.values(*w).astype(np.float32)).cuda().t()).cpu().double().numpy() for w in (g, u))
    want = mo.silu(gv) * uv
    half, smallest = {"f16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 0.0)}[tag]
    off = 2.0 ** -21 + 7 * 2.0 ** -24 * np.minimum(np.abs(gv), 90.0)
    bound = (half + off) * np.abs(want) + 2.0 ** -126 * np.abs(gv * uv) + smallest
    assert np.all(np.abs(got - want) <= bound)
    assert np.any(np.abs(want) > bound)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_blocks_of_zeros_that_are_nan(M):
    """A scale of 255 makes the block NaN whatever its codes."""
    import torch
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(M)
    K, N = 288, 4100
    codes, scales = _weights(rng, N, K, 0, 200)
    codes[7, 16:32], codes[4099, 128:144] = 0, 0x88
    scales[7, 1], scales[4099, 8] = 255, 255
    for x_kind in ("f16", "bf16", "mx"):
        given, _, tag = _inputs(rng, M, K, x_kind, 0)
        bad = torch.isnan(wq.MXLinear(_mx(codes, scales)).gemm(given, dtype=_dt(tag)))
        assert bad[:, [7, 4099]].all() and int(bad.sum()) == 2 * M


def test_weights_of_zeros_alone():
    import torch
    import weight_only_quantized_amd as wq
    rng = np.random.default_rng(0)
    codes, scales = rng.choice(ZEROS, (70, 48)), np.full((70, 3), 254, np.uint8)
    for M in (1, 200):
        for x_kind in ("f16", "bf16", "mx"):
            given, _, tag = _inputs(rng, M, 96, x_kind, 0)
            assert not wq.MXLinear(_mx(codes, scales)).gemm(given, dtype=_dt(tag)).any()

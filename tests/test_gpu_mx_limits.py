"""Microscaled operators at the largest sizes that the header allows: inputs, outputs, rows and strides.  Values are ones,
zeros and minus ones, so that float32 sums are exact (fewer than 2^24 of them) and results compare bit by bit."""
import pytest

pytestmark = pytest.mark.gpu
ONE, MINUS = 2, 10


def _signs(shape, gen):
    import torch
    return torch.randint(-1, 2, shape, device="cuda", generator=gen, dtype=torch.int8)


def _mx(v):
    """Signs as codes under scales of 1."""
    import torch
    import weight_only_quantized_amd as wq
    n = torch.where(v == 1, ONE, torch.where(v == -1, MINUS, 0)).to(torch.uint8)
    return wq.MXTensor(n[:, 0::2] | n[:, 1::2] << 4, torch.full((v.shape[0], v.shape[1] // 32), 127, dtype=torch.uint8, device="cuda"))


def _gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("M", [1, 16, 40, 64, 70, 200])
def test_most_inputs(M):
    """2^20 inputs, rows of x up to 2^21 values apart, against three tiles of outputs."""
    import torch
    import weight_only_quantized_amd as wq
    K, N, gen = 1 << 20, 40, _gen(M)
    w, x = _signs((N, K), gen), _signs((M, K), gen)
    want = x.float() @ w.float().t()
    layer = wq.MXLinear(_mx(w))
    room = torch.full((M, 1 << 21), float("nan"), dtype=torch.float16, device="cuda")
    room[:, :K] = x
    for given in (room[:, :K], x.bfloat16(), _mx(x)):
        dt = getattr(given, "dtype", torch.bfloat16)
        assert torch.equal(layer.gemm(given, dtype=dt), want.to(dt))
    t = wq.MXTensor.quantize(room[:, :K])
    assert torch.equal(t.dequantize(torch.float16), x.half())


@pytest.mark.parametrize("M", [1, 20, 48, 64, 70, 130])
def test_most_outputs(M):
    import torch
    import weight_only_quantized_amd as wq
    K, N, gen = 32, 1 << 20, _gen(M)
    w, x = _signs((N, K), gen), _signs((M, K), gen)
    want = x.float() @ w.float().t()
    layer, pair = wq.MXLinear(_mx(w)), wq.MXGatedLinear(_mx(w), _mx(w))
    for given in (x.half(), x.bfloat16(), _mx(x)):
        dt = getattr(given, "dtype", torch.bfloat16)
        assert torch.equal(layer.gemm(given, dtype=dt), want.to(dt))
        gated, ref = pair.gemm(given, dtype=dt).float(), want * torch.sigmoid(want) * want
        # half a step of the type, and eight float32 roundings on either side, of arguments up to 32
        half = 2.0 ** -11 if dt == torch.float16 else 2.0 ** -8
        assert bool(((gated - ref).abs() <= (half + 2.0 ** -17) * ref.abs() + 2.0 ** -25).all())


@pytest.mark.parametrize("N", [1, 70])
def test_most_rows(N):
    import torch
    import weight_only_quantized_amd as wq
    K, M, gen = 32, 1 << 24, _gen(N)
    w, x = _signs((N, K), gen), _signs((M, K), gen).bfloat16()
    layer = wq.MXLinear(_mx(w))
    want = (x.float() @ w.float().t()).bfloat16()
    assert torch.equal(layer.gemm(x), want)
    t = wq.MXTensor.quantize(x)
    assert torch.equal(layer.gemm(t), want)
    assert torch.equal(t.dequantize(torch.bfloat16), x)
    with pytest.raises(wq.GPTQError):
        layer.gemm(torch.zeros((M + 1, K), dtype=torch.bfloat16, device="cuda"))


def test_rows_that_repeat_one():
    """Expanded rows lie no elements apart: they are copied."""
    import torch
    import weight_only_quantized_amd as wq
    gen = _gen(0)
    w, row = _signs((70, 96), gen), _signs((1, 96), gen).half()
    layer, t = wq.MXLinear(_mx(w)), wq.MXTensor.quantize(row.expand(75, 96))
    want = (row.float() @ w.float().t()).half().expand(75, 70)
    assert torch.equal(layer.gemm(row.expand(75, 96)), want) and torch.equal(layer.gemm(t, dtype=torch.float16), want)


def test_two_streams_share_a_layer():
    """A layer holds nothing that a call writes: calls at once on several streams, captured or not."""
    import torch
    import weight_only_quantized_amd as wq
    gen = _gen(1)
    w = _signs((1000, 4096), gen)
    layer, pair = wq.MXLinear(_mx(w)), wq.MXGatedLinear(_mx(w), _mx(w.flip(0)))
    xs = [torch.randn((m, 4096), device="cuda", generator=gen).bfloat16() for m in (1, 48, 300, 700)]

    def both(x):
        q = wq.MXTensor.quantize(x)
        return layer.gemm(x), pair.gemm(x), layer.gemm(q), pair.gemm(q), q.dequantize(torch.float32)

    want = [both(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    graphs = []
    for x, s in zip(xs, streams):
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = both(x)
        graphs.append((graph, out))
    for _ in range(5):
        eager = []
        for x, s, (graph, _) in zip(xs, streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
            eager.append(both(x))
        torch.cuda.synchronize()
        for a, b, (_, c) in zip(want, eager, graphs):
            assert all(torch.equal(p, q) and torch.equal(p, r) for p, q, r in zip(a, b, c))

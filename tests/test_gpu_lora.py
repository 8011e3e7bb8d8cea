"""Low-rank adapters of many requests beside a projection, against the float64 oracle.

Bound: out is rounded once (half a unit of its type), A x is kept to 16 bits or more, and both sums
run in float32 over products of at most 2^20 terms in an order of the kernel's own: their error is
within 2^-16 of the sum of the terms' magnitudes."""
import sys

import numpy as np
import pytest

import oracle.serving_oracle as so

pytestmark = pytest.mark.gpu

HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_amd as wq
    wq.load_library()
    yield


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def tdtype(tag):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16}[tag]


def host(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


def make(M, K, N, rank, adapters, tag, seed, ids=None, x_std=1.0):
    import torch
    import weight_only_quantized_amd as wq
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, std):
        return torch.empty(shape, device="cuda").normal_(0, std, generator=g).to(tdtype(tag))

    x, y = normal((M, K), x_std), normal((M, N), 1.0)
    a, b = normal((adapters, rank, K), K ** -0.5), normal((adapters, N, rank), 0.5 * rank ** -0.5)
    scale = torch.empty(adapters, device="cuda").uniform_(0.5, 2.0, generator=g)
    if ids is None:
        ids = np.random.default_rng(seed).integers(-1, adapters, M)
    ids = np.asarray(ids, np.int32)
    return wq.LoraBank(a, b, scale), x, y, torch.from_numpy(ids).cuda(), ids


def check(got, bank, x, y, ids, tag, columns=None, label=""):
    b = host(bank.b) if columns is None else host(bank.b[:, columns])
    yy = host(y) if columns is None else host(y[:, columns])
    want, weight = so.lora(yy, host(x), host(bank.a), b, host(bank.scale), ids)
    out = host(got) if columns is None else host(got[:, columns])
    bound = HALF[tag] * np.abs(want) + 2.0 ** -16 * (weight + np.abs(yy)) + 1e-7
    err = np.abs(out - want)
    assert np.all(np.isfinite(out)), label
    assert np.all(err <= bound), (label, float((err / bound).max()), np.argwhere(err > bound)[:4].tolist())


# (rows, K, N, rank, adapters, type)
CASES = [
    (1, 32, 32, 8, 1, "f16"), (1, 4096, 1024, 16, 3, "bf16"), (2, 64, 96, 24, 5, "f16"), (3, 288, 160, 40, 2, "bf16"),
    (15, 1024, 544, 64, 4, "f16"), (16, 2048, 256, 16, 16, "bf16"), (17, 96, 2080, 128, 3, "f16"),
    (33, 4096, 416, 32, 40, "bf16"), (64, 512, 512, 8, 64, "f16"), (65, 544, 1056, 56, 7, "bf16"),
    (130, 256, 320, 104, 2, "f16"), (257, 1056, 288, 16, 5, "bf16"), (500, 128, 96, 64, 9, "f16"),
    (5, 14336, 128, 16, 2, "f16"), (1, 28672, 64, 128, 2, "bf16"),
    (16, 5120, 480, 32, 16, "f16"), (16, 5152, 480, 24, 16, "bf16"), (9, 5088, 7328, 8, 9, "f16"), (8, 96, 8192, 32, 8, "bf16"),
    (9, 96, 8192, 32, 9, "f16"), (127, 1024, 96, 32, 30, "bf16"), (128, 1056, 288, 40, 3, "f16"), (129, 1056, 288, 40, 3, "f16"),
    (192, 512, 320, 16, 90, "bf16"), (255, 288, 1056, 72, 4, "f16"), (256, 1024, 544, 64, 300, "bf16"), (256, 256, 128, 8, 1, "f16"),
]


@pytest.mark.parametrize("case", CASES, ids=["_".join(map(str, c)) for c in CASES])
def test_against_oracle(case):
    M, K, N, rank, adapters, tag = case
    say("lora", case)
    bank, x, y, idt, ids = make(M, K, N, rank, adapters, tag, seed=M + K)
    check(bank.add(y, x, idt), bank, x, y, ids, tag, label=case)
    # one adapter for all rows, runs of rows, and no adapter at all
    for other in (np.zeros(M), np.repeat(np.arange(-1, adapters), M // (adapters + 1) + 1)[:M], -np.ones(M)):
        bank, x, y, idt, ids = make(M, K, N, rank, adapters, tag, seed=M + K + 1, ids=other)
        check(bank.add(y, x, idt), bank, x, y, ids, tag, label=(case, "runs"))


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_ids_outside_the_bank_keep_y(M):
    import torch
    ids = np.random.default_rng(3).choice([-1, -100, 4, 5, 1 << 30, -(1 << 31)], M)
    bank, x, y, idt, ids = make(M, 256, 192, 16, 4, "bf16", seed=9, ids=ids)
    assert torch.equal(bank.add(y, x, idt), y)


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("M,rank", [(1, 8), (40, 64), (300, 24)])
def test_infinite_sums_stay_infinite(M, rank, tag):
    """A row whose A x is infinite (one sign) gives infinities where B's values have one sign, and a row
    beside it keeps its values."""
    import torch
    bank, x, y, idt, ids = make(M, 256, 192, rank, 2, tag, seed=21, ids=np.ones(M))
    bank.a.abs_().add_(1e-3)
    bank.b.abs_().add_(1e-3)
    plain = bank.add(y, x, idt)
    x[M // 2, 7] = float("inf")
    got = bank.add(y, x, idt)
    assert bool((got[M // 2] == float("inf")).all())
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(got[keep], plain[keep])


def test_no_rows():
    import torch
    bank, x, y, idt, ids = make(1, 256, 192, 16, 2, "f16", seed=1)
    assert bank.add(y[:0], x[:0], idt[:0]).shape == (0, 192)


def test_in_place_streams_and_equal_bits():
    import torch
    bank, x, y, idt, ids = make(37, 1024, 512, 16, 6, "f16", seed=5)
    want = bank.add(y, x, idt)
    check(want, bank, x, y, ids, "f16")
    ws = torch.full((bank.workspace_size(37) + 256,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(bank.add(y, x, idt, workspace=ws), want)
    side = torch.cuda.Stream()
    got = bank.add(y, x, idt, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    mine = y.clone()
    assert bank.add(mine, x, idt, out=mine) is mine and torch.equal(mine, want)
    assert bank.add(y[:0], x[:0], idt[:0]).shape == (0, 512)


@pytest.mark.parametrize("tag,power", [("bf16", 40), ("bf16", -40), ("f16", 8)])
@pytest.mark.parametrize("M", [3, 200])
def test_wide_ranges(tag, power, M):
    """Inputs far from one: A x beyond float16's range or deep below it."""
    import torch
    bank, x, y, idt, ids = make(M, 512, 256, 16, 3, tag, seed=6)
    x = (x.float() * 2.0 ** power).to(x.dtype)
    if tag == "f16":                     # A x is about 2^18: over what float16 holds
        bank.a.mul_(2.0 ** 10)
        bank.b.mul_(2.0 ** -13)
    else:
        y = (y.float() * 2.0 ** power).to(y.dtype)
    check(bank.add(y, x, idt), bank, x, y, ids, tag)
    assert torch.isfinite(bank.add(y, x, idt)).all()


@pytest.mark.parametrize("M", [2, 40, 200])
def test_non_finite_rows_stay_in_their_row(M):
    import torch
    bank, x, y, idt, ids = make(M, 256, 128, 16, 3, "f16", seed=7, ids=np.arange(M) % 3)
    want = bank.add(y, x, idt)
    x = x.clone()
    x[1, 7] = float("inf")
    got = bank.add(y, x, idt)
    assert not bool(torch.isfinite(got[1]).any())
    keep = torch.arange(M, device="cuda") != 1
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("M", [4, 100])
def test_graph(M):
    import torch
    bank, x, y, idt, _ = make(M, 1024, 512, 16, 6, "bf16", seed=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bank.add(y, x, idt)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = bank.add(y, x, idt)
    for i in range(4):
        x.normal_()
        idt.copy_(torch.randint(-1, 6, (M,), device="cuda", dtype=torch.int32))
        want = bank.add(y, x, idt)
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_beside_a_quantized_projection():
    """The use: y = the quantized layer's output, the adapters' sum added in place."""
    import torch
    import gptq_inputs as gi
    from gpu_util import repack_layer
    L = gi.make_layer(512, 256, 4, 128, desc_act=False, scales_dtype="f16", seed=gi.seed_for(9, 1))
    h = repack_layer(L)
    bank, x, _, idt, ids = make(20, 512, 256, 16, 4, "f16", seed=10)
    y = h.gemm(x)
    base = y.clone()
    out = bank.add(y, x, idt, out=y)
    check(out, bank, x, base, ids, "f16")
    h.close()
    assert torch.isfinite(out).all()

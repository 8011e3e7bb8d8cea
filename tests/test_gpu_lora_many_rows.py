"""Low-rank adapters of hundreds to thousands of rows, against the float64 oracle with the bound of
test_gpu_lora.py.  Rows run from 129 to 4099 in every kind of check, so that each form the library may choose
by the number of rows is met, wherever it changes from one to the other."""
import numpy as np
import pytest

from test_gpu_lora import check, make, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_amd as wq
    wq.load_library()
    yield


def ids_of(kind, M, adapters, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "mixed":                  # no order, about one in `adapters` without
        return rng.integers(-1, adapters, M)
    if kind == "runs":                   # prompts: runs of any length, one without an adapter
        cuts = np.sort(rng.integers(0, M + 1, 2 * adapters))
        return (np.searchsorted(cuts, np.arange(M), side="right") % (adapters + 1)) - 1
    if kind == "tail":                   # a prompt, then single rows of other requests
        return np.concatenate([np.zeros(M - 40, int), rng.integers(-1, adapters, 40)])
    if kind == "one":
        return np.full(M, adapters - 1)
    return np.full(M, -1)                # "none"


# (rows, K, N, rank, adapters, type)
CASES = [
    (129, 96, 288, 8, 5, "bf16"), (257, 544, 96, 128, 3, "f16"), (513, 288, 544, 72, 4, "bf16"), (1000, 160, 32, 40, 6, "f16"),
    (1024, 96, 160, 24, 9, "bf16"), (1025, 96, 160, 24, 9, "bf16"), (1025, 288, 544, 64, 5, "f16"), (1056, 544, 96, 8, 4, "f16"),
    (1056, 96, 288, 128, 3, "bf16"), (1100, 1056, 288, 40, 7, "f16"), (1100, 32, 32, 16, 2, "bf16"), (1153, 288, 96, 72, 4, "f16"),
    (1217, 2080, 64, 128, 3, "f16"), (1217, 96, 1056, 72, 2, "bf16"), (1300, 4096, 96, 64, 3, "bf16"), (1300, 160, 2080, 32, 5, "f16"),
    (2049, 288, 160, 128, 4, "f16"), (2049, 96, 288, 56, 5, "bf16"), (2100, 544, 544, 16, 20, "f16"), (4099, 64, 96, 104, 3, "bf16"),
    (4099, 96, 64, 24, 4, "f16"),
]


@pytest.mark.parametrize("case", CASES, ids=["_".join(map(str, c)) for c in CASES])
@pytest.mark.parametrize("kind", ["mixed", "runs", "tail", "one", "none"])
def test_against_oracle(kind, case):
    import torch
    M, K, N, rank, adapters, tag = case
    say("lora rows", kind, case)
    bank, x, y, idt, ids = make(M, K, N, rank, adapters, tag, seed=M + K, ids=ids_of(kind, M, adapters, seed=M))
    got = bank.add(y, x, idt)
    check(got, bank, x, y, ids, tag, label=(kind, case))
    if kind == "none":
        assert torch.equal(got, y)
    mine = y.clone()
    assert torch.equal(bank.add(mine, x, idt, out=mine), got)                       # in place
    ws = torch.full((bank.workspace_size(M) + 256,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(bank.add(y, x, idt, workspace=ws), got)                      # whatever the workspace held


ROWS = [300, 1030, 1500, 2070]


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("rank", [24, 128])
@pytest.mark.parametrize("M", ROWS)
def test_non_finite_rows_stay_in_their_row(M, rank, tag):
    import torch
    bank, x, y, idt, ids = make(M, 256, 192, rank, 3, tag, seed=7, ids=ids_of("mixed", M, 3))
    bad = np.flatnonzero(ids >= 0)[[0, 5, -1]]
    want = bank.add(y, x, idt)
    x = x.clone()
    x[bad[0], 7], x[bad[1], 0], x[bad[2], 255] = float("inf"), float("nan"), -float("inf")
    got = bank.add(y, x, idt)
    assert not bool(torch.isfinite(got[torch.from_numpy(bad).cuda()]).any())
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[torch.from_numpy(bad).cuda()] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("tag,power", [("bf16", 40), ("bf16", -40), ("f16", 8)])
@pytest.mark.parametrize("M", ROWS)
def test_wide_ranges(M, tag, power):
    """Inputs far from one: A x beyond float16's range or deep below it, every row by another power."""
    import torch
    bank, x, y, idt, ids = make(M, 96, 160, 40, 5, tag, seed=6, ids=ids_of("mixed", M, 5))
    each = 2.0 ** (torch.arange(M, device="cuda") % 5 - 2)[:, None]
    x = (x.float() * each * 2.0 ** power).to(x.dtype)
    if tag == "f16":                     # A x is about 2^18: over what float16 holds
        bank.a.mul_(2.0 ** 10)
        bank.b.mul_(2.0 ** -13)
    else:
        y = (y.float() * 2.0 ** power).to(y.dtype)
    check(bank.add(y, x, idt), bank, x, y, ids, tag)


@pytest.mark.parametrize("M", ROWS)
def test_ids_outside_the_bank_keep_y(M):
    import torch
    ids = np.random.default_rng(3).choice([-1, -100, 4, 5, 1 << 30, -(1 << 31)], M)
    bank, x, y, idt, ids = make(M, 96, 160, 16, 4, "bf16", seed=9, ids=ids)
    assert torch.equal(bank.add(y, x, idt), y)


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("M", ROWS)
def test_streams_and_graph(M, tag):
    import torch
    bank, x, y, idt, _ = make(M, 288, 160, 40, 6, tag, seed=8, ids=ids_of("runs", M, 6))
    want = bank.add(y, x, idt)
    side = torch.cuda.Stream()
    got = bank.add(y, x, idt, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bank.add(y, x, idt)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = bank.add(y, x, idt)
    for i in range(3):
        x.normal_()
        idt.copy_(torch.from_numpy(ids_of(("mixed", "tail", "one")[i], M, 6).astype(np.int32)))
        want = bank.add(y, x, idt)
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i

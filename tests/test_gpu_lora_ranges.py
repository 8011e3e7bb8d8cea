"""Low-rank adapters whose ranks differ widely in size, against the float64 oracle with the bound of
test_gpu_lora.py: what a small one adds is not lost beside a large one that an output does not take."""
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


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("rank", [8, 40, 128])
@pytest.mark.parametrize("M", [1, 16, 40, 300, 1100, 2050])
def test_ranks_of_very_different_size(M, rank, tag):
    """A x of the first rank 2^31 times that of the others, and B's column for it zero."""
    import torch
    say("ranks", M, rank, tag)
    bank, x, y, idt, ids = make(M, 256, 96, rank, 3, tag, seed=M + rank)
    bank.a[:, 0].mul_(2.0 ** 17)
    bank.a[:, 1:].mul_(2.0 ** -14)
    bank.b.mul_(2.0 ** 15)
    bank.b[:, :, 0] = 0
    y.zero_()
    got = bank.add(y, x, idt)
    assert bool(torch.isfinite(got).all())
    check(got, bank, x, y, ids, tag, label=(M, rank, tag))

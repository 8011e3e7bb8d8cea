"""Attention over the paged 8-bit cache at the edges of the sizes it takes."""
import numpy as np
import pytest

from test_gpu_kv_cache import Pool, dev, offsets, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_amd as wq
    wq.load_library()
    yield


@pytest.mark.parametrize("length", [40, 9000], ids=["short", "long"])
def test_no_rows_of_any_sequence(length):
    """max_q 0 with rows: all of them are absent, and out stays as it is."""
    import torch
    say("max_q 0", length)
    pool = Pool([length, 20], 16, 2, 64, seed=3)
    q = dev(np.ones((3, 4, 64)), torch.float16)
    out = torch.full_like(q, 7.0)
    got = pool.cache().attention(q, dev(pool.table), dev(np.asarray([length, 20], np.int32)), dev(offsets([2, 1])), max_q=0,
                                 out=out)
    torch.cuda.synchronize()
    assert got is out and bool((out == 7.0).all())

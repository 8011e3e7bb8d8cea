"""Attention over the paged 8-bit cache at the edges of the sizes it takes."""
import numpy as np
import pytest

from test_gpu_kv_cache import Pool, check_attention, dev, host, offsets, say

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


def test_short_sequences_in_a_wide_table():
    """2^12 units over a table of 2^24 tokens each: what a call can see is 64 tokens."""
    import torch
    batch, hkv = 512, 8
    rng = np.random.default_rng(8)
    lens = rng.integers(1, 65, batch).astype(np.int32)
    say("wide table", batch)
    pool = Pool(lens.tolist(), 256, hkv, 64, seed=4)
    table = torch.full((batch, 1 << 16), -1, dtype=torch.int32, device="cuda")
    table[:, :pool.table.shape[1]] = dev(pool.table)
    cu = offsets([1] * batch)
    q = dev(rng.normal(0, 1.5, (batch, hkv, 64)), torch.float16)
    out = pool.cache().attention(q, table, dev(lens), dev(cu), max_q=1, max_kv=64)
    check_attention(host(out), host(q), pool, lens, cu, "f16", 64 ** -0.5)


def test_a_workspace_on_the_host_is_refused():
    import torch
    import weight_only_quantized_amd as wq
    say("host workspace")
    pool = Pool([6000], 16, 2, 64, seed=5)
    q, host_ws = dev(np.ones((1, 4, 64)), torch.float16), torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace"):
        pool.cache().attention(q, dev(pool.table), dev(np.asarray([6000], np.int32)), dev(offsets([1])), max_q=1,
                               workspace=host_ws)
    a, b = (torch.zeros(s, dtype=torch.float16, device="cuda") for s in ((2, 64, 64), (2, 32, 64)))
    bank = wq.LoraBank(a, b, torch.ones(2, device="cuda"))
    x, y = (torch.zeros(s, dtype=torch.float16, device="cuda") for s in ((40, 64), (40, 32)))
    with pytest.raises(ValueError, match="workspace"):
        bank.add(y, x, torch.zeros(40, dtype=torch.int32, device="cuda"), workspace=host_ws)

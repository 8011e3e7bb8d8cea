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


# (lengths, cu, max_q) of four rows over two sequences of 64 cached tokens -> what each row gives: None where it
# stays as it was, 0 where it sees nothing, else (sequence, tokens that it sees)
BOUNDS = {
    "all_rows": ([64, 64], [0, 2, 4], 4, [(0, 63), (0, 64), (1, 63), (1, 64)]),
    "first_rows": ([64, 64], [0, 2, 4], 1, [(0, 63), None, (1, 63), None]),
    "past_the_table": ([1 << 30, 64], [0, 2, 4], 4, [(0, 64), (0, 64), (1, 63), (1, 64)]),
    "no_tokens": ([-4, 0], [0, 2, 4], 4, [0, 0, 0, 0]),
    "more_rows_than_tokens": ([1, 2], [0, 2, 4], 4, [0, (0, 1), (1, 1), (1, 2)]),
    "rows_that_descend": ([64, 64], [0, -9, 4], 4, [None, None, None, None]),
    "rows_past_the_last": ([64, 64], [9, 12, 15], 4, [None, None, None, None]),
}


@pytest.mark.parametrize("hkv,heads", [(1, 2), (1, 40), (16, 1024)], ids=["few_heads", "heads", "many_heads"])
@pytest.mark.parametrize("case", BOUNDS)
def test_each_row_within_the_stated_bounds(case, hkv, heads):
    """Rows that are absent stay as they were, rows that see nothing are zero, all others are right."""
    import torch
    lens, cu, max_q, rows = BOUNDS[case]
    say("bounds", case, heads)
    pool = Pool([64, 64], 16, hkv, 64, seed=71)
    q = dev(np.random.default_rng(3).normal(0, 1.5, (4, heads, 64)), torch.float16)
    out = torch.full_like(q, 77.0)
    pool.cache().attention(q, dev(pool.table), dev(np.asarray(lens, np.int32)), dev(np.asarray(cu, np.int32)), max_q=max_q,
                           out=out)
    got = host(out)
    for i, row in enumerate(rows):
        if row is None:
            assert np.all(got[i] == 77.0), (case, i)
        elif row == 0:
            assert np.all(got[i] == 0.0), (case, i)
        else:
            one = Pool([64], 16, hkv, 64, seed=71)
            for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
                setattr(one, name, getattr(pool, name))
            one.table = pool.table[row[0]:row[0] + 1]
            check_attention(got[i:i + 1], host(q)[i:i + 1], one, [row[1]], offsets([1]), "f16", 64 ** -0.5, label=(case, i))


def test_a_page_that_fills_token_by_token():
    """Each growth of a page's scale rounds its older codes once more, by half a code of the new scale, and
    what they were off before shrinks with the ratio: a value is off by half a code for its own rounding and
    half for each growth after it, and a few float32 roundings of 127 codes."""
    import torch
    rng = np.random.default_rng(9)
    steps, page = 96, 32
    pool = Pool([steps], page, 2, 64, seed=51)
    cache, table, cu = pool.cache(), dev(pool.table), dev(offsets([1]))
    grow = np.exp(np.arange(steps) / 40.0)[:, None, None]                    # values that grow all along
    x = dev(rng.normal(0, 0.3, (steps, 2, 64)) * grow, torch.float16)
    growths = np.zeros((steps, 2))
    before = None
    for t in range(steps):
        cache.append(x[t:t + 1], x[t:t + 1], table, dev(np.asarray([t], np.int32)), cu, max_new=1)
        now = host(cache.k_scale)[pool.table[0, t // page]]
        if t % page:
            growths[t - t % page:t] += now > before
        before = now
    k, v = cache.read(table, dev(np.zeros(1, np.int32)), dev(offsets([steps])), rows=steps, max_rows=steps, dtype=torch.float32)
    unit = host(cache.k_scale)[pool.table[0, np.arange(steps) // page]]
    bound = unit[..., None] * (0.5 * (1 + growths) + (1 + growths) * 127 * 4 * 2.0 ** -23)[..., None]
    assert growths.max() > 3
    for got in (k, v):
        assert np.all(np.abs(host(got) - host(x)) <= bound), float((np.abs(host(got) - host(x)) / bound).max())


def test_bounds_past_32_bits():
    """max_kv and window are upper bounds: any that is large enough is as good as none."""
    import torch
    say("large bounds")
    pool = Pool([300, 40], 16, 2, 64, seed=6)
    q, cu = dev(np.random.default_rng(4).normal(0, 1, (6, 4, 64)), torch.float16), dev(offsets([5, 1]))
    lens = dev(np.asarray([300, 40], np.int32))
    want = pool.cache().attention(q, dev(pool.table), lens, cu, max_q=5)
    for kw in (dict(max_kv=1 << 31), dict(max_kv=1 << 40), dict(window=1 << 31), dict(window=1 << 40, max_kv=1 << 33)):
        assert torch.equal(pool.cache().attention(q, dev(pool.table), lens, cu, max_q=5, **kw), want), kw

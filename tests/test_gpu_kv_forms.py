"""Attention over the paged 8-bit cache in the forms that a call's sizes choose, each in both types and both
head sizes, against the float64 oracle with the bound of test_gpu_kv_cache.py."""
import numpy as np
import pytest

from test_gpu_kv_cache import Pool, attend, check_attention, dev, host, offsets, say, tdtype

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
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("case", [([5000, 3000, 0, 1500], [40, 70, 0, 3], 2, 8, 0, True),
                                  ([4000, 2500], [65, 64], 2, 12, 1700, True),
                                  ([2300], [33], 1, 3, 0, False),
                                  ([1800, 1200], [100, 9], 1, 2, 0, True)], ids=["ragged", "window", "all", "two"])
def test_many_columns_with_the_keys_split(case, dim, tag):
    """More than 16 (row, head) columns over enough tokens that the keys are split."""
    lens, ns, hkv, hq, window, causal = case
    say("columns, keys split", case, dim, tag)
    attend(Pool(lens, 16, hkv, dim, seed=dim + len(lens)), lens, ns, hq, tag, causal=causal, window=window)


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("case", [([4200], [4200], 3, 48, 128, 0), ([3100, 900, 2000], [2700, 200, 1100], 2, 40, 128, 700),
                                  ([4099, 700], [4099, 700], 2, 32, 64, 0)], ids=["prompt", "ragged", "heads64"])
def test_large_prompts(case, tag):
    """Over 131072 (row, head) columns; sampled rows against the oracle, each as a sequence of its own."""
    import torch
    lens, ns, hkv, hq, dim, window = case
    say("large prompts", case, tag)
    pool = Pool(lens, 32, hkv, dim, seed=hq)
    cu = offsets(ns)
    q = torch.empty((int(cu[-1]), hq, dim), dtype=tdtype(tag), device="cuda")
    q.normal_(0, 1.5)
    out = pool.cache().attention(q, dev(pool.table), dev(np.asarray(lens, np.int32)), dev(cu), max_q=max(ns), window=window)
    rng = np.random.default_rng(2)
    for b, (n, length) in enumerate(zip(ns, lens)):
        pick = np.unique(np.concatenate([[0, 1, 63, 64, n - 1], rng.integers(0, n, 8)]))
        some = Pool([], 32, hkv, dim, seed=0)
        for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
            setattr(some, name, getattr(pool, name))
        some.table = np.repeat(pool.table[b:b + 1], len(pick), 0)
        rows = torch.from_numpy(pick + cu[b])
        check_attention(host(out[rows]), host(q[rows]), some, (pick + length - n + 1).astype(np.int32),
                        np.arange(len(pick) + 1), tag, dim ** -0.5, window=window, label=b)


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompts_and_single_tokens_in_one_call(dim, tag):
    """A chunk of a prompt beside other requests' single tokens and drafts, short and long."""
    lens = [450, 1, 37, 2600, 900, 0, 64, 1500, 3, 130]
    ns = [310, 1, 1, 1, 5, 0, 1, 1, 3, 1]
    say("mixed", dim, tag)
    for hkv, hq in ((4, 16), (1, 4)):
        attend(Pool(lens, 16, hkv, dim, seed=dim + hq), lens, ns, hq, tag)

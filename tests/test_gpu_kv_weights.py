"""Attention's probabilities in the second product: calls of up to sixteen (row, head) columns a sequence and kv
head keep them to 21 bits and more.

Bound, beside out's own rounding (half a unit of its type, half of float16's smallest step): the first 11 bits
of a weight are exact, what is left of them is rounded to 11 bits again, 2^-21 of the weight, and the sum of
weights and the exponential add a few 2^-23: 2^-20 of sum_j p_j |v_j| in all, the scores' 2^-19 (1 + most) as in
test_gpu_kv_cache.py (most is below one here), and 2^-31 of the largest token's codes for weights below
float16's smallest step, as in test_gpu_kv_ranges.py."""
import numpy as np
import pytest

import oracle.serving_oracle as so
from test_gpu_kv_cache import HALF, Pool, dev, host, offsets, say, tdtype
from test_gpu_kv_ranges import smallest_steps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_amd as wq
    wq.load_library()
    yield


# (lengths, rows of each, kv heads, q heads, dim, window)
FORMS = {
    "one": ([777], [1], 2, 8, 128, 0),
    "short": ([50, 17, 5], [1, 1, 1], 2, 16, 64, 0),
    "drafts": ([90, 33, 300], [5, 2, 0], 3, 3, 64, 0),
    "window": ([1900, 700], [5, 8], 2, 2, 64, 90),
    "split": ([6000, 700], [1, 1], 1, 8, 128, 0),
    "drafts_split": ([5000, 4100], [5, 3], 2, 2, 64, 0),
    "batch": ([40 + i for i in range(70)], [1] * 70, 4, 4, 128, 0),
    "batch_split": ([90 * i + 1 for i in range(40)], [1] * 40, 3, 15, 64, 0),
    "eight_heads": ([333, 2000], [1, 1], 2, 16, 128, 0),
    "sixteen_heads": ([777, 40], [1, 1], 2, 32, 128, 0),
    "nine": ([600, 130], [3, 2], 2, 6, 64, 0),
    "drafts_of_four": ([5000, 4100], [3, 4], 1, 4, 64, 0),
    "long_sixteen": ([7000, 300], [1, 1], 1, 16, 128, 0),
    "batch_of_twelve": ([40 + i for i in range(70)], [1] * 70, 2, 24, 64, 0),
    "batch_of_sixteen": ([900 - 9 * i for i in range(70)], [4] * 70, 1, 4, 128, 200),
}


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("form", FORMS)
def test_small_calls_keep_their_probabilities(form, tag):
    lens, ns, hkv, hq, dim, window = FORMS[form]
    say("weights", form, tag)
    pool = Pool(lens, 16, hkv, dim, seed=len(lens) + dim)
    cu = offsets(ns)
    q = dev(np.random.default_rng(6).normal(0, 0.1, (int(cu[-1]), hq, dim)), tdtype(tag))
    out = host(pool.cache().attention(q, dev(pool.table), dev(np.asarray(lens, np.int32)), dev(cu), max_q=max(ns),
                                      window=window))
    want, weight, most = so.attention(host(q), pool.k_codes, pool.v_codes, pool.k_scale, pool.v_scale, pool.table, lens,
                                      cu, dim ** -0.5, True, window)
    bound = HALF[tag] * np.abs(want) + (2.0 ** -20 + 2.0 ** -19 * (1 + most[..., None])) * weight + 2.0 ** -25
    bound += smallest_steps(host(q), pool, lens, cu, dim ** -0.5, window)
    err = np.abs(out - want)
    assert np.all(err <= bound), (form, float((err / bound).max()), np.argwhere(err > bound)[:4].tolist())

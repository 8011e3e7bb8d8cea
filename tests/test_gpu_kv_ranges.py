"""The paged 8-bit cache at the ends of its scales' range: attention over pages whose value scales are far
from one or far from each other, against the float64 oracle with bounds relative to the values themselves.

Bound, beside that of test_gpu_kv_cache.py: the logarithm of a value scale stands in a weight's exponent
through four float32 roundings at a magnitude below 128, 2^-18 each, so weights err by at most 2^-15 of
themselves more; out is bfloat16, whose smallest step is 2^-133.  Weights are float16, relative to the
column's largest, which is at least 2^6: one far below it errs by half of float16's smallest step, 2^-25, so
beside a token of a large page the codes of the others count with an error of 2^-31 of that token's."""
import numpy as np
import pytest

import oracle.serving_oracle as so
from test_gpu_kv_cache import HALF, Pool, dev, host, offsets, say

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
    "one": ([50, 17], [1, 1], 2, 8, 64, 0),                                   # short units, one launch
    "drafts": ([90, 33], [3, 2], 1, 4, 128, 0),
    "split": ([6000, 700], [1, 1], 1, 4, 128, 0),                             # keys split, parts joined
    "batch": ([40 + i for i in range(70)], [1] * 70, 4, 4, 128, 0),            # a wave a unit
    "rows_split": ([2600], [40], 2, 16, 64, 0),                                # two column tiles, keys split
    "prompt": ([260, 200], [260, 90], 5, 20, 128, 0),                          # through all keys
    "prompt_window": ([330, 100], [330, 100], 5, 20, 64, 20),                  # later rows do not see the first pages
}


def scales(pattern, pool):
    """Value scales [pages, heads], by each page's place in its sequence (unused pages: 1)."""
    rng, shape = np.random.default_rng(5), pool.v_scale.shape
    place = np.zeros(shape[0], int)
    for row in pool.table:
        for j, p in enumerate(row):
            if p >= 0:
                place[p] = j
    near = np.exp(rng.normal(0, 0.25, shape)) / 36
    first = (place == 0)[:, None]
    return {"tiny": near * 1e-22, "smaller": near * 1e-35, "large": near * 1e30,
            "first_tiny": near * np.where(first, 1e-30, 1.0), "first_zero": near * np.where(first, 0.0, 1e-22),
            "first_large": near * np.where(first, 1.0, 1e-25),
            "spread": 2.0 ** rng.uniform(-38, 38, shape)}[pattern].astype(np.float32)


def smallest_steps(q, pool, lens, cu, scale, window):
    """2^-31 max_j p_j s_j sum_j |code_j| of each output (causal calls)."""
    out, group = np.zeros_like(q), q.shape[1] // pool.heads
    for b, (n, length) in enumerate(zip(np.diff(cu), lens)):
        k, _ = so.values(pool.k_codes, pool.k_scale, pool.table, b, length)
        code, _ = so.values(pool.v_codes, np.ones_like(pool.v_scale), pool.table, b, length)
        s = pool.v_scale[pool.table[b, np.arange(length) // pool.page]].astype(np.float64)
        for i in range(n):
            at = length - n + i
            see = slice(max(0, at - window + 1) if window else 0, at + 1)
            for h in range(q.shape[1]):
                t = k[see, h // group] @ q[cu[b] + i, h] * scale
                p = np.exp(t - t.max())
                p /= p.sum()
                out[cu[b] + i, h] = 2.0 ** -31 * (p * s[see, h // group]).max() * np.abs(code[see, h // group]).sum(0)
    return out


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("pattern", ["tiny", "smaller", "large", "first_tiny", "first_zero", "first_large", "spread"])
def test_value_scales_far_from_one(pattern, form):
    import torch
    lens, ns, hkv, hq, dim, window = FORMS[form]
    say("value scales", pattern, form)
    pool = Pool(lens, 16, hkv, dim, seed=len(lens) + dim)
    pool.v_scale = scales(pattern, pool)
    cu = offsets(ns)
    q = dev(np.random.default_rng(6).normal(0, 1.5, (int(cu[-1]), hq, dim)), torch.bfloat16)
    out = host(pool.cache().attention(q, dev(pool.table), dev(np.asarray(lens, np.int32)), dev(cu), max_q=max(ns),
                                      window=window))
    want, weight, most = so.attention(host(q), pool.k_codes, pool.v_codes, pool.k_scale, pool.v_scale, pool.table, lens,
                                      cu, dim ** -0.5, True, window)
    bound = HALF["bf16"] * np.abs(want) + (2.0 ** -11 + 2.0 ** -15 + 2.0 ** -19 * (1 + most[..., None])) * weight + 2.0 ** -133
    bound += smallest_steps(host(q), pool, lens, cu, dim ** -0.5, window)
    err = np.abs(out - want)
    assert np.all(np.isfinite(out))
    assert np.all(err <= bound), (pattern, form, float((err / bound).max()), np.argwhere(err > bound)[:4].tolist())


@pytest.mark.parametrize("n", [1, 40], ids=["token", "rows"])
@pytest.mark.parametrize("had", [0.3, 2.0], ids=["grows", "stays"])
@pytest.mark.parametrize("size", [1e-35, 1e-37, 1e-38, 3e-39])
def test_append_of_values_near_the_smallest(size, had, n):
    """Pages whose scale has no float32 inverse.  Bounds: a scale is within 4 float32 roundings and half of
    the smallest subnormal step, 2^-150, of the ideal, and the codes follow it."""
    import torch
    starts, ns = [5, 0, 16], [n, n, n]
    pool = Pool([s + n for s in starts], 16, 2, 64, seed=n)
    pool.k_scale[:] = pool.v_scale[:] = np.float32(had * size / 127)
    cache, cu, rng = pool.cache(), offsets(ns), np.random.default_rng(n)
    say("append", size, had, n)
    k, v = (dev(np.clip(rng.normal(0, 0.4, (3 * n, 2, 64)), -1, 1) * size, torch.bfloat16) for _ in "kv")
    cache.append(k, v, dev(pool.table), dev(np.asarray(starts, np.int32)), dev(cu), max_new=n)
    for name, x in (("k", k), ("v", v)):
        ideal, scale = so.append(getattr(pool, name + "_codes"), getattr(pool, name + "_scale"), host(x), pool.table, starts, cu)
        got, got_scale = host(getattr(cache, name + "_codes")), host(getattr(cache, name + "_scale"))
        assert np.all(np.abs(got_scale - scale) <= scale * 4 * 2.0 ** -23 + 2.0 ** -150)
        off = 0.5 + 127 * (16 * 2.0 ** -24 + 2.0 ** -150 / np.maximum(scale, 2.0 ** -149))[:, :, None, None]
        assert np.all(np.abs(got - ideal) <= off), (name, float(np.abs(got - ideal).max()))


@pytest.mark.parametrize("form", [([1500], [1], 1, 4), ([1500, 40], [300, 40], 5, 20), ([1500], [60], 1, 8)],
                         ids=["token", "prompt", "rows"])
def test_small_values_after_many_zeros(form):
    """Over 1024 tokens of pages whose value scale is zero, then values near 1e-33."""
    import torch
    lens, ns, hkv, hq = form
    say("zeros first", form)
    pool = Pool(lens, 16, hkv, 64, seed=3)
    pool.v_scale = scales("smaller", pool)
    pool.v_scale[pool.table[0, :70]] = 0.0
    cu = offsets(ns)
    q = dev(np.random.default_rng(6).normal(0, 1.5, (int(cu[-1]), hq, 64)), torch.bfloat16)
    out = host(pool.cache().attention(q, dev(pool.table), dev(np.asarray(lens, np.int32)), dev(cu), max_q=max(ns)))
    want, weight, most = so.attention(host(q), pool.k_codes, pool.v_codes, pool.k_scale, pool.v_scale, pool.table, lens,
                                      cu, 64 ** -0.5)
    bound = HALF["bf16"] * np.abs(want) + (2.0 ** -11 + 2.0 ** -15 + 2.0 ** -19 * (1 + most[..., None])) * weight + 2.0 ** -133
    bound += smallest_steps(host(q), pool, lens, cu, 64 ** -0.5, 0)
    err = np.abs(out - want)
    assert np.all(err <= bound), (form, float((err / bound).max()), np.argwhere(err > bound)[:4].tolist())

"""The paged 8-bit cache on the GPU (append with rotation, read back, attention) against the float64
oracle (oracle/serving_oracle.py), through the package's entry points.

Bounds, from the operators' definitions and the formats alone:
 * a written code is the rounding of a value known to a few float32 roundings: within half a code and
   127 * 16 * 2^-24 of the ideal; a page's scale within 4 float32 roundings;
 * read back: bit-exact, one float32 product and one rounding;
 * attention: out is rounded once (half a unit of its type), each probability once to 11 bits, and
   scores, which are sums of at most 128 products in float32, err by at most 2^-20 of the sum of
   their terms' magnitudes: |err| <= half_ulp(out) + (2^-11 + 2^-19 (1 + most)) sum_j p_j |v_j|."""
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
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[tag]


def host(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


class Pool:
    """A cache with its page tables on the host and the device."""

    def __init__(self, lengths, page, heads, dim, seed, spare=3, v_spread=0.25):
        rng = np.random.default_rng(seed)
        self.rng, self.page, self.heads, self.dim = rng, page, heads, dim
        counts = [-(-n // page) for n in lengths]
        pages = sum(counts) + spare
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(lengths), max(max(counts, default=1), 1)), -1, np.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = order[at:at + c]
            at += c
        shape = (pages, heads, page, dim)
        self.k_codes, self.v_codes = (np.clip(np.rint(rng.normal(0, 36, shape)), -127, 127).astype(np.int8) for _ in "kv")
        self.k_scale = (np.exp(rng.normal(0, 0.25, shape[:2])) / 36).astype(np.float32)
        self.v_scale = (np.exp(rng.normal(0, v_spread, shape[:2])) / 36).astype(np.float32)

    def cache(self):
        import weight_only_quantized_amd as wq
        return wq.KVCache(dev(self.k_codes), dev(self.v_codes), dev(self.k_scale), dev(self.v_scale))


def offsets(ns):
    return np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)


def check_attention(got, q, pool, lens, cu, tag, scale, causal=True, window=0, rows=None, label=""):
    want, weight, most = so.attention(q, pool.k_codes, pool.v_codes, pool.k_scale, pool.v_scale, pool.table, lens, cu,
                                      scale, causal, window)
    bound = HALF[tag] * np.abs(want) + (2.0 ** -11 + 2.0 ** -19 * (1 + most[..., None])) * weight + 1e-7
    err = np.abs(got - want)
    if rows is not None:
        err, bound = err[rows], bound[rows]
    assert np.all(np.isfinite(err)), label
    assert np.all(err <= bound), (label, float((err / bound).max()), np.argwhere(err > bound)[:4].tolist())


def attend(pool, lens, ns, q_heads, tag, seed=0, causal=True, window=0, scale=None, q_std=1.5, check=True, **kw):
    rng = np.random.default_rng(seed + 1000)
    cu = offsets(ns)
    q = dev(rng.normal(0, q_std, (int(cu[-1]), q_heads, pool.dim)), tdtype(tag))
    out = pool.cache().attention(q, dev(pool.table), dev(np.asarray(lens, np.int32)), dev(cu), max_q=max(ns, default=0),
                                 causal=causal, window=window, scale=scale, **kw)
    if check:
        check_attention(host(out), host(q), pool, lens, cu, tag, pool.dim ** -0.5 if scale is None else scale, causal,
                        window, label=(lens, ns))
    return q, out


# (lengths, rows of each, page, kv heads, q heads, dim, type, causal, window)
ATTENTION = [
    ([1], [1], 16, 1, 1, 64, "bf16", True, 0),
    ([16], [1], 16, 2, 8, 128, "f16", True, 0),
    ([17, 0, 5], [1, 1, 1], 16, 2, 4, 128, "bf16", True, 0),          # a sequence without tokens
    ([33, 64, 65], [1, 0, 1], 32, 8, 8, 64, "f16", True, 0),          # a sequence without rows
    ([257, 31, 15, 128], [1, 1, 1, 1], 64, 2, 16, 128, "bf16", True, 0),
    ([1000], [1], 16, 1, 64, 64, "f16", True, 0),                     # 64 query heads on one head
    ([1300, 700], [1, 1], 128, 4, 4, 128, "bf16", True, 100),
    ([5000], [1], 16, 2, 8, 128, "f16", True, 0),                     # split over the keys
    ([4097, 3, 2000], [1, 1, 1], 256, 1, 3, 64, "bf16", True, 0),
    ([40, 77, 300], [3, 5, 7], 16, 2, 6, 128, "f16", True, 0),        # a few rows each
    ([40, 77, 300], [5, 1, 16], 32, 2, 2, 64, "bf16", True, 17),
    ([2, 3], [5, 9], 16, 2, 4, 64, "f16", True, 0),                   # rows before the first token
    ([65], [65], 16, 1, 2, 128, "bf16", True, 0),
    ([130, 1, 200], [70, 1, 33], 64, 2, 8, 64, "f16", True, 0),
    ([300, 129], [150, 129], 16, 2, 4, 128, "bf16", True, 64),
    ([96, 160], [40, 64], 32, 1, 7, 128, "f16", False, 0),            # not causal
    ([96, 160], [1, 2], 128, 2, 4, 64, "bf16", False, 0),
    ([257], [257], 256, 1, 1, 64, "bf16", True, 1),                   # a window of the token itself
    ([520, 64, 511], [260, 64, 1], 16, 1, 4, 128, "f16", True, 300),
    ([1025], [33], 16, 1, 32, 64, "f16", True, 0),
    ([5000, 3000, 0, 1500], [40, 70, 0, 3], 16, 2, 8, 128, "bf16", True, 0),     # many columns, keys split
    ([2200, 90], [300, 90], 64, 1, 4, 64, "f16", True, 0),
    ([4000, 2500], [65, 64], 32, 2, 12, 128, "f16", True, 1700),
    ([1800], [200], 128, 1, 2, 128, "bf16", False, 0),
    ([600, 500, 40], [90, 200, 40], 16, 3, 12, 128, "bf16", True, 0),            # short: not split
]


@pytest.mark.parametrize("case", ATTENTION, ids=[str(i) for i in range(len(ATTENTION))])
def test_attention_against_oracle(case):
    lens, ns, page, hkv, hq, dim, tag, causal, window = case
    say("attention", case)
    pool = Pool(lens, page, hkv, dim, seed=len(lens) * 7 + page)
    attend(pool, lens, ns, hq, tag, causal=causal, window=window)


@pytest.mark.parametrize("seed", range(24))
def test_attention_random_shapes(seed):
    rng = np.random.default_rng(77 + seed)
    batch = int(rng.integers(1, 6))
    many = seed % 2
    ns = [int(rng.integers(0, 140 if many else 9)) for _ in range(batch)]
    lens = [max(0, n + int(rng.integers(-2, 600 if many else 1500))) for n in ns]
    page, dim = int(rng.choice([16, 32, 64, 128, 256])), int(rng.choice([64, 128]))
    hkv, group = int(rng.integers(1, 4)), int(rng.choice([1, 2, 3, 4, 5, 8, 12]))
    window = int(rng.choice([0, 0, 1, 30, 129]))
    tag = str(rng.choice(["f16", "bf16"]))
    causal = bool(rng.random() < 0.8)
    say("attention random", seed, ns, lens, page, dim, hkv, group, window, tag, causal)
    if sum(ns) == 0:
        ns[0] = 1
    pool = Pool(lens, page, hkv, dim, seed=seed)
    attend(pool, lens, ns, hkv * group, tag, seed=seed, causal=causal, window=window,
           scale=None if seed % 3 else 0.3)


@pytest.mark.parametrize("case", [(120, 4, 8, 128, 16, "bf16", 0, 1), (90, 6, 6, 64, 32, "f16", 0, 2),
                                  (130, 3, 12, 128, 64, "f16", 50, 5), (70, 8, 16, 64, 16, "bf16", 90, 1)])
def test_many_short_sequences(case):
    """Batches whose sequences are short and many, some without rows or tokens."""
    batch, hkv, hq, dim, page, tag, window, most = case
    rng = np.random.default_rng(batch)
    ns = [int(n) for n in rng.integers(0, most + 1, batch)]
    lens = [max(0, int(n + rng.choice([0, 0, 1, 15, 33, 100, 190]) + rng.integers(-1, 40))) for n in ns]
    say("short sequences", case)
    attend(Pool(lens, page, hkv, dim, seed=batch), lens, ns, hq, tag, window=window)


@pytest.mark.parametrize("batch", [0, 3])
def test_calls_without_rows(batch):
    """No rows, with and without sequences: empty outputs, and the cache as it was."""
    import torch
    pool = Pool([5, 9, 16], 16, 2, 64, seed=2)
    cache, table = pool.cache(), dev(pool.table[:batch])
    at, cu = dev(np.zeros(batch, np.int32)), dev(np.zeros(batch + 1, np.int32))
    k, q = (torch.zeros((0, h, 64), dtype=torch.float16, device="cuda") for h in (2, 4))
    cos, sin = tables(16, 32)
    before = cache.k_codes.clone()
    cache.append(k, k, table, at, cu, max_new=0)
    got = cache.append(k, k, table, at, cu, max_new=0, q=q, cos=dev(cos), sin=dev(sin))
    assert got.shape == q.shape
    assert [t.shape for t in cache.read(table, at, cu, rows=0, max_rows=0)] == [k.shape, k.shape]
    assert cache.attention(q, table, at, cu, max_q=0).shape == q.shape
    assert torch.equal(cache.k_codes, before)


def test_calls_that_differ_in_causality_only():
    """With a window the keys that a call may see, and its workspace with them, follow from causality too."""
    import torch
    pool = Pool([6000, 2000], 16, 2, 64, seed=8)
    for causal in (True, False, True):
        cache = pool.cache() if causal else cache  # the same object for the first two calls
        cu, lens = offsets([1, 1]), [6000, 2000]
        q = dev(np.random.default_rng(1).normal(0, 1, (2, 4, 64)), torch.float16)
        out = cache.attention(q, dev(pool.table), dev(np.asarray(lens, np.int32)), dev(cu), max_q=1, window=40, causal=causal)
        check_attention(host(out), host(q), pool, lens, cu, "f16", 64 ** -0.5, causal, 40)


@pytest.mark.parametrize("seed", range(16))
def test_attention_prompts_random(seed):
    """Prompts with enough (row, head) columns to go through the keys a workgroup each, ragged, with
    contexts, windows and pages of all sizes."""
    rng = np.random.default_rng(900 + seed)
    batch, hkv, group = int(rng.integers(2, 6)), int(rng.integers(4, 7)), int(rng.choice([3, 4, 5, 8]))
    ns = [int(rng.integers(0, 220)) for _ in range(batch)]
    ns[0] = int(rng.integers(180, 330))
    lens = [max(0, n + int(rng.integers(-3, 500))) for n in ns]
    page, dim = int(rng.choice([16, 32, 64, 128, 256])), int(rng.choice([64, 128]))
    window = int(rng.choice([0, 0, 1, 65, 200]))
    tag, causal = str(rng.choice(["f16", "bf16"])), bool(rng.random() < 0.8)
    say("prompts", seed, ns, lens, page, dim, hkv, group, window, tag, causal)
    assert batch * hkv * -(-ns[0] * group // 16) > 256
    pool = Pool(lens, page, hkv, dim, seed=seed)
    attend(pool, lens, ns, hkv * group, tag, seed=seed, causal=causal, window=window)


@pytest.mark.parametrize("seed", range(12))
def test_attention_few_rows_long(seed):
    """A few rows each over thousands of tokens, sequences of very different lengths among them."""
    rng = np.random.default_rng(500 + seed)
    batch = int(rng.integers(1, 9))
    ns = [int(rng.integers(0, 6 if seed % 3 == 0 else 2)) for _ in range(batch)]
    ns[0] = 1
    lens = [max(0, n + int(2 ** rng.uniform(0, 12))) for n in ns]
    lens[0] = [1023, 1024, 1025, 1056, 2047, 2049, 4097][seed % 7]
    page, dim = int(rng.choice([16, 32, 64, 128, 256])), int(rng.choice([64, 128]))
    hkv, group = int(rng.integers(1, 12)), int(rng.choice([1, 2, 3, 4, 8]))
    window = int(rng.choice([0, 0, 1100, 1500]))
    tag = str(rng.choice(["f16", "bf16"]))
    say("attention few rows", seed, ns, lens, page, dim, hkv, group, window, tag)
    pool = Pool(lens, page, hkv, dim, seed=seed)
    attend(pool, lens, ns, hkv * group, tag, seed=seed, window=window)


@pytest.mark.parametrize("case", [(4200, 0, 32, 1, 16, 0), (3000, 1500, 48, 3, 128, 0), (4500, 77, 32, 2, 32, 700)],
                         ids=["prompt", "chunk", "window"])
def test_long_prompts(case):
    """Over 131072 (row, head) columns; sampled rows against the oracle, each as a call of its own."""
    import torch
    rows, start, hq, hkv, page, window = case
    say("long prompt", case)
    pool = Pool([rows + start], page, hkv, 128, seed=rows)
    q = torch.empty((rows, hq, 128), dtype=torch.bfloat16, device="cuda")
    q.normal_(0, 1.5)
    out = pool.cache().attention(q, dev(pool.table), dev(np.asarray([rows + start], np.int32)), dev(offsets([rows])),
                                 max_q=rows, window=window)
    pick = np.unique(np.concatenate([[0, 1, 63, 64, 65, rows - 1], np.random.default_rng(1).integers(0, rows, 18)]))
    some = Pool([], page, hkv, 128, seed=0)
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        setattr(some, name, getattr(pool, name))
    some.table = np.repeat(pool.table, len(pick), 0)
    check_attention(host(out[pick]), host(q[pick]), some, (pick + start + 1).astype(np.int32),
                    np.arange(len(pick) + 1), "bf16", 128 ** -0.5, window=window)


@pytest.mark.parametrize("ns", [[1, 1, 1], [40, 3, 90]], ids=["tokens", "rows"])
def test_absent_pages_and_unused_memory(ns):
    """Pages missing in the middle are not seen; codes and scales that no visible token owns (unused
    pages, and a page's tokens past the length) may hold anything, NaN and infinities included."""
    lens = [200, 50, 333]
    pool = Pool(lens, 16, 2, 128, seed=5)
    pool.table[0, 3] = -1
    pool.table[0, 12] = -7                        # the page of the last token
    pool.table[2, 0] = 1 << 30                    # past the pool
    pool.table[2, 5:9] = -1
    used = set(pool.table[(pool.table >= 0) & (pool.table < pool.k_codes.shape[0])].tolist())
    for p in range(pool.k_codes.shape[0]):
        if p not in used:
            pool.k_scale[p], pool.v_scale[p] = np.nan, np.inf
    say("absent pages", ns)
    attend(pool, lens, ns, 8, "bf16")
    # a whole sequence absent: zeros
    pool.table[1] = -1
    q, out = attend(pool, lens, ns, 8, "f16")
    cu = offsets(ns)
    assert np.all(host(out)[cu[1]:cu[2]] == 0)


@pytest.mark.parametrize("ns", [[1, 1], [30, 64]], ids=["tokens", "rows"])
@pytest.mark.parametrize("tag", ["f16", "bf16"])
def test_values_of_very_different_scale(ns, tag):
    """Value scales from 1e-6 to 1e3 between the pages of one sequence, some pages all zero."""
    lens = [700, 129]
    pool = Pool(lens, 16, 2, 64, seed=9)
    pool.v_scale[:] = np.exp(pool.rng.uniform(np.log(1e-6), np.log(1e1), pool.v_scale.shape)).astype(np.float32)
    pool.v_scale[::5] = 0.0
    pool.k_scale[::7] = 0.0
    attend(pool, lens, ns, 4, tag)


@pytest.mark.parametrize("n", [1, 50], ids=["tokens", "rows"])
def test_large_and_flat_scores(n):
    """Scores of hundreds (one token takes all), a zero scale (the mean of what is seen), a negative
    scale, and bf16 queries far outside float16's range."""
    import torch
    pool = Pool([400], 32, 2, 128, seed=11)
    attend(pool, [400], [n], 4, "bf16", scale=2.0)
    attend(pool, [400], [n], 4, "f16", scale=0.0)
    attend(pool, [400], [n], 4, "f16", scale=-0.11)
    rng = np.random.default_rng(3)
    cu = offsets([n])
    for power in (-70, 60):
        q = dev(rng.normal(0, 1.0, (n, 4, 128)), torch.bfloat16) * 2.0 ** power
        scale = 0.1 * 2.0 ** -power
        out = pool.cache().attention(q, dev(pool.table), dev(np.asarray([400], np.int32)), dev(cu), max_q=n, scale=scale)
        check_attention(host(out), host(q), pool, [400], cu, "bf16", scale, label=power)


@pytest.mark.parametrize("n", [1, 40], ids=["tokens", "rows"])
def test_non_finite_queries_stay_in_their_row(n):
    import torch
    pool = Pool([90], 16, 1, 64, seed=12)
    rng = np.random.default_rng(4)
    cu = offsets([n])
    q = dev(rng.normal(0, 1.5, (n, 8, 64)), torch.float16)
    bad = [(0, 1), (n - 1, 3)]
    q[0, 1, 5] = float("nan")
    q[n - 1, 3, 0] = float("inf")
    out = host(pool.cache().attention(q, dev(pool.table), dev(np.asarray([90], np.int32)), dev(cu), max_q=n))
    clean = q.clone()
    for r, h in bad:
        clean[r, h] = 0
    want = host(pool.cache().attention(clean, dev(pool.table), dev(np.asarray([90], np.int32)), dev(cu), max_q=n))
    for r, h in bad:
        assert np.all(np.isnan(out[r, h]))
        out[r, h] = want[r, h] = 0
    assert np.array_equal(out, want)


def test_offsets_past_32_bits():
    """Pages whose codes lie past 2^32 bytes, and past 2^31 elements of the packed tensors."""
    import torch
    import weight_only_quantized_amd as wq
    pages, page, heads, dim = 37000, 128, 8, 128          # 4.8 GB of codes a half
    cache = wq.KVCache.allocate(pages, page, heads, dim)
    small = Pool([300, 200], page, heads, dim, seed=21, spare=0)
    where = np.arange(small.k_codes.shape[0])
    far = pages - 1 - where * 3
    for t, s in ((cache.k_codes, small.k_codes), (cache.v_codes, small.v_codes), (cache.k_scale, small.k_scale),
                 (cache.v_scale, small.v_scale)):
        t[torch.from_numpy(far).cuda()] = dev(s)
    table = np.where(small.table >= 0, far[np.maximum(small.table, 0)], -1).astype(np.int32)
    for ns in ([1, 1], [70, 20]):
        cu = offsets(ns)
        q = dev(np.random.default_rng(5).normal(0, 1.5, (sum(ns), 8, dim)), torch.float16)
        out = cache.attention(q, dev(table), dev(np.asarray([300, 200], np.int32)), dev(cu), max_q=max(ns))
        check_attention(host(out), host(q), small, [300, 200], cu, "f16", dim ** -0.5)
    k, v = cache.read(dev(table), dev(np.zeros(2, np.int32)), dev(offsets([300, 200])), rows=500, max_rows=300,
                      dtype=torch.float32)
    want = np.concatenate([so.values(small.k_codes, small.k_scale, small.table, b, n)[0] for b, n in ((0, 300), (1, 200))])
    assert np.array_equal(host(k), want.astype(np.float32).astype(np.float64))
    x = dev(np.random.default_rng(6).normal(0, 1.0, (2, heads, dim)), torch.float16)
    cache.append(x, x, dev(table), dev(np.asarray([299, 199], np.int32)), dev(offsets([1, 1])), max_new=1)
    k, v = cache.read(dev(table), dev(np.asarray([299, 199], np.int32)), dev(offsets([1, 1])), rows=2, max_rows=1,
                      dtype=torch.float32)
    top = np.abs(host(x)).max(-1, keepdims=True)
    s = cache.k_scale[torch.from_numpy(far[[small.table[0, 2], small.table[1, 1]]]).cuda()].cpu().numpy()[..., None]
    assert np.all(np.abs(host(k) - host(x)) <= s * 0.5001) and np.all(s * 127.001 >= top)


def test_strided_tensors_and_out():
    """q, k and v as slices of one fused projection's rows, and out as a slice too; unaligned views
    are copied."""
    import torch
    hq, hkv, dim, lens, ns = 4, 2, 64, [50, 33], [2, 1]
    pool = Pool(lens, 16, hkv, dim, seed=31)
    cu = offsets(ns)
    fused = dev(np.random.default_rng(7).normal(0, 1, (3, (hq + 2 * hkv) * dim)), torch.bfloat16)
    q = fused[:, :hq * dim].view(3, hq, dim)
    wide = torch.full((3, hq + 3, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 1:1 + hq]
    got = pool.cache().attention(q, dev(pool.table), dev(np.asarray(lens, np.int32)), dev(cu), max_q=2, out=out)
    assert got is out
    check_attention(host(out), host(q), pool, lens, cu, "bf16", dim ** -0.5)
    assert bool((wide[:, 0] == 9).all()) and bool((wide[:, hq + 1:] == 9).all())
    odd = torch.empty(3 * hq * dim + 1, dtype=torch.bfloat16, device="cuda")[1:].view(3, hq, dim)
    odd.copy_(q)
    again = pool.cache().attention(odd, dev(pool.table), dev(np.asarray(lens, np.int32)), dev(cu), max_q=2)
    assert bool((again == out).all())
    swapped = q.transpose(0, 1).contiguous().transpose(0, 1)
    again = pool.cache().attention(swapped, dev(pool.table), dev(np.asarray(lens, np.int32)), dev(cu), max_q=2)
    assert bool((again == out).all())


def test_attention_bits_do_not_change():
    """The same call gives the same bits, on another stream and with another workspace's contents;
    a call without rows launches nothing."""
    import torch
    lens, ns = [6000, 10, 900], [1, 1, 1]
    pool = Pool(lens, 16, 2, 128, seed=41)
    cache, table = pool.cache(), dev(pool.table)
    kv, cu = dev(np.asarray(lens, np.int32)), dev(offsets(ns))
    q = dev(np.random.default_rng(8).normal(0, 1.5, (3, 8, 128)), torch.float16)
    one = cache.attention(q, table, kv, cu, max_q=1)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(one, cache.attention(q, table, kv, cu, max_q=1, workspace=ws))
    side = torch.cuda.Stream()
    other = cache.attention(q, table, kv, cu, max_q=1, stream=side)
    side.synchronize()
    assert torch.equal(one, other)
    none = cache.attention(q[:0], table[:0], kv[:0], dev(np.zeros(1, np.int32)), max_q=0)
    assert none.shape == (0, 8, 128)


# ---- append and read -----------------------------------------------------------------------------

# (starts, rows, page, kv heads, q heads, dim, rot, interleaved, type)
APPEND = [
    ([0], [1], 16, 1, 1, 64, 64, False, "f16"),
    ([15, 16, 17, 0], [1, 1, 1, 1], 16, 2, 4, 128, 128, False, "bf16"),
    ([3, 200, 64], [1, 0, 1], 64, 8, 8, 64, 32, True, "f16"),
    ([0, 5, 31], [33, 70, 1], 16, 2, 6, 128, 64, True, "bf16"),
    ([100, 0], [200, 257], 32, 1, 2, 64, 16, False, "f16"),
    ([7], [300], 128, 3, 3, 128, 128, False, "bf16"),
    ([250, 600], [20, 100], 256, 2, 2, 128, 128, True, "f16"),
    ([250, 600], [1, 1], 256, 1, 5, 64, 48, False, "bf16"),
]


def tables(positions, half, seed=0):
    at = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(half) / max(half, 1))
    return np.cos(at).astype(np.float32), np.sin(at).astype(np.float32)


def check_append(pool, cache, starts, cu, k, v, what=""):
    for name, x in (("k", k), ("v", v)):
        ideal, scale = so.append(getattr(pool, name + "_codes"), getattr(pool, name + "_scale"), x, pool.table, starts, cu)
        got_scale = host(getattr(cache, name + "_scale"))
        got = host(getattr(cache, name + "_codes"))
        assert np.all(np.abs(got_scale - scale) <= scale * 4 * 2.0 ** -23), (what, name)
        assert np.all(np.abs(got - ideal) <= 0.5 + 127 * 16 * 2.0 ** -24), \
            (what, name, float(np.abs(got - ideal).max()))


@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
@pytest.mark.parametrize("big", [0.3, 4.0], ids=["small", "grows"])
def test_append_against_oracle(case, big):
    import torch
    starts, ns, page, hkv, hq, dim, rot, inter, tag = case
    say("append", case, big)
    rng = np.random.default_rng(page + dim)
    pool = Pool([s + n for s, n in zip(starts, ns)], page, hkv, dim, seed=page)
    cache = pool.cache()
    cu = offsets(ns)
    T = int(cu[-1])
    cos, sin = tables(max(s + n for s, n in zip(starts, ns)), rot // 2)
    k, v, q = (dev(rng.normal(0, big, (T, h, dim)), tdtype(tag)) for h in (hkv, hkv, hq))
    got = cache.append(k, v, dev(pool.table), dev(np.asarray(starts, np.int32)), dev(cu), max_new=max(ns), q=q,
                       cos=dev(cos), sin=dev(sin), interleaved=inter)
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, ns)])
    want = so.rotate(host(q), cos[pos], sin[pos], inter)
    both = np.abs(host(q)).max(-1, keepdims=True) * 2
    assert np.all(np.abs(host(got) - want) <= HALF[tag] * np.abs(want) + both * 4 * 2.0 ** -24 + 2.0 ** -25)
    check_append(pool, cache, starts, cu, so.rotate(host(k), cos[pos], sin[pos], inter), host(v), case)
    # in place, and with no rotation
    q2 = q.clone()
    back = cache.append(k, v, dev(pool.table), dev(np.asarray(starts, np.int32)), dev(cu), max_new=max(ns), q=q2,
                        cos=dev(cos), sin=dev(sin), interleaved=inter, q_out=q2)
    assert back is q2 and torch.equal(q2, got)
    plain = pool.cache()
    assert plain.append(k, v, dev(pool.table), dev(np.asarray(starts, np.int32)), dev(cu), max_new=max(ns)) is None
    check_append(pool, plain, starts, cu, host(k), host(v), case)


@pytest.mark.parametrize("tag", ["f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
def test_rotation_rounds_each_product(tag, inter):
    """Products and sums of the rotation are float32 operations rounded one by one: the same bits as on
    the CPU, so codes do not depend on how a compiler joins operations."""
    import torch
    rng = np.random.default_rng(31)
    rows, heads, dim = 700, 4, 128
    cos, sin = (torch.from_numpy(t) for t in tables(rows, dim // 2))
    x = torch.from_numpy(rng.normal(0, 2, (rows, heads, dim))).to(torch.float16 if tag == "f16" else torch.bfloat16)
    cache, kv = Pool([rows], 64, 1, dim, seed=1), torch.zeros((rows, 1, dim), dtype=x.dtype, device="cuda")
    got = cache.cache().append(kv, kv, dev(cache.table), dev(np.zeros(1, np.int32)), dev(offsets([rows])), max_new=rows,
                               q=x.cuda(), cos=cos.cuda(), sin=sin.cuda(), interleaved=inter)
    f, c, s = x.float(), cos[:, None], sin[:, None]
    a, b = (f[..., 0::2], f[..., 1::2]) if inter else (f[..., :dim // 2], f[..., dim // 2:])
    ac, bs, bc, as_ = a * c, b * s, b * c, a * s
    lo, hi = ac - bs, bc + as_
    want = torch.stack((lo, hi), -1).flatten(-2) if inter else torch.cat((lo, hi), -1)
    assert torch.equal(got.cpu(), want.to(x.dtype))


@pytest.mark.parametrize("batch,many", [(65, False), (200, False), (300, True), (70, True)])
def test_many_sequences(batch, many):
    """More sequences than a wave has lanes: appended, read back and attended to, some without rows or
    tokens."""
    import torch
    rng = np.random.default_rng(batch)
    ns = [int(n) for n in (rng.integers(0, 6, batch) if many else rng.integers(0, 2, batch))]
    starts = [int(s) for s in rng.integers(0, 80, batch)]
    ns[0], ns[-1] = 1, 1
    lens = [s + n for s, n in zip(starts, ns)]
    pool = Pool(lens, 16, 2, 64, seed=batch)
    cache, cu = pool.cache(), offsets(ns)
    T, table = int(cu[-1]), dev(pool.table)
    cos, sin = tables(100, 32)
    k, v, q = (dev(rng.normal(0, 1, (T, h, 64)), torch.float16) for h in (2, 2, 6))
    got = cache.append(k, v, table, dev(np.asarray(starts, np.int32)), dev(cu), max_new=max(ns), q=q, cos=dev(cos),
                       sin=dev(sin))
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(starts, ns)])
    check_append(pool, cache, starts, cu, so.rotate(host(k), cos[pos], sin[pos], False), host(v), batch)
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        setattr(pool, name, getattr(cache, name).cpu().numpy())
    out = cache.attention(got, table, dev(np.asarray(lens, np.int32)), dev(cu), max_q=max(ns))
    check_attention(host(out), host(got), pool, lens, cu, "f16", 64 ** -0.5)
    kk, _ = cache.read(table, dev(np.asarray(starts, np.int32)), dev(cu), rows=T, max_rows=max(ns), dtype=torch.float32)
    want = np.concatenate([so.values(pool.k_codes, pool.k_scale, pool.table, b, s + n)[0][s:] for b, (s, n) in
                           enumerate(zip(starts, ns))])
    assert np.array_equal(host(kk), want.astype(np.float32).astype(np.float64))


def test_append_again_changes_nothing_and_pages_fill_token_by_token():
    import torch
    pool = Pool([64, 64], 32, 2, 64, seed=51)
    cache, table = pool.cache(), dev(pool.table)
    x = dev(np.random.default_rng(9).normal(0, 1, (96, 2, 64)), torch.float16)
    start = np.asarray([10, 0], np.int32)
    cu = offsets([1, 1])
    for _ in range(2):
        cache.append(x[:2], x[2:4], table, dev(start), dev(cu), max_new=1)
        state = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)]
    cache.append(x[:2], x[2:4], table, dev(start), dev(cu), max_new=1)
    for t, u in zip(state, (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)):
        assert torch.equal(t, u)
    # token by token, each step against the oracle's step from the same cache
    for step in range(40):
        start = np.asarray([step, step + 3], np.int32)
        rows = x[2 * step:2 * step + 2]
        for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
            setattr(pool, name, getattr(cache, name).cpu().numpy())
        cache.append(rows, rows * 0.5, table, dev(start), dev(cu), max_new=1)
        check_append(pool, cache, start, cu, host(rows), host(rows * 0.5), step)
    # every value within one and a half steps of what was appended
    k, _ = cache.read(table, dev(np.zeros(2, np.int32)), dev(offsets([40, 0])), rows=40, max_rows=40, dtype=torch.float32)
    unit = cache.k_scale[table[0, :2].long()].repeat_interleave(32, 0)[:40, :, None]
    off = ((k - x[0:80:2].float()).abs() / unit).max().item()
    assert off < 3.0, off


def test_append_zeros_infinities_and_absent_pages():
    import torch
    pool = Pool([48, 48, 48], 16, 1, 64, seed=52)
    pool.table[1, 1] = -1
    pool.table[2, 0] = 99999
    cache = pool.cache()
    rng = np.random.default_rng(10)
    starts, ns = [0, 4, 0], [48, 40, 20]
    cu = offsets(ns)
    k = rng.normal(0, 1, (108, 1, 64)).astype(np.float32)
    k[:16] = 0                                    # a page of zeros
    k[20, 0, 3], k[21, 0, 4], k[22, 0, 5] = np.inf, -np.inf, np.nan
    kt = dev(k, torch.float16)
    cache.append(kt, kt, dev(pool.table), dev(np.asarray(starts, np.int32)), dev(cu), max_new=48)
    check_append(pool, cache, starts, cu, host(kt), host(kt), "special")
    codes, p = cache.k_codes.cpu().numpy(), pool.table
    assert codes[p[0, 1], 0, 4, 3] == 127 and codes[p[0, 1], 0, 5, 4] == -127 and codes[p[0, 1], 0, 6, 5] == 0
    assert np.all(codes[p[0, 0]] == 0) and float(cache.k_scale[int(p[0, 0]), 0]) == 0.0
    # reading back: absent tokens are zeros
    k2, v2 = cache.read(dev(pool.table), dev(np.zeros(3, np.int32)), dev(offsets([48, 48, 48])), rows=144, max_rows=48,
                        dtype=torch.float32)
    assert bool((k2[48 + 16:48 + 32] == 0).all()) and bool((v2[96:112] == 0).all()) and bool((k2[112:116] != 0).any())


@pytest.mark.parametrize("tag", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("page,heads,dim", [(16, 3, 64), (64, 8, 128), (256, 1, 64)])
def test_read_is_exact(tag, page, heads, dim):
    import torch
    lens = [70, 0, 300]
    pool = Pool(lens, page, heads, dim, seed=61)
    starts, ns = [5, 0, 17], [65, 0, 283]
    k, v = pool.cache().read(dev(pool.table), dev(np.asarray(starts, np.int32)), dev(offsets(ns)), rows=348, max_rows=283,
                             dtype=tdtype(tag))
    for got, codes, scale in ((k, pool.k_codes, pool.k_scale), (v, pool.v_codes, pool.v_scale)):
        want = np.concatenate([so.values(codes, scale, pool.table, b, s + n)[0][s:] for b, (s, n) in
                               enumerate(zip(starts, ns))])
        assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).to(tdtype(tag)))


def test_rows_past_the_stated_bounds_are_left_alone():
    """max_rows, the table's width and rows bound what a call touches, whatever cu and at hold."""
    import torch
    pool = Pool([64, 64], 16, 1, 64, seed=71)
    cache = pool.cache()
    before = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)]
    x = dev(np.ones((4, 1, 64)), torch.float16)
    for start, cu in (([64, 500], [0, 2, 4]), ([-5, 1 << 30], [0, 2, 4]), ([0, 0], [0, -3, 9]), ([0, 0], [7, 9, 4])):
        cache.append(x, x, dev(pool.table), dev(np.asarray(start, np.int32)), dev(np.asarray(cu, np.int32)), max_new=4)
    torch.cuda.synchronize()
    for t, u in zip(before, (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)):
        assert torch.equal(t, u)
    q = dev(np.ones((4, 2, 64)), torch.float16)
    for kv, cu in (([1 << 30, 64], [0, 2, 4]), ([-4, 0], [0, 2, 4]), ([64, 64], [0, -9, 4]), ([64, 64], [9, 12, 15])):
        for max_q in (1, 4):
            out = cache.attention(q, dev(pool.table), dev(np.asarray(kv, np.int32)), dev(np.asarray(cu, np.int32)),
                                  max_q=max_q, out=torch.zeros_like(q))
            assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("ns", [[1, 1], [40, 90]], ids=["tokens", "rows"])
def test_graph_of_a_step(ns):
    """Append and attention captured in one graph and replayed over changed inputs, with eager work
    between the replays: every replay equals the eager calls on a copy of the cache."""
    import torch
    import weight_only_quantized_amd as wq
    starts = [1500, 30]
    pool = Pool([s + n + 8 for s, n in zip(starts, ns)], 16, 2, 128, seed=81)
    cache, table, cu = pool.cache(), dev(pool.table), dev(offsets(ns))
    T = sum(ns)
    cos, sin = (dev(t) for t in tables(2000, 64))
    rng = np.random.default_rng(11)
    start = dev(np.asarray(starts, np.int32))
    length = torch.empty_like(start)
    add = dev(np.asarray(ns, np.int32))
    k, v, q = (torch.empty((T, h, 128), dtype=torch.bfloat16, device="cuda") for h in (2, 2, 8))

    def step(c):
        torch.add(start, add, out=length)
        r = c.append(k, v, table, start, cu, max_new=max(ns), q=q, cos=cos, sin=sin)
        return c.attention(r, table, length, cu, max_q=max(ns))

    def fill():
        for t in (k, v, q):
            t.copy_(dev(rng.normal(0, 1, tuple(t.shape)), torch.bfloat16))

    fill()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(cache)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache)
    for i in range(4):
        fill()
        start.add_(1)
        twin = wq.KVCache(*(t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)))
        want = step(twin)
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert torch.equal(cache.k_codes, twin.k_codes) and torch.equal(cache.v_scale, twin.v_scale), i

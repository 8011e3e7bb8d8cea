"""Timing cases of the serving operators that stand next to the quantized projections of a decoder
layer: low-rank adapters of many requests beside a shared projection, appending rotated keys and
values to a paged 8-bit cache, and attention over that cache.

`run` computes one pass, either in plain torch operations in 32 bits (`own` false) or through the
package's entry points (`own` true); both take the same state.  The cache is kept as the package
documents it: codes int8 [pages, kv_heads, page, dim], one float32 scale for each page and head,
value = code * scale.  Lengths and adapter ids follow from the case alone, values from the seed.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_BASE = 500000.0          # rotation base


# ---- cases ---------------------------------------------------------------------------------------

def _attention(name, batch, max_q, max_kv, q_heads, kv_heads, dim, page, window, dtype, ragged, mix):
    return {"name": name, "op": "attention", "batch": batch, "max_q": max_q, "max_kv": max_kv, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "window": window, "dtype": dtype, "ragged": ragged,
            "mix": mix}


def _append(name, batch, max_new, max_start, q_heads, kv_heads, dim, page, rot, interleaved, dtype, mix):
    return {"name": name, "op": "append", "batch": batch, "max_new": max_new, "max_start": max_start,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "rot": rot,
            "interleaved": interleaved, "dtype": dtype, "mix": mix}


def _lora(name, rows, inner, outer, rank, adapters, runs, dtype, mix):
    return {"name": name, "op": "lora", "rows": rows, "inner": inner, "outer": outer, "rank": rank,
            "adapters": adapters, "runs": runs, "dtype": dtype, "mix": mix}


def listed():
    return [
        # one user chatting: a single query over a short context, where only latency counts
        _attention("attention_one_token", 1, 1, 777, 32, 8, 128, 16, 0, "bf16", False, 1),
        # an ordinary serving batch: 64 requests of very different lengths, one new token each
        _attention("attention_decode_batch", 64, 1, 4096, 32, 8, 128, 16, 0, "bf16", True, 2),
        # few requests over long documents: the cache's bytes are everything
        _attention("attention_decode_long", 6, 1, 70001, 64, 8, 128, 64, 0, "f16", True, 3),
        # drafted tokens checked five at a time, every head its own keys, a sliding window
        _attention("attention_drafts_window", 24, 5, 5003, 16, 16, 64, 32, 2000, "bf16", True, 4),
        # chunks of several prompts in one batch, some with a long context before them
        _attention("attention_prefill_ragged", 5, 1301, 4500, 32, 8, 128, 16, 0, "f16", True, 5),
        # one long prompt, the compute-bound end
        _attention("attention_prefill_long", 1, 8192, 8192, 32, 8, 128, 64, 0, "bf16", False, 6),
        # the decode step's append: one token for each of 64 requests, most into a part-filled page
        _append("append_decode_batch", 64, 1, 4000, 32, 8, 128, 16, 128, False, "bf16", 7),
        # a prompt chunk of odd lengths, half of each head rotated, neighbouring pairs
        _append("append_prefill_ragged", 7, 2500, 3000, 64, 8, 128, 64, 64, True, "f16", 8),
        # one row and its adapter beside a 4096 x 14336 projection: latency
        _lora("lora_one_row", 1, 4096, 14336, 16, 4, 0, "f16", 9),
        # a decode batch in which nearly every request has another adapter
        _lora("lora_decode_mixed", 61, 8192, 28672, 32, 48, 0, "bf16", 10),
        # prompts of a few requests, each one run of rows
        _lora("lora_prefill_runs", 4001, 4096, 14336, 64, 6, 9, "bf16", 11),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype, mix = rng.choice(["bf16", "f16"]), rng.randrange(1 << 30)
    kind = rng.choice(["attention_decode", "attention_prefill", "append", "lora_decode", "lora_prefill"])
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 4, 8])
    dim, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if kind == "attention_decode":
        max_kv = _log_int(rng, 1, 70001)
        batch = _log_int(rng, 1, max(1, min(128, 420000 // max_kv)))
        max_q = min(max_kv, rng.choice([1, 1, 1, 1, 2, 4, 7]))
        window = rng.choice([0, 0, 0, _log_int(rng, 1, max_kv)])
        return _attention("drawn", batch, max_q, max_kv, q_heads, kv_heads, dim, page, window, dtype, True, mix)
    if kind == "attention_prefill":
        max_q = _log_int(rng, 9, 4096)
        max_kv = max_q + _log_int(rng, 1, 4096) - 1
        batch = _log_int(rng, 1, max(1, min(16, (1 << 30) // (max_q * max_kv * q_heads))))
        window = rng.choice([0, 0, 0, _log_int(rng, 1, max_kv)])
        return _attention("drawn", batch, max_q, max_kv, q_heads, kv_heads, dim, page, window, dtype, True, mix)
    if kind == "append":
        max_new = rng.choice([1, 1, _log_int(rng, 2, 4096)])
        batch = _log_int(rng, 1, max(1, min(128, 14000 // max_new)))
        rot = rng.choice([dim, dim, dim // 2])
        return _append("drawn", batch, max_new, _log_int(rng, 1, 8000) - 1, q_heads, kv_heads, dim, page, rot,
                       rng.random() < 0.4, dtype, mix)
    inner, outer = 32 * _log_int(rng, 8, 256), 32 * _log_int(rng, 8, 448)
    if kind == "lora_decode":
        return _lora("drawn", _log_int(rng, 1, 128), inner, outer, rng.choice([8, 16, 32, 64]), _log_int(rng, 1, 48), 0,
                     dtype, mix)
    rows = _log_int(rng, 129, 4001)
    return _lora("drawn", rows, min(inner, 4096), outer, rng.choice([8, 16, 32, 64]), rng.randrange(1, 7),
                 rng.randrange(1, 10), dtype, mix)


def _spans(case):
    """[(tokens of this call, tokens cached before them)] of each sequence."""
    r = random.Random(case["mix"])
    if case["op"] == "attention":
        got = [(case["max_q"], case["max_kv"] - case["max_q"])]
        for _ in range(case["batch"] - 1):
            if not case["ragged"]:
                got.append(got[0])
                continue
            n = case["max_q"] if case["max_q"] <= 8 else _log_int(r, 1, case["max_q"])
            got.append((n, _log_int(r, max(n, case["max_kv"] // 16), case["max_kv"]) - n))
        return got
    got = [(case["max_new"], case["max_start"])]
    for _ in range(case["batch"] - 1):
        n = 1 if case["max_new"] == 1 else _log_int(r, 1, case["max_new"])
        got.append((n, r.randrange(case["max_start"] + 1)))
    return got


def _ids(case):
    """Adapter of each row: none (-1) for about one row or run in eight."""
    r = random.Random(case["mix"])
    pick = lambda: -1 if r.random() < 0.125 else r.randrange(case["adapters"])  # noqa: E731
    if not case["runs"]:
        ids = [pick() for _ in range(case["rows"])]
    else:
        cuts = sorted(r.randrange(case["rows"] + 1) for _ in range(case["runs"] - 1))
        ids = []
        for lo, hi in zip([0] + cuts, cuts + [case["rows"]]):
            ids += [pick()] * (hi - lo)
    if max(ids) < 0:
        ids[0] = 0
    return ids


def _visible(case):
    """(keys that some query of a sequence sees, summed; pairs of query and key that count)."""
    keys = pairs = 0
    for n, start in _spans(case):
        w = case["window"] or start + n
        pairs += sum(min(start + i + 1, w) for i in range(n))
        keys += min(start + n, w + n - 1)
    return keys, pairs


def work(case):
    if case["op"] == "attention":
        keys, pairs = _visible(case)
        tokens = sum(n for n, _ in _spans(case))
        cache = keys * case["kv_heads"] * case["dim"] * 2 + keys // case["page"] * case["kv_heads"] * 8
        return {"bytes": cache + tokens * case["q_heads"] * case["dim"] * 4,
                "flops": 4 * pairs * case["q_heads"] * case["dim"]}
    if case["op"] == "append":
        # q in and out, k and v in; codes of the touched pages out, of their older tokens in too;
        # and the touched pages' values, read back
        spans, p = _spans(case), case["page"]
        new, old = sum(n for n, _ in spans), sum(s % p for _, s in spans)
        head = case["kv_heads"] * case["dim"]
        size = new * case["q_heads"] * case["dim"] * 4 + new * head * 4 + (new + 2 * old) * head * 2
        return {"bytes": size + (new + old) * head * (2 + 4),
                "flops": 3 * new * case["rot"] * (case["q_heads"] + case["kv_heads"]) + 4 * (new + old) * head}
    ids = _ids(case)
    used, rows = len({i for i in ids if i >= 0}), sum(i >= 0 for i in ids)
    size = rows * case["inner"] * 2 + case["rows"] * case["outer"] * 4
    return {"bytes": size + used * case["rank"] * (case["inner"] + case["outer"]) * 2,
            "flops": 2 * rows * case["rank"] * (case["inner"] + case["outer"])}


# ---- state ---------------------------------------------------------------------------------------

def _cache(spans, page, kv_heads, dim, gen, dev):
    """A filled cache: every sequence's pages scattered over the pool, codes as the quantization of
    normal values leaves them, and the page table (-1 where a sequence has no page)."""
    counts = [max(1, -(-(n + s) // page)) for n, s in spans]
    pages = sum(counts) + 3
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(spans), max(counts)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    shape = (pages, kv_heads, page, dim)

    def codes():
        x = torch.empty(shape, dtype=torch.float16, device=dev).normal_(0.0, 36.0, generator=gen)
        return x.round_().clamp_(-127, 127).to(torch.int8)

    def scales(mean):
        return torch.empty(shape[:2], device=dev).normal_(0.0, 0.25, generator=gen).exp_().mul_(mean / 36.0)

    return {"k_codes": codes(), "v_codes": codes(), "k_scale": scales(1.0), "v_scale": scales(0.7),
            "page_table": table}


def _offsets(lengths, dev):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32).to(dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 2 + 1)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=dt, device=dev).normal_(0.0, std, generator=gen)

    state = {"case": case}
    if case["op"] == "lora":
        n, r, k, m = case["adapters"], case["rank"], case["inner"], case["outer"]
        state |= {"x": normal(case["rows"], k), "y": normal(case["rows"], m), "a": normal(n, r, k, std=k ** -0.5),
                  "b": normal(n, m, r, std=0.3 * r ** -0.5),
                  "scale": torch.empty(n, device=dev).uniform_(0.5, 2.0, generator=gen),
                  "ids": torch.tensor(_ids(case), dtype=torch.int32).to(dev)}
        return state
    spans = _spans(case)
    state |= _cache(spans, case["page"], case["kv_heads"], case["dim"], gen, dev)
    tokens = sum(n for n, _ in spans)
    state["cu"] = _offsets([n for n, _ in spans], dev)
    state["q"] = normal(tokens, case["q_heads"], case["dim"], std=1.5)
    if case["op"] == "attention":
        state["kv_len"] = torch.tensor([n + s for n, s in spans], dtype=torch.int32).to(dev)
        return state
    half, p = case["rot"] // 2, case["page"]
    state["k"] = normal(tokens, case["kv_heads"], case["dim"])
    state["v"] = normal(tokens, case["kv_heads"], case["dim"], std=0.7)
    state["start"] = torch.tensor([s for _, s in spans], dtype=torch.int32).to(dev)
    at = torch.arange(max(n + s for n, s in spans), device=dev, dtype=torch.float64)[:, None]
    angle = at * _BASE ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
    state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
    # the touched pages, from the first token of the first to the newest one
    state["read_start"] = torch.tensor([s - s % p for _, s in spans], dtype=torch.int32).to(dev)
    state["read_cu"] = _offsets([n + s % p for n, s in spans], dev)
    state["read_rows"] = sum(n + s % p for n, s in spans)
    state["read_max"] = max(n + s % p for n, s in spans)
    return state


# ---- the plain forms -----------------------------------------------------------------------------

def _places(cu, rows):
    """(sequence, place in it) of each of `rows` packed rows."""
    at = torch.arange(rows, device=cu.device)
    cu = cu.long()
    seq = torch.searchsorted(cu[1:].contiguous(), at, right=True)
    return seq, at - cu[seq]


def _plain_attention(s):
    c = s["case"]
    batch, hkv, dim, max_q = c["batch"], c["kv_heads"], c["dim"], c["max_q"]
    group, tokens = c["q_heads"] // hkv, s["q"].shape[0]
    table = s["page_table"].clamp(min=0).long()

    def whole(codes, scale):
        x = codes[table].float() * scale[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(batch, hkv, -1, dim)

    k, v = whole(s["k_codes"], s["k_scale"]), whole(s["v_codes"], s["v_scale"])
    length, cu = s["kv_len"].long(), s["cu"].long()
    i = torch.arange(max_q, device=cu.device)
    rows = (cu[:-1, None] + i).clamp(max=tokens - 1)
    q = s["q"][rows].float().reshape(batch, max_q, hkv, group, dim).permute(0, 2, 3, 1, 4)
    score = torch.matmul(q.reshape(batch, hkv, group * max_q, dim), k.transpose(-1, -2)) * dim ** -0.5
    score = score.reshape(batch, hkv, group, max_q, -1)
    at = (length - (cu[1:] - cu[:-1]))[:, None, None] + i[None, :, None]      # each query's position
    key = torch.arange(score.shape[-1], device=cu.device)[None, None, :]
    seen = (key <= at) & (key < length[:, None, None])
    if c["window"]:
        seen = seen & (key > at - c["window"])
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.reshape(batch, hkv, group * max_q, -1), v).reshape(batch, hkv, group, max_q, dim)
    out = out / torch.where(total > 0, total, torch.ones_like(total))
    seq, place = _places(s["cu"], tokens)
    return out.permute(0, 3, 1, 2, 4)[seq, place].reshape(tokens, c["q_heads"], dim).to(s["q"].dtype)


def _rotated(x, cos, sin, interleaved):
    """x [T, H, D] in 32 bits with the pairs of its first 2 * half values turned; cos, sin [T, half]."""
    half = cos.shape[1]
    x = x.float()
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _plain_append(s):
    c = s["case"]
    page, tokens = c["page"], s["k"].shape[0]
    dev, dt = s["k"].device, s["k"].dtype
    start, cu, table = s["start"].long(), s["cu"].long(), s["page_table"].long()
    seq, place = _places(s["cu"], tokens)
    cos, sin = s["cos"][start[seq] + place], s["sin"][start[seq] + place]
    q = _rotated(s["q"], cos, sin, c["interleaved"]).to(dt)
    # every page that a sequence's new tokens touch; the last one again where a sequence has fewer
    new = cu[1:] - cu[:-1]
    first, last = start // page, (start + new - 1) // page
    j = torch.minimum(first[:, None] + torch.arange((c["max_new"] + page - 2) // page + 1, device=dev), last[:, None])
    pos = j[..., None] * page + torch.arange(page, device=dev)
    fresh = ((pos >= start[:, None, None]) & (pos < (start + new)[:, None, None]))[:, :, None, :, None]
    old = (pos < start[:, None, None])[:, :, None, :, None]
    row = (cu[:-1, None, None] + pos - start[:, None, None]).clamp(0, tokens - 1)
    where = table.gather(1, j)

    def put(x, codes, scale):
        x = x[row].transpose(2, 3) * fresh                               # [B, pages, heads, page, dim]
        had = torch.where(old.any(3).squeeze(-1), scale[where], torch.zeros_like(scale[where]))
        unit = torch.maximum(had, x.abs().amax((3, 4)) / 127.0)
        inverse = torch.where(unit > 0, 1.0 / unit, torch.zeros_like(unit))
        moved = torch.round(codes[where].float() * (had * inverse)[..., None, None])
        kept = torch.where((unit > had)[..., None, None], moved, codes[where].float())
        made = torch.round(x * inverse[..., None, None]).clamp(-127, 127)
        codes[where] = torch.where(fresh, made, kept).to(torch.int8)
        scale[where] = unit

    put(_rotated(s["k"], cos, sin, c["interleaved"]), s["k_codes"], s["k_scale"])
    put(s["v"].float(), s["v_codes"], s["v_scale"])
    seq, place = _places(s["read_cu"], s["read_rows"])
    pos = s["read_start"].long()[seq] + place
    where = table[seq, pos // page]

    def values(codes, scale):
        return (codes[where, :, pos % page].float() * scale[where][..., None]).to(dt)

    return {"q": q, "k": values(s["k_codes"], s["k_scale"]), "v": values(s["v_codes"], s["v_scale"])}


def _plain_lora(s):
    # x A^T for all adapters at once, each row's own kept, then one product with all B
    n, r, k = s["a"].shape
    low = torch.matmul(s["x"].float(), s["a"].reshape(n * r, k).float().t()).reshape(-1, n, r)
    mine = (s["ids"][:, None] == torch.arange(n, device=low.device)[None]).float() * s["scale"][None]
    low = (low * mine[..., None]).reshape(-1, n * r)
    up = s["b"].float().permute(0, 2, 1).reshape(n * r, -1)
    return (s["y"].float() + torch.matmul(low, up)).to(s["y"].dtype)


# ---- the package's entry points ------------------------------------------------------------------

def _own_run(s):
    import weight_only_quantized_amd as wq
    c = s["case"]
    if c["op"] == "lora":
        if "bank" not in s:
            s["bank"] = wq.LoraBank(s["a"], s["b"], s["scale"])
        return s["bank"].add(s["y"], s["x"], s["ids"])
    if "cache" not in s:
        s["cache"] = wq.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    if c["op"] == "attention":
        return s["cache"].attention(s["q"], s["page_table"], s["kv_len"], s["cu"], max_q=c["max_q"],
                                    max_kv=c["max_kv"], window=c["window"])
    q = s["cache"].append(s["k"], s["v"], s["page_table"], s["start"], s["cu"], max_new=c["max_new"], q=s["q"],
                          cos=s["cos"], sin=s["sin"], interleaved=c["interleaved"])
    k, v = s["cache"].read(s["page_table"], s["read_start"], s["read_cu"], rows=s["read_rows"],
                           max_rows=s["read_max"], dtype=s["k"].dtype)
    return {"q": q, "k": k, "v": v}


def run(state):
    if own:
        return _own_run(state)
    return {"attention": _plain_attention, "append": _plain_append, "lora": _plain_lora}[state["case"]["op"]](state)


# ---- 64 bits, from the definitions ---------------------------------------------------------------

def _exact_attention(c, s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    page, group = c["page"], c["q_heads"] // c["kv_heads"]
    at = 0
    for b, (n, start) in enumerate(_spans(c)):
        length = n + start
        pages = s["page_table"][b, :-(-length // page)].long()
        qpos = torch.arange(start, length, device=out.device)[:, None]
        kpos = torch.arange(length, device=out.device)[None]
        hidden = kpos > qpos
        if c["window"]:
            hidden |= kpos <= qpos - c["window"]
        for h in range(c["kv_heads"]):
            k = (s["k_codes"][pages, h].double() * s["k_scale"][pages, h].double()[:, None, None]).flatten(0, 1)
            v = (s["v_codes"][pages, h].double() * s["v_scale"][pages, h].double()[:, None, None]).flatten(0, 1)
            for g in range(h * group, (h + 1) * group):
                score = s["q"][at:at + n, g].double() @ k[:length].t() / math.sqrt(c["dim"])
                out[at:at + n, g] = torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ v[:length]
        at += n
    return out


def _exact_append(c, s):
    page, dim, half = c["page"], c["dim"], c["rot"] // 2
    pair = [(2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half) for i in range(half)]
    left, right = [a for a, _ in pair], [b for _, b in pair]
    found = {"q": [], "k": [], "v": []}
    at = 0
    for b, (n, start) in enumerate(_spans(c)):
        where = slice(start, start + n)
        cos, sin = s["cos"][where].double()[:, None], s["sin"][where].double()[:, None]

        def turn(x):
            x = x.double()
            y = x.clone()
            y[..., left] = x[..., left] * cos - x[..., right] * sin
            y[..., right] = x[..., left] * sin + x[..., right] * cos
            return y

        found["q"].append(turn(s["q"][at:at + n]))
        first, skip = start // page, start % page
        pages = s["page_table"][b, first:-(-(start + n) // page)].long()
        for name, x in (("k", turn(s["k"][at:at + n])), ("v", s["v"][at:at + n].double())):
            codes = s[name + "_codes"][pages].double().transpose(1, 2).reshape(-1, c["kv_heads"], dim).clone()
            base = s[name + "_scale"][pages].double().clone()
            if skip == 0:
                base[0] = 0
            base[1:] = 0
            full = torch.zeros_like(codes)
            full[skip:skip + n] = x
            most = full.abs().reshape(len(pages), page, c["kv_heads"], dim).amax((1, 3)) / 127
            unit = torch.maximum(base, most)
            ratio = torch.where(unit > 0, base / unit, torch.zeros_like(unit))[0]
            each = unit.repeat_interleave(page, 0)[..., None]
            fresh = torch.where(each > 0, (full / each).round(), torch.zeros_like(full))
            fresh[:skip] = (codes[:skip] * ratio[None, :, None]).round()
            found[name].append((fresh * each)[:skip + n])
        at += n
    return {name: torch.cat(x) for name, x in found.items()}


def _exact_lora(c, s):
    out = s["y"].double()
    ids = torch.tensor(_ids(c), device=out.device)
    for i in sorted(set(_ids(c)) - {-1}):
        rows = (ids == i).nonzero().flatten()
        low = s["x"][rows].double() @ s["a"][i].double().t()
        out[rows] += float(s["scale"][i]) * (low @ s["b"][i].double().t())
    return out


def exact(case, seed):
    state = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "lora": _exact_lora}[case["op"]](case, state)

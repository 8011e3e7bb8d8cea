"""Refusals of the serving entry points (host checks: no GPU, no launch), and pins of their oracle."""
import ctypes

import numpy as np
import pytest

import oracle.serving_oracle as so
import weight_only_quantized_amd as wq

A = 1 << 20          # a well-aligned address: the checks only compare addresses, nothing is read
P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class Cache(ctypes.Structure):
    _fields_ = [("k_codes", P), ("v_codes", P), ("k_scale", P), ("v_scale", P), ("num_pages", I64), ("kv_heads", I32),
                ("page_size", I32), ("head_dim", I32), ("reserved", I32)]


class Batch(ctypes.Structure):
    _fields_ = [("page_table", P), ("at", P), ("cu", P), ("rows", I64), ("batch", I32), ("table_width", I32),
                ("max_rows", I32), ("reserved", I32)]


class Rope(ctypes.Structure):
    _fields_ = [("cos", P), ("sin", P), ("rows", I32), ("dim", I32), ("interleaved", I32), ("reserved", I32)]


class Attention(ctypes.Structure):
    _fields_ = [("q_heads", I32), ("dtype", I32), ("scale", ctypes.c_float), ("causal", I32), ("window", I32),
                ("max_kv", I32), ("q_stride", I64), ("out_stride", I64)]


class Bank(ctypes.Structure):
    _fields_ = [("a", P), ("b", P), ("scale", P), ("adapters", I32), ("rank", I32), ("in_features", I32),
                ("out_features", I32), ("dtype", I32), ("reserved", I32)]


def test_the_binding_packs_the_header_structures():
    from weight_only_quantized_amd import serving as s
    pairs = ((s._CACHE, Cache, range(1, 10)), (s._BATCH, Batch, range(1, 9)), (s._ROPE, Rope, range(1, 7)),
             (s._ATTENTION, Attention, (1, 2, 0.5, 4, 5, 6, 7, 8)), (s._BANK, Bank, range(1, 10)))
    for packed, structure, values in pairs:
        assert packed.size == ctypes.sizeof(structure)
        assert packed.pack(*values) == bytes(structure(*values)), structure


def cache(**kw):
    c = Cache(A, A + (64 << 20), A + (128 << 20), A + (129 << 20), 8, 2, 16, 64, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def batch(**kw):
    b = Batch(A, A, A, 4, 2, 3, 4, 0)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


FREE = A + (512 << 20)      # past every buffer of the cache


def append(c=None, b=None, k=FREE, ks=128, v=FREE + (1 << 20), vs=128, q=None, qs=0, heads=0, out=None, os_=0, dtype=0,
           rope=None):
    lib = wq.load_library()
    ref = lambda s: ctypes.byref(s) if s is not None else None  # noqa: E731
    c, b = (cache() if c is None else c), (batch() if b is None else b)
    return wq.STATUS[lib.gptq_kv_append(ref(c), ref(b), k, ks, v, vs, q, qs, heads, out, os_, dtype, ref(rope), None)]


def rope(**kw):
    r = Rope(A, A, 100, 64, 0, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def test_append_refusals():
    lib = wq.load_library()
    assert wq.STATUS[lib.gptq_kv_append(None, ctypes.byref(batch()), FREE, 128, FREE, 128, None, 0, 0, None, 0, 0, None,
                                        None)] == "E_INVALID_ARG"
    for kw, want in ((dict(page_size=24), "E_UNSUPPORTED"), (dict(page_size=8), "E_UNSUPPORTED"),
                     (dict(page_size=512), "E_UNSUPPORTED"), (dict(head_dim=96), "E_UNSUPPORTED"),
                     (dict(kv_heads=0), "E_SHAPE"), (dict(num_pages=0), "E_SHAPE"), (dict(reserved=1), "E_INVALID_ARG"),
                     (dict(k_codes=None), "E_INVALID_ARG"), (dict(v_codes=A + 8), "E_INVALID_ARG"),
                     (dict(v_scale=A + 2), "E_INVALID_ARG")):
        assert append(c=cache(**kw)) == want, kw
    for kw, want in ((dict(rows=-1), "E_SHAPE"), (dict(max_rows=5), "E_SHAPE"), (dict(batch=-1), "E_SHAPE"),
                     (dict(table_width=0), "E_SHAPE"), (dict(cu=None), "E_INVALID_ARG"), (dict(at=None), "E_INVALID_ARG"),
                     (dict(page_table=A + 1), "E_INVALID_ARG"), (dict(reserved=2), "E_INVALID_ARG"),
                     (dict(rows=0, max_rows=0), "OK"), (dict(batch=0), "OK")):
        assert append(b=batch(**kw)) == want, kw
    for kw in (dict(k=None), dict(k=FREE + 8), dict(ks=120), dict(ks=132), dict(vs=64), dict(dtype=2), dict(dtype=7),
               dict(k=A), dict(q=FREE + (2 << 20), qs=128, heads=2, out=FREE + (3 << 20), os_=128),
               dict(q=FREE + (2 << 20), qs=128, heads=2, rope=rope()),
               dict(q=FREE + (2 << 20), qs=128, heads=2, out=FREE + (2 << 20) + 64, os_=128, rope=rope()),
               dict(q=FREE + (2 << 20), qs=128, heads=2, out=FREE, os_=128, rope=rope()),
               dict(q=FREE + (2 << 20), qs=128, heads=2, out=A, os_=128, rope=rope()),
               dict(rope=rope(cos=None)), dict(rope=rope(sin=A + 4)), dict(rope=rope(interleaved=2)),
               dict(rope=rope(reserved=1))):
        assert append(**kw) == "E_INVALID_ARG", kw
    assert append(rope=rope(dim=80)) == "E_UNSUPPORTED" and append(rope=rope(dim=24)) == "E_UNSUPPORTED"
    assert append(rope=rope(rows=0)) == "E_SHAPE"
    # q, k and v as slices of one fused row, q rotated in place: taken (what stops it is the device)
    assert append(k=FREE + 256, ks=384, v=FREE + 512, vs=384, q=FREE, qs=384, heads=2, out=FREE, os_=384,
                  rope=rope()) in ("E_HIP", "E_DEVICE")
    assert append(k=FREE + 128, ks=384, v=FREE + 512, vs=384, q=FREE, qs=384, heads=2, out=FREE, os_=384,
                  rope=rope()) == "E_INVALID_ARG"


def attention(c=None, b=None, q=FREE, out=FREE + (1 << 20), ws=None, ws_bytes=0, **kw):
    lib = wq.load_library()
    a = Attention(4, 0, 0.125, 1, 0, 48, 256, 256)
    for k, v in kw.items():
        setattr(a, k, v)
    c, b = (cache() if c is None else c), (batch() if b is None else b)
    return wq.STATUS[lib.gptq_kv_attention(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), q, out, ws, ws_bytes, None)]


def test_attention_refusals():
    for kw, want in ((dict(q_heads=3), "E_SHAPE"), (dict(q_heads=0), "E_SHAPE"), (dict(q_heads=130), "E_SHAPE"),
                     (dict(dtype=2), "E_INVALID_ARG"), (dict(scale=float("nan")), "E_INVALID_ARG"),
                     (dict(scale=float("inf")), "E_INVALID_ARG"), (dict(causal=2), "E_INVALID_ARG"),
                     (dict(window=-1), "E_INVALID_ARG"), (dict(max_kv=-1), "E_INVALID_ARG"), (dict(q=None), "E_INVALID_ARG"),
                     (dict(out=FREE + (1 << 20) + 8), "E_INVALID_ARG"), (dict(q_stride=252), "E_INVALID_ARG"),
                     (dict(out_stride=128), "E_INVALID_ARG"), (dict(out=FREE), "E_INVALID_ARG"),
                     (dict(out=A), "E_INVALID_ARG"), (dict(b=batch(rows=0, max_rows=0)), "OK"),
                     (dict(c=cache(head_dim=32)), "E_UNSUPPORTED")):
        assert attention(**kw) == want, kw
    lib, n = wq.load_library(), ctypes.c_size_t()
    a = Attention(4, 0, 0.125, 1, 0, 48, 256, 256)
    assert lib.gptq_kv_attention_workspace_size(ctypes.byref(cache()), ctypes.byref(batch()), ctypes.byref(a), None) == 1
    assert lib.gptq_kv_attention_workspace_size(None, ctypes.byref(batch()), ctypes.byref(a), ctypes.byref(n)) == 1


def test_attention_workspace_is_checked():
    """One sequence over a long cache splits its keys: a missing, short or misaligned workspace is
    refused."""
    lib, n = wq.load_library(), ctypes.c_size_t()
    c, b = cache(num_pages=4096), batch(rows=1, max_rows=1, batch=1, table_width=4096)
    c.v_codes, c.k_scale, c.v_scale = A + (64 << 20), A + (128 << 20), A + (129 << 20)
    a = Attention(4, 0, 0.125, 1, 0, 65536, 256, 256)
    assert lib.gptq_kv_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), ctypes.byref(n)) == 0
    if n.value:
        ws = FREE + (64 << 20)
        for kw in (dict(), dict(ws=ws, ws_bytes=n.value - 1), dict(ws=ws + 128, ws_bytes=n.value)):
            assert attention(c=c, b=b, max_kv=65536, **kw) == "E_WORKSPACE"
        assert attention(c=c, b=b, max_kv=65536, ws=FREE, ws_bytes=n.value) == "E_INVALID_ARG"


def test_read_refusals():
    lib = wq.load_library()
    ok = dict(k=FREE, v=FREE + (1 << 20), dtype=0)

    def read(c=None, b=None, **kw):
        a = ok | kw
        return wq.STATUS[lib.gptq_kv_read(ctypes.byref(c or cache()), ctypes.byref(b or batch()), a["k"], a["v"], a["dtype"],
                                          None)]
    for kw in (dict(k=None, v=None), dict(k=FREE + 4), dict(dtype=3), dict(v=FREE), dict(k=A)):
        assert read(**kw) == "E_INVALID_ARG", kw
    assert read(b=batch(rows=0, max_rows=0)) == "OK" and read(c=cache(page_size=17)) == "E_UNSUPPORTED"


def test_lora_refusals():
    lib = wq.load_library()
    n = ctypes.c_size_t()

    def bank(**kw):
        k = Bank(A, A + (1 << 20), A + (2 << 20), 3, 16, 64, 96, 0, 0)
        for f, v in kw.items():
            setattr(k, f, v)
        return k

    def call(k=None, x=FREE, y=FREE + (1 << 20), ids=FREE + (2 << 20), M=5, out=FREE + (3 << 20), ws=FREE + (4 << 20),
             size=1 << 30):
        return wq.STATUS[lib.gptq_lora_add(ctypes.byref(k or bank()), x, y, ids, M, out, ws, size, None)]

    for kw, want in ((dict(rank=4), "E_UNSUPPORTED"), (dict(rank=20), "E_UNSUPPORTED"), (dict(rank=136), "E_UNSUPPORTED"),
                     (dict(adapters=0), "E_SHAPE"), (dict(in_features=40), "E_SHAPE"), (dict(out_features=0), "E_SHAPE"),
                     (dict(dtype=2), "E_INVALID_ARG"), (dict(reserved=1), "E_INVALID_ARG"), (dict(a=None), "E_INVALID_ARG"),
                     (dict(b=A + (1 << 20) + 8), "E_INVALID_ARG"), (dict(scale=A + 1), "E_INVALID_ARG")):
        assert call(bank(**kw)) == want, kw
    for kw, want in ((dict(x=None), "E_INVALID_ARG"), (dict(ids=None), "E_INVALID_ARG"), (dict(y=FREE + (1 << 20) + 4), "E_INVALID_ARG"),
                     (dict(M=-1), "E_SHAPE"), (dict(M=(1 << 24) + 1), "E_SHAPE"), (dict(out=FREE), "E_INVALID_ARG"),
                     (dict(out=FREE + (1 << 20) + 16), "E_INVALID_ARG"), (dict(out=A), "E_INVALID_ARG"),
                     (dict(M=0), "OK")):
        assert call(**kw) == want, kw
    for kw, want in ((dict(ws=None), "E_WORKSPACE"), (dict(size=0), "E_WORKSPACE"), (dict(ws=FREE + (4 << 20) + 8), "E_WORKSPACE"),
                     (dict(ws=FREE), "E_INVALID_ARG")):
        assert call(bank(rank=64), **kw) == want, kw
    assert call() in ("E_HIP", "E_DEVICE")
    assert call(out=FREE + (1 << 20)) in ("E_HIP", "E_DEVICE")          # in place
    assert lib.gptq_lora_workspace_size(ctypes.byref(bank(rank=64)), 5, ctypes.byref(n)) == 0 and n.value > 0
    # few rows of small adapters: one launch, no workspace
    assert lib.gptq_lora_workspace_size(ctypes.byref(bank()), 5, ctypes.byref(n)) == 0 and n.value == 0
    assert call(ws=None, size=0) in ("E_HIP", "E_DEVICE")
    assert lib.gptq_lora_workspace_size(ctypes.byref(bank()), 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.gptq_lora_workspace_size(ctypes.byref(bank()), 5, None) == 1


def test_binding_refuses_wrong_tensors():
    import torch
    codes, scale = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        wq.KVCache(codes, codes[:3], scale, scale)
    with pytest.raises(ValueError):
        wq.KVCache(codes.float(), codes, scale, scale)
    with pytest.raises(ValueError):
        wq.KVCache(codes, codes, scale.half(), scale)
    a, b, s = torch.zeros(2, 8, 64, dtype=torch.float16), torch.zeros(2, 32, 8, dtype=torch.float16), torch.zeros(2)
    wq.LoraBank(a, b, s)
    with pytest.raises(ValueError):
        wq.LoraBank(a, b.transpose(1, 2), s)
    with pytest.raises(ValueError):
        wq.LoraBank(a, b, s.half())
    with pytest.raises(TypeError):
        wq.LoraBank(a.float(), b.float(), s)
    bank = wq.LoraBank(a, b, s)
    y, x, ids = torch.zeros(3, 32, dtype=torch.float16), torch.zeros(3, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    for bad in (dict(x=x[:2]), dict(x=x.float()), dict(ids=ids.long()), dict(ids=ids[:2]), dict(out=y.t())):
        with pytest.raises((TypeError, ValueError)):
            bank.add(**(dict(y=y, x=x, ids=ids) | bad))


# ---- pins of the oracle --------------------------------------------------------------------------

def test_oracle_rotation_is_a_turn_of_pairs():
    rng = np.random.default_rng(0)
    x, angle = rng.normal(size=(3, 2, 8)), rng.normal(size=(3, 3))
    for inter in (False, True):
        y = so.rotate(x, np.cos(angle), np.sin(angle), inter)
        a, b = ((0, 1), (2, 3), (4, 5)) if inter else ((0, 3), (1, 4), (2, 5)), None
        for i, (p, r) in enumerate(a):
            z = (x[..., p] + 1j * x[..., r]) * np.exp(1j * angle[:, i])[:, None]
            assert np.allclose(y[..., p], z.real) and np.allclose(y[..., r], z.imag)
        assert np.array_equal(y[..., 6:], x[..., 6:])


def test_oracle_append_and_attention_by_hand():
    codes, scale = np.zeros((3, 1, 2, 2), np.int8), np.zeros((3, 1), np.float32)
    codes[2, 0, 0], scale[2, 0] = [100, -50], 0.01                     # one older token: (1, -0.5)
    table = np.asarray([[2, 0]], np.int32)
    x = np.asarray([[[2.54, 0.0]], [[0.0, 1.27]]])
    ideal, unit = so.append(codes, scale, x, table, [1], [0, 2])
    assert np.allclose(unit[:, 0], [0.01, 0, 0.02]) and np.allclose(ideal[2, 0, 0], [50, -25])
    assert np.allclose(ideal[2, 0, 1], [127, 0]) and np.allclose(ideal[0, 0, 0], [0, 127])
    k = np.asarray([[[[1, 0], [0, 1]]], [[[1, 1], [9, 9]]]], np.int8)
    one = np.ones((2, 1), np.float32)
    q = np.asarray([[[np.log(3.0), 0.0]], [[0.0, 0.0]]])
    out, _, _ = so.attention(q, k, k, one, one, np.asarray([[0, 1]], np.int32), [3], [0, 2], 1.0)
    assert np.allclose(out[0, 0], [0.75, 0.25]) and np.allclose(out[1, 0], [2 / 3, 2 / 3])
    out, _, _ = so.attention(q, k, k, one, one, np.asarray([[0, -1]], np.int32), [3], [0, 2], 1.0, window=1)
    assert np.allclose(out[0, 0], [0, 1]) and np.allclose(out[1, 0], [0, 0])


def test_oracle_lora_by_hand():
    out, w = so.lora([[1.0, 2.0], [5.0, 6.0]], [[1.0, -1.0], [1.0, 1.0]], [[[2.0, 1.0]]], [[[3.0], [-1.0]]], [0.5], [0, -1])
    assert np.allclose(out, [[2.5, 1.5], [5, 6]]) and np.allclose(w, [[4.5, 1.5], [0, 0]])

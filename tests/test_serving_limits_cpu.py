"""Sizes at the edges of what the serving entry points take, as the host sees them (no GPU, no launch)."""
import ctypes

import pytest

import weight_only_quantized_amd as wq
from test_serving_cpu import A, FREE, Attention, Bank, append, attention, batch, cache, rope


def workspace(c, b, **kw):
    """(status, bytes) of an attention call's workspace."""
    a = Attention(4, 0, 0.125, 1, 0, 48, 256, 256)
    for k, v in kw.items():
        setattr(a, k, v)
    n = ctypes.c_size_t(12345)
    st = wq.load_library().gptq_kv_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), ctypes.byref(n))
    return wq.STATUS[st], n.value


@pytest.mark.parametrize("max_kv", [48, 65536])
def test_no_rows_of_any_sequence(max_kv):
    """max_rows 0 says that every row is absent: nothing to do, however long the table."""
    b = batch(max_rows=0, table_width=4096)
    assert workspace(cache(), b, max_kv=max_kv) == ("OK", 0)
    assert attention(b=b, max_kv=max_kv) == "OK"


def test_steps_count_by_what_a_call_can_see():
    """A wide table is no reason to refuse short sequences; what cannot be counted is refused by both
    entry points, as a size."""
    c = cache(kv_heads=8, page_size=256, num_pages=4096)
    b = batch(rows=1 << 20, max_rows=1, batch=1 << 20, table_width=1 << 16)
    wide = dict(q_heads=8, q_stride=512, out_stride=512)
    assert workspace(c, b, max_kv=64, **wide) == ("OK", 0)
    assert workspace(c, b, max_kv=1 << 24, window=40, **wide) == ("OK", 0)
    assert workspace(c, b, max_kv=1 << 24, **wide)[0] == "E_SHAPE"
    assert attention(c=c, b=b, max_kv=1 << 24, **wide) == "E_SHAPE"
    # any number of sequences, columns and tokens
    b = batch(rows=1 << 24, max_rows=1 << 24, batch=1 << 20, table_width=1 << 22)
    c.kv_heads = 1024
    for q_heads in (1024, 65536):
        huge = dict(q_heads=q_heads, q_stride=q_heads * 64, out_stride=q_heads * 64, max_kv=1 << 30)
        assert workspace(c, b, **huge)[0] == "E_SHAPE" and attention(c=c, b=b, **huge) == "E_SHAPE"


def test_launches_that_cannot_number_their_threads():
    lib, n = wq.load_library(), ctypes.c_size_t()
    c, b = cache(kv_heads=1024, num_pages=4096), batch(rows=1 << 24, max_rows=1 << 24, batch=1)
    far = FREE + (1 << 45)
    assert append(c=c, b=b, ks=65536, v=far, vs=65536) == "E_SHAPE"
    assert wq.STATUS[lib.gptq_kv_read(ctypes.byref(c), ctypes.byref(b), FREE, far, 0, None)] == "E_SHAPE"
    bank = Bank(A, A + (1 << 20), A + (2 << 20), 3, 16, 64, 1 << 20, 0, 0)
    assert wq.STATUS[lib.gptq_lora_workspace_size(ctypes.byref(bank), 1 << 24, ctypes.byref(n))] == "E_SHAPE"
    assert wq.STATUS[lib.gptq_lora_add(ctypes.byref(bank), FREE, far, FREE, 1 << 24, far, None, 0, None)] == "E_SHAPE"


def test_tensors_on_the_host_are_refused():
    """The kernels would be given host addresses."""
    import torch
    c = wq.KVCache.allocate(4, 16, 2, 64, device="cpu")
    at, table, cu = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32)
    k, q = torch.zeros(1, 2, 64, dtype=torch.float16), torch.zeros(1, 4, 64, dtype=torch.float16)
    bank = wq.LoraBank(torch.zeros(2, 8, 64).half(), torch.zeros(2, 32, 8).half(), torch.zeros(2))
    for call in (lambda: c.append(k, k, table, at, cu, max_new=1), lambda: c.attention(q, table, at, cu, max_q=1),
                 lambda: c.read(table, at, cu, rows=1, max_rows=1),
                 lambda: bank.add(torch.zeros(3, 32).half(), torch.zeros(3, 64).half(), torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_a_workspace_is_a_whole_tensor_of_the_device():
    """(Pointer, bytes) that the library may write to: not host memory, not a view that repeats itself."""
    import torch
    from weight_only_quantized_amd import serving
    t = torch.zeros(16, dtype=torch.float32)                    # get_device() of the host is -1
    assert serving._scratch(t, -1) == (t.data_ptr(), 64)
    for bad, device in ((t, 0), (t[:1].expand(1 << 20), -1), (t[::2], -1)):
        with pytest.raises(ValueError, match="workspace"):
            serving._scratch(bad, device)


def test_outputs_do_not_overlap_tables():
    """Page tables, lengths, rotation tables, ids and adapters' scales are read while outputs and
    workspaces are written."""
    lib, n = wq.load_library(), ctypes.c_size_t()
    here = FREE + (8 << 20)
    for table in ("page_table", "at", "cu"):
        b = batch(**{table: here})
        assert attention(b=b, out=here) == "E_INVALID_ARG", table
        assert append(b=b, q=FREE + (2 << 20), qs=128, heads=2, out=here, os_=128, rope=rope()) == "E_INVALID_ARG", table
        for k, v in ((here, None), (None, here)):
            assert wq.STATUS[lib.gptq_kv_read(ctypes.byref(cache()), ctypes.byref(b), k, v, 0, None)] == "E_INVALID_ARG", table
        long = batch(rows=1, max_rows=1, batch=1, table_width=4096, **{table: here})
        assert workspace(cache(), long, max_kv=65536)[1] > 0
        assert attention(b=long, max_kv=65536, ws=here, ws_bytes=1 << 30) == "E_INVALID_ARG", table
    for table in ("cos", "sin"):
        assert append(q=FREE + (2 << 20), qs=128, heads=2, out=here, os_=128, rope=rope(**{table: here})) == "E_INVALID_ARG", table

    def lora(scale=A + (2 << 20), ids=FREE + (2 << 20), out=FREE + (3 << 20), ws=FREE + (4 << 20)):
        bank = Bank(A, A + (1 << 20), scale, 3, 64, 64, 96, 0, 0)
        return wq.STATUS[lib.gptq_lora_add(ctypes.byref(bank), FREE, FREE + (1 << 20), ids, 5, out, ws, 1 << 20, None)]
    assert lora() in ("E_HIP", "E_DEVICE")
    for kw in (dict(scale=here, out=here), dict(scale=here, ws=here), dict(ids=here, ws=here), dict(ids=here, out=here)):
        assert lora(**kw) == "E_INVALID_ARG", kw


@pytest.mark.parametrize("batch_size,max_rows,tokens", [(1, 1, 65536), (64, 1, 4096), (4, 64, 16000)])
def test_a_split_call_needs_its_workspace(batch_size, max_rows, tokens):
    """Calls whose keys are split: a missing, short, misaligned or overlapping workspace is refused."""
    rows = batch_size * max_rows
    c = cache(kv_heads=8, num_pages=512)
    b = batch(rows=rows, max_rows=max_rows, batch=batch_size, table_width=4096)
    far = FREE + (1 << 30)
    kw = dict(max_kv=tokens, q_heads=32, q_stride=2048, out_stride=2048)
    status, need = workspace(c, b, **kw)
    assert status == "OK" and need > 0
    for ws in (dict(), dict(ws=far, ws_bytes=need - 1), dict(ws=far + 128, ws_bytes=need)):
        assert attention(c=c, b=b, out=FREE + (64 << 20), **ws, **kw) == "E_WORKSPACE", ws
    assert attention(c=c, b=b, out=FREE + (64 << 20), ws=FREE, ws_bytes=need, **kw) == "E_INVALID_ARG"
    assert attention(c=c, b=b, out=FREE + (64 << 20), ws=far, ws_bytes=need, **kw) in ("E_HIP", "E_DEVICE")

"""Sizes at the edges of what the serving entry points take, as the host sees them (no GPU, no launch)."""
import ctypes

import pytest

import weight_only_quantized_amd as wq
from test_serving_cpu import Attention, attention, batch, cache


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

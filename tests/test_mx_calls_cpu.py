"""Calls on microscaled tensors that the binding refuses before anything runs (no GPU)."""
import pytest
import torch

import weight_only_quantized_amd as wq


@pytest.mark.parametrize("K", [(1 << 31) - 32, 1 << 31, (1 << 32) + 256])
def test_rows_longer_than_the_library_can_be_told(K):
    """Rows past 2^20 inputs are GPTQ_E_SHAPE, also where K does not fit the structure's 32 bits."""
    try:
        t = wq.MXTensor(torch.empty((0, K // 2), dtype=torch.uint8), torch.empty((0, K // 32), dtype=torch.uint8))
    except wq.GPTQError as e:
        assert K >= 1 << 31 and e.name == "E_SHAPE"
    else:
        assert K < 1 << 31
        assert wq.STATUS[wq.load_library().gptq_mx_dequantize(t._c, 1 << 20, 1, None)] == "E_SHAPE"

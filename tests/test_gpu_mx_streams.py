"""Weights in the format that were made on another stream than the one that lays them out."""
import numpy as np
import pytest

import oracle.mx_oracle as mo

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("made", ["given", "quantized"])
@pytest.mark.parametrize("gated", [False, True])
def test_sources_of_another_stream_may_be_freed(gated, made):
    """Their memory is not handed out again on their own stream before the layout, held back here, has read it."""
    import torch
    import weight_only_quantized_amd as wq
    N, K = 1000, 4096
    side = torch.cuda.Stream()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    w32 = [torch.randn((N, K), device="cuda", generator=gen) for _ in range(2 if gated else 1)]
    x = torch.randn((3, K), device="cuda", generator=gen).bfloat16()
    make = wq.MXGatedLinear if gated else wq.MXLinear
    want = make(*(wq.MXTensor.quantize(w) for w in w32)).gemm(x)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sources = [wq.MXTensor.quantize(w) for w in w32]
        if made == "given":
            sources = [wq.MXTensor(t.codes.clone(), t.scales.contiguous()) for t in sources]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    held = {(p.untyped_storage().data_ptr(), p.untyped_storage().nbytes()) for t in sources for p in t._keep}
    torch.cuda._sleep(1 << 27)
    layer = make(*sources)
    del sources
    with torch.cuda.stream(side):
        for _, size in sorted(held) * 2:
            new = torch.empty(size, dtype=torch.uint8, device="cuda")
            a = new.data_ptr()
            assert all(a + size <= b or b + n <= a for b, n in held)
            new.fill_(0x77)
    assert torch.equal(layer.gemm(x), want)
    torch.cuda.synchronize()
    host = [mo.values(*mo.quantize(w.cpu().double().numpy())) for w in w32]
    xv = x.cpu().double().numpy()
    exact = mo.gated(xv, *host, "silu") if gated else mo.gemm(xv, host[0])
    got = want.cpu().double().numpy()
    assert np.linalg.norm(got - exact) <= 1.02 * 2.0 ** -8 * np.linalg.norm(exact)

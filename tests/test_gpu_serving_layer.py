"""The example layer (examples/serve_layer.py): projections, adapters, cache and attention as they are
used together, prompts and then tokens, against the oracles composed in float64."""
import importlib.util
import os

import numpy as np
import pytest

import oracle.serving_oracle as so

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("serve_layer", os.path.join(ROOT, "examples", "serve_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def host(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


def weight(h):
    """W [N, K] in float64 of a repacked layer with float16 scales and groups of 128."""
    d = h.decode()
    scale = d["scales"].astype(np.uint16).view(np.float16).astype(np.float64)
    g = np.arange(h.K) // 128
    return ((d["codes"].astype(np.float64) - d["zeros"][g]) * scale[g]).T


def test_layer_against_composed_oracles(example):
    """Every stage's output is rounded to float16 as the layer's is; codes may differ by one where a
    value lies at a rounding boundary, so the result is compared as a whole: 1 % of its norm, which is
    a small multiple of 8-bit and float16 rounding, and what a swapped row, head or page exceeds."""
    import torch
    hidden, hq, hkv, dim, page = 256, 4, 2, 64, 16
    layer = example.random_layer(hidden, hq, hkv, dim, 24, page, 128, 3, 8, torch.float16, seed=3)
    pages = example.Pages(24, page, 3, 6)
    Wqkv, Wout = weight(layer.qkv), weight(layer.out)
    banks = [[host(t) for t in (b.a, b.b, b.scale)] for b in (layer.qkv_bank, layer.out_bank)]
    cos, sin = host(layer.cos), host(layer.sin)
    codes = [np.zeros((24, hkv, page, dim)) for _ in "kv"]
    scales = [np.zeros((24, hkv)) for _ in "kv"]
    rng = np.random.default_rng(4)
    adapter = np.asarray([-1, 2, 0], np.int32)
    length = np.zeros(3, np.int32)
    half = lambda t: t.astype(np.float16).astype(np.float64)  # noqa: E731
    for counts in ([37, 5, 16], [1, 1, 1], [1, 0, 1], [2, 30, 1], [1, 1, 1]):
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        ids = np.repeat(adapter, counts).astype(np.int32)
        x = half(rng.normal(0, 1, (int(cu[-1]), hidden)))
        table = pages.grow((length + counts).tolist())
        z = layer(torch.from_numpy(x).cuda().half(), table, torch.from_numpy(length).cuda(), torch.from_numpy(cu).cuda(),
                  max(counts), torch.from_numpy(ids).cuda())
        y = half(so.lora(half(x @ Wqkv.T), x, *banks[0], ids)[0])
        pos = np.concatenate([np.arange(s, s + n) for s, n in zip(length, counts)])
        q, k, v = (y[:, a:b].reshape(-1, h, dim) for a, b, h in
                   ((0, hq * dim, hq), (hq * dim, (hq + hkv) * dim, hkv), ((hq + hkv) * dim, None, hkv)))
        q = half(so.rotate(q, cos[pos], sin[pos], False))
        host_table = pages.table.numpy()
        for i, t in enumerate((so.rotate(k, cos[pos], sin[pos], False), v)):
            ideal, scales[i] = so.append(codes[i], scales[i], t, host_table, length, cu)
            codes[i] = np.rint(ideal)
        length = (length + counts).astype(np.int32)
        a, _, _ = so.attention(q, codes[0], codes[1], scales[0], scales[1], host_table, length, cu, dim ** -0.5)
        a = half(a.reshape(-1, hq * dim))
        want = so.lora(half(a @ Wout.T), a, *banks[1], ids)[0]
        err = np.linalg.norm(host(z) - want) / np.linalg.norm(want)
        assert err < 0.01, (counts, err)


def test_pages_come_back(example):
    p = example.Pages(8, 16, 2, 4)
    p.grow([40, 17])
    assert len(p.free) == 3
    p.release(0)
    assert len(p.free) == 6 and bool((p.table[0] == -1).all())


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_command_runs(example, graph, capsys):
    argv = ["--requests", "3", "--prompt", "90", "--tokens", "12"] + (["--graph"] if graph else [])
    x = example.main(argv)
    assert "us a step" in capsys.readouterr().out
    if graph:
        import torch
        assert torch.equal(x, example.main(argv[:-1]))

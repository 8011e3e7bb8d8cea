#!/usr/bin/env python3
"""One attention layer of a served decoder on an MI355X: quantized projections with the requests' own
low-rank adapters beside them, a paged 8-bit cache, prompts first and then token by token; with
--feed-forward the layer's feed-forward block too, its weights in microscaled 4-bit floating point.

    python examples/serve_layer.py                      # Llama-3-8B-shaped layer, 4 requests
    python examples/serve_layer.py --requests 64 --tokens 100 --graph
    python examples/serve_layer.py --requests 64 --feed-forward 14336 --graph

Weights, adapters and inputs are random: the layer shows how the calls go together and prints times.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_amd as wq  # noqa: E402


def rotation_tables(positions, dim, base=500000.0, device="cuda"):
    """cos and sin of each position's angles, float32 [positions, dim / 2]."""
    freq = base ** (-torch.arange(dim // 2, device=device, dtype=torch.float64) / (dim // 2))
    angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


class Pages:
    """The pages of a cache and which sequence has which: the host's side of a paged cache."""

    def __init__(self, num_pages, page_size, requests, width, device="cuda"):
        self.free = list(range(num_pages))[::-1]
        self.page_size, self.held = page_size, [[] for _ in range(requests)]
        self.table = torch.full((requests, width), -1, dtype=torch.int32)
        self.on_device = self.table.to(device)
        self.changed = False

    def grow(self, lengths):
        """Give every sequence pages for its length; the table on the device follows when it changed."""
        for b, n in enumerate(lengths):
            while len(self.held[b]) * self.page_size < n:
                self.held[b].append(self.free.pop())
                self.table[b, len(self.held[b]) - 1] = self.held[b][-1]
                self.changed = True
        if self.changed:
            self.on_device.copy_(self.table)
            self.changed = False
        return self.on_device

    def release(self, b):
        self.free += self.held[b]
        self.held[b] = []
        self.table[b] = -1
        self.changed = True


class AttentionLayer:
    """x -> attention(x) of one layer: qkv and output projections are repacked quantized layers, each with
    a bank of adapters (or None); keys and values go into `cache`."""

    def __init__(self, qkv, out, q_heads, cache, cos, sin, qkv_bank=None, out_bank=None):
        self.qkv, self.out, self.q_heads, self.cache = qkv, out, q_heads, cache
        self.cos, self.sin, self.qkv_bank, self.out_bank = cos, sin, qkv_bank, out_bank

    def __call__(self, x, page_table, start, cu, max_new, ids=None):
        """x [T, hidden]: the packed new tokens; sequence b has start[b] tokens in the cache and gets rows
        cu[b] .. cu[b + 1]; ids [T]: each row's adapter."""
        cache, hq, hkv, dim = self.cache, self.q_heads, self.cache.kv_heads, self.cache.head_dim
        T = x.shape[0]
        y = self.qkv.gemm(x)
        if self.qkv_bank is not None:
            self.qkv_bank.add(y, x, ids, out=y)
        # q, k and v are slices of the projection's rows; q is rotated in place, k on its way into the cache
        q = y[:, :hq * dim].view(T, hq, dim)
        k = y[:, hq * dim:(hq + hkv) * dim].view(T, hkv, dim)
        v = y[:, (hq + hkv) * dim:].view(T, hkv, dim)
        cache.append(k, v, page_table, start, cu, max_new=max_new, q=q, cos=self.cos, sin=self.sin, q_out=q)
        o = cache.attention(q, page_table, start + (cu[1:] - cu[:-1]), cu, max_q=max_new).view(T, hq * dim)
        z = self.out.gemm(o)
        if self.out_bank is not None:
            self.out_bank.add(z, o, ids, out=z)
        return z


class FeedForward:
    """x -> down(act(x Wg^T) * (x Wu^T)) with weights in the format.  Few rows are multiplied as they are (the
    weights' bytes take the time), many in 4 bits too (four times the rate of 16-bit products)."""

    def __init__(self, gate, up, down, activation="silu", many=256):
        self.gate_up, self.down, self.many = wq.MXGatedLinear(gate, up, activation), wq.MXLinear(down), many

    def __call__(self, x):
        quantized = wq.MXTensor.quantize if x.shape[0] > self.many else lambda t: t
        return self.down.gemm(quantized(self.gate_up.gemm(quantized(x), dtype=x.dtype)), dtype=x.dtype)


def random_feed_forward(hidden, inner, seed=2):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def weights(N, K):
        return wq.MXTensor.quantize(torch.empty((N, K), device="cuda").normal_(0, K ** -0.5, generator=gen))

    return FeedForward(weights(inner, hidden), weights(inner, hidden), weights(hidden, inner))


def random_projection(K, N, gen, bits=4, group=128):
    """A repacked 4-bit layer of random codes with weights of about K ** -0.5."""
    G = K // group
    qweight = torch.randint(-2 ** 31, 2 ** 31, (K // 32 * bits, N), generator=gen, device="cuda").to(torch.int32)
    qzeros = torch.full((G, N // 32 * bits), 0x77777777, dtype=torch.int32, device="cuda")
    scales = torch.empty((G, N), device="cuda").uniform_(0.8, 1.2, generator=gen).mul_(K ** -0.5 / 4.6).half()
    return wq.repack(qweight, qzeros, scales, bits=bits, group_size=group)


def random_bank(K, N, adapters, rank, dtype, gen):
    a = torch.empty((adapters, rank, K), device="cuda").normal_(0, K ** -0.5, generator=gen).to(dtype)
    b = torch.empty((adapters, N, rank), device="cuda").normal_(0, 0.3 * rank ** -0.5, generator=gen).to(dtype)
    return wq.LoraBank(a, b, torch.ones(adapters, device="cuda"))


def random_layer(hidden, q_heads, kv_heads, dim, pages, page_size, positions, adapters, rank, dtype, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    qkv_n, out_k = (q_heads + 2 * kv_heads) * dim, q_heads * dim
    cos, sin = rotation_tables(positions, dim)
    return AttentionLayer(random_projection(hidden, qkv_n, gen), random_projection(out_k, hidden, gen), q_heads,
                          wq.KVCache.allocate(pages, page_size, kv_heads, dim), cos, sin,
                          random_bank(hidden, qkv_n, adapters, rank, dtype, gen),
                          random_bank(out_k, hidden, adapters, rank, dtype, gen))


def offsets(counts, device="cuda"):
    return torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).to(device)


def main(argv=None):
    p = argparse.ArgumentParser()
    p.add_argument("--requests", type=int, default=4)
    p.add_argument("--prompt", type=int, default=700, help="the longest prompt")
    p.add_argument("--tokens", type=int, default=32, help="tokens to generate")
    p.add_argument("--page", type=int, default=16)
    p.add_argument("--rank", type=int, default=16)
    p.add_argument("--feed-forward", type=int, default=0, help="width of the feed-forward block, a multiple of 32 (0: none)")
    p.add_argument("--graph", action="store_true", help="replay the token step as one HIP graph")
    a = p.parse_args(argv)
    hidden, q_heads, kv_heads, dim, dtype = 4096, 32, 8, 128, torch.bfloat16
    prompts = [max(1, a.prompt * (i + 1) // a.requests) for i in range(a.requests)]
    longest = max(prompts) + a.tokens
    width = -(-longest // a.page)
    layer = random_layer(hidden, q_heads, kv_heads, dim, width * a.requests, a.page, longest, 8, a.rank, dtype)
    block = random_feed_forward(hidden, a.feed_forward) if a.feed_forward else None
    pages = Pages(width * a.requests, a.page, a.requests, width)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    adapter = torch.arange(a.requests, dtype=torch.int32, device="cuda") % 9 - 1      # -1: none

    # the prompts, all in one call
    x = torch.empty((sum(prompts), hidden), dtype=dtype, device="cuda").normal_(generator=gen)
    cu = offsets(prompts)
    start = torch.zeros(a.requests, dtype=torch.int32, device="cuda")
    table = pages.grow(prompts)
    ids = adapter.repeat_interleave(torch.tensor(prompts, device="cuda"))
    torch.cuda.synchronize()
    t = time.perf_counter()
    z = layer(x, table, start, cu, max(prompts), ids)
    if block is not None:
        z = z + block(z)
    torch.cuda.synchronize()
    print(f"prompts of {sum(prompts)} tokens: {1e3 * (time.perf_counter() - t):.2f} ms (first call)")

    # token by token: each request's last output (scaled) is its next input
    length = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    one = torch.arange(a.requests + 1, dtype=torch.int32, device="cuda")
    x = z[(cu[1:] - 1).long()].contiguous()

    def step():
        z = layer(x, table, length, one, 1, adapter)
        if block is not None:
            z = z + block(z)
        z.mul_(z.float().pow(2).mean(-1, keepdim=True).rsqrt().to(z.dtype))
        length.add_(1)
        x.copy_(z)

    # once before the clock starts, since kernels are loaded at their first use (a token that is appended
    # again leaves the cache as it is)
    graph = None
    pages.grow([n + 1 for n in prompts])
    keep = [t.clone() for t in (x, length)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    if a.graph:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    x.copy_(keep[0])
    length.copy_(keep[1])
    torch.cuda.synchronize()
    t = time.perf_counter()
    for i in range(a.tokens):
        pages.grow([n + i + 1 for n in prompts])
        graph.replay() if graph is not None else step()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens of {a.requests} requests: {1e6 * (time.perf_counter() - t) / a.tokens:.1f} us a step"
          + (" (graph)" if graph is not None else ""))
    assert torch.isfinite(x).all()
    return x


if __name__ == "__main__":
    main()

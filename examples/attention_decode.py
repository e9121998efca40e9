"""One attention layer of the 9B-class stack, served from packed weights and a
4-bit key/value cache: hidden 4096, 32 query heads and 8 key/value heads of 128.

    python examples/attention_decode.py [--batch 8] [--prompt 1500] [--steps 32] [--window 0]

A prompt enters through the batched products (vbq_gemm), its keys and values go
into the cache (kv4_append), it attends to itself (kv4_attention, many rows) and
leaves through the output projection. Then tokens are decoded one at a time:
the q, k and v GEMVs in one launch (vbq_gemv_batched), the append, the attention
of one query a sequence, the output projection; the step is a HIP graph that is
replayed while the lengths grow on the device. The last step is checked against
attention in float32 over the values that kv4_read returns.

There is no model around the layer: weights are random, positions are not
encoded (a model with rotary positions turns q and k before the append), and a
step's input is the last output with noise.
"""
import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import packed_decode_gemv_amd as vbq  # noqa: E402


class AttentionLayer:
    def __init__(self, hidden=4096, heads=32, kv_heads=8, dim=128, seed=0):
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)

        def packed(n, k):
            widths = rng.choice(np.array([1, 2, 4, 8], np.uint8), size=(n, k // 64), p=[0.1, 0.2, 0.4, 0.3])
            return vbq.vbq_pack(torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5, widths)

        self.q, self.k, self.v = packed(heads * dim, hidden), packed(kv_heads * dim, hidden), packed(kv_heads * dim, hidden)
        self.o = packed(hidden, heads * dim)


class Session:
    """A batch of sequences decoded through one layer: the cache, its block table, and what a step keeps."""

    def __init__(self, layer, batch, max_tokens, page_tokens=64, window=0, sinks=0):
        self.layer, self.batch, self.window, self.sinks = layer, batch, window, sinks
        width = -(-max_tokens // page_tokens)
        self.max_tokens = width * page_tokens
        self.cache = vbq.Kv4Cache(batch * width, page_tokens, layer.kv_heads, layer.dim)
        # sequence b owns pages b, b + batch, ...: any table does
        self.table = (torch.arange(width, device="cuda")[None, :] * batch
                      + torch.arange(batch, device="cuda")[:, None]).int().contiguous()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.one_each = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
        self.workspace = vbq.kv4_attention_workspace(self.cache, batch, batch, layer.heads, 1, self.max_tokens, window,
                                                     sinks)
        self.x = torch.zeros(batch, layer.hidden, dtype=torch.float16, device="cuda")
        self.y = torch.zeros(batch, layer.hidden, device="cuda")
        self.attended = torch.zeros(batch, layer.heads, layer.dim, dtype=torch.float16, device="cuda")
        self.query = torch.zeros_like(self.attended)

    def prompt(self, x):
        """x [batch][n][hidden] bf16: all sequences take n tokens; returns the layer's output, float32."""
        ly, n = self.layer, x.shape[1]
        rows = x.reshape(-1, ly.hidden)
        q = vbq.vbq_gemm(ly.q, rows).view(-1, ly.heads, ly.dim).bfloat16()
        k = vbq.vbq_gemm(ly.k, rows).view(-1, ly.kv_heads, ly.dim)
        v = vbq.vbq_gemm(ly.v, rows).view(-1, ly.kv_heads, ly.dim)
        cu = torch.arange(0, self.batch * n + 1, n, dtype=torch.int32, device="cuda")
        vbq.kv4_append(self.cache, k, v, self.table, self.lens, cu, max_tokens=n)
        self.lens += n
        out = vbq.kv4_attention(self.cache, q, self.table, self.lens, cu, n, self.max_tokens, window=self.window,
                                sinks=self.sinks)
        return vbq.vbq_gemm(ly.o, out.view(-1, ly.heads * ly.dim)).view(self.batch, n, ly.hidden)

    def step(self):
        """One token a sequence: reads self.x, writes self.y, moves the lengths on. Fit for capture."""
        ly = self.layer
        q, k, v = vbq.vbq_gemv_batched([ly.q, ly.k, ly.v], [self.x, self.x, self.x])
        vbq.kv4_append(self.cache, k.view(-1, ly.kv_heads, ly.dim), v.view(-1, ly.kv_heads, ly.dim), self.table,
                       self.lens, self.one_each, max_tokens=1)
        self.lens += 1
        self.query.copy_(q.view(-1, ly.heads, ly.dim))
        vbq.kv4_attention(self.cache, self.query, self.table, self.lens, self.one_each, 1, self.max_tokens,
                          window=self.window, sinks=self.sinks, out=self.attended, workspace=self.workspace)
        vbq.vbq_gemv(ly.o, self.attended.view(self.batch, -1), out=self.y)

    def reference(self):
        """The last step's attention in float32 over the values read back."""
        ly, n = self.layer, int(self.lens[0])
        cu = torch.arange(0, self.batch * n + 1, n, dtype=torch.int32, device="cuda")
        k, v = vbq.kv4_read(self.cache, self.table, torch.zeros_like(self.lens), cu, self.batch * n, torch.float32,
                            max_tokens=n)
        shape = (self.batch, n, ly.kv_heads, ly.dim)
        k, v = k.view(shape).transpose(1, 2).contiguous(), v.view(shape).transpose(1, 2).contiguous()
        q = self.query.float().view(self.batch, ly.kv_heads, -1, ly.dim)
        s = torch.matmul(q, k.transpose(2, 3).contiguous()) * ly.dim ** -0.5
        if self.window:
            j = torch.arange(n, device="cuda")
            s = s.masked_fill(~((j > n - 1 - self.window) | (j < self.sinks)), float("-inf"))
        return torch.matmul(torch.softmax(s, -1), v).view(self.batch, ly.heads, ly.dim)


def run(batch=8, prompt=1500, steps=32, window=0, sinks=4, layer=None):
    if not 1 <= batch <= vbq.MAX_BATCH:
        raise ValueError(f"batch {batch} outside 1..{vbq.MAX_BATCH}")
    layer = layer or AttentionLayer()
    gen = torch.Generator(device="cuda").manual_seed(1)
    s = Session(layer, batch, prompt + steps + 1, window=window, sinks=sinks if window else 0)
    x = torch.randn(batch, prompt, layer.hidden, generator=gen, device="cuda").bfloat16()
    y = s.prompt(x)
    s.x.copy_(y[:, -1])
    s.step()                      # eagerly once, before the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(steps):
        s.x.copy_(s.y + torch.randn(s.y.shape, generator=gen, device="cuda"))
        graph.replay()
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t) / steps * 1e3
    s.cache.check()
    ref = s.reference()
    err = float((s.attended.float() - ref).norm() / ref.norm())
    return dict(tokens=int(s.lens[0]), step_ms=ms, rel_l2=err, cache_bytes=s.cache.nbytes,
                bf16_bytes=s.cache.n_pages * s.cache.page_tokens * layer.kv_heads * layer.dim * 4)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1500)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--window", type=int, default=0)
    a = ap.parse_args()
    r = run(a.batch, a.prompt, a.steps, a.window)
    print(f"{a.batch} sequences, {r['tokens']} tokens each: {r['step_ms']:.3f} ms per step, attention rel-L2 "
          f"{r['rel_l2']:.1e} against float32, cache {r['cache_bytes'] / 2 ** 20:.1f} MiB "
          f"({r['bf16_bytes'] / 2 ** 20:.1f} MiB in bf16)")

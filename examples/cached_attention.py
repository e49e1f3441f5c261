"""One decoder layer's self-attention with 4-bit weights and a 4-bit KV cache, as a serving program runs it.

The Q, K and V projections of the new tokens are one grouped launch into one [rows, 3 d] buffer; their K and
V columns are quantised into a paged cache, their Q columns attend over it, and the output projection follows.
A prompt goes through in one call, then tokens one by one from a CUDA graph whose lengths live on the device.

    python examples/cached_attention.py --fmt q4_0 --batch 4 --prompt 300 --steps 32
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_weight_quantized_matmul_gb300 import wq  # noqa: E402


class CachedAttention:
    """Self-attention of `heads` heads of `dim` elements: weights packed in weight_fmt ('q4_0', 'nvfp4', 'nf4' ...),
    keys and values in cache_fmt ('q4_0' or 'nvfp4')."""

    def __init__(self, wqkv, wo, heads, dim, batch, capacity, weight_fmt="q4_0", cache_fmt="q4_0", page=64, g=None):
        self.heads, self.dim, self.batch, self.weight_fmt = heads, dim, batch, weight_fmt
        self.d = heads * dim
        self.qkv, self.out = wq.pack(weight_fmt, wqkv), wq.pack(weight_fmt, wo)
        per = -(-capacity // page)
        table = torch.randperm(batch * per, device="cuda").to(torch.int32).view(batch, per).contiguous()   # any pages will do
        self.cache = wq.kv_alloc(cache_fmt, batch * per, page, heads, dim, table, *(g or (None, None)))
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")      # tokens held by each sequence

    def __call__(self, x, counts=None):
        """x bf16 [batch, tokens, d]: the next tokens of every sequence (the first counts[b] of them, if given)."""
        batch, tokens, d = x.shape
        rows = torch.empty((batch * tokens, 3 * d), dtype=torch.bfloat16, device=x.device)
        # one launch; the three projections are one stacked weight, their columns land side by side
        wq.linear_grouped_ex([(x.view(-1, d), *self.qkv, 3 * d, d, None, [(rows, 3 * d)])], self.weight_fmt)
        q, k, v = (rows.view(batch, tokens, 3, self.heads, self.dim)[:, :, i] for i in range(3))
        wq.kv_append(self.cache, k, v, start=self.lens, counts=counts)
        self.lens += tokens if counts is None else counts
        att = wq.attend(self.cache, q, self.lens, counts=counts)
        return wq.linear(att.view(-1, d), *self.out, self.weight_fmt, d, d).view(batch, tokens, d)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--fmt", default="q4_0", choices=["q4_0", "nvfp4"])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--heads", type=int, default=20)
    ap.add_argument("--dim", type=int, default=64)
    a = ap.parse_args()
    torch.manual_seed(0)
    d = a.heads * a.dim
    layer = CachedAttention(torch.randn(3 * d, d, device="cuda") * 0.02, torch.randn(d, d, device="cuda") * 0.02, a.heads,
                            a.dim, a.batch, a.prompt + a.steps + 4, a.fmt, a.fmt)
    y = layer(torch.randn(a.batch, a.prompt, d, device="cuda").bfloat16())
    x = y[:, -1:].contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):              # warm up off the capture: three tokens that count as any other
        for _ in range(3):
            layer(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps):
        graph.replay()
        x.copy_(out)
    end.record()
    torch.cuda.synchronize()
    assert wq.last_device_status() == 0
    print(f"{a.fmt}: {a.batch} sequences, {a.prompt} prompt tokens, {a.steps} steps: {begin.elapsed_time(end) / a.steps * 1e3:.1f} us a step; "
          f"every sequence holds {int(layer.lens[0])} tokens, |y| {out.float().abs().mean():.4f}")


if __name__ == "__main__":
    main()

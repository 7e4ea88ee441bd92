"""One attention layer served from 4-bit weights and an 8-bit cache.

A batch of prompts of different lengths goes through the layer, then a number
of single tokens of every sequence, as a serving loop runs them:

  projections   bf16_w4_gemm_nt for few tokens; for a prompt the weights are
                widened once (dequantize_b_w4) and multiplied by bf16_gemm_nt
  cache         kv8_append
  attention     kv8_attention

The single-token step is captured into a graph once and replayed: all lengths
live on the device, and the captured work follows them as the sequences grow.
Weights and activations are random; `python examples/serve_layer.py` prints
the time of a step, and how far the layer is from the same layer in fp32.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_nt_amd as dg  # noqa: E402


class Layer:
    """Weights of one attention layer, [rows, hidden] in 4 bits."""

    def __init__(self, hidden, h_q, h_kv, d, fmt="u4", group=64, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.h_q, self.h_kv, self.d = hidden, h_q, h_kv, d
        qkv = torch.randn((h_q + 2 * h_kv) * d, hidden, generator=gen, device="cuda") * hidden ** -0.5
        out = torch.randn(hidden, h_q * d, generator=gen, device="cuda") * (h_q * d) ** -0.5
        self.qkv, self.out = (dg.quantize_b_w4(w.bfloat16(), fmt, group) for w in (qkv, out))

    def project(self, x, w):
        y = torch.empty((x.shape[0], w[0].shape[0]), dtype=torch.bfloat16, device=x.device)
        if x.shape[0] <= 64:
            return dg.bf16_w4_gemm_nt(x, w, y)
        return dg.bf16_gemm_nt(x, dg.dequantize_b_w4(w), y)


class Cache:
    """The layer's cache and where each sequence stands in it."""

    def __init__(self, layer, batch, most, block=64):
        per = -(-most // block)
        self.codes = dg.empty_kv8_cache(batch * per, layer.h_kv, layer.d, block)
        self.table = torch.randperm(batch * per, device="cuda").int().view(batch, per).contiguous()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")


def forward(layer, cache, x, cu, most):
    """x bf16 [tokens, hidden], the new tokens of every sequence one after the
    other with running sums cu; returns the layer's output and moves the cache on."""
    qkv = layer.project(x, layer.qkv).view(x.shape[0], -1, layer.d)
    q, k, v = qkv.split((layer.h_q, layer.h_kv, layer.h_kv), 1)
    dg.kv8_append(k, v, cache.codes, cache.table, cache.lens, cu, most)
    cache.lens += cu[1:] - cu[:-1]
    y = torch.empty((x.shape[0], layer.h_q, layer.d), dtype=torch.bfloat16, device=x.device)
    dg.kv8_attention(q, cache.codes, cache.table, cache.lens, cu, most, y)
    return layer.project(y.view(x.shape[0], -1), layer.out)


def reference(layer, tokens):
    """The same layer in fp32 on one sequence's tokens [n, hidden]: 4-bit weights as they stand, keys and values unrounded."""
    n, h_q, h_kv, d = tokens.shape[0], layer.h_q, layer.h_kv, layer.d
    qkv = tokens.float() @ dg.dequantize_b_w4(layer.qkv).float().t()
    q, k, v = qkv.view(n, -1, d).split((h_q, h_kv, h_kv), 1)
    k, v = (t.repeat_interleave(h_q // h_kv, 1).transpose(0, 1).contiguous() for t in (k, v))
    s = torch.matmul(q.transpose(0, 1).contiguous(), k.transpose(1, 2).contiguous()) * d ** -0.5
    s = s.masked_fill(torch.ones(n, n, device=s.device).triu(1).bool(), float("-inf"))
    y = torch.matmul(torch.softmax(s, -1), v).transpose(0, 1).reshape(n, -1)
    return y @ dg.dequantize_b_w4(layer.out).float().t()


def serve(hidden=2048, h_q=16, h_kv=4, d=128, prompts=(300, 77, 512, 1), steps=16, seed=0):
    """Runs the loop; returns (relative error against fp32, seconds a step)."""
    layer = Layer(hidden, h_q, h_kv, d, seed=seed)
    batch = len(prompts)
    cache = Cache(layer, batch, max(prompts) + steps)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = [torch.randn(n + steps, hidden, generator=gen, device="cuda").bfloat16() for n in prompts]

    cu = torch.tensor([0] + list(prompts), device="cuda").cumsum(0).int()
    got = [[y] for y in forward(layer, cache, torch.cat([t[:n] for t, n in zip(x, prompts)]), cu, max(prompts)).split(list(prompts))]

    one = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    token = torch.empty((batch, hidden), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    dg.reserve_workspace(max(dg.kv8_attention_workspace_size(d),
                             *(dg.bf16_w4_workspace_size(batch, w[0].shape[0], 2 * w[0].shape[1], 64, "u4")
                               for w in (layer.qkv, layer.out))), side)
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = forward(layer, cache, token, one, 1)
    spent = 0.0
    for i in range(steps):
        token.copy_(torch.stack([t[n + i] for t, n in zip(x, prompts)]))
        torch.cuda.synchronize()
        start = time.perf_counter()
        graph.replay()
        torch.cuda.synchronize()
        spent += time.perf_counter() - start
        for s in range(batch):
            got[s].append(y[s:s + 1].clone())
    off = size = 0.0
    for s in range(batch):
        want = reference(layer, x[s])
        off += (torch.cat(got[s]).float() - want).square().sum().item()
        size += want.square().sum().item()
    return (off / size) ** 0.5, spent / steps


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    prompts = tuple(max(1, a.prompt - 97 * i) for i in range(a.batch))
    error, step = serve(a.hidden, a.heads, a.kv_heads, 128, prompts, a.steps)
    print(f"{a.batch} sequences of {min(prompts)}..{max(prompts)} tokens: {step * 1e6:.1f} us a step, "
          f"relative error against fp32 keys and values {error:.4f}")


if __name__ == "__main__":
    main()

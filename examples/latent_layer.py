"""One layer of latent attention, served from a paged cache of latents.

A batch of prompts of different lengths goes through the layer in chunks, then
a number of single tokens of every sequence, as a serving loop runs them:

  projections   bf16_gemm_nt: the joint down-projection (latent and rope part)
                and the queries' projection
  cache         latent_append: norm and rotation on the way, the queries'
                rope parts rotated by the same call
  prompts       latent_gather, the up-projection by bf16_gemm_nt, and
                latent_expanded_attention
  single tokens latent_attention on queries that have taken in the
                up-projection's key weights; its value weights follow

The single-token step is captured into a graph once and replayed: all lengths
live on the device.  Weights and activations are random; `python
examples/latent_layer.py` prints the time of a step, and how far the layer is
from the same layer in fp32.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_nt_amd as dg  # noqa: E402

EPS = 1e-6


class Layer:
    """bf16 weights; heads of D + D values and rope parts of D / 2 for latents of 4 D."""

    def __init__(self, hidden, heads, latent, positions, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda rows, k: (torch.randn(rows, k, generator=gen, device="cuda") * k ** -0.5).bfloat16()  # noqa: E731
        self.hidden, self.heads, self.L, self.D, self.P = hidden, heads, latent, latent // 4, latent // 8
        self.joint = new(latent + self.P, hidden)
        self.query = new(heads * (self.D + self.P), hidden)
        self.up = new(heads * 2 * self.D, latent)
        self.out = new(hidden, heads * self.D)
        self.norm = (1 + 0.1 * torch.randn(latent, generator=gen, device="cuda")).bfloat16()
        # the up-projection's two halves by head, as batched products take them
        by_head = self.up.view(heads, 2, self.D, latent)
        self.up_k, self.up_v = by_head[:, 0].contiguous(), by_head[:, 1].transpose(1, 2).contiguous()
        f = 10000.0 ** (-torch.arange(self.P // 2, dtype=torch.float64, device="cuda") * 2 / self.P)
        a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
        self.angles = torch.cat((a.cos(), a.sin()), 1).float()

    def project(self, x, w):
        return dg.bf16_gemm_nt(x, w, torch.empty((x.shape[0], w.shape[0]), dtype=torch.bfloat16, device=x.device))


class Cache:
    """The layer's cache and where each sequence stands in it."""

    def __init__(self, layer, batch, most, block, fmt):
        per = -(-most // block)
        self.pool = dg.empty_latent_cache(batch * per, layer.L, block, fmt)
        self.table = torch.randperm(batch * per, device="cuda").int().view(batch, per).contiguous()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")


def project_and_append(layer, cache, x, cu, most):
    """The queries [tokens, heads, D + P] of x, rotated; its latents go into the cache."""
    joint = layer.project(x, layer.joint)
    q = layer.project(x, layer.query).view(x.shape[0], layer.heads, -1)
    dg.latent_append(joint[:, :layer.L], joint[:, layer.L:], cache.pool, cache.table, cache.lens, cu, most, layer.angles,
                     norm=layer.norm, eps=EPS, q_rope=q[..., layer.D:])
    cache.lens += cu[1:] - cu[:-1]
    return q


def prompts(layer, cache, x, cu, most, cu_kv, keys):
    """New tokens of every sequence behind what it has cached; cu_kv, keys: running
    sums and number of all cached tokens with the new ones."""
    q = project_and_append(layer, cache, x, cu, most)
    rows = torch.empty((keys, layer.L), dtype=torch.bfloat16, device=x.device)
    rope = torch.empty((keys, layer.P), dtype=torch.bfloat16, device=x.device)
    dg.latent_gather(cache.pool, cache.table, cu_kv, rows, rope)
    kv = layer.project(rows, layer.up).view(keys, layer.heads, 2 * layer.D)
    y = torch.empty((x.shape[0], layer.heads, layer.D), dtype=torch.bfloat16, device=x.device)
    dg.latent_expanded_attention(q, kv, rope, cu, cu_kv, most, y)
    return layer.project(y.view(x.shape[0], -1), layer.out)


def tokens(layer, cache, x, cu):
    """One new token of every sequence."""
    q = project_and_append(layer, cache, x, cu, 1)
    latent_q = torch.bmm(q[..., :layer.D].transpose(0, 1).contiguous(), layer.up_k)          # [heads, tokens, L]
    seen = torch.empty_like(latent_q)
    dg.latent_attention(latent_q.transpose(0, 1), q[..., layer.D:], cache.pool, cache.table, cache.lens, cu, 1,
                        seen.transpose(0, 1))
    y = torch.bmm(seen, layer.up_v).transpose(0, 1).contiguous()
    return layer.project(y.view(x.shape[0], -1), layer.out)


def reference(layer, x):
    """The same layer in fp32 on one sequence's tokens [n, hidden]: latents unrounded."""
    n, h, D, L = x.shape[0], layer.heads, layer.D, layer.L
    joint = x.float() @ layer.joint.float().t()
    c = joint[:, :L]
    c = c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS) * layer.norm.float()
    cos, sin = (t[:, None] for t in layer.angles[:n].chunk(2, 1))

    def turn(t):
        a, b = t[..., 0::2], t[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)

    q = (x.float() @ layer.query.float().t()).view(n, h, -1)
    q = torch.cat((q[..., :D], turn(q[..., D:])), 2).transpose(0, 1).contiguous()
    kv = (c @ layer.up.float().t()).view(n, h, 2 * D)
    k = torch.cat((kv[..., :D], turn(joint[:, None, L:]).expand(n, h, -1)), 2).permute(1, 2, 0).contiguous()
    s = torch.matmul(q, k) * (D + layer.P) ** -0.5
    s = s.masked_fill(torch.ones(n, n, device=x.device).triu(1).bool(), float("-inf"))
    y = torch.matmul(torch.softmax(s, -1), kv[..., D:].transpose(0, 1).contiguous()).transpose(0, 1).reshape(n, -1)
    return y @ layer.out.float().t()


def running(lens):
    return torch.tensor([0] + list(lens), device="cuda").cumsum(0).int()


def serve(hidden=2048, heads=8, latent=512, lens=(300, 77, 512, 1), steps=16, fmt="e4m3", chunk=256, seed=0):
    """Runs the loop; returns (relative error against fp32, seconds a step)."""
    layer = Layer(hidden, heads, latent, max(lens) + steps, seed)
    batch = len(lens)
    cache = Cache(layer, batch, max(lens) + steps, 64, fmt)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = [torch.randn(n + steps, hidden, generator=gen, device="cuda").bfloat16() for n in lens]

    got = [[] for _ in lens]
    for at in range(0, max(lens), chunk):
        now = [min(max(n - at, 0), chunk) for n in lens]
        cached = [min(n, at + chunk) for n in lens]
        y = prompts(layer, cache, torch.cat([t[at:at + n] for t, n in zip(x, now)]), running(now), max(now), running(cached),
                    sum(cached))
        for s, part in enumerate(y.split(now)):
            got[s].append(part)

    one = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    token = torch.empty((batch, hidden), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    need = [dg.latent_attention_workspace_size(latent, 1, heads)]
    for w in (layer.joint, layer.query, layer.out):
        need.append(dg.dense_workspace_size(batch, *w.shape, "bf16"))
    dg.reserve_workspace(max(need), side)
    before = cache.lens.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                       # libraries set themselves up outside the capture
        token.zero_()
        tokens(layer, cache, token, one)
        cache.lens.copy_(before)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = tokens(layer, cache, token, one)
    spent = 0.0
    for i in range(steps):
        token.copy_(torch.stack([t[n + i] for t, n in zip(x, lens)]))
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
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--heads", type=int, default=128)
    ap.add_argument("--latent", type=int, default=512, choices=(256, 512))
    ap.add_argument("--cache", default="e4m3", choices=("bf16", "e4m3"))
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    lens = tuple(max(1, a.prompt - 97 * i) for i in range(a.batch))
    error, step = serve(a.hidden, a.heads, a.latent, lens, a.steps, a.cache)
    print(f"{a.batch} sequences of {min(lens)}..{max(lens)} tokens: {step * 1e6:.1f} us a step, "
          f"relative error against fp32 latents {error:.4f}")


if __name__ == "__main__":
    main()

"""The attention half of a decoder layer, decoded token by token within a budget.

    python examples/decode_attention.py [--rows 8] [--steps 200] [--budget 128] [--r 4] [--cache bf16|fp8]

The layer's qkv and o products run on the r-bit child of nested 8-bit parents; between them
the new keys and values go into a paged cache (normalised as Qwen3-8B does, rotated), the new
token attends to it, and when a sequence grows past its budget the tokens that attention
has cared least about make room.  Weights and inputs are random, with the shapes of the
Llama-3.1-8B and Qwen3-8B attention (32 query heads, 8 key-value heads of 128).
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nested_bit_weight_amd as nbw  # noqa: E402


def random_parent(n: int, k: int, seed: int):
    """Planes and scales of a random 8-bit parent [n][k], values of about 1/sqrt(k)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(n, k // 128, generator=g, device="cuda") + 0.5) / (74.0 * k ** 0.5)
    return nbw.pack_bitplanes(codes), scales.to(torch.bfloat16)


class AttentionHalf:
    """Weights of one layer's attention and one batch's cache, `rows` sequences of at most
    `budget` tokens (and the one that arrives)."""

    def __init__(self, rows, budget, *, r=4, heads=32, kv=8, dim=128, page=16, sink=4, recent=32, positions=4096,
                 cache="bf16", seed=0):
        self.rows, self.budget, self.r, self.heads, self.kv, self.dim = rows, budget, r, heads, kv, dim
        self.sink, self.recent = sink, recent
        hidden = heads * dim
        self.qkv, self.qkv_scales = random_parent((heads + 2 * kv) * dim, hidden, seed)
        self.o, self.o_scales = random_parent(hidden, hidden, seed + 1)
        self.q_norm = self.k_norm = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
        angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * \
            500000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
        self.rope = torch.cat([angle.cos(), angle.sin()], dim=1).float()

        width = -(-(budget + 1) // page)  # pages of a sequence
        kind = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
        pools = [torch.zeros((rows * width, kv, page, dim), dtype=kind, device="cuda") for _ in "kv"]
        # a normalised key's elements are within sqrt(dim), the values here within a few units
        factors = (None, None) if cache == "bf16" else [torch.full((kv,), f, device="cuda") for f in (dim ** 0.5 / 448, 0.02)]
        table = torch.randperm(rows * width, device="cuda", dtype=torch.int32).view(rows, width)
        self.cache = nbw.KVCache(*pools, table, *factors)
        # totals, positions and lengths before and after an eviction take turns
        track = (rows, kv, self.cache.capacity)
        self.acc = [torch.zeros(track, device="cuda") for _ in range(2)]
        self.pos = [torch.zeros(track, dtype=torch.int32, device="cuda") for _ in range(2)]
        self.lens = [torch.zeros(rows, dtype=torch.int32, device="cuda") for _ in range(2)]
        self.seen = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.tokens = 0

    def decode(self, x: torch.Tensor) -> torch.Tensor:
        """One new token for each sequence: x bf16 [rows][hidden] -> fp32 [rows][hidden]."""
        d, now, then = self.dim, 0, 1
        y = nbw.qgemm(x, self.qkv.slice_view(self.r), self.qkv_scales, self.r, out_dtype=torch.bfloat16)
        q, k, v = (t.unflatten(1, (-1, d)) for t in y.split([self.heads * d, self.kv * d, self.kv * d], dim=1))
        q, lens = nbw.kv_append(self.cache, k, v, self.lens[now], self.seen, q=q, rope=self.rope, q_norm=self.q_norm,
                                k_norm=self.k_norm, pos=self.pos[now], acc=self.acc[now], lens_out=self.lens[then])
        self.seen += 1
        self.tokens += 1
        most = min(self.tokens, self.budget + 1)
        out = nbw.kv_attend(self.cache, q, lens, acc=self.acc[now], max_len=most)
        if self.tokens > self.budget:
            nbw.kv_evict(self.cache, self.acc[now], self.pos[now], lens, self.budget, sink=self.sink, recent=self.recent,
                         acc_out=self.acc[then], pos_out=self.pos[then], lens_out=self.lens[now], max_len=most)
            self.acc.reverse()
            self.pos.reverse()
        else:
            self.lens.reverse()
        return nbw.qgemm(out.view(self.rows, -1), self.o.slice_view(self.r), self.o_scales, self.r)


def main(argv=None) -> int:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--rows", type=int, default=8)
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--budget", type=int, default=128)
    p.add_argument("--r", type=int, default=4)
    p.add_argument("--cache", choices=("bf16", "fp8"), default="bf16")
    a = p.parse_args(argv)
    layer = AttentionHalf(a.rows, a.budget, r=a.r, cache=a.cache, positions=a.steps, sink=min(4, a.budget // 4),
                          recent=a.budget // 4)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.rows, layer.heads * layer.dim, generator=g, device="cuda")
    began = time.perf_counter()
    for _ in range(a.steps):
        # the next input follows from the last output, as the next token would
        x = torch.nn.functional.normalize(x, dim=1) * x.shape[1] ** 0.5
        x = 0.5 * x + layer.decode(x.to(torch.bfloat16))
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    kept = layer.pos[0][0, 0, :int(layer.lens[0][0])].sort().values.tolist()
    print(f"{a.steps} tokens for each of {a.rows} sequences in {took:.3f} s, {len(kept)} kept for each head")
    print(f"positions that the first head kept: {kept[:8]} .. {kept[-8:]}")
    return 0


if __name__ == "__main__":
    sys.exit(main())

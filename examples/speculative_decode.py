"""A decoder layer whose narrow child drafts tokens and whose wide child checks them.

    python examples/speculative_decode.py [--rows 8] [--steps 40] [--drafts 4] [--r-draft 3] [--r 8] [--prompt 256]

All sequences answer the same prompt: its keys and values are in the cache once, on pages that every
row's table names, and are attended to once for all of them.  In a step the r-draft-bit child of the
nested parents drafts a few tokens for each sequence, the r-bit child of the same planes takes
them all at once, and what it does not accept is taken back: the lengths say so, and the next step's
reservation gives the pages back.  Nothing is copied to the host between steps.  Weights are random,
with the head shapes of the Llama-3.1-8B and Qwen3-8B attention unless told otherwise.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nested_bit_weight_amd as nbw  # noqa: E402

I32 = torch.int32


def random_parent(n: int, k: int, seed: int):
    """Planes and scales of a random 8-bit parent [n][k], values of about 1/sqrt(k)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(n, k // 128, generator=g, device="cuda") + 0.5) / (74.0 * k ** 0.5)
    return nbw.pack_bitplanes(codes), scales.to(torch.bfloat16)


class Speculation:
    """One layer and a vocabulary, `rows` sequences behind one prompt, `drafts` tokens drafted a step."""

    def __init__(self, rows, drafts, *, r_draft=3, r=8, heads=32, kv=8, dim=128, vocab=4096, page=16, room=512, prompt=256,
                 sharpness=3.0, seed=0):
        if prompt % page:
            raise ValueError("the prompt ends with a page, so that no sequence writes to what it shares")
        self.rows, self.drafts, self.heads, self.kv, self.dim, self.vocab = rows, drafts, heads, kv, dim, vocab
        self.r_draft, self.r, self.prompt, self.page, self.sharpness = r_draft, r, prompt, page, sharpness
        hidden = heads * dim
        self.qkv, self.qkv_scales = random_parent((heads + 2 * kv) * dim, hidden, seed)
        self.o, self.o_scales = random_parent(hidden, hidden, seed + 1)
        self.head, self.head_scales = random_parent(vocab, hidden, seed + 2)
        self.gen = torch.Generator(device="cuda").manual_seed(seed + 3)
        self.embedding = torch.randn(vocab, hidden, generator=self.gen, device="cuda")
        width = -(-(prompt + room) // page)
        angle = torch.arange(width * page, device="cuda", dtype=torch.float64)[:, None] * \
            500000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
        self.rope = torch.cat([angle.cos(), angle.sin()], dim=1).float()

        pages = prompt // page + rows * (width - prompt // page)
        pools = [torch.zeros((pages, kv, page, dim), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        self.table = torch.full((rows, width), -1, dtype=I32, device="cuda")
        self.table[:, :prompt // page] = torch.arange(prompt // page, dtype=I32, device="cuda")
        self.cache = nbw.KVCache(*pools, self.table)
        # the free pages, the first one on top
        self.free = torch.arange(pages - 1, prompt // page - 1, -1, dtype=I32, device="cuda")
        self.free = torch.cat([self.free, torch.full((prompt // page,), -1, dtype=I32, device="cuda")])
        self.count = torch.tensor([pages - prompt // page], dtype=I32, device="cuda")
        ints = lambda x: torch.full((rows,), x, dtype=I32, device="cuda")  # noqa: E731
        self.lens, self.held, self.shared, self.want = ints(prompt), ints(prompt // page), ints(prompt // page), ints(drafts + 1)
        self.last = torch.zeros(rows, dtype=I32, device="cuda")
        self.runs = torch.arange(rows, dtype=I32, device="cuda") * (drafts + 1)
        self.groups = torch.tensor([0, rows], dtype=I32, device="cuda")
        self.prefix = torch.tensor([prompt], dtype=I32, device="cuda")
        self.accepted = torch.zeros((), dtype=torch.int64, device="cuda")

    def layer(self, ids, r, lens, positions, cu, groups, prefix, cache=None):
        """Hidden states [tokens][hidden] after the layer's attention, by the r-bit child."""
        d, cache = self.dim, cache or self.cache
        x = self.embedding[ids.long()]
        y = nbw.qgemm(x.to(torch.bfloat16), self.qkv.slice_view(r), self.qkv_scales, r, out_dtype=torch.bfloat16)
        q, k, v = (t.unflatten(1, (-1, d)) for t in y.split([self.heads * d, self.kv * d, self.kv * d], dim=1))
        q, lens = nbw.kv_append(cache, k, v, lens, positions, q=q, cu=cu, rope=self.rope)
        a = nbw.kv_attend_shared(cache, q, lens, cu=cu, groups=groups, prefix=prefix)
        return x + nbw.qgemm(a.flatten(1), self.o.slice_view(r), self.o_scales, r)

    def probabilities(self, h, r):
        """The r-bit child's distribution of the token after each hidden state: fp32 [tokens][vocab]."""
        h = torch.nn.functional.normalize(h, dim=1) * (h.shape[1] ** 0.5 * self.sharpness)
        return torch.softmax(nbw.qgemm(h.to(torch.bfloat16), self.head.slice_view(r), self.head_scales, r), dim=1)

    def read_prompt(self, ids):
        """The prompt's keys and values, into the pages that all rows name; each row's first token is sampled."""
        one = nbw.KVCache(self.cache.k, self.cache.v, self.table[:1])
        n = ids.numel()
        cu = torch.tensor([0, n], dtype=I32, device="cuda")
        h = self.layer(ids, self.r, torch.zeros(1, dtype=I32, device="cuda"), torch.arange(n, dtype=I32, device="cuda"), cu, None,
                       None, one)
        p = self.probabilities(h[-1:], self.r).expand(self.rows, -1).contiguous()
        self.last = nbw.verify_drafts(p, None, torch.rand(self.rows, generator=self.gen, device="cuda"))[1]

    def step(self):
        """One step: drafts, their check, and what stands: (accepted, next), int32 [rows].

        A row that is granted no place, as the pages are used up or it has reached its capacity, stays as it is, with
        nothing accepted and the next token it had."""
        rows, n = self.rows, self.drafts + 1
        got = nbw.kv_reserve(self.cache, self.lens, self.want, self.held, self.free, self.count, rows * n, shared=self.shared)
        u = torch.rand(rows, 2 * n, generator=self.gen, device="cuda")
        ids = torch.empty(rows, n, dtype=I32, device="cuda")
        draft = torch.empty(rows, n, self.vocab, device="cuda")  # the last line of a row is not read
        # a row without places drafts past its capacity: nothing is stored, and what it drafts is not looked at
        served = got.granted > 0
        first = torch.where(served, self.lens, self.cache.capacity)
        ids[:, 0] = self.last
        for i in range(self.drafts):
            lens = first + i
            h = self.layer(ids[:, i], self.r_draft, lens, lens, None, self.groups, self.prefix)
            draft[:, i] = self.probabilities(h, self.r_draft)
            ids[:, i + 1] = nbw.verify_drafts(draft[:, i], None, u[:, n + i].contiguous())[1].clamp_(min=0)
        # Rows with places have n each, side by side in their order: the row of each run of places (any, behind the last).
        # The wide child's keys and values take the places of the drafts'.
        row = torch.searchsorted(got.cu[1:], self.runs, right=True).clamp_(max=rows - 1)
        ids, draft = ids[row].flatten(), draft[row].flatten(0, 1)
        h = self.layer(ids, self.r, self.lens, got.positions, got.cu, self.groups, self.prefix)
        accepted, after = nbw.verify_drafts(self.probabilities(h, self.r), ids, u[row, :n].flatten(), draft=draft, cu=got.cu)
        self.lens = torch.where(served, self.lens + accepted + 1, self.lens)
        self.last = torch.where(served, after, self.last)
        self.held, self.count = got.held, got.count
        self.accepted += accepted.sum()
        return accepted, self.last


def main(argv=None) -> int:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--rows", type=int, default=8)
    p.add_argument("--steps", type=int, default=40)
    p.add_argument("--drafts", type=int, default=4)
    p.add_argument("--r-draft", type=int, default=3)
    p.add_argument("--r", type=int, default=8)
    p.add_argument("--prompt", type=int, default=256)
    a = p.parse_args(argv)
    s = Speculation(a.rows, a.drafts, r_draft=a.r_draft, r=a.r, prompt=a.prompt, room=a.steps * (a.drafts + 1) + 16)
    s.read_prompt(torch.randint(0, s.vocab, (a.prompt,), generator=s.gen, device="cuda", dtype=I32))
    began = time.perf_counter()
    for _ in range(a.steps):
        s.step()
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    stood, drafted = int(s.accepted), a.rows * a.steps * a.drafts
    print(f"{a.steps} steps of {a.rows} sequences in {took:.3f} s: {stood} of {drafted} drafts stood, "
          f"{(stood + a.rows * a.steps) / (a.rows * a.steps):.2f} tokens a step")
    return 0


if __name__ == "__main__":
    sys.exit(main())

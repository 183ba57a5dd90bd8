"""Beam search over a paged 8-bit cache, with attention over the blocks that a cheap score selects.

    python examples/beam_step.py

One layer's calls, as a serving loop makes them for every new token:

  1. the beams that go on take over their parents' pages: full ones are shared, a partly
     filled one that several would write to is copied, beams that end free theirs
     (``cache_fork``, ``cache_copy``);
  2. the new token's keys and values go into the cache, and the bounds of the block that they
     lie in are brought up to date (``cache_write``, ``cache_bounds``);
  3. every block of the context gets a score, the best are selected, and each query attends
     to them, the first and the last block always among them (``block_scores``,
     ``topk_indices``, ``block_attention``);
  4. now and then the pages in use are moved together (``cache_compact``, ``cache_copy``).

Weights are not needed to show the calls: queries, keys, values and the beams' choices are random.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_attention_topk_gb300 as tks  # noqa: E402


class Beams:
    """A layer's cache with the bounds of its blocks, and the page tables of the beams of some prompts."""

    def __init__(self, prompts, beams, room, pages, kv_heads, head_dim, page_size, block, seed=0):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        self.beams, self.pages, self.page_size, self.block = beams, pages, page_size, block
        self.kv_heads, self.head_dim = kv_heads, head_dim
        shape = (pages, page_size, kv_heads, head_dim)
        self.k_cache = torch.zeros(shape, dtype=torch.int8, device="cuda")
        self.v_cache = torch.zeros(shape, dtype=torch.int8, device="cuda")
        self.scales = torch.zeros((pages, page_size, kv_heads, 2), device="cuda")
        self.bounds = torch.zeros((pages, page_size // block, kv_heads, 2, head_dim), dtype=torch.bfloat16, device="cuda")
        width = -(-(max(prompts) + room) // page_size)
        self.table = torch.empty((0, width), dtype=torch.int32, device="cuda")
        self.lens = torch.empty(0, dtype=torch.int32, device="cuda")
        # one sequence for each prompt, from nothing
        self.fork(torch.full((len(prompts),), -1, dtype=torch.int32, device="cuda"), torch.tensor(prompts, dtype=torch.int32, device="cuda"))
        seq = torch.repeat_interleave(torch.arange(len(prompts), device="cuda"), self.lens.long())
        pos = torch.cat([torch.arange(n, device="cuda") for n in prompts])
        self.write(seq, pos, torch.zeros_like(self.lens))
        # which become the beams of each prompt
        self.fork(torch.arange(len(prompts), dtype=torch.int32, device="cuda").repeat_interleave(beams), self.lens.repeat_interleave(beams))

    def random(self, *shape):
        return torch.randn(*shape, device="cuda", generator=self.gen).to(torch.bfloat16)

    def copy(self, src, dst, count=None):
        tks.cache_copy(src, dst, self.k_cache, self.v_cache, scales=self.scales, bounds=self.bounds, count=count)

    def fork(self, parents, lens):
        self.table, src, dst = tks.cache_fork(self.table, self.lens, parents, lens, self.pages, self.page_size)
        self.lens = lens
        self.copy(src, dst)

    def write(self, seq, pos, start):
        """Puts a token at position `pos` of each of the sequences `seq`; start: the sequences' lengths before."""
        kv = self.random(len(seq), 2, self.kv_heads, self.head_dim)
        slots = (self.table[seq, pos // self.page_size] * self.page_size + pos % self.page_size).to(torch.int32)
        tks.cache_write(kv[:, 0], kv[:, 1], self.k_cache, self.v_cache, slots, scales=self.scales)
        tks.cache_bounds(self.k_cache, self.table, self.lens, self.bounds, start=start, scales=self.scales)

    def step(self, parents, q, selected):
        """One new token of every beam; parents: the beam that each goes on from. Returns (blocks, outputs)."""
        self.fork(parents, self.lens[parents.long()] + 1)
        self.write(torch.arange(len(parents), device="cuda"), (self.lens - 1).long(), self.lens - 1)
        kv_len = self.lens.unsqueeze(1)
        scores, seen = tks.block_scores(q, self.bounds, self.table, kv_len, self.block, first=1, last=1)
        blocks = tks.topk_indices(scores.flatten(0, 2), selected, row_len=seen.flatten()).view(*seen.shape, selected)
        return blocks, tks.block_attention(q, self.k_cache, self.v_cache, self.table, blocks, self.block, kv_len=kv_len, scales=self.scales)

    def compact(self):
        """Moves the pages in use to the lowest ones; returns how many are."""
        self.table, src, dst, count = tks.cache_compact(self.table, self.lens, self.pages, self.page_size, out=self.table)
        self.copy(src, dst, count)
        return int(count[1])


def main():
    prompts, beams, q_heads = [65536, 30000, 4096], 4, 32
    layer = Beams(prompts, beams, 64, 3000, kv_heads=8, head_dim=128, page_size=64, block=64)
    group = beams * torch.arange(len(prompts), device="cuda").repeat_interleave(beams)
    for step in range(5):
        parents = (group + torch.randint(beams, group.shape, device="cuda", generator=layer.gen)).to(torch.int32)
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        ev[0].record()
        blocks, out = layer.step(parents, layer.random(len(group), 1, q_heads, 128), 32)
        ev[1].record()
        status = tks.device_status()
        if status != tks.TKS_OK:
            raise tks.TksError(status, "beam step")
        print(f"step {step}: {ev[0].elapsed_time(ev[1]) * 1e3:.0f} us for {len(group)} beams over up to {int(layer.lens.max())} positions, "
              f"of which each head attends to {blocks.shape[-1] * layer.block}; {layer.compact()} of {layer.pages} pages in use")


if __name__ == "__main__":
    main()

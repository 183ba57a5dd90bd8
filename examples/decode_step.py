"""One layer's speculative decode step over a paged 8-bit cache, from prompt to accepted tokens.

    python examples/decode_step.py

The calls of the package as a serving loop makes them:

  1. the prompt's keys and values are written into the cache (``cache_write``);
  2. a tree of drafted tokens goes behind each sequence's context, and every draft
     attends to the whole context and to its ancestors (``tree_attention``);
  3. sparsely, as DeepSeek Sparse Attention does it: the indexer's logits select the
     positions that each draft attends to (``topk_indices``, ``selected_attention``);
  4. the accepted path's rows, which lie among the rest of the tree, are read back and
     written right behind the context, where the next step expects them (``cache_read``,
     ``cache_write``).

Weights are not needed to show the calls: queries, keys, values and logits are random.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_attention_topk_gb300 as tks  # noqa: E402


class Layer:
    """A layer's cache and the page tables of its sequences."""

    def __init__(self, context, room, kv_heads, head_dim, page_size, seed=0):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        self.page_size, self.kv_heads, self.head_dim = page_size, kv_heads, head_dim
        need = [-(-(n + room) // page_size) for n in context]
        pages = sum(need)
        shape = (pages, page_size, kv_heads, head_dim)
        self.k_cache = torch.zeros(shape, dtype=torch.int8, device="cuda")
        self.v_cache = torch.zeros(shape, dtype=torch.int8, device="cuda")
        self.scales = torch.zeros((pages, page_size, kv_heads, 2), device="cuda")
        # pages are handed out in no order; a table's unused entries are never looked at
        free = torch.randperm(pages, generator=self.gen, device="cuda").to(torch.int32)
        self.table = torch.full((len(context), max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = free[at:at + n]
            at += n
        self.ctx_len = torch.tensor(context, dtype=torch.int32, device="cuda")

    def slots(self, seq, pos):
        """The cache slots of positions `pos` of sequences `seq`."""
        return (self.table[seq, pos // self.page_size] * self.page_size + pos % self.page_size).to(torch.int32)

    def random(self, *shape):
        return torch.randn(*shape, device="cuda", generator=self.gen).to(torch.bfloat16)

    def write(self, k, v, slots):
        tks.cache_write(k, v, self.k_cache, self.v_cache, slots, scales=self.scales)

    def prompt(self):
        for b, n in enumerate(self.ctx_len.tolist()):
            # one fused projection's output: keys and values are views of it, read in place
            kv = self.random(n, 2, self.kv_heads, self.head_dim)
            self.write(kv[:, 0], kv[:, 1], self.slots(b, torch.arange(n, device="cuda")))

    def draft(self, tokens):
        """Puts `tokens` drafted tokens behind every context."""
        batch = self.ctx_len.numel()
        seq = torch.arange(batch, device="cuda").repeat_interleave(tokens)
        pos = (self.ctx_len[:, None] + torch.arange(tokens, device="cuda")).reshape(-1)
        kv = self.random(batch * tokens, 2, self.kv_heads, self.head_dim)
        self.write(kv[:, 0], kv[:, 1], self.slots(seq, pos))

    def dense(self, q, bits):
        return tks.tree_attention(q, self.k_cache, self.v_cache, self.table, self.ctx_len, tree=bits, scales=self.scales)

    def sparse(self, q, logits, k):
        """logits: [batch, tokens, at least the longest context], of which a sequence's first ctx_len count."""
        batch, tokens, n = logits.shape
        lens = self.ctx_len.repeat_interleave(tokens)
        idx = tks.topk_indices(logits.view(batch * tokens, n), k, row_len=lens).view(batch, tokens, k)
        out = tks.selected_attention(q, self.k_cache, self.v_cache, self.table, idx, kv_len=self.ctx_len, scales=self.scales)
        return idx, out

    def accept(self, paths):
        """paths: for every sequence, the accepted drafts from the root down. Moves their rows behind the context."""
        seq = torch.tensor([b for b, path in enumerate(paths) for _ in path], dtype=torch.int64, device="cuda")
        draft = torch.tensor([d for path in paths for d in path], dtype=torch.int32, device="cuda")
        place = torch.tensor([i for path in paths for i in range(len(path))], dtype=torch.int32, device="cuda")
        base = self.ctx_len[seq]
        # (in 32 bits: the codes of what is read are those that it was read from)
        k, v = tks.cache_read(self.k_cache, self.v_cache, self.slots(seq, base + draft), scales=self.scales, dtype=torch.float32)
        self.write(k, v, self.slots(seq, base + place))
        self.ctx_len += torch.tensor([len(path) for path in paths], dtype=torch.int32, device="cuda")


def path_to(parents, leaf):
    path = []
    while leaf >= 0:
        path.append(leaf)
        leaf = parents[leaf]
    return path[::-1]


def main():
    context = [65536, 40001, 8192, 777]
    tokens, q_heads, k = 8, 32, 2048
    layer = Layer(context, 64, kv_heads=8, head_dim=128, page_size=64)
    layer.prompt()
    parents = [[-1, 0, 0, 1, 1, 2, 3, 6]] * len(context)  # two branches, one of them five deep
    bits = tks.tree_mask(torch.tensor(parents, device="cuda"))
    logits = torch.randn(len(context), tokens, max(context) + 64, device="cuda", generator=layer.gen)  # (contexts grow)
    for step in range(3):
        layer.draft(tokens)
        q = layer.random(len(context), tokens, q_heads, 128)
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
        ev[0].record()
        dense = layer.dense(q, bits)
        ev[1].record()
        idx, sparse = layer.sparse(q, logits, k)
        ev[2].record()
        layer.accept([path_to(parents[b], 7 if b % 2 else 5) for b in range(len(context))])
        status = tks.device_status()
        if status != tks.TKS_OK:
            raise tks.TksError(status, "decode step")
        apart = (dense.float() - sparse.float()).abs().mean().item() / dense.float().abs().mean().item()
        print(f"step {step}: over everything {ev[0].elapsed_time(ev[1]) * 1e3:.0f} us, selection and attention over {k} positions "
              f"{ev[1].elapsed_time(ev[2]) * 1e3:.0f} us, mean difference {apart:.2f} of the mean output; contexts now {layer.ctx_len.tolist()}")


if __name__ == "__main__":
    main()

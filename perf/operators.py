"""The cases on which the cache and attention operators are measured.

The top-k selector is the second of three steps of sparse attention; these
operators are what stands around it in a decode step: the new tokens' keys and
values go into a paged cache (held as bfloat16, or as 8-bit integers with one
scale for each token and head) and are read back from it, a tree of drafted
tokens attends to its context in the cache, and queries attend to the positions
that the selector chose.

    listed(), draw(rng)     cases: dicts of plain values
    prepare(case, seed)     the tensors a program has in hand before the call
    run(state)              one pass through an operator, and its outputs
    exact(case, seed)       the same outputs from the definitions, in 64 bits
    work(case)              the bytes and operations a pass cannot do without

``own`` chooses what run() does: False computes the plain forms with elementary
torch operations in 32 bits, True calls the package.
"""

import math

import torch

own = False

#: An 8-bit row is code * scale with scale = amax * (1 / 127); amax is held to this range.
AMAX_LOW, AMAX_HIGH = 2.0 ** -40, 2.0 ** 80

_BYTES = {"int8": 1, "bf16": 2, "f32": 4}
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8}


def listed():
    def cache(name, tokens, heads, dim, src, held, page):
        return {"name": name, "op": "cache", "tokens": tokens, "heads": heads, "dim": dim, "src": src, "held": held, "page": page}

    def tree(name, batch, drafts, q_heads, kv_heads, dim, context, ragged, held, page):
        return {"name": name, "op": "tree", "batch": batch, "drafts": drafts, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
                "context": context, "ragged": ragged, "held": held, "page": page}

    def selected(name, batch, queries, q_heads, kv_heads, dim, context, ragged, k, held, page):
        return {"name": name, "op": "selected", "batch": batch, "queries": queries, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
                "context": context, "ragged": ragged, "k": k, "held": held, "page": page}

    return [
        # the one new token of a decode step: latency
        cache("cache_one_token", 1, 8, 128, "bf16", "int8", 64),
        # an odd chunk of a prompt, computed in 32 bits, small heads and small pages
        cache("cache_odd_chunk", 5003, 4, 64, "f32", "int8", 16),
        # a whole prompt of the length of the repository's prefill workload, written and read back for the layers that want bfloat16
        cache("cache_prompt_32k", 32768, 8, 128, "bf16", "int8", 64),
        # one token over a short context (the selector's smallest row): latency
        tree("tree_one_4k", 1, 1, 32, 8, 128, 4096, False, "int8", 64),
        # a few odd sequences with a small tree each, a group of 6 heads, small pages
        tree("tree_odd_small", 5, 13, 12, 2, 64, 777, True, "bf16", 16),
        # speculative decoding of a batch of ragged contexts (the lengths of the repository's ragged batch)
        tree("tree_batch_ragged", 8, 8, 32, 8, 128, 65536, True, "bf16", 64),
        # a wide tree: the matrix products outweigh the cache's bytes
        tree("tree_wide_32k", 2, 64, 64, 8, 128, 32768, False, "int8", 64),
        # one token over the longest context (the selector's longest row): the cache is read at the memory's rate
        tree("tree_one_1m", 1, 1, 32, 4, 128, 1048576, False, "int8", 64),
        # the selector's decode row of 128K: 2048 positions for one token
        selected("selected_one_128k", 1, 1, 32, 8, 128, 131072, False, 2048, "int8", 64),
        # a batch of decode rows, ragged as in the repository's ragged batch
        selected("selected_batch64", 64, 1, 16, 2, 128, 65536, True, 2048, "bf16", 64),
        # the 512 causal rows over 32K of the repository's prefill workload, all heads on one shared key and value head
        selected("selected_prefill", 1, 512, 64, 1, 128, 32768, False, 2048, "int8", 64),
        # four rows of 1M, every position far from the next
        selected("selected_4x1m", 4, 1, 64, 1, 128, 1048576, False, 2048, "bf16", 64),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("cache", "tree", "selected"))
    dim, held, page = rng.choice((64, 128, 128)), rng.choice(("int8", "bf16")), rng.choice((16, 32, 64, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    if op == "cache":
        return {"op": op, "tokens": _log(rng, 1, 32768), "heads": kv_heads, "dim": dim, "src": rng.choice(("bf16", "f32")) if held == "int8" else "bf16",
                "held": held, "page": page}
    if op == "tree":
        batch, drafts, group = _log(rng, 1, 16), _log(rng, 1, 64), rng.choice((1, 2, 4, 6, 8))
        keys = (1 << 30) // (batch * kv_heads * dim * 2 * _BYTES[held])  # at most 1 GB of cache,
        keys = min(keys, 34_000_000_000 // (batch * kv_heads * group * drafts * dim))  # and 4 * this many operations
        return {"op": op, "batch": batch, "drafts": drafts, "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
                "context": _log(rng, 1, max(1, min(1048576, keys))), "ragged": rng.random() < 0.5, "held": held, "page": page}
    batch, queries, group = _log(rng, 1, 16), _log(rng, 1, 64), rng.choice((1, 4, 8, 16, 64))
    context = _log(rng, 100, max(100, min(1048576, (1 << 30) // (batch * kv_heads * dim * 2 * _BYTES[held]))))
    k = _log(rng, 16, 4096)
    while queries > 1 and batch * queries * k * kv_heads * dim > 134_000_000:
        queries = (queries + 1) // 2
    return {"op": op, "batch": batch, "queries": queries, "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
            "context": context, "ragged": rng.random() < 0.5, "k": k, "held": held, "page": page}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _lengths(case):
    """Context lengths: the full one first, then, where ragged, others spread below it."""
    n, b = case["context"], case["batch"]
    return [n if i == 0 or not case["ragged"] else max(1, int(n * ((i * 0.6180339887) % 1.0))) for i in range(b)]


def _draft_counts(case):
    t, b = case["drafts"], case["batch"]
    return [t if i == 0 or not case["ragged"] else t - (5 * i) % (t // 2 + 1) for i in range(b)]


def _hold(x, held):
    """Rows of x as the cache holds them: (what is stored, its scales)."""
    if held == "bf16":
        return x.to(torch.bfloat16), None
    x = x.float()
    amax = x.abs().amax(-1).clamp(AMAX_LOW, AMAX_HIGH)
    scale = amax * (1.0 / 127.0)
    codes = (x * scale.reciprocal().unsqueeze(-1)).round().clamp(-127, 127)
    return codes.to(torch.int8), scale


def _empty_cache(pages, page, heads, dim, held, g):
    """A cache that nothing was written to: what it holds is not to be used."""
    shape = (pages, page, heads, dim)
    if held == "bf16":
        return torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda"), torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda"), None
    k, v = (torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g) for _ in range(2))
    return k, v, torch.full(shape[:3] + (2,), math.nan, dtype=torch.float32, device="cuda")


def _tensors(case, lengths, g):
    """A cache whose sequence b holds lengths[b] tokens in pages of random order, and its page table."""
    page, heads, dim, held = case["page"], case["kv_heads"], case["dim"], case["held"]
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + 3
    kc, vc, sc = _empty_cache(pages, page, heads, dim, held, g)
    order = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    table = torch.full((len(lengths), max(need)), -1, dtype=torch.int32, device="cuda")
    # keys with channels of different sizes, as projections give them; values of different sizes from token to token
    channel = torch.exp(0.4 * torch.randn(heads, dim, device="cuda", generator=g))
    at = 0
    for b, n in enumerate(lengths):
        table[b, : need[b]] = order[at : at + need[b]]
        at += need[b]
        pos = torch.arange(n, device="cuda")
        slots = table[b][pos // page].long() * page + pos % page
        for c, plane, size in ((kc, 0, channel), (vc, 1, None)):
            x = torch.randn(n, heads, dim, device="cuda", generator=g)
            x *= size if size is not None else torch.exp(0.5 * torch.randn(n, heads, 1, device="cuda", generator=g))
            x, scale = _hold(x, held)
            c.view(pages * page, heads, dim)[slots] = x
            if scale is not None:
                sc.view(pages * page, heads, 2)[slots, :, plane] = scale
            del x
    return {"k_cache": kc, "v_cache": vc, "scales": sc, "page_table": table}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    heads, dim = case.get("heads", case.get("kv_heads")), case["dim"]
    s = {"op": case["op"], "page": case["page"], "held": case["held"]}
    if case["op"] == "cache":
        n, page = case["tokens"], case["page"]
        pages = -(-n // page) + 8
        kc, vc, sc = _empty_cache(pages, page, heads, dim, case["held"], g)
        slots = torch.randperm(pages, device="cuda", generator=g)[torch.arange(n, device="cuda") // page] * page + torch.arange(n, device="cuda") % page
        # keys and values of one projection: two strided halves of one tensor
        kv = torch.randn(n, 2, heads, dim, device="cuda", generator=g) * torch.exp(torch.randn(n, 2, heads, 1, device="cuda", generator=g))
        kv = kv.to(_TYPES[case["src"]])
        return {**s, "k": kv[:, 0], "v": kv[:, 1], "k_cache": kc, "v_cache": vc, "scales": sc, "slots": slots.to(torch.int32)}

    lengths = _lengths(case)
    batch, width = case["batch"], case["drafts"] if case["op"] == "tree" else case["queries"]
    q = (1.5 * torch.randn(batch, width, case["q_heads"], dim, device="cuda", generator=g)).to(torch.bfloat16)
    s.update(q=q, softmax_scale=dim ** -0.5, width=max(lengths) + (width if case["op"] == "tree" else 0))
    if case["op"] == "tree":
        counts = _draft_counts(case)
        s.update(_tensors(case, [n + t for n, t in zip(lengths, counts)], g))
        # a random tree: each drafted token's parent is an earlier one, or the context's last token (-1)
        parents = (torch.rand(batch, width, device="cuda", generator=g) * (torch.arange(width, device="cuda") + 1)).long() - 1
        reach = torch.eye(width, dtype=torch.bool, device="cuda").repeat(batch, 1, 1)
        for i in range(1, width):  # a token attends to itself and to what its parent attends to
            p = parents[:, i]
            reach[:, i] |= reach[torch.arange(batch, device="cuda"), p.clamp(min=0)] & (p >= 0).unsqueeze(-1)
        words = -(-width // 32)
        bits = torch.zeros(batch, width, words * 32, dtype=torch.int64, device="cuda")
        bits[:, :, :width] = reach
        bits = (bits.view(batch, width, words, 32) << torch.arange(32, device="cuda")).sum(-1)
        s.update(parents=parents, tree=torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32),
                 ctx_len=torch.tensor(lengths, dtype=torch.int32, device="cuda"), draft_len=torch.tensor(counts, dtype=torch.int32, device="cuda"))
        return s
    s.update(_tensors(case, lengths, g))
    # each query's k positions, all different, in no order, among those before it; -1 where it has fewer than k
    seen = torch.tensor(lengths, device="cuda").view(-1, 1) - width + 1 + torch.arange(width, device="cuda")
    k = case["k"]
    idx = torch.full((batch, width, k), -1, dtype=torch.int32, device="cuda")
    take = min(k, max(lengths))
    for b in range(batch):
        logits = torch.rand(width, max(lengths), device="cuda", generator=g).masked_fill_(torch.arange(max(lengths), device="cuda") >= seen[b].view(-1, 1), -1.0)
        top = logits.topk(take, dim=-1)
        at = torch.where(top.values >= 0, top.indices, -1)
        idx[b, :, :take] = at[:, torch.randperm(take, device="cuda", generator=g)].to(torch.int32)
    s.update(indices=idx, kv_len=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    return s


# ---------------------------------------------------------------------------
# One pass: the plain forms, and the package's operators
# ---------------------------------------------------------------------------


def _rows(cache, scales, plane, slots):
    """The rows a cache holds at `slots`, as the 32-bit values they stand for."""
    heads, dim = cache.shape[2:]
    x = cache.view(-1, heads, dim)[slots].float()
    return x if scales is None else x * scales.view(-1, heads, 2)[slots][..., plane].unsqueeze(-1)


def _attend(q, k, v, seen, scale):
    """q [n, heads, rows, dim], k and v [n, heads, keys, dim], seen [n, 1 or heads, rows, keys]: the rows' outputs and log-sum-exps.
    Keys that a row does not see count for nothing, whatever they hold; a row that sees none gives 0 and -inf."""
    x = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.where(total > 0, (x @ v) / total, 0.0)
    return out, (total.log() + top).squeeze(-1)


def _plain_cache(s):
    slots = s["slots"].long()
    for x, cache, plane in ((s["k"], s["k_cache"], 0), (s["v"], s["v_cache"], 1)):
        rows, scale = _hold(x, s["held"])
        cache.view(-1, *cache.shape[2:])[slots] = rows
        if scale is not None:
            s["scales"].view(-1, cache.shape[2], 2)[slots, :, plane] = scale
    k, v = (_rows(c, s["scales"], p, slots).to(s["k"].dtype) for c, p in ((s["k_cache"], 0), (s["v_cache"], 1)))
    return k, v


def _plain_tree(s):
    q, page = s["q"], s["page"]
    batch, width, q_heads, dim = q.shape
    heads = s["k_cache"].shape[2]
    pos = torch.arange(s["width"], device=q.device)
    ctx, count = s["ctx_len"].view(-1, 1), s["draft_len"].view(-1, 1)
    held = pos < ctx + count  # [batch, keys]
    at = (pos // page).clamp(max=s["page_table"].shape[1] - 1)
    slots = torch.where(held, s["page_table"][:, at] * page + pos % page, 0).long()
    k, v = (torch.where(held[..., None, None], _rows(c, s["scales"], p, slots), 0.0).transpose(1, 2) for c, p in ((s["k_cache"], 0), (s["v_cache"], 1)))
    draft = pos - ctx  # [batch, keys]
    inside = ((draft >= 0) & (draft < width)).unsqueeze(1)
    word = s["tree"].gather(2, (draft.clamp(0, width - 1) // 32).unsqueeze(1).expand(-1, width, -1))
    bit = (word >> (draft.clamp(0, width - 1) % 32).unsqueeze(1)) & 1
    rows_in_use = (torch.arange(width, device=q.device) < count).unsqueeze(-1)
    seen = held.unsqueeze(1) & ((draft < 0).unsqueeze(1) | (inside & (bit == 1))) & rows_in_use  # [batch, width, keys]
    group = q_heads // heads
    rows = q.float().view(batch, width, heads, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, heads, width * group, dim)
    out, lse = _attend(rows, k, v, seen.unsqueeze(1).repeat_interleave(group, dim=2), s["softmax_scale"])
    out = out.view(batch, heads, width, group, dim).permute(0, 2, 1, 3, 4).reshape(q.shape).to(q.dtype)
    return out, lse.view(batch, heads, width, group).permute(0, 2, 1, 3).reshape(batch, width, q_heads)


def _plain_selected(s):
    q, idx, page = s["q"], s["indices"], s["page"]
    batch, width, q_heads, dim = q.shape
    heads, k_sel = s["k_cache"].shape[2], idx.shape[2]
    seen = (idx >= 0) & (idx < s["kv_len"].view(-1, 1, 1))
    pos = torch.where(seen, idx, 0).long()
    pages = s["page_table"].gather(1, (pos // page).view(batch, -1)).view(pos.shape)
    slots = torch.where(seen, pages * page + pos % page, 0).view(batch * width, k_sel)
    seen = seen.view(batch * width, 1, 1, k_sel)
    k, v = (torch.where(seen.view(-1, k_sel, 1, 1), _rows(c, s["scales"], p, slots), 0.0).transpose(1, 2) for c, p in ((s["k_cache"], 0), (s["v_cache"], 1)))
    group = q_heads // heads
    out, lse = _attend(q.float().view(batch * width, heads, group, dim), k, v, seen, s["softmax_scale"])
    return out.reshape(q.shape).to(q.dtype), lse.reshape(batch, width, q_heads)


def run(s):
    if own:
        import sparse_attention_topk_gb300 as tks

        if s["op"] == "cache":
            tks.cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], scales=s["scales"])
            k, v = tks.cache_read(s["k_cache"], s["v_cache"], s["slots"], scales=s["scales"], dtype=s["k"].dtype)
        elif s["op"] == "tree":
            out, lse = tks.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["ctx_len"], tree=s["tree"], draft_len=s["draft_len"],
                                          scales=s["scales"], softmax_scale=s["softmax_scale"], return_lse=True)
        else:
            out, lse = tks.selected_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["indices"], kv_len=s["kv_len"],
                                              scales=s["scales"], softmax_scale=s["softmax_scale"], return_lse=True)
    elif s["op"] == "cache":
        k, v = _plain_cache(s)
    else:
        out, lse = _plain_tree(s) if s["op"] == "tree" else _plain_selected(s)
    if s["op"] == "cache":
        # the updated cache: its scales, or, where it holds bfloat16, itself
        held = {"scales": s["scales"]} if s["scales"] is not None else {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        return {"k": k, "v": v, **held}
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, and the work
# ---------------------------------------------------------------------------


def _softmax_row_block(q, k, v, allowed, scale):
    """q [r, d], k and v [n, d] in 64 bits, allowed [r, n]: softmax(q k^T scale) v over the allowed keys, by the log-sum-exp."""
    s = (q @ k.T) * scale
    s[~allowed] = -math.inf
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse.isinf(), 0.0, lse).unsqueeze(-1))
    return p @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    page = case["page"]
    if case["op"] == "cache":
        back = []
        planes = []
        for x in (s["k"], s["v"]):
            x = x.double()
            if case["held"] == "bf16":
                back.append(x)
                continue
            step = x.abs().amax(-1, keepdim=True).clamp(AMAX_LOW, AMAX_HIGH) / 127
            back.append(torch.clamp(torch.round(x / step), -127, 127) * step)
            planes.append(step[..., 0])
        slots = s["slots"].long()
        if case["held"] == "bf16":
            for name, x in (("k_cache", back[0]), ("v_cache", back[1])):
                s[name] = s[name].double()
                s[name].view(-1, *s[name].shape[2:])[slots] = x
            return {"k": back[0], "v": back[1], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        scales = s["scales"].double()
        scales.view(-1, case["heads"], 2)[slots] = torch.stack(planes, -1)
        return {"k": back[0], "v": back[1], "scales": scales}

    q = s["q"].double()
    batch, width, q_heads, dim = q.shape
    heads = case["kv_heads"]
    group = q_heads // heads
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=q.device)

    def values(cache, plane, slots, head):
        x = cache.view(-1, heads, dim)[slots, head].double()
        return x if s["scales"] is None else x * s["scales"].view(-1, heads, 2)[slots, head, plane].double().unsqueeze(-1)

    for b in range(batch):
        table = s["page_table"][b].long()
        if case["op"] == "tree":
            n, t = int(s["ctx_len"][b]), int(s["draft_len"][b])
            pos = torch.arange(n + t, device=q.device)
            allowed = torch.zeros(t, n + t, dtype=torch.bool)
            allowed[:, :n] = True
            parents = s["parents"][b].tolist()
            for i in range(t):
                j = i
                while j >= 0:  # up the tree
                    allowed[i, n + j] = True
                    j = parents[j]
            blocks = [(slice(0, t), pos, allowed.to(q.device))]
        else:
            blocks = []
            for i in range(width):
                pos = s["indices"][b, i]
                pos = pos[pos >= 0].long()
                blocks.append((slice(i, i + 1), pos, torch.ones(1, len(pos), dtype=torch.bool, device=q.device)))
        for rows, pos, allowed in blocks:
            slots = table[pos // page] * page + pos % page
            for h in range(heads if len(pos) else 0):
                hs = slice(h * group, (h + 1) * group)
                k, v = values(s["k_cache"], 0, slots, h), values(s["v_cache"], 1, slots, h)
                rq = q[b, rows, hs].reshape(-1, dim)
                o, l = _softmax_row_block(rq, k, v, allowed.repeat_interleave(group, 0), s["softmax_scale"])
                out[b, rows, hs] = o.view(-1, group, dim)
                lse[b, rows, hs] = l.view(-1, group)
    return {"out": out, "lse": lse}


def work(case):
    dim = case["dim"]
    row = 2 * (dim * _BYTES[case["held"]] + (4 if case["held"] == "int8" else 0))  # one token's key and value of one head, as held
    if case["op"] == "cache":
        rows = case["tokens"] * case["heads"]
        # the new rows are read and written as held, read back from there and written out again
        return {"bytes": rows * (2 * row + 4 * dim * _BYTES[case["src"]]) + 8 * case["tokens"], "flops": 8 * rows * dim}
    lengths, heads, q_heads = _lengths(case), case["kv_heads"], case["q_heads"]
    width = case["drafts"] if case["op"] == "tree" else case["queries"]
    ends = case["batch"] * width * q_heads * (4 * dim + 4)  # queries, outputs, log-sum-exps
    if case["op"] == "tree":
        counts = _draft_counts(case)
        keys = sum(n + t for n, t in zip(lengths, counts))
        pairs = sum((n + (t + 1) / 2) * t for n, t in zip(lengths, counts))
        table = sum(-(-(n + t) // case["page"]) for n, t in zip(lengths, counts)) + case["batch"] * (2 + width * -(-width // 32))
        return {"bytes": keys * heads * row + ends + 4 * table, "flops": 4 * dim * q_heads * pairs}
    each = [[max(0, min(case["k"], n - width + 1 + i)) for i in range(width)] for n in lengths]
    keys = sum(min(sum(e), n) for e, n in zip(each, lengths))  # each position that is chosen at all, once
    return {"bytes": keys * heads * row + ends + 4 * case["batch"] * width * case["k"] + 4 * min(keys, sum(-(-n // case["page"]) for n in lengths)),
            "flops": 4 * dim * q_heads * sum(map(sum, each))}

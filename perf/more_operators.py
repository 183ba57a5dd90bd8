"""The cases on which the operators over a cache's pages and blocks are measured.

Sparse attention by blocks: a cheap score of every block of a paged cache, by the
least and largest value of its keys in each channel, selects the blocks that a
query attends to (the top-k selector stands between the two).  And what a serving
loop does with the pages themselves between its steps: sequences fork, grow, end,
and what is left is moved together.

    bounds      the least and largest key of the blocks that new tokens lie in
    scores      each query's score of every block: no key in it has a larger product with the query
    attend      attention of each query and key/value head over its own list of blocks
    fork        the page tables of a step's new sequences, and copies of the pages that two would write to
    compact     page tables and pages after moving what is in use to the lowest pages

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

_BYTES = {"int8": 1, "bf16": 2}
_NONE = 2 ** 31 - 1


def listed():
    def bounds(name, batch, context, ragged, new, heads, dim, held, page, block):
        return {"name": name, "op": "bounds", "batch": batch, "context": context, "ragged": ragged, "new": new, "kv_heads": heads, "dim": dim,
                "held": held, "page": page, "block": block}

    def scores(name, batch, queries, q_heads, kv_heads, dim, context, ragged, page, block):
        return {"name": name, "op": "scores", "batch": batch, "queries": queries, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
                "context": context, "ragged": ragged, "page": page, "block": block}

    def attend(name, batch, queries, q_heads, kv_heads, dim, context, ragged, chosen, held, page, block):
        return {"name": name, "op": "attend", "batch": batch, "queries": queries, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
                "context": context, "ragged": ragged, "chosen": chosen, "held": held, "page": page, "block": block}

    def fork(name, groups, beams, survivors, context, ragged, heads, dim, held, page):
        return {"name": name, "op": "fork", "groups": groups, "beams": beams, "survivors": survivors, "context": context, "ragged": ragged,
                "kv_heads": heads, "dim": dim, "held": held, "page": page}

    def compact(name, pages, fill, batch, heads, dim, held, page):
        return {"name": name, "op": "compact", "pages": pages, "fill": fill, "batch": batch, "kv_heads": heads, "dim": dim, "held": held, "page": page}

    return [
        # one decode step of a ragged batch (the lengths of the repository's ragged batch): each sequence's last block changes; latency
        bounds("bounds_step64", 64, 65536, True, 1, 8, 128, "int8", 64, 64),
        # a whole prompt of the length of the repository's prefill workload
        bounds("bounds_prompt_32k", 1, 32768, False, 32768, 8, 128, "int8", 64, 64),
        # one token over the selector's row of 128K: latency
        scores("scores_one_128k", 1, 1, 32, 8, 128, 131072, False, 64, 64),
        # a batch of decode rows, ragged, smaller blocks: the bounds are read at the memory's rate
        scores("scores_batch64", 64, 1, 16, 2, 128, 65536, True, 64, 32),
        # a chunk of a long prompt, causal: matrix products
        scores("scores_chunk_2048", 1, 2048, 32, 8, 128, 131072, False, 64, 64),
        # one token over 32 blocks of a context of 128K, each head its own: latency
        attend("attend_one_128k", 1, 1, 32, 8, 128, 131072, False, 32, "int8", 64, 64),
        # a batch of decode rows, ragged, smaller blocks over a bfloat16 cache
        attend("attend_batch64", 64, 1, 16, 2, 128, 65536, True, 64, "bf16", 64, 32),
        # the 512 causal rows over 32K of the repository's prefill workload
        attend("attend_prefill", 1, 512, 64, 4, 128, 32768, False, 32, "int8", 64, 64),
        # a few odd beams over short contexts, small heads and pages: latency
        fork("fork_beams_odd", 3, 5, 2, 777, True, 4, 64, "bf16", 16),
        # beam search of a ragged batch of long contexts
        fork("fork_beams_64k", 16, 4, 2, 65536, True, 8, 128, "int8", 64),
        # a small pool after some of its sequences have ended
        compact("compact_small", 639, 0.6, 7, 4, 64, "bf16", 16),
        # half of a pool of a gigabyte in use, in no order
        compact("compact_pool", 8192, 0.5, 33, 8, 128, "int8", 64),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("bounds", "scores", "attend", "fork", "compact"))
    dim, held, page = rng.choice((64, 128, 128)), rng.choice(("int8", "bf16")), rng.choice((16, 32, 64, 128))
    heads, block = rng.choice((1, 2, 4, 8)), rng.choice([n for n in (8, 16, 32, 64, 128) if n <= page])
    row = 2 * heads * dim * _BYTES[held]  # one token's keys and values
    if op == "bounds":
        batch = _log(rng, 1, 64)
        context = _log(rng, 1, min(65536, (1 << 29) // (batch * row)))
        return {"op": op, "batch": batch, "context": context, "ragged": rng.random() < 0.5, "new": _log(rng, 1, min(context, 33_000_000 // (batch * row) + 1)),
                "kv_heads": heads, "dim": dim, "held": held, "page": page, "block": block}
    if op == "scores":
        batch, queries, group = _log(rng, 1, 64), _log(rng, 1, 1000), rng.choice((1, 2, 4, 7, 8, 16))
        while batch * queries > 2048:
            queries = (queries + 1) // 2
        blocks = min(16384, (100 << 20) // (batch * heads * dim * 4), 134_000_000 // (batch * queries * heads * group * dim // 128 + 1),
                     33_000_000 // (batch * queries * heads))
        return {"op": op, "batch": batch, "queries": queries, "q_heads": heads * group, "kv_heads": heads, "dim": dim,
                "context": max(queries, _log(rng, 1, max(1, blocks * block))), "ragged": rng.random() < 0.5, "page": page, "block": block}
    if op == "attend":
        batch, queries, group = _log(rng, 1, 16), _log(rng, 1, 64), rng.choice((1, 4, 7, 8, 16, 32))
        context = max(queries, _log(rng, 100, max(100, min(1048576, (1 << 30) // (batch * row)))))
        chosen = max(1, _log(rng, 16, 4096) // block)
        while queries > 1 and batch * queries * chosen * block * heads * dim > 134_000_000:
            queries = (queries + 1) // 2
        return {"op": op, "batch": batch, "queries": queries, "q_heads": heads * group, "kv_heads": heads, "dim": dim, "context": context,
                "ragged": rng.random() < 0.5, "chosen": chosen, "held": held, "page": page, "block": block}
    if op == "fork":
        groups, beams = _log(rng, 1, 24), rng.choice((1, 2, 3, 4, 5, 8))
        context = _log(rng, 1, max(1, min(65536, (1 << 30) // (groups * (1 + beams) * row))))
        return {"op": op, "groups": groups, "beams": beams, "survivors": rng.randint(1, beams), "context": context, "ragged": rng.random() < 0.5,
                "kv_heads": heads, "dim": dim, "held": held, "page": page}
    return {"op": op, "pages": _log(rng, 50, min(8192, (1 << 30) // (page * row))), "fill": rng.choice((0.1, 0.3, 0.5, 0.7, 0.9)), "batch": _log(rng, 1, 40),
            "kv_heads": heads, "dim": dim, "held": held, "page": page}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _lengths(case):
    """Context lengths: the full one first, then, where ragged, others spread below it."""
    n, b = case["context"], case.get("batch", case.get("groups"))
    least = case.get("queries", 1)
    return [n if i == 0 or not case["ragged"] else max(least, int(n * ((i * 0.6180339887) % 1.0))) for i in range(b)]


def _rows(shape, held, g, channel=None):
    """Rows [.., heads, dim] of keys (channels of different sizes) or values (tokens of different sizes), as a cache holds them, and their scales."""
    x = torch.randn(shape, device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), device="cuda", generator=g)) if channel is None else channel
    if held == "bf16":
        return x.to(torch.bfloat16), None
    scale = x.abs().amax(-1) * (1.0 / 127.0)
    return (x / scale.unsqueeze(-1)).round_().clamp_(-127, 127).to(torch.int8), scale


def _cache(case, pages, written, g):
    """A cache of `pages` pages; slots outside `written` (bool [pages * page]) hold nothing that may be used."""
    page, heads, dim, held = case["page"], case["kv_heads"], case["dim"], case["held"]
    channel = torch.exp(0.4 * torch.randn(heads, dim, device="cuda", generator=g))
    s = {}
    scales = []
    for name, size in (("k_cache", channel), ("v_cache", None)):
        c, scale = _rows((pages, page, heads, dim), held, g, size)
        if held == "bf16":
            c.view(pages * page, heads, dim)[~written] = math.nan
        else:
            scale.view(pages * page, heads)[~written] = math.nan
            scales.append(scale)
        s[name] = c
    s["scales"] = torch.stack(scales, -1) if scales else None
    return s


def _tables(case, lengths, g, room=0):
    """A page table whose sequence b holds lengths[b] tokens in pages of random order, the number of pages, and which slots are written."""
    page = case["page"]
    need = torch.tensor([-(-(n + room) // page) for n in lengths], device="cuda")
    pages = int(need.sum()) + 3
    order = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    column = torch.arange(int(need.max()), device="cuda")
    at = (need.cumsum(0) - need).unsqueeze(1) + column
    held = column < need.unsqueeze(1)
    table = torch.where(held, order[torch.where(held, at, 0)], -1)
    pos = column.view(1, -1, 1) * page + torch.arange(page, device="cuda")  # [1, pages of a sequence, page]
    there = pos < torch.tensor(lengths, device="cuda").view(-1, 1, 1)
    written = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    written[table[held].long()] = there[held]
    return table, pages, written.view(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, heads, dim, page = case["op"], case["kv_heads"], case["dim"], case["page"]
    s = {"op": op, "page": page, "block": case.get("block")}
    if op == "fork":
        return {**s, **_forked(case, g)}
    if op == "compact":
        return {**s, **_fragmented(case, g)}
    lengths = _lengths(case)
    table, pages, written = _tables(case, lengths, g)
    s.update(page_table=table)
    blocks = page // case["block"]
    if op == "bounds":
        s.update(_cache(case, pages, written, g))
        end = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        s.update(end=end, start=(end - case["new"]).clamp(min=0).to(torch.int32),
                 bounds=torch.zeros(pages, blocks, heads, 2, dim, dtype=torch.bfloat16, device="cuda"))
        return s
    batch, width, q_heads = case["batch"], case["queries"], case["q_heads"]
    q = (1.5 * torch.randn(batch, width, q_heads, dim, device="cuda", generator=g)).to(torch.bfloat16)
    last = torch.tensor(lengths, device="cuda").view(-1, 1)
    kv_len = (last - width + 1 + torch.arange(width, device="cuda")).to(torch.int32)  # each token sees those before it, and itself
    s.update(q=q, kv_len=kv_len)
    if op == "scores":
        # bounds of blocks of keys whose channels have different sizes and middles
        channel = torch.exp(0.4 * torch.randn(heads, dim, device="cuda", generator=g))
        middle = 0.5 * torch.randn(pages, blocks, heads, dim, device="cuda", generator=g)
        half = 1.5 + 1.5 * torch.rand(pages, blocks, heads, dim, device="cuda", generator=g)
        s["bounds"] = torch.stack((channel * (middle - half), channel * (middle + half)), 3).to(torch.bfloat16)
        s["bounds"][~written.view(pages, blocks, -1).any(-1)] = math.nan  # blocks without a token
        return s
    s.update(_cache(case, pages, written, g), softmax_scale=dim ** -0.5)
    # each query's and head's blocks: the first, the last and others among those it sees, all different, in no order; -1 where there are fewer
    n, chosen = -(-max(lengths) // case["block"]), case["chosen"]
    take = min(chosen, n)
    column = torch.arange(n, device="cuda")
    lists = torch.full((batch, width, heads, chosen), -1, dtype=torch.int32, device="cuda")
    for b in range(batch):
        seen = -(-kv_len[b] // case["block"]).view(-1, 1, 1)
        x = torch.rand(width, heads, n, device="cuda", generator=g)
        x = torch.where((column == 0) | (column == seen - 1), 2.0, x).masked_fill_(column >= seen, -1.0)
        top = x.topk(take, dim=-1)
        at = torch.where(top.values >= 0, top.indices, -1)
        lists[b, :, :, :take] = at[..., torch.randperm(take, device="cuda", generator=g)].to(torch.int32)
    s["blocks"] = lists
    return s


def _forked(case, g):
    """Groups of beams that share their prompt's pages (three quarters of the context) and have their own behind; `survivors` of each go on."""
    page, beams, heads, dim = case["page"], case["beams"], case["kv_heads"], case["dim"]
    lengths = _lengths(case)
    need = [-(-n // page) for n in lengths]
    shared = [(3 * n // 4) // page for n in lengths]
    pages = sum(s + beams * (n - s) for n, s in zip(need, shared)) + 2 * beams * len(need) + 5
    order = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    table = torch.full((beams * len(need), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    parents, at = [], 0
    for b, (n, s) in enumerate(zip(need, shared)):
        rows = slice(b * beams, (b + 1) * beams)
        table[rows, :s] = order[at : at + s]
        table[rows, s:n] = order[at + s : at + s + beams * (n - s)].view(beams, n - s)
        at += s + beams * (n - s)
        # every survivor has a child, the other children are theirs at random
        alive = torch.randperm(beams, device="cuda", generator=g)[: case["survivors"]]
        more = alive[torch.randint(case["survivors"], (beams - case["survivors"],), device="cuda", generator=g)]
        mine = torch.cat((alive, more))[torch.randperm(beams, device="cuda", generator=g)]
        parents.append(mine + b * beams)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda").repeat_interleave(beams)
    s = _cache(case, pages, torch.ones(pages * page, dtype=torch.bool, device="cuda"), g)
    s.update(page_table=table, lens=lens, parents=torch.cat(parents).to(torch.int32), new_lens=lens + 1, pages=pages,
             bounds=torch.randn(pages, 1, heads, 2, dim, device="cuda", generator=g).to(torch.bfloat16))
    return s


def _used(case):
    """The pages of each sequence of a pool, as sizes."""
    total, b = max(1, int(case["pages"] * case["fill"])), min(case["batch"], max(1, int(case["pages"] * case["fill"])))
    cuts = [total * (i * i + i) // (b * b + b) for i in range(b)] + [total]
    return [cuts[i + 1] - cuts[i] for i in range(b)]


def _fragmented(case, g):
    page, pages, heads, dim = case["page"], case["pages"], case["kv_heads"], case["dim"]
    used = torch.tensor(_used(case), device="cuda")
    order = torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    column = torch.arange(int(used.max()) + 1, device="cuda")
    held = column < used.unsqueeze(1)
    table = torch.where(held, order[torch.where(held, (used.cumsum(0) - used).unsqueeze(1) + column, 0)], -1)
    less = torch.randint(page, used.shape, device="cuda", generator=g)
    s = _cache(case, pages, torch.ones(pages * page, dtype=torch.bool, device="cuda"), g)
    s.update(page_table=table, lens=(used * page - less).clamp(min=0).to(torch.int32), pages=pages,
             bounds=torch.randn(pages, 1, heads, 2, dim, device="cuda", generator=g).to(torch.bfloat16))
    return s


# ---------------------------------------------------------------------------
# One pass: the plain forms, and the package's operators
# ---------------------------------------------------------------------------


def _slots(s, pos):
    """The cache slots of positions [batch, ...] of each sequence; those of a position without a page are not to be used."""
    page, table = s["page"], s["page_table"]
    pages = table.gather(1, (pos // page).clamp(max=table.shape[1] - 1).flatten(1).long()).view(pos.shape)
    return (pages.clamp(min=0) * page + pos % page).long()


def _values(s, name, plane, slots):
    """The rows of a cache at `slots`, as the 32-bit values they stand for."""
    cache = s[name]
    heads, dim = cache.shape[2:]
    x = cache.view(-1, heads, dim)[slots].float()
    return x if s["scales"] is None else x * s["scales"].view(-1, heads, 2)[slots][..., plane].unsqueeze(-1)


def _plain_bounds(s):
    block = s["block"]
    start, end = s["start"].long(), s["end"].long()
    first = start // block
    count = torch.where(start < end, -(-end // block) - first, 0)
    # all new blocks of all sequences, one after the other
    seq = torch.repeat_interleave(torch.arange(len(start), device=start.device), count)
    number = first[seq] + torch.arange(len(seq), device=seq.device) - (count.cumsum(0) - count)[seq]
    pos = number.unsqueeze(1) * block + torch.arange(block, device=seq.device)  # [blocks, block]
    there = (pos < end[seq].unsqueeze(1))[..., None, None]
    pages = s["page_table"][seq, number * block // s["page"]].long()
    x = _values(s, "k_cache", 0, pages.unsqueeze(1) * s["page"] + pos % s["page"])
    low, high = torch.where(there, x, math.inf).amin(1), torch.where(there, x, -math.inf).amax(1)
    s["bounds"][pages, number % (s["page"] // block)] = torch.stack((low, high), 2).to(torch.bfloat16)
    return {"bounds": s["bounds"]}


def _plain_scores(s):
    q, bounds = s["q"], s["bounds"]
    batch, width, q_heads, dim = q.shape
    heads = bounds.shape[2]
    group, n = q_heads // heads, s["page_table"].shape[1] * bounds.shape[1]
    mine = bounds[s["page_table"].clamp(min=0).long()].view(batch, n, heads, 2, dim)
    low, high = (mine[:, :, :, i].permute(0, 2, 3, 1).float() for i in (0, 1))  # [batch, heads, dim, n]
    rows = q.float().view(batch, width, heads, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, heads, width * group, dim)
    x = rows.clamp(min=0) @ high
    x += rows.clamp(max=0) @ low
    x = x.view(batch, heads, width, group, n).amax(3).transpose(1, 2)  # [batch, width, heads, n]
    seen = -(-s["kv_len"] // s["block"])
    x = torch.where(torch.arange(n, device=q.device) < seen.view(batch, width, 1, 1), x, -math.inf)
    return {"scores": x, "row_len": seen.unsqueeze(-1).expand(batch, width, heads).to(torch.int32).contiguous()}


def _plain_attend(s):
    q, block, lists = s["q"], s["block"], s["blocks"]
    batch, width, q_heads, dim = q.shape
    heads = s["k_cache"].shape[2]
    group = q_heads // heads
    pos = (lists.unsqueeze(-1) * block + torch.arange(block, device=q.device)).flatten(3)  # [batch, width, heads, keys]
    seen = (pos >= 0) & (lists >= 0).repeat_interleave(block, -1) & (pos < s["kv_len"].view(batch, width, 1, 1))
    slots = _slots(s, pos.clamp(min=0))
    head = torch.arange(heads, device=q.device).view(heads, 1)
    k, v = (torch.where(seen.unsqueeze(-1), _of_head(s, name, plane, slots, head), 0.0) for name, plane in (("k_cache", 0), ("v_cache", 1)))
    x = (q.float().view(batch, width, heads, group, dim) @ k.transpose(-1, -2)).mul_(s["softmax_scale"])
    x.masked_fill_(~seen.unsqueeze(3), -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.where(total > 0, (x @ v) / total, 0.0)
    return {"out": out.reshape(q.shape).to(q.dtype), "lse": (total.log() + top).reshape(batch, width, q_heads)}


def _of_head(s, name, plane, slots, head):
    """As _values, for slots [..., heads, keys] of which each head has its own."""
    cache = s[name]
    heads, dim = cache.shape[2:]
    x = cache.view(-1, heads, dim)[slots, head].float()
    return x if s["scales"] is None else x.mul_(s["scales"].view(-1, heads, 2)[slots, head, plane].unsqueeze(-1))


def _moved(s, src, dst):
    """Copies whole pages; pairs with a negative page are none."""
    real = src >= 0
    src, dst = src[real].long(), dst[real].long()
    for name in ("k_cache", "v_cache", "scales", "bounds"):
        if s[name] is not None:
            s[name][dst] = s[name][src]


def _plain_fork(s):
    table, page, pages, parents = s["page_table"], s["page"], s["pages"], s["parents"].long()
    kept = torch.minimum(s["lens"][parents], s["new_lens"])
    have, need = -(-kept // page), -(-s["new_lens"] // page)
    column = torch.arange(table.shape[1], device=table.device)
    rows = table[parents]
    held = column < have.unsqueeze(1)
    # a page that a sequence would write to is its own: its last, partly filled one
    writes = (kept % page != 0) & (s["new_lens"] > kept)
    last = writes.unsqueeze(1) & (column == have.unsqueeze(1) - 1)
    owner = torch.full((pages,), _NONE, dtype=torch.int64, device=table.device)
    number = torch.arange(len(parents), device=table.device).unsqueeze(1).expand(rows.shape)
    owner.scatter_reduce_(0, rows[held].long(), torch.where(last, number, -1)[held], "amin")
    tail = rows.gather(1, (have - 1).clamp(min=0).unsqueeze(1).long()).squeeze(1)
    copied = writes & (owner[tail.clamp(min=0).long()] != number[:, 0])
    # free pages go to those who want one, in order
    wants = (last & copied.unsqueeze(1)) | ((column >= have.unsqueeze(1)) & (column < need.unsqueeze(1)))
    rank = (wants.flatten().cumsum(0) - 1).view(wants.shape)
    free = torch.nonzero(owner == _NONE).squeeze(1)
    given = free[torch.where(wants, rank, 0)].to(torch.int32)
    new = torch.where(wants, given, torch.where(held, rows, -1))
    src = torch.where(copied, tail, -1)
    dst = torch.where(copied, new.gather(1, (have - 1).clamp(min=0).unsqueeze(1).long()).squeeze(1), -1)
    _moved(s, src, dst)
    return {"table": new, "src": src, "dst": dst}


def _plain_compact(s):
    table, page, pages = s["page_table"], s["page"], s["pages"]
    held = torch.arange(table.shape[1], device=table.device) < (-(-s["lens"] // page)).unsqueeze(1)
    used = torch.zeros(pages, dtype=torch.bool, device=table.device)
    used[table[held].long()] = True
    count = used.sum()
    number = torch.arange(pages, device=table.device)
    moves, holes = used & (number >= count), ~used & (number < count)
    source, target = (torch.nonzero(x).squeeze(1).to(torch.int32) for x in (moves, holes))
    target = target[: len(source)]
    place = number.to(torch.int32)
    place[source.long()] = target
    src, dst = (torch.full((pages // 2,), -1, dtype=torch.int32, device=table.device) for _ in range(2))
    src[: len(source)], dst[: len(source)] = source, target
    _moved(s, src, dst)
    new = torch.where(held, place[table.clamp(min=0).long()], -1)
    return {"table": new, "src": src, "dst": dst, "count": torch.stack((moves.sum(), count)).to(torch.int32)}


def run(s):
    op = s["op"]
    if own:
        import sparse_attention_topk_gb300 as tks

        if op == "bounds":
            tks.cache_bounds(s["k_cache"], s["page_table"], s["end"], s["bounds"], start=s["start"], scales=s["scales"])
            return {"bounds": s["bounds"]}
        if op == "scores":
            scores, row_len = tks.block_scores(s["q"], s["bounds"], s["page_table"], s["kv_len"], s["block"])
            return {"scores": scores, "row_len": row_len}
        if op == "attend":
            out, lse = tks.block_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["blocks"], s["block"], kv_len=s["kv_len"],
                                           scales=s["scales"], softmax_scale=s["softmax_scale"], return_lse=True)
            return {"out": out, "lse": lse}
        if op == "fork":
            table, src, dst = tks.cache_fork(s["page_table"], s["lens"], s["parents"], s["new_lens"], s["pages"], s["page"])
            tks.cache_copy(src, dst, s["k_cache"], s["v_cache"], scales=s["scales"], bounds=s["bounds"])
            r = {"table": table, "src": src, "dst": dst}
        else:
            table, src, dst, count = tks.cache_compact(s["page_table"], s["lens"], s["pages"], s["page"])
            tks.cache_copy(src, dst, s["k_cache"], s["v_cache"], scales=s["scales"], bounds=s["bounds"], count=count)
            r = {"table": table, "src": src, "dst": dst, "count": count}
    elif op == "bounds":
        return _plain_bounds(s)
    elif op == "scores":
        return _plain_scores(s)
    elif op == "attend":
        return _plain_attend(s)
    else:
        r = _plain_fork(s) if op == "fork" else _plain_compact(s)
    # the pool as it is now (8-bit codes are copied as they are)
    r.update({name: s[name] for name in ("k_cache", "v_cache", "scales", "bounds") if s[name] is not None})
    return r


# ---------------------------------------------------------------------------
# The definitions in 64 bits, and the work
# ---------------------------------------------------------------------------


def _exact_pages(s, pairs):
    for name in ("k_cache", "v_cache", "scales", "bounds"):
        if s[name] is None:
            continue
        x = s[name].double() if s[name].is_floating_point() else s[name]
        if pairs:
            to, of = (torch.tensor(p, device=x.device) for p in zip(*pairs))
            x[to] = x[of]
        s[name] = x
    return {name: s[name] for name in ("k_cache", "v_cache", "scales", "bounds") if s[name] is not None}


def _exact_fork(s):
    page, lens, new_lens, parents = s["page"], s["lens"].tolist(), s["new_lens"].tolist(), s["parents"].tolist()
    rows = s["page_table"].tolist()
    width = len(rows[0])
    holders = {}  # page: the new sequences that hold it, and which of them write to it
    kept = []
    for i, p in enumerate(parents):
        n = min(lens[p], new_lens[i])
        mine = rows[p][: -(-n // page)]
        kept.append((n, mine))
        for j, e in enumerate(mine):
            holders.setdefault(e, []).append((i, j == len(mine) - 1 and n % page != 0 and new_lens[i] > n))
    free = iter([p for p in range(s["pages"]) if p not in holders])
    out, src, dst = [], [], []
    for i, (n, mine) in enumerate(kept):
        mine, a, b = list(mine), -1, -1
        if mine and (i, True) in holders[mine[-1]] and not (all(w for _, w in holders[mine[-1]]) and min(holders[mine[-1]])[0] == i):
            a, b = mine[-1], next(free)
            mine[-1] = b
        mine += [next(free) for _ in range(-(-new_lens[i] // page) - len(mine))]
        out.append(mine + [-1] * (width - len(mine)))
        src.append(a)
        dst.append(b)
    r = {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in (("table", out), ("src", src), ("dst", dst))}
    return {**r, **_exact_pages(s, [(b, a) for a, b in zip(src, dst) if a >= 0])}


def _exact_compact(s):
    page, rows = s["page"], s["page_table"].tolist()
    mine = [row[: -(-n // page)] for row, n in zip(rows, s["lens"].tolist())]
    used = sorted({e for row in mine for e in row})
    count = len(used)
    among = set(used)
    holes = [p for p in range(count) if p not in among]
    to = dict(zip([p for p in used if p >= count], holes))
    none = [-1] * (s["pages"] // 2 - len(to))
    r = {"table": [[to.get(e, e) for e in row] + [-1] * (len(rows[0]) - len(row)) for row in mine], "src": list(to) + none, "dst": list(to.values()) + none,
         "count": [len(to), count]}
    r = {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in r.items()}
    return {**r, **_exact_pages(s, [(b, a) for a, b in to.items()])}


def exact(case, seed):
    s = prepare(case, seed)
    page, block, heads = case["page"], case.get("block"), case["kv_heads"]
    if case["op"] == "fork":
        return _exact_fork(s)
    if case["op"] == "compact":
        return _exact_compact(s)

    def rows(name, plane, slots, head):
        """The rows at `slots` of a cache, of one head or of all."""
        x = s[name].flatten(0, 1)[slots][:, head].double()
        return x if s["scales"] is None else x * s["scales"].flatten(0, 1)[slots][:, head, plane].double().unsqueeze(-1)

    if case["op"] == "bounds":
        bounds = s["bounds"].double()
        for table, start, end in zip(s["page_table"].long(), s["start"].tolist(), s["end"].tolist()):
            for at in range(start // block * block, end, 4096 * block):  # some thousand blocks at a time
                pos = torch.arange(at, min(at + 4096 * block, end), device="cuda")
                x = rows("k_cache", 0, table[pos // page] * page + pos % page, slice(None))
                fill = -len(pos) % block
                x = torch.cat((x, x[-1:].expand(fill, -1, -1))).unflatten(0, (-1, block))  # (the last row again changes neither)
                first = pos[::block]
                bounds[table[first // page], first % page // block, :, 0] = x.min(1).values
                bounds[table[first // page], first % page // block, :, 1] = x.max(1).values
        return {"bounds": bounds}

    q = s["q"].double()
    batch, width, q_heads, dim = q.shape
    group = q_heads // heads
    if case["op"] == "scores":
        n = s["page_table"].shape[1] * (page // block)
        out = torch.full((batch, width, heads, n), -math.inf, dtype=torch.float64, device="cuda")
        row_len = -(-s["kv_len"] // block)
        for b in range(batch):
            number = torch.arange(int(row_len[b].max()), device="cuda")
            table = s["page_table"][b].long()
            mine = s["bounds"][table[number * block // page], number % (page // block)].double()  # [blocks, heads, 2, dim]
            step = max(1, 300_000_000 // (len(number) * dim * group))
            for h in range(heads):
                low, high = mine[:, h, 0], mine[:, h, 1]
                for t in range(0, width, step):
                    x = q[b, t : t + step, h * group : (h + 1) * group].unsqueeze(2)  # [tokens, group, 1, dim]
                    y = torch.maximum(x * low, x * high).sum(-1).amax(1)  # [tokens, blocks]
                    out[b, t : t + step, h, : len(number)] = torch.where(number < row_len[b, t : t + step].unsqueeze(1), y, -math.inf)
        return {"scores": out, "row_len": row_len.unsqueeze(-1).repeat(1, 1, heads).to(torch.int32)}

    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for b in range(batch):
        table = s["page_table"][b].long()
        for t in range(width):
            limit = int(s["kv_len"][b, t])
            for h in range(heads):
                mine = s["blocks"][b, t, h]
                pos = (mine[mine >= 0].long().unsqueeze(1) * block + torch.arange(block, device="cuda")).flatten()
                pos = pos[pos < limit]
                slots = table[pos // page] * page + pos % page
                x = q[b, t, h * group : (h + 1) * group] @ rows("k_cache", 0, slots, h).T * s["softmax_scale"]
                lse[b, t, h * group : (h + 1) * group] = torch.logsumexp(x, -1)
                out[b, t, h * group : (h + 1) * group] = torch.softmax(x, -1) @ rows("v_cache", 1, slots, h)
    return {"out": out, "lse": lse}


def work(case):
    op, heads, dim, page = case["op"], case["kv_heads"], case["dim"], case["page"]
    if op in ("fork", "compact"):
        held = _BYTES[case["held"]]
        one = page * heads * (2 * dim * held + (8 if case["held"] == "int8" else 0)) + 4 * heads * dim  # a page's keys, values, scales and bounds
        if op == "compact":
            used = _used(case)
            total = sum(used)
            moves = total * (case["pages"] - total) // case["pages"]
            return {"bytes": 2 * moves * one + 4 * (total + len(used) * (max(used) + 2) + 2 * (case["pages"] // 2) + 2), "flops": total}
        lengths = _lengths(case)
        copies = sum(case["beams"] - case["survivors"] for n in lengths if n % page)
        need = [-(-n // page) for n in lengths]
        rows = case["beams"] * len(lengths)
        entries = case["survivors"] * sum(need) + rows * (max(need) + 1)
        return {"bytes": 2 * copies * one + 4 * (entries + 5 * rows), "flops": entries}
    block, lengths = case["block"], _lengths(case)
    if op == "bounds":
        row = dim * _BYTES[case["held"]] + (4 if case["held"] == "int8" else 0)
        first = [max(0, n - case["new"]) // block * block for n in lengths]
        keys, blocks = sum(n - f for n, f in zip(lengths, first)), sum(-(-n // block) - f // block for n, f in zip(lengths, first))
        return {"bytes": heads * (keys * row + blocks * 4 * dim) + 4 * (blocks * block // page + 3 * case["batch"]), "flops": 3 * heads * keys * dim}
    width, q_heads = case["queries"], case["q_heads"]
    seen = [[n - width + 1 + t for t in range(width)] for n in lengths]
    if op == "scores":
        blocks = sum(-(-n // block) for n in lengths)
        pairs = sum(-(-n // block) for e in seen for n in e)
        columns = max(-(-n // page) for n in lengths) * (page // block)
        ends = case["batch"] * width * (2 * q_heads * dim + heads * (4 * columns + 4) + 4)
        return {"bytes": blocks * heads * 4 * dim + ends + 4 * sum(-(-n // page) for n in lengths), "flops": 4 * dim * q_heads * pairs}
    row = 2 * (dim * _BYTES[case["held"]] + (4 if case["held"] == "int8" else 0))
    each = [[min(case["chosen"] * block, n) for n in e] for e in seen]
    keys = sum(min(sum(e), n) for e, n in zip(each, lengths))  # each position that is chosen at all, once
    ends = case["batch"] * width * (q_heads * (4 * dim + 4) + 4 * heads * case["chosen"] + 4)
    return {"bytes": keys * heads * row + ends + 4 * sum(-(-n // page) for n in lengths), "flops": 4 * dim * q_heads * sum(map(sum, each))}

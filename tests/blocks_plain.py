"""Plain implementations of the block and page operators: 64-bit scores, and page
tables one entry at a time. Written from the definitions, without the package."""

import math

import torch

BF16_MAX = torch.finfo(torch.bfloat16).max


def bounds_of(keys, block):
    """keys [n, heads, dim] in 32 bits, of one sequence from its start: bfloat16 [blocks, heads, 2, dim]."""
    out = []
    for at in range(0, keys.shape[0], block):
        x = keys[at : at + block]
        out.append(torch.stack((x.amin(0), x.amax(0)), 1))  # (a NaN goes through both)
    return torch.stack(out).clamp(-BF16_MAX, BF16_MAX).to(torch.bfloat16)


def scores_of(q, bounds):
    """q [heads of a group, dim], bounds [blocks, 2, dim]: the scores, and the sum of magnitudes that their error is relative to."""
    q, lo, hi = q.double().unsqueeze(1), bounds[:, 0].double(), bounds[:, 1].double()
    each = torch.maximum(q * lo, q * hi)
    size = (q.abs() * torch.maximum(lo.abs(), hi.abs())).sum(-1).amax(0)
    x = each.sum(-1)
    bad = x.isnan().any(0)
    return torch.where(bad, math.inf, torch.nan_to_num(x, nan=-math.inf, posinf=math.inf, neginf=-math.inf).amax(0)), size


def fork(table, lens, parents, new_lens, pages, page, keep=None):
    """Returns (table, src, dst, status bits: "row_len", "index", "no_page")."""
    width = len(table[0]) if table else 0
    room, status = width * page, set()

    def held(n):
        r = min(max(n, 0), room)
        if r != n:
            status.add("row_len")
        return r

    kept = []
    for p, wanted in zip(parents, new_lens):
        wanted = held(wanted)
        had, row = 0, []
        if 0 <= p < len(lens):
            had, row = held(lens[p]), table[p]
        elif p >= 0:
            status.add("index")
        n = min(had, wanted)
        mine = list(row[: -(-n // page)])
        kept.append((n, wanted, mine, n % page != 0 and wanted > n))
        if any(not 0 <= e < pages for e in mine):
            status.add("index")
    holders = {}
    for i, (_, _, mine, writes) in enumerate(kept):
        for j, e in enumerate(mine):
            if 0 <= e < pages:
                holders.setdefault(e, []).append((i, writes and j == len(mine) - 1))
    pinned = {p for p in range(pages) if keep is not None and keep[p]}
    free = [p for p in range(pages) if p not in holders and p not in pinned]

    def take():
        if free:
            return free.pop(0)
        status.add("no_page")
        return -1

    out, src, dst = [], [], []
    for i, (n, wanted, mine, writes) in enumerate(kept):
        a = b = -1
        if writes and 0 <= mine[-1] < pages:
            who = holders[mine[-1]]
            if mine[-1] in pinned or not (all(w for _, w in who) and min(who)[0] == i):
                b = take()
                a = mine[-1] if b >= 0 else -1
                mine[-1] = b
        mine += [take() for _ in range(-(-wanted // page) - len(mine))]
        out.append(mine + [-1] * (width - len(mine)))
        src.append(a)
        dst.append(b)
    return out, src, dst, status


def compact(table, lens, pages, page, keep=None):
    """Returns (table, src, dst, [moves, used], status)."""
    width = len(table[0]) if table else 0
    status, mine = set(), []
    for row, n in zip(table, lens):
        r = min(max(n, 0), width * page)
        if r != n:
            status.add("row_len")
        mine.append(list(row[: -(-r // page)]))
        if any(not 0 <= e < pages for e in mine[-1]):
            status.add("index")
    pinned = {p for p in range(pages) if keep is not None and keep[p]}
    used = {e for row in mine for e in row if 0 <= e < pages} | pinned
    n = len(used)
    moves = dict(zip([p for p in range(n, pages) if p in used and p not in pinned], [p for p in range(n) if p not in used]))
    none = [-1] * (pages // 2 - len(moves))
    out = [[moves.get(e, e) for e in row] + [-1] * (width - len(row)) for row in mine]
    return out, list(moves) + none, list(moves.values()) + none, [len(moves), n], status

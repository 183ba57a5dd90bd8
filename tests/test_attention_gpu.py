"""Tree attention and attention over selected positions, against plain implementations in 64 bits."""

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402
from tests.attention_plain import PagedCache, check_rows  # noqa: E402


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert tks.device_status() == tks.TKS_OK


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand_rows(n, heads, dim, g):
    return torch.randn(n, heads, dim, device="cuda", generator=g) * torch.exp(0.7 * torch.randn(n, heads, 1, device="cuda", generator=g))


def random_parents(batch, drafts, g):
    return (torch.rand(batch, drafts, device="cuda", generator=g) * (torch.arange(drafts, device="cuda") + 1)).long() - 1


def ancestors(parents):
    """bool [drafts, drafts] of one sequence, by walking up."""
    t = len(parents)
    a = torch.zeros(t, t, dtype=torch.bool)
    for i in range(t):
        j = i
        while j >= 0:
            a[i, j] = True
            j = parents[j]
    return a


def tree_case(ctx, drafts, q_heads, kv_heads, dim, held, page, layout="tokens", tree="random", counts=None, seed=0, scale=None,
              spread=1.5, room=1):
    g = gen(seed)
    batch = len(ctx)
    counts = [drafts] * batch if counts is None else counts
    lens = [c + d for c, d in zip(ctx, counts)]
    pages = sum(-(-n // page) for n in lens) + 2
    cache = PagedCache(pages, page, kv_heads, dim, held, layout, seed)
    width = max(1, max(-(-n // page) for n in lens) + room)  # (`room`: columns of the page table without a page)
    tables, held_rows = [], []
    for n in lens:
        t, k, v = cache.fill(rand_rows(n, kv_heads, dim, g), rand_rows(n, kv_heads, dim, g), width)
        tables.append(t)
        held_rows.append((k, v))
    q = (spread * torch.randn(batch, drafts, q_heads, dim, device="cuda", generator=g)).to(torch.bfloat16)
    parents = random_parents(batch, drafts, g)
    bits = tks.tree_mask(parents) if tree == "random" else None
    scale = dim ** -0.5 if scale is None else scale
    dl = torch.tensor(counts, dtype=torch.int32, device="cuda")
    out, lse = tks.tree_attention(q, cache.k, cache.v, torch.stack(tables), torch.tensor(ctx, dtype=torch.int32, device="cuda"), tree=bits,
                                  draft_len=dl, scales=cache.scales, softmax_scale=scale, return_lse=True)
    group = q_heads // kv_heads
    for b in range(batch):
        up = ancestors(parents[b].tolist()) if tree == "random" else torch.ones(drafts, drafts).tril().bool()
        seen = torch.zeros(drafts, lens[b], dtype=torch.bool)
        seen[:, : ctx[b]] = True
        seen[:, ctx[b] :] = up[:, : counts[b]]
        seen[counts[b] :] = False
        seen = seen.cuda().repeat_interleave(group, 0)
        for h in range(kv_heads):
            hs = slice(h * group, (h + 1) * group)
            k, v = held_rows[b][0][:, h], held_rows[b][1][:, h]
            check_rows(out[b, :, hs].reshape(-1, dim), lse[b, :, hs].reshape(-1), q[b, :, hs].reshape(-1, dim).double(), k, v, seen, scale, held)
    return out, lse


HELD = ["int8", "bf16"]


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("ctx", [0, 1, 14, 15, 16, 47, 62, 63, 64, 127, 128, 1000])
def test_one_token(ctx, dim, held):
    tree_case([ctx], 1, 8, 2, dim, held, 16, seed=ctx)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("q_heads, kv_heads", [(1, 1), (3, 1), (8, 8), (6, 2), (14, 2), (32, 2), (34, 2), (64, 1), (130, 1)])
def test_head_layouts(q_heads, kv_heads, held):
    tree_case([300, 5], 1, q_heads, kv_heads, 128, held, 32, seed=q_heads)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("drafts", [2, 3, 7, 16, 31, 33, 64, 100])
def test_trees(drafts, dim, held):
    tree_case([130, 0, 777], drafts, 8, 2, dim, held, 16, seed=drafts)


@pytest.mark.parametrize("held", HELD)
def test_many_drafts_of_a_wide_group(held):
    tree_case([2000, 129], 64, 16, 2, 128, held, 64, seed=3)
    tree_case([70], 300, 4, 2, 64, held, 64, seed=4)


@pytest.mark.parametrize("held", HELD)
def test_chain_without_a_mask(held):
    tree_case([50, 3], 9, 4, 2, 128, held, 16, tree=None)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("page", [1, 2, 8, 16, 64, 1024])
@pytest.mark.parametrize("layout", ["tokens", "heads", "side by side"])
def test_pages_and_layouts(layout, page, held):
    tree_case([333, 70], 5, 6, 3, 64, held, page, layout=layout, seed=page)
    tree_case([333, 70], 9, 32, 4, 128, held, page, layout=layout, seed=page)


@pytest.mark.parametrize("held", HELD)
def test_ragged_batch_and_draft_counts(held):
    tree_case([0, 1, 5000, 63, 64, 65, 0, 812], 6, 8, 2, 128, held, 16, counts=[6, 0, 3, 1, 6, 2, 0, 5])
    tree_case([0, 1, 5000, 63, 64, 65, 0, 812], 40, 8, 1, 64, held, 16, counts=[40, 0, 3, 1, 33, 2, 0, 39])


@pytest.mark.parametrize("held", HELD)
def test_more_sequences_than_a_warp(held):
    tree_case([(37 * i) % 301 for i in range(75)], 2, 4, 1, 64, held, 16)


@pytest.mark.parametrize("held", HELD)
def test_long_contexts_are_split(held):
    tree_case([50003], 1, 8, 1, 128, held, 64)
    tree_case([30011, 17], 8, 16, 1, 64, held, 64)
    tree_case([30011], 20, 16, 1, 128, held, 64)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("drafts, heads, kv_heads", [(1, 8, 2), (3, 4, 4), (30, 8, 2), (70, 4, 2)])
def test_page_tables_with_room_to_spare(drafts, heads, kv_heads, held):
    """Short sequences that could be long: blocks split by the lengths on the device."""
    tree_case([700, 0, 33, 1, 450], drafts, heads, kv_heads, 64, held, 16, counts=[drafts, drafts, 0, 1, drafts], room=2000)
    tree_case([130], drafts, heads, kv_heads, 128, held, 16, room=2000)


@pytest.mark.parametrize("held", HELD)
def test_more_units_than_blocks(held):
    tree_case([(61 * i) % 200 for i in range(90)], 1, 8, 4, 64, held, 16, room=600)
    tree_case([(61 * i) % 200 for i in range(45)], 9, 16, 4, 64, held, 16)
    tree_case([3000, 5] + [1] * 60, 9, 8, 4, 64, held, 64, room=300)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_softmax_scales(scale, held):
    tree_case([200], 3, 4, 2, 64, held, 16, scale=scale, spread=0.5)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("spread", [1e-6, 30.0])
def test_small_and_large_queries(spread, held):
    tree_case([500], 3, 4, 1, 128, held, 16, spread=spread)
    tree_case([500], 30, 4, 1, 128, held, 16, spread=spread)


@pytest.mark.parametrize("held", HELD)
def test_a_row_that_sees_nothing(held):
    """No context, and a mask without a bit for some rows."""
    g = gen(1)
    for drafts, heads in ((4, 4), (40, 8)):
        cache = PagedCache(8, 16, 1, 128, held)
        table, k, v = cache.fill(rand_rows(drafts, 1, 128, g), rand_rows(drafts, 1, 128, g))
        q = torch.randn(1, drafts, heads, 128, device="cuda", generator=g).to(torch.bfloat16)
        bits = torch.ones(1, drafts, (drafts + 31) // 32, dtype=torch.int32, device="cuda")  # bit 0 of each word
        bits[0, 1::2] = 0
        out, lse = tks.tree_attention(q, cache.k, cache.v, table[None], torch.zeros(1, dtype=torch.int32, device="cuda"), tree=bits,
                                      scales=cache.scales, return_lse=True)
        seen = torch.zeros(drafts, drafts, dtype=torch.bool, device="cuda")
        seen[0::2, 0::32] = True
        check_rows(out[0].reshape(-1, 128), lse[0].reshape(-1), q[0].reshape(-1, 128).double(), k[:, 0], v[:, 0],
                   seen.repeat_interleave(heads, 0), 128 ** -0.5, held)
        assert (lse[0, 1::2] == -math.inf).all()


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("drafts, heads", [(5, 2), (5, 32), (37, 8)])
def test_masked_drafts_have_no_influence(drafts, heads, what, held):
    """Siblings of one parent: each sees only itself, and one of them is poisoned."""
    g = gen(2)
    ctx = 100
    cache = PagedCache(16, 16, 1, 64, held)
    table, k, v = cache.fill(rand_rows(ctx + drafts, 1, 64, g), rand_rows(ctx + drafts, 1, 64, g))
    q = torch.randn(1, drafts, heads, 64, device="cuda", generator=g).to(torch.bfloat16)
    bad = 3
    pg, tok = table[(ctx + bad) // 16].item(), (ctx + bad) % 16
    if held == "int8":
        cache.scales[pg, tok] = what
    else:
        cache.k[pg, tok, 0, 7] = what
        cache.v[pg, tok, 0, 9] = what
    bits = tks.tree_mask(torch.full((1, drafts), -1, dtype=torch.int64, device="cuda"))
    out, lse = tks.tree_attention(q, cache.k, cache.v, table[None], torch.tensor([ctx], dtype=torch.int32, device="cuda"), tree=bits,
                                  scales=cache.scales, return_lse=True)
    seen = torch.cat([torch.ones(drafts, ctx, dtype=torch.bool), torch.eye(drafts).bool()], 1).cuda()
    good = [i for i in range(drafts) if i != bad]
    k[ctx + bad] = v[ctx + bad] = 0.0
    check_rows(out[0, good].reshape(-1, 64), lse[0, good].reshape(-1), q[0, good].reshape(-1, 64).double(), k[:, 0], v[:, 0],
               seen[good].repeat_interleave(heads, 0), 64 ** -0.5, held)
    if math.isnan(what):
        assert out[0, bad].isnan().any(-1).all() and lse[0, bad].isnan().all()


@pytest.mark.parametrize("heads", [4, 40])
def test_infinite_values_reach_the_rows_that_attend(heads):
    g = gen(3)
    cache = PagedCache(16, 16, 1, 64, "bf16")
    table, k, v = cache.fill(rand_rows(60, 1, 64, g), rand_rows(60, 1, 64, g))
    for pos, d, x in ((10, 3, math.inf), (58, 5, -math.inf), (59, 6, math.nan)):  # one in the context, two among the drafts
        cache.v[table[pos // 16], pos % 16, 0, d] = x
    q = 0.1 * torch.randn(1, 4, heads, 64, device="cuda", generator=g)
    out = tks.tree_attention(q.to(torch.bfloat16), cache.k, cache.v, table[None], torch.tensor([56], dtype=torch.int32, device="cuda"))
    assert (out[..., 3] == math.inf).all()
    assert (out[0, 2:, :, 5] == -math.inf).all() and out[0, :2, :, 5].isfinite().all()
    assert out[0, 3, :, 6].isnan().all() and out[0, :3, :, 6].isfinite().all()


@pytest.mark.parametrize("held", HELD)
def test_a_nan_query_touches_only_its_rows(held):
    g = gen(4)
    for drafts, heads in ((2, 4), (16, 16)):
        cache = PagedCache(16, 16, 1, 128, held)
        table, k, v = cache.fill(rand_rows(100, 1, 128, g), rand_rows(100, 1, 128, g))
        q = torch.randn(1, drafts, heads, 128, device="cuda", generator=g).to(torch.bfloat16)
        q[0, 1, 2, 5] = math.nan
        out, lse = tks.tree_attention(q, cache.k, cache.v, table[None], torch.tensor([100 - drafts], dtype=torch.int32, device="cuda"),
                                      scales=cache.scales, return_lse=True)
        assert out[0, 1, 2].isnan().all() and lse[0, 1, 2].isnan()
        out[0, 1, 2] = 0
        assert not out.isnan().any()


@pytest.mark.parametrize("held", HELD)
def test_rows_of_very_different_scales(held):
    """Values of one token far larger than the rest, and a dominant token with tiny values (an attention sink)."""
    g = gen(5)
    for heads in (4, 48):
        cache = PagedCache(64, 16, 1, 64, held)
        k, v = rand_rows(400, 1, 64, g), rand_rows(400, 1, 64, g)
        v[7] *= 1e6
        v[0] *= 1e-6
        q = torch.randn(1, 1, heads, 64, device="cuda", generator=g)
        k[0, 0] = 8 * q[0, 0, 0]
        k[7] *= 0.01
        table, kh, vh = cache.fill(k, v)
        q = q.to(torch.bfloat16)
        out, lse = tks.tree_attention(q, cache.k, cache.v, table[None], torch.tensor([399], dtype=torch.int32, device="cuda"),
                                      scales=cache.scales, return_lse=True)
        check_rows(out[0, 0], lse[0, 0], q[0, 0].double(), kh[:, 0], vh[:, 0], torch.ones(heads, 400, dtype=torch.bool, device="cuda"), 0.125, held)


def test_offsets_beyond_32_bits():
    """A cache whose last pages lie more than 2^32 bytes behind its first."""
    g = gen(6)
    page, heads, dim = 64, 8, 128
    pages = (1 << 32) // (page * heads * dim) + 64
    k = torch.empty((pages, page, heads, dim), dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    scales = torch.empty((pages, page, heads, 2), device="cuda")
    n = 700
    table = (pages - 1 - torch.arange(-(-n // page), device="cuda")).to(torch.int32)
    table[3] = 5
    pos = torch.arange(n, device="cuda")
    slots = (table[pos // page].long() * page + pos % page).to(torch.int32)
    ks, vs = (rand_rows(n, heads, dim, g).to(torch.bfloat16) for _ in range(2))
    tks.cache_write(ks, vs, k, v, slots, scales=scales)
    kh, vh = (x.double() for x in tks.cache_read(k, v, slots, scales=scales, dtype=torch.float32))
    assert (kh - ks.double()).abs().max() < 0.51 * ks.abs().max() / 127 * 1.01
    for q_heads in (16, 192):
        q = torch.randn(1, 1, q_heads, dim, device="cuda", generator=g).to(torch.bfloat16)
        out, lse = tks.tree_attention(q, k, v, table[None], torch.tensor([n - 1], dtype=torch.int32, device="cuda"), scales=scales, return_lse=True)
        idx = torch.randperm(n, device="cuda", generator=g)[:300].to(torch.int32)
        sel, slse = tks.selected_attention(q, k, v, table[None], idx.view(1, 1, -1), scales=scales, return_lse=True)
        group = q_heads // heads
        for h in range(heads):
            hs = slice(h * group, (h + 1) * group)
            ones = torch.ones(group, n, dtype=torch.bool, device="cuda")
            check_rows(out[0, 0, hs], lse[0, 0, hs], q[0, 0, hs].double(), kh[:, h], vh[:, h], ones, dim ** -0.5, "int8")
            check_rows(sel[0, 0, hs], slse[0, 0, hs], q[0, 0, hs].double(), kh[idx.long(), h], vh[idx.long(), h], ones[:, :300], dim ** -0.5, "int8")


# ---------------------------------------------------------------------------
# Selected positions
# ---------------------------------------------------------------------------


def selected_case(lens, tokens, k, q_heads, kv_heads, dim, held, page, layout="tokens", seed=0, fill=1.0, limit=True):
    g = gen(seed)
    batch = len(lens)
    cache = PagedCache(sum(-(-n // page) for n in lens) + 2, page, kv_heads, dim, held, layout, seed)
    width = max(1, max(-(-n // page) for n in lens))
    tables, rows = [], []
    for n in lens:
        t, kk, vv = cache.fill(rand_rows(n, kv_heads, dim, g), rand_rows(n, kv_heads, dim, g), width)
        tables.append(t)
        rows.append((kk, vv))
    q = torch.randn(batch, tokens, q_heads, dim, device="cuda", generator=g).to(torch.bfloat16)
    idx = torch.full((batch, tokens, k), -1, dtype=torch.int32, device="cuda")
    for b in range(batch):
        for t in range(tokens):
            take = min(lens[b], int(k * fill))
            at = torch.randperm(k, device="cuda", generator=g)[:take]
            idx[b, t, at] = torch.randperm(max(lens[b], 1), device="cuda", generator=g)[:take].to(torch.int32)
    out, lse = tks.selected_attention(q, cache.k, cache.v, torch.stack(tables), idx,
                                      kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda") if limit else None,
                                      scales=cache.scales, return_lse=True)
    group = q_heads // kv_heads
    for b in range(batch):
        for t in range(tokens):
            at = idx[b, t][idx[b, t] >= 0].long()
            for h in range(kv_heads):
                hs = slice(h * group, (h + 1) * group)
                check_rows(out[b, t, hs], lse[b, t, hs], q[b, t, hs].double(), rows[b][0][at, h], rows[b][1][at, h],
                           torch.ones(group, len(at), dtype=torch.bool, device="cuda"), dim ** -0.5, held)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("k", [1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 300, 2048])
def test_selected_list_lengths(k, dim, held):
    selected_case([4096], 1, k, 8, 2, dim, held, 64, seed=k)
    selected_case([4096], 2, k, 64, 1, dim, held, 64, seed=k)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("q_heads, kv_heads", [(1, 1), (5, 1), (16, 1), (17, 1), (32, 8), (64, 2), (128, 1), (129, 1), (300, 1)])
def test_selected_head_layouts(q_heads, kv_heads, held):
    selected_case([500, 77], 2, 100, q_heads, kv_heads, 128, held, 16, seed=q_heads)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("layout", ["tokens", "heads", "side by side"])
@pytest.mark.parametrize("page", [1, 4, 64])
def test_selected_pages_and_layouts(page, layout, held):
    selected_case([200, 333], 3, 90, 4, 2, 64, held, page, layout=layout)
    selected_case([200, 333], 3, 90, 64, 2, 128, held, page, layout=layout)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("q_heads", [4, 64])
def test_selected_padding_and_short_rows(q_heads, held):
    """-1 among the entries, rows with fewer positions than k, and rows with none."""
    selected_case([3, 0, 400], 2, 200, q_heads, 1, 64, held, 16, fill=0.6)
    selected_case([3, 0, 400], 2, 200, q_heads, 1, 64, held, 16, limit=False)


@pytest.mark.parametrize("held", HELD)
def test_selected_many_tokens(held):
    selected_case([1000], 100, 64, 8, 1, 64, held, 16)
    selected_case([1000], 60, 200, 64, 1, 128, held, 16)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("q_heads, kv_heads", [(4, 2), (40, 1)])
def test_selected_long_lists_and_many_units(q_heads, kv_heads, held):
    selected_case([12000], 1, 9001, q_heads, kv_heads, 64, held, 64)
    selected_case([12000, 700], 2, 5000, q_heads, kv_heads, 128, held, 64)
    selected_case([300], 170, 70, q_heads, kv_heads, 64, held, 16)


@pytest.mark.parametrize("q_heads", [4, 64])
def test_positions_listed_twice_count_twice(q_heads):
    g = gen(9)
    cache = PagedCache(8, 16, 1, 64, "bf16")
    table, k, v = cache.fill(rand_rows(50, 1, 64, g), rand_rows(50, 1, 64, g))
    q = torch.randn(1, 1, q_heads, 64, device="cuda", generator=g).to(torch.bfloat16)
    at = torch.tensor([3, 3, 3, 17, 44, 17], device="cuda")
    out, lse = tks.selected_attention(q, cache.k, cache.v, table[None], at.to(torch.int32).view(1, 1, -1), return_lse=True)
    check_rows(out[0, 0], lse[0, 0], q[0, 0].double(), k[at, 0], v[at, 0], torch.ones(q_heads, 6, dtype=torch.bool, device="cuda"), 0.125, "bf16")


def test_no_entries_no_queries_no_sequences():
    cache = PagedCache(2, 16, 1, 64, "bf16")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    q = torch.ones(1, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = tks.selected_attention(q, cache.k, cache.v, table, torch.empty(1, 2, 0, dtype=torch.int32, device="cuda"), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    empty = torch.empty(1, 0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert tks.tree_attention(empty, cache.k, cache.v, table, torch.zeros(1, dtype=torch.int32, device="cuda")).shape == empty.shape
    none = torch.empty(0, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert tks.tree_attention(none, cache.k, cache.v, table[:0], torch.zeros(0, dtype=torch.int32, device="cuda")).shape == none.shape
    no_table = torch.empty(1, 0, dtype=torch.int32, device="cuda")
    out = tks.tree_attention(q, cache.k, cache.v, no_table, torch.zeros(1, dtype=torch.int32, device="cuda"),
                             draft_len=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert (out == 0).all()


# ---------------------------------------------------------------------------
# How they are called
# ---------------------------------------------------------------------------


def _small(held="int8", heads=8, drafts=3, ctx=100, seed=0):
    g = gen(seed)
    cache = PagedCache(16, 16, 2, 64, held, seed=seed)
    table, k, v = cache.fill(rand_rows(ctx + drafts, 2, 64, g), rand_rows(ctx + drafts, 2, 64, g))
    q = torch.randn(1, drafts, heads, 64, device="cuda", generator=g).to(torch.bfloat16)
    return cache, table[None], q, torch.tensor([ctx], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("heads", [8, 64])
def test_strided_queries(heads):
    cache, table, q, ctx = _small(heads=heads)
    want = tks.tree_attention(q, cache.k, cache.v, table, ctx, scales=cache.scales)
    fused = torch.randn(1, 3, 3 * heads, 64, device="cuda").to(torch.bfloat16)
    fused[:, :, heads : 2 * heads] = q
    assert torch.equal(tks.tree_attention(fused[:, :, heads : 2 * heads], cache.k, cache.v, table, ctx, scales=cache.scales), want)
    odd = torch.randn(1, 3, heads, 67, device="cuda").to(torch.bfloat16)  # rows that start anywhere
    odd[..., 1:65] = q
    assert torch.equal(tks.tree_attention(odd[..., 1:65], cache.k, cache.v, table, ctx, scales=cache.scales), want)
    out = torch.empty_like(q)
    assert tks.tree_attention(q, cache.k, cache.v, table, ctx, scales=cache.scales, out=out) is out and torch.equal(out, want)


@pytest.mark.parametrize("heads", [8, 64])
def test_streams_graphs_and_repeats_agree(heads):
    cache, table, q, ctx = _small(heads=heads)
    want = tks.tree_attention(q, cache.k, cache.v, table, ctx, scales=cache.scales)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = tks.tree_attention(q, cache.k, cache.v, table, ctx, scales=cache.scales, stream=s)
    b = tks.tree_attention(q, cache.k, cache.v, table, ctx, scales=cache.scales, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c = tks.tree_attention(q, cache.k, cache.v, table, ctx, scales=cache.scales)
    for _ in range(3):
        c.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want)
    assert tks.device_status(s) == tks.TKS_OK


def test_calls_of_mixed_shapes_back_to_back():
    """One stream's workspace, reused across shapes and kernels without waiting between."""
    cases = []
    for i, (held, heads, drafts, ctx) in enumerate([("int8", 8, 3, 100), ("bf16", 2, 1, 200), ("int8", 64, 8, 30), ("bf16", 64, 2, 150), ("int8", 4, 1, 0)]):
        cache, table, q, c = _small(held, heads, drafts, ctx, seed=i)
        cases.append((q, cache.k, cache.v, table, c, cache.scales))
    call = lambda x: tks.tree_attention(*x[:5], scales=x[5])  # noqa: E731
    want = []
    for x in cases:
        want.append(call(x))
        torch.cuda.synchronize()
    for _ in range(5):
        got = [call(x) for x in cases]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("heads", [4, 64])
def test_positions_outside_the_cache_are_skipped_and_reported(heads):
    cache, table, q, ctx = _small("bf16", heads=heads)
    idx = torch.tensor([5, 6, 99], dtype=torch.int32, device="cuda").view(1, 1, -1).expand(1, 3, 3).contiguous()
    want = tks.selected_attention(q, cache.k, cache.v, table, idx)
    more = torch.tensor([5, 103, 6, -7, 99, 2 ** 31 - 1, 120], dtype=torch.int32, device="cuda").view(1, 1, -1).expand(1, 3, 7).contiguous()
    n = torch.tensor([103], dtype=torch.int32, device="cuda")
    got = tks.selected_attention(q, cache.k, cache.v, table, more, kv_len=n)
    assert tks.device_status() == tks.TKS_E_INDEX and tks.device_status() == tks.TKS_OK
    assert torch.allclose(got.float(), want.float(), rtol=2 ** -6, atol=2 ** -6)
    # pages outside the cache
    bad = table.clone()
    bad[0, 0], bad[0, 2] = 16, -1
    got = tks.tree_attention(q, cache.k, cache.v, bad, ctx)
    assert tks.device_status() == tks.TKS_E_INDEX
    keep = [p for p in range(103) if p // 16 not in (0, 2)]
    for t in range(3):
        at = torch.tensor([p for p in keep if p <= 100 + t], dtype=torch.int32, device="cuda").view(1, 1, -1)
        want = tks.selected_attention(q[:, t : t + 1], cache.k, cache.v, table, at)
        assert torch.allclose(got[:, t : t + 1].float(), want.float(), rtol=2 ** -6, atol=2 ** -6)


def test_lengths_out_of_range_are_held_and_reported():
    cache, table, q, ctx = _small("bf16")
    full = torch.tensor([table.shape[1] * 16], dtype=torch.int32, device="cuda")
    got = tks.tree_attention(q, cache.k, cache.v, table, full + 5)
    assert tks.device_status() == tks.TKS_E_ROW_LEN
    assert (got == 0).all()  # no room for a draft, so no query
    got = tks.tree_attention(q, cache.k, cache.v, table, ctx, draft_len=torch.tensor([9], dtype=torch.int32, device="cuda"))
    assert tks.device_status() == tks.TKS_E_ROW_LEN
    assert torch.equal(got, tks.tree_attention(q, cache.k, cache.v, table, ctx))
    tks.tree_attention(q, cache.k, cache.v, table, ctx - 200)
    assert tks.device_status() == tks.TKS_E_ROW_LEN


def test_refusals():
    cache, table, q, ctx = _small("int8")
    ok = dict(scales=cache.scales)
    idx = torch.zeros(1, 3, 4, dtype=torch.int32, device="cuda")
    tree = lambda **k: tks.tree_attention(**{**dict(q=q, k_cache=cache.k, v_cache=cache.v, page_table=table, ctx_len=ctx, **ok), **k})  # noqa: E731
    sel = lambda **k: tks.selected_attention(**{**dict(q=q, k_cache=cache.k, v_cache=cache.v, page_table=table, indices=idx, **ok), **k})  # noqa: E731
    tree(), sel()
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q=q[..., :32]), dict(q=q[:, :, :7]), dict(q=q.cpu()), dict(scales=None),
                dict(scales=cache.scales.double()), dict(k_cache=cache.k.float(), v_cache=cache.v.float()), dict(v_cache=cache.v[:3]),
                dict(k_cache=cache.k[:, :12], v_cache=cache.v[:, :12], scales=cache.scales[:, :12]), dict(page_table=table.long()),
                dict(page_table=table[0]), dict(softmax_scale=math.inf), dict(out=q.float()), dict(out=q[:, :2])):
        for call in (tree, sel):
            with pytest.raises(ValueError):
                call(**bad)
    for bad in (dict(ctx_len=ctx.long()), dict(ctx_len=ctx.cpu()), dict(draft_len=ctx.repeat(2)), dict(tree=torch.zeros(1, 3, 2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            tree(**bad)
    for bad in (dict(indices=idx[0]), dict(indices=idx.long()), dict(indices=idx[:, :2]), dict(kv_len=ctx.long())):
        with pytest.raises(ValueError):
            sel(**bad)
    with pytest.raises(ValueError):
        many = torch.zeros(1, tks.TKS_DRAFTS_MAX + 1, 8, 64, dtype=torch.bfloat16, device="cuda")
        tks.tree_attention(many, cache.k, cache.v, table, ctx, scales=cache.scales)


@pytest.mark.parametrize("held", HELD)
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_sound(held):
    """The lookups of each block's first tile are never announced, so its other warps' waits run out."""
    cache, table, q, ctx = _small(held, heads=64)
    want = tks.tree_attention(q, cache.k, cache.v, table, ctx, scales=cache.scales)
    assert tks.device_status() == tks.TKS_OK
    tks.set_option(tks.TKS_OPT_SPIN_LIMIT_NS, 20_000_000)
    tks.set_option(tks.TKS_OPT_TEST_SKIP_ARRIVE, 1)
    try:
        tks.tree_attention(q, cache.k, cache.v, table, ctx, scales=cache.scales)
        assert tks.device_status() == tks.TKS_E_TIMEOUT
    finally:
        tks.set_option(tks.TKS_OPT_TEST_SKIP_ARRIVE, 0)
        tks.set_option(tks.TKS_OPT_SPIN_LIMIT_NS, 1_000_000_000)
    assert torch.equal(tks.tree_attention(q, cache.k, cache.v, table, ctx, scales=cache.scales), want)

"""Bounds of blocks, scores and attention over selected blocks, against plain implementations in 64 bits."""

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402
from tests.attention_plain import PagedCache, check_rows  # noqa: E402
from tests.blocks_plain import BF16_MAX, bounds_of, scores_of  # noqa: E402

HELD = ["int8", "bf16"]


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert tks.device_status() == tks.TKS_OK


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(lens, page, heads, dim, held, layout="tokens", seed=0, room=1):
    """A cache with sequences of these lengths, its page table, and each one's keys and values in 64 bits."""
    g = gen(seed)
    cache = PagedCache(sum(-(-n // page) for n in lens) + 2, page, heads, dim, held, layout, seed)
    width = max(1, max(-(-n // page) for n in lens) + room)
    tables, rows = [], []
    for n in lens:
        k, v = (torch.randn(n, heads, dim, device="cuda", generator=g) * torch.exp(0.7 * torch.randn(n, heads, 1, device="cuda", generator=g)) for _ in range(2))
        t, *kv = cache.fill(k, v, width)
        tables.append(t)
        rows.append(kv)
    return cache, torch.stack(tables), rows


def keys_of(cache, table, n):
    """The keys of a sequence's first n positions, in 32 bits, as a cache stands for them."""
    pos = torch.arange(n, device="cuda")
    pg, tok = table[pos // cache.page].long(), pos % cache.page
    x = cache.k[pg, tok].float()
    return x if cache.scales is None else x * cache.scales[pg, tok, :, 0].unsqueeze(-1)


def new_bounds(cache, block, value=math.nan):
    pages, page, heads, dim = cache.k.shape
    return torch.full((pages, page // block, heads, 2, dim), value, dtype=torch.bfloat16, device="cuda")


def sequence_bounds(bounds, table, page, blocks):
    """The bounds of a sequence's first blocks: [blocks, heads, 2, dim]."""
    of_page = bounds.shape[1]
    j = torch.arange(blocks, device="cuda")
    return bounds[table[j // of_page].long(), j % of_page]


# ---------------------------------------------------------------------------
# Bounds
# ---------------------------------------------------------------------------


def check_bounds(cache, table, lens, starts, block, bounds, before):
    """Blocks of [start, end) are exact; all others as they were."""
    left = torch.ones(bounds.shape[:2], dtype=torch.bool, device="cuda")
    of_page = bounds.shape[1]
    for b, (a, n) in enumerate(zip(starts, lens)):
        if a >= n:
            continue
        want = bounds_of(keys_of(cache, table[b], n), block)
        j = torch.arange(a // block, -(-n // block), device="cuda")
        pg, at = table[b][j // of_page].long(), j % of_page
        assert torch.equal(bounds[pg, at].float(), want[j].float())
        left[pg, at] = False
    assert torch.equal(bounds[left].view(torch.int16), before[left].view(torch.int16))


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page, block", [(1, 1), (4, 2), (16, 16), (64, 8), (64, 64), (128, 32), (256, 256)])
def test_bounds(page, block, dim, held):
    lens = [1, 200, page, block + 1, 777]
    cache, table, _ = filled(lens, page, 3, dim, held, seed=page)
    for starts in (None, [0, 199, page - 1, block, 300], [1, 13, 0, 0, 776]):
        bounds = new_bounds(cache, block, 7.0)
        before = bounds.clone()
        tks.cache_bounds(cache.k, table, ints(lens), bounds, start=None if starts is None else ints(starts), scales=cache.scales)
        check_bounds(cache, table, lens, starts or [0] * len(lens), block, bounds, before)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("layout", ["heads", "side by side"])
def test_bounds_of_other_layouts(layout, held):
    lens = [77, 300]
    cache, table, _ = filled(lens, 32, 2, 128, held, layout)
    bounds = new_bounds(cache, 16)
    tks.cache_bounds(cache.k, table, ints(lens), bounds, scales=cache.scales)
    check_bounds(cache, table, lens, [0, 0], 16, bounds, bounds.clone())


@pytest.mark.parametrize("held", HELD)
def test_bounds_token_by_token_are_those_of_the_whole(held):
    lens = [0, 5]
    cache, table, _ = filled([40, 45], 16, 2, 64, held)
    whole, steps = new_bounds(cache, 8, 0.0), new_bounds(cache, 8, 0.0)
    for n in range(1, 41):
        tks.cache_bounds(cache.k, table, ints([lens[0] + n, lens[1] + n]), steps, start=ints([lens[0] + n - 1, lens[1] + n - 1 if n > 1 else 0]), scales=cache.scales)
    tks.cache_bounds(cache.k, table, ints([40, 45]), whole, scales=cache.scales)
    assert torch.equal(whole, steps)


def test_bounds_of_many_ragged_sequences():
    lens = [(97 * i) % 61 for i in range(700)]
    starts = [(13 * i) % 70 for i in range(700)]
    cache, table, _ = filled(lens, 16, 1, 64, "int8")
    bounds = new_bounds(cache, 8, 1.0)
    before = bounds.clone()
    tks.cache_bounds(cache.k, table, ints(lens), bounds, start=ints(starts), scales=cache.scales)
    check_bounds(cache, table, lens, starts, 8, bounds, before)


def test_bounds_of_infinities_and_nans():
    cache, table, _ = filled([40], 16, 1, 64, "bf16")
    slot = lambda i: (table[0][i // 16].long(), i % 16)  # noqa: E731
    for i, d, x in ((3, 0, math.inf), (5, 1, -math.inf), (20, 2, math.nan), (21, 3, 3.3895e38), (39, 4, math.nan)):
        cache.k[slot(i)][0, d] = x
    bounds = new_bounds(cache, 8)
    tks.cache_bounds(cache.k, table, ints([40]), bounds)
    got = sequence_bounds(bounds, table[0], 16, 5)[:, 0].float()
    want = bounds_of(keys_of(cache, table[0], 40), 8)[:, 0].float()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
    assert got[0, 1, 0] == BF16_MAX and got[0, 0, 1] == -BF16_MAX and got[2, :, 2].isnan().all() and got.isnan().sum() == 4
    cache, table, _ = filled([40], 16, 2, 64, "int8")
    cache.scales[table[0][1].long(), 9, 1, 0] = math.nan  # a whole row of one head: position 25
    bounds = new_bounds(cache, 8)
    tks.cache_bounds(cache.k, table, ints([40]), bounds, scales=cache.scales)
    bad = sequence_bounds(bounds, table[0], 16, 5).isnan()
    assert bad[3, 1].all() and bad.sum() == 2 * 64


def test_bounds_of_wrong_lengths_and_pages():
    cache, table, _ = filled([40, 40], 16, 1, 64, "int8", room=0)
    bounds = new_bounds(cache, 8, 5.0)
    before = bounds.clone()
    tks.cache_bounds(cache.k, table, ints([10 ** 6, -4]), bounds, start=ints([30, -9]), scales=cache.scales)  # the first is held to 48
    assert tks.device_status() == tks.TKS_E_ROW_LEN
    assert torch.equal(bounds[table[1].long()], before[table[1].long()])
    assert (sequence_bounds(bounds, table[0], 16, 6)[3:5] != 5.0).any()
    wrong = table.clone()
    wrong[0, 1], wrong[1, 2] = cache.k.shape[0], -1
    tks.cache_bounds(cache.k, wrong, ints([40, 40]), bounds, scales=cache.scales)
    assert tks.device_status() == tks.TKS_E_INDEX
    for b, there in ((0, [0, 1, 4]), (1, [0, 1, 2, 3])):
        want = bounds_of(keys_of(cache, table[b], 40), 8)
        got = sequence_bounds(bounds, table[b], 16, 5)
        assert all(torch.equal(got[j].float(), want[j].float()) for j in there)


# ---------------------------------------------------------------------------
# Scores
# ---------------------------------------------------------------------------


def score_case(seen, tokens, q_heads, kv_heads, dim, page, block, seed=0, first=0, last=0, n=None, width=None, spread=1.0):
    """seen: for each sequence, the last token's length (the token before sees one less), or a list of lengths."""
    g = gen(seed)
    kv = [x if isinstance(x, list) else [max(0, x - tokens + 1 + t) for t in range(tokens)] for x in seen]
    of_page = page // block
    need = [-(-max(x) // page) for x in kv]
    pages = sum(need) + 3
    width = max(1, max(need)) + 1 if width is None else width
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(kv), width), -1, dtype=torch.int32, device="cuda")
    bounds = torch.full((pages, of_page, kv_heads, 2, dim), math.nan, dtype=torch.bfloat16, device="cuda")
    at = 0
    for b, x in enumerate(need):
        table[b, :x] = order[at : at + x]
        at += x
        j = torch.arange(-(-max(kv[b]) // block), device="cuda")
        a, c = (spread * torch.randn(len(j), kv_heads, dim, device="cuda", generator=g) for _ in range(2))
        bounds[table[b][j // of_page].long(), j % of_page] = torch.stack((torch.minimum(a, c), torch.maximum(a, c)), 2).to(torch.bfloat16)
    q = torch.randn(len(kv), tokens, q_heads, dim, device="cuda", generator=g).to(torch.bfloat16)
    scores, row_len = tks.block_scores(q, bounds, table, ints(kv), block, first=first, last=last, n=n)
    columns = width * of_page if n is None else n
    assert scores.shape == (len(kv), tokens, kv_heads, columns) and row_len.shape == scores.shape[:3]
    group = q_heads // kv_heads
    worst = 0.0
    for b in range(len(kv)):
        blocks = -(-max(kv[b]) // block)
        mine = sequence_bounds(bounds, table[b], page, blocks)
        for t in range(tokens):
            vis = -(-kv[b][t] // block)
            assert (row_len[b, t] == vis).all()
            assert (scores[b, t, :, vis:] == -math.inf).all()
            for h in range(kv_heads):
                want, size = scores_of(q[b, t, h * group : (h + 1) * group], mine[:, h])
                got = scores[b, t, h, :vis].double()
                forced = torch.zeros(vis, dtype=torch.bool, device="cuda")
                forced[:first] = True
                forced[max(0, vis - last) :] = True
                assert (got[forced] == math.inf).all()
                # 2 * dim products, exact in 32 bits, added one after the other in at most 2^-23 of their magnitudes each
                worst = max([worst] + ((got - want[:vis]).abs() / (2 * dim * 2.0 ** -23 * size[:vis] + 1e-30))[~forced].tolist())
    assert worst <= 1.0, f"scores off by {worst:.2f} of their bound"
    return scores, row_len


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length", [1, 7, 8, 9, 63, 64, 255, 256, 257, 1025, 5000])
def test_scores_of_one_token(length, dim):
    score_case([length], 1, 8, 2, dim, 16, 8, seed=length)


@pytest.mark.parametrize("q_heads, kv_heads", [(1, 1), (3, 1), (8, 8), (14, 2), (16, 1), (17, 1), (34, 2), (64, 1), (130, 1), (300, 1)])
@pytest.mark.parametrize("tokens", [1, 3])
def test_score_heads(q_heads, kv_heads, tokens):
    score_case([300, 20], tokens, q_heads, kv_heads, 128, 32, 16, seed=q_heads)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens", [2, 5, 16, 17, 33, 100, 131])
def test_scores_of_chunks(tokens, dim):
    score_case([200, tokens, 1000], tokens, 8, 2, dim, 16, 8, seed=tokens)


@pytest.mark.parametrize("tokens, q_heads, kv_heads", [(130, 16, 2), (257, 4, 4), (65, 6, 2), (40, 7, 1), (300, 1, 1)])
def test_scores_of_long_chunks(tokens, q_heads, kv_heads):
    score_case([4000, 513], tokens, q_heads, kv_heads, 128, 64, 16, seed=tokens)


@pytest.mark.parametrize("page, block", [(1, 1), (8, 2), (64, 64), (256, 32), (16, 1)])
def test_score_pages(page, block):
    score_case([333, 70], 2, 6, 3, 64, page, block, seed=page)
    score_case([333, 70], 20, 6, 3, 64, page, block, seed=page)


@pytest.mark.parametrize("tokens, q_heads", [(3, 4), (40, 8)])
def test_score_lengths_in_no_order_and_empty(tokens, q_heads):
    score_case([[(37 * t + 11 * b) % 400 if t % 3 else 0 for t in range(tokens)] for b in range(3)] + [[0] * tokens], tokens, q_heads, 2, 128, 32, 16)


@pytest.mark.parametrize("tokens, q_heads", [(2, 4), (70, 8)])
@pytest.mark.parametrize("first, last", [(1, 1), (0, 2), (3, 0), (1000, 0), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_first_and_last_blocks_are_forced(first, last, tokens, q_heads):
    score_case([300, [1] * tokens], tokens, q_heads, 2, 64, 16, 8, first=first, last=last)


@pytest.mark.parametrize("tokens, q_heads", [(1, 4), (50, 8)])
@pytest.mark.parametrize("n", [38, 39, 40, 61])
def test_rows_shorter_than_the_table(n, tokens, q_heads):
    score_case([300], tokens, q_heads, 2, 64, 16, 8, n=n, width=40)
    score_case([100], tokens, q_heads, 2, 64, 16, 8, width=2000)  # a table with room for much more


@pytest.mark.parametrize("tokens, q_heads", [(1, 4), (50, 8)])
@pytest.mark.parametrize("spread", [1e-6, 1e4])
def test_scores_of_small_and_large_bounds(spread, tokens, q_heads):
    score_case([300], tokens, q_heads, 2, 64, 16, 8, spread=spread)


@pytest.mark.parametrize("tokens, q_heads", [(1, 4), (50, 8)])
def test_score_lengths_that_do_not_fit(tokens, q_heads):
    g = gen(3)
    bounds = torch.randn(4, 2, 2, 2, 64, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(1, tokens, q_heads, 64, device="cuda", generator=g).to(torch.bfloat16)
    table = ints([[3, 1, 0, 2]])
    good, n_good = tks.block_scores(q, bounds, table, ints([[64] * tokens]), 8)
    many, n_many = tks.block_scores(q, bounds, table, ints([[65] * tokens]), 8)
    assert tks.device_status() == tks.TKS_E_ROW_LEN and torch.equal(good, many) and torch.equal(n_good, n_many)
    none, n_none = tks.block_scores(q, bounds, table, ints([[-5] * tokens]), 8)
    assert tks.device_status() == tks.TKS_E_ROW_LEN and (none == -math.inf).all() and (n_none == 0).all()
    all_, n_all = tks.block_scores(q, bounds, table, None, 8)
    assert torch.equal(good, all_) and torch.equal(n_all, n_good)
    short, n_short = tks.block_scores(q, bounds, table, None, 8, n=5)
    assert torch.equal(good[..., :5], short) and (n_short == 5).all()
    wrong, _ = tks.block_scores(q, bounds, ints([[3, 4, -1, 2]]), ints([[64] * tokens]), 8)
    assert tks.device_status() == tks.TKS_E_INDEX
    assert (wrong[..., 2:6] == -math.inf).all() and torch.equal(wrong[..., [0, 1, 6, 7]], good[..., [0, 1, 6, 7]])
    hidden, _ = tks.block_scores(q, bounds, ints([[3, 4, -1, 2]]), ints([[10] * tokens]), 8)  # (beyond what the tokens see)
    assert torch.equal(hidden[..., :2], good[..., :2])


@pytest.mark.parametrize("tokens, q_heads", [(1, 4), (50, 8), (1, 40)])
def test_scores_that_are_no_numbers_are_picked(tokens, q_heads):
    g = gen(4)
    bounds = torch.randn(4, 2, 2, 2, 64, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(1, tokens, q_heads, 64, device="cuda", generator=g).to(torch.bfloat16)
    table = ints([[0, 1, 2, 3]])
    good, _ = tks.block_scores(q, bounds, table, None, 8)
    bounds[1, 1, 0, 1, 17] = math.nan  # block 3 of head 0
    got, _ = tks.block_scores(q, bounds, table, None, 8)
    assert (got[:, :, 0, 3] == math.inf).all()
    rest = torch.ones_like(got, dtype=torch.bool)
    rest[:, :, 0, 3] = False
    assert torch.equal(got[rest], good[rest])
    q[0, 0, 1, 5] = math.nan  # one query head, of head 0
    got, _ = tks.block_scores(q, bounds, table, None, 8)
    assert (got[0, 0, 0] == math.inf).all() and torch.equal(got[0, 1:, 1], good[0, 1:, 1]) and torch.equal(got[0, 0, 1], good[0, 0, 1])


@pytest.mark.parametrize("tokens, q_heads, kv_heads", [(3, 40, 1), (2, 257, 1), (9, 100, 2), (20, 128, 1), (7, 129, 1)])
def test_scores_of_wide_groups_in_chunks(tokens, q_heads, kv_heads):
    score_case([300, 20], tokens, q_heads, kv_heads, 64, 32, 16, seed=tokens, first=1)


def test_scores_of_many_tiles():
    """More tiles of tokens than are counted before the work is split, and several tiles of blocks for each."""
    g = gen(12)
    bounds = torch.randn(300, 1, 1, 2, 64, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(30, 300, 8, 64, device="cuda", generator=g).to(torch.bfloat16)
    table = torch.randint(300, (30, 200), device="cuda", generator=g).to(torch.int32)
    lens = torch.randint(0, 1601, (30, 300), device="cuda", generator=g).to(torch.int32)
    scores, seen = tks.block_scores(q, bounds, table, lens, 8)
    assert torch.equal(seen[..., 0], (lens + 7) // 8)
    for b in (0, 13, 29):
        lo, hi = (bounds[table[b].long(), 0, 0, i].double() for i in (0, 1))
        x = q[b].double()
        want = (x.clamp(min=0) @ hi.T + x.clamp(max=0) @ lo.T).amax(1)
        size = (x.abs() @ torch.maximum(lo.abs(), hi.abs()).T).amax(1)
        there = torch.arange(200, device="cuda") < seen[b]
        assert (scores[b, :, 0][~there] == -math.inf).all()
        assert ((scores[b, :, 0].double() - want).abs() <= 128 * 2.0 ** -23 * size)[there].all()


def test_a_wait_that_runs_out_is_reported():
    """(Of the kernel for many rows: a warp does not say that it has read the first tile.)"""
    g = gen(13)
    bounds = torch.randn(50, 1, 1, 2, 64, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(1, 40, 8, 64, device="cuda", generator=g).to(torch.bfloat16)
    table = torch.randint(50, (1, 128 * 1000), device="cuda", generator=g).to(torch.int32)  # six tiles or more a thread block
    want, _ = tks.block_scores(q, bounds, table, None, 8)
    assert tks.device_status() == tks.TKS_OK
    tks.set_option(tks.TKS_OPT_SPIN_LIMIT_NS, 20_000_000)
    tks.set_option(tks.TKS_OPT_TEST_SKIP_ARRIVE, 1)
    try:
        tks.block_scores(q, bounds, table, None, 8)
        assert tks.device_status() == tks.TKS_E_TIMEOUT
    finally:
        tks.set_option(tks.TKS_OPT_TEST_SKIP_ARRIVE, 0)
        tks.set_option(tks.TKS_OPT_SPIN_LIMIT_NS, 1_000_000_000)
    assert torch.equal(want, tks.block_scores(q, bounds, table, None, 8)[0])


def test_scores_bound_every_product():
    lens = [500, 61]
    cache, table, rows = filled(lens, 32, 2, 64, "bf16")
    bounds = new_bounds(cache, 16)
    tks.cache_bounds(cache.k, table, ints(lens), bounds)
    q = torch.randn(2, 1, 8, 64, device="cuda", generator=gen(1)).to(torch.bfloat16)
    scores, seen = tks.block_scores(q, bounds, table, ints([[n] for n in lens]), 16)
    for b, n in enumerate(lens):
        for h in range(8):
            x = rows[b][0][:, h // 4] @ q[b, 0, h].double()
            for j in range(seen[b, 0, 0]):
                assert x[16 * j : 16 * j + 16].max() <= scores[b, 0, h // 4, j] + 1e-4


def test_scores_of_strided_queries_and_tables():
    g = gen(9)
    bounds = torch.randn(40, 2, 2, 2, 64, device="cuda", generator=g).to(torch.bfloat16)
    fused = torch.randn(2, 3, 24, 64, device="cuda", generator=g).to(torch.bfloat16)
    table = torch.randint(40, (2, 30), device="cuda", generator=g).to(torch.int32)
    lens = ints([[100, 101, 102], [7, 8, 9]])
    a = tks.block_scores(fused[:, :, 8:16], bounds, table[:, 3:17], lens, 8)
    b = tks.block_scores(fused[:, :, 8:16].contiguous(), bounds, table[:, 3:17].contiguous(), lens, 8)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    out = torch.empty_like(a[0])
    assert tks.block_scores(fused[:, :, 8:16], bounds, table[:, 3:17], lens, 8, out=out)[0] is out and torch.equal(out, a[0])
    odd = torch.zeros(2, 3, 8, 67, dtype=torch.bfloat16, device="cuda")
    odd[..., 1:65] = fused[:, :, 8:16]
    assert torch.equal(tks.block_scores(odd[..., 1:65], bounds, table[:, 3:17], lens, 8)[0], out)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------


def attend_case(seen, tokens, q_heads, kv_heads, dim, held, page, block, chosen, layout="tokens", seed=0, lists=None, scale=None):
    g = gen(seed + 100)
    kv = [x if isinstance(x, list) else [max(0, x - tokens + 1 + t) for t in range(tokens)] for x in seen]
    lens = [max(x) for x in kv]
    cache, table, rows = filled(lens, page, kv_heads, dim, held, layout, seed)
    q = (1.5 * torch.randn(len(kv), tokens, q_heads, dim, device="cuda", generator=g)).to(torch.bfloat16)
    if lists is None:
        lists = torch.full((len(kv), tokens, kv_heads, chosen), -1, dtype=torch.int32, device="cuda")
        for b in range(len(kv)):
            for t in range(tokens):
                n = -(-kv[b][t] // block)
                for h in range(kv_heads):
                    x = torch.randperm(n, device="cuda", generator=g)[:chosen]
                    at = torch.randperm(chosen, device="cuda", generator=g)[: len(x)]
                    lists[b, t, h, at] = x.to(torch.int32)
    scale = dim ** -0.5 if scale is None else scale
    out, lse = tks.block_attention(q, cache.k, cache.v, table, lists, block, kv_len=ints(kv), scales=cache.scales, softmax_scale=scale, return_lse=True)
    group = q_heads // kv_heads
    for b in range(len(kv)):
        for t in range(tokens):
            for h in range(kv_heads):
                x = lists[b, t, h]
                pos = (x[x >= 0].long().unsqueeze(1) * block + torch.arange(block, device="cuda")).flatten()
                pos = pos[pos < kv[b][t]]
                hs = slice(h * group, (h + 1) * group)
                check_rows(out[b, t, hs], lse[b, t, hs], q[b, t, hs].double(), rows[b][0][pos, h], rows[b][1][pos, h],
                           torch.ones(group, len(pos), dtype=torch.bool, device="cuda"), scale, held)
    return out, lse


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length", [1, 15, 16, 17, 100, 1000])
def test_block_attention_of_one_token(length, dim, held):
    attend_case([length], 1, 8, 2, dim, held, 16, 16, 5, seed=length)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("q_heads, kv_heads", [(1, 1), (8, 8), (14, 2), (32, 2), (34, 2), (64, 1), (130, 1), (12, 3)])
def test_block_attention_heads(q_heads, kv_heads, held):
    attend_case([300, 20], 2, q_heads, kv_heads, 128, held, 32, 16, 7, seed=q_heads)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("page, block", [(1, 1), (16, 1), (1, 16), (16, 64), (64, 8), (64, 128), (256, 32), (8, 2)])
@pytest.mark.parametrize("layout", ["tokens", "heads", "side by side"])
def test_block_attention_pages_and_layouts(layout, page, block, held):
    """(Blocks of attention need not go with the pages.)"""
    attend_case([333, 70], 2, 6, 3, 64, held, page, block, max(2, 100 // block), layout=layout, seed=page)
    attend_case([333, 70], 2, 40, 2, 128, held, page, block, max(2, 100 // block), layout=layout, seed=page)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("q_heads, kv_heads", [(8, 2), (48, 2)])
def test_block_attention_of_chunks(q_heads, kv_heads, held):
    attend_case([400, 37], 37, q_heads, kv_heads, 64, held, 16, 16, 6)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("q_heads", [4, 40])
def test_long_lists(q_heads, held):
    attend_case([30000], 1, q_heads, 2, 128, held, 64, 64, 300)
    attend_case([70000], 1, q_heads, 1, 64, held, 64, 64, 1100)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("q_heads", [4, 40])
def test_lists_without_a_block_and_lengths_of_zero(q_heads, held):
    lists = torch.full((2, 3, 2, 9), -1, dtype=torch.int32, device="cuda")
    lists[0, 0, 0, 4] = 2
    lists[0, 1, 1, 8] = 0
    lists[1, 2] = torch.arange(9, device="cuda")
    attend_case([[48, 5, 0], [0, 0, 144]], 3, q_heads, 2, 64, held, 16, 16, 9, lists=lists)
    attend_case([100], 1, q_heads, 2, 64, held, 16, 16, 0)
    attend_case([100], 1, q_heads, 2, 64, held, 16, 16, 3, lists=torch.full((1, 1, 2, 3), -2 ** 31, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("q_heads", [4, 40])
def test_a_block_listed_twice_counts_twice(q_heads, held):
    attend_case([100], 1, q_heads, 2, 128, held, 16, 16, 4, lists=ints([[[[3, 3, 0, -1], [6, 6, 6, 6]]]]))


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("q_heads", [4, 40])
def test_blocks_beyond_the_length_are_skipped_and_reported(q_heads, held):
    cache, table, _ = filled([100], 16, 1, 64, held)
    q = torch.randn(1, 1, q_heads, 64, device="cuda", generator=gen(5)).to(torch.bfloat16)
    call = lambda x, kv: tks.block_attention(q, cache.k, cache.v, table, ints([[[x]]]), 16, kv_len=ints([[kv]]), scales=cache.scales, return_lse=True)  # noqa: E731
    good = call([2, 0, -1, -1], 41)
    for wrong in ([2, 0, 3, -1], [2, 0, 2 ** 31 - 1, 2 ** 27], [2, 0, 2 ** 28, -1]):
        got = call(wrong, 41)
        assert tks.device_status() == tks.TKS_E_INDEX and all(torch.equal(a, b) for a, b in zip(good, got))
    assert (call([-1, -1, -1, -1], -3)[0] == 0).all() and tks.device_status() == tks.TKS_E_ROW_LEN
    whole = call([0, 1, 2, 3], 10 ** 6)
    assert tks.device_status() == tks.TKS_E_ROW_LEN
    assert all(torch.equal(a, b) for a, b in zip(whole, call([0, 1, 2, 3], 64)))
    none = tks.block_attention(q, cache.k, cache.v, table, ints([[[[0, 1, 2, 3]]]]), 16, scales=cache.scales, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(whole, none))


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("q_heads", [4, 40])
def test_what_lies_behind_the_length_has_no_influence(q_heads, held):
    cache, table, _ = filled([96], 16, 1, 64, held)
    q = torch.randn(1, 1, q_heads, 64, device="cuda", generator=gen(6)).to(torch.bfloat16)
    call = lambda: tks.block_attention(q, cache.k, cache.v, table, ints([[[[2, 5, 0]]]]), 16, kv_len=ints([[83]]), scales=cache.scales, return_lse=True)  # noqa: E731
    good = call()
    pg = table[0][5].long()
    for c in (cache.k, cache.v):
        c[pg, 3:] = math.nan if held == "bf16" else 127
    if held == "int8":
        cache.scales[pg, 3:] = math.nan
    assert all(torch.equal(a, b) for a, b in zip(good, call()))


@pytest.mark.parametrize("held", HELD)
def test_blocks_are_the_positions_they_stand_for(held):
    """The same bits as selected attention over the positions written out."""
    for q_heads in (8, 48):
        cache, table, _ = filled([640], 64, 2, 128, held)
        q = torch.randn(1, 1, q_heads, 128, device="cuda", generator=gen(7)).to(torch.bfloat16)
        blocks = ints([9, 3, 0, 7])
        a = tks.block_attention(q, cache.k, cache.v, table, blocks.expand(1, 1, 2, 4).contiguous(), 64, kv_len=ints([[640]]), scales=cache.scales, return_lse=True)
        pos = (blocks.unsqueeze(1) * 64 + torch.arange(64, dtype=torch.int32, device="cuda")).view(1, 1, -1)
        b = tks.selected_attention(q, cache.k, cache.v, table, pos, kv_len=ints([640]), scales=cache.scales, return_lse=True)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# ---------------------------------------------------------------------------
# All of them together, and what is refused
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("tokens, q_heads", [(1, 8), (40, 8), (1, 64)])
def test_write_bounds_scores_selection_attention(tokens, q_heads, held):
    """As a step makes the calls; with as many blocks as there are, it is attention over everything."""
    lens, page, block, heads, dim = [300, 45 + tokens, tokens], 32, 16, 2, 128
    cache, table, rows = filled(lens, page, heads, dim, held, room=0)
    bounds = new_bounds(cache, block)
    tks.cache_bounds(cache.k, table, ints(lens), bounds, scales=cache.scales)
    q = torch.randn(3, tokens, q_heads, dim, device="cuda", generator=gen(8)).to(torch.bfloat16)
    kv = ints([[n - tokens + 1 + t for t in range(tokens)] for n in lens])
    for n in (4, 20):
        scores, seen = tks.block_scores(q, bounds, table, kv, block, first=1, last=1)
        picked = tks.topk_indices(scores.flatten(0, 2), n, row_len=seen.flatten()).view(*seen.shape, n)
        out, lse = tks.block_attention(q, cache.k, cache.v, table, picked, block, kv_len=kv, scales=cache.scales, return_lse=True)
        assert tks.device_status() == tks.TKS_OK
        group = q_heads // heads
        for b in range(3):
            for t in range(tokens):
                count = int(seen[b, t, 0])
                for h in range(heads):
                    mine = picked[b, t, h]
                    mine = mine[mine >= 0].long()
                    assert len(mine) == min(n, count) and 0 in mine and count - 1 in mine
                    want = torch.topk(scores[b, t, h, :count], min(n, count)).values
                    assert torch.equal(scores[b, t, h][mine].sort().values, want.sort().values)
                    pos = (mine.unsqueeze(1) * block + torch.arange(block, device="cuda")).flatten()
                    pos = pos[pos < kv[b, t]]
                    hs = slice(h * group, (h + 1) * group)
                    check_rows(out[b, t, hs], lse[b, t, hs], q[b, t, hs].double(), rows[b][0][pos, h], rows[b][1][pos, h],
                               torch.ones(group, len(pos), dtype=torch.bool, device="cuda"), dim ** -0.5, held)


def test_streams_graphs_and_repeats():
    lens = [900, 61]
    cache, table, _ = filled(lens, 32, 2, 128, "int8")
    bounds, kv, q = new_bounds(cache, 16), ints([[n] for n in lens]), torch.randn(2, 1, 8, 128, device="cuda", generator=gen(2)).to(torch.bfloat16)

    def step(stream=None):
        tks.cache_bounds(cache.k, table, kv.view(-1), bounds, scales=cache.scales, stream=stream)
        scores, seen = tks.block_scores(q, bounds, table, kv, 16, last=1, stream=stream)
        picked = tks.topk_indices(scores.flatten(0, 2), 6, row_len=seen.flatten(), stream=stream, sorted=True).view(*seen.shape, 6)
        return scores, picked, tks.block_attention(q, cache.k, cache.v, table, picked, 16, kv_len=kv, scales=cache.scales, stream=stream)

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    bounds.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
        step(s.cuda_stream)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = step()
    for _ in range(3):
        bounds.zero_()
        for x in held:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))
    assert tks.device_status(s) == tks.TKS_OK


def test_nothing_to_do():
    cache, table, _ = filled([10], 16, 2, 64, "bf16")
    bounds = new_bounds(cache, 8)
    q = torch.empty(0, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, 1, dtype=torch.int32, device="cuda")
    tks.cache_bounds(cache.k, table[:0], none[:, 0], bounds)
    scores, seen = tks.block_scores(q, bounds, table[:0], none, 8)
    assert scores.shape == (0, 1, 2, 4) and seen.shape == (0, 1, 2)
    assert tks.block_attention(q, cache.k, cache.v, table[:0], torch.empty(0, 1, 2, 3, dtype=torch.int32, device="cuda"), 8, kv_len=none).shape == q.shape
    q = torch.randn(1, 1, 4, 64, device="cuda").to(torch.bfloat16)
    scores, seen = tks.block_scores(q, bounds, table, ints([[0]]), 8, n=0)
    assert scores.shape == (1, 1, 2, 0) and (seen == 0).all()
    scores, seen = tks.block_scores(q, bounds, table[:, :0], ints([[0]]), 8)
    assert scores.shape == (1, 1, 2, 0) and (seen == 0).all()


def test_refusals():
    cache, table, _ = filled([40], 16, 2, 64, "int8")
    bounds, end = new_bounds(cache, 8), ints([40])
    q, kv, lists = torch.randn(1, 1, 4, 64, device="cuda").to(torch.bfloat16), ints([[40]]), ints([[[[0, 1], [2, 3]]]])
    good_b = dict(k_cache=cache.k, page_table=table, end=end, bounds=bounds, start=None, scales=cache.scales)
    good_s = dict(q=q, bounds=bounds, page_table=table, kv_len=kv, block=8)
    good_a = dict(q=q, k_cache=cache.k, v_cache=cache.v, page_table=table, blocks=lists, block=8, kv_len=kv, scales=cache.scales)
    tks.cache_bounds(**good_b), tks.block_scores(**good_s), tks.block_attention(**good_a)
    for call, good, bads in (
            (tks.cache_bounds, good_b, [dict(scales=None), dict(page_table=table.long()), dict(page_table=table.cpu()), dict(page_table=table[0]),
                                        dict(page_table=table.t()), dict(end=end.long()), dict(end=ints([1, 2])), dict(start=ints([1, 2])),
                                        dict(bounds=bounds.float()), dict(bounds=bounds[1:]), dict(bounds=bounds[:, :, :1].contiguous()), dict(bounds=bounds[0]),
                                        dict(bounds=bounds.transpose(1, 2)), dict(bounds=bounds[..., :32].contiguous()), dict(end=None),
                                        dict(bounds=bounds.repeat(1, 16, 1, 1, 1)), dict(bounds=bounds.cpu())]),
            (tks.block_scores, good_s, [dict(q=q.float()), dict(q=q[0]), dict(q=q[..., :32]), dict(q=q[:, :, :3]), dict(q=q.cpu()), dict(kv_len=kv[0]),
                                        dict(kv_len=kv.long()), dict(block=0), dict(block=3), dict(block=-8), dict(first=-1), dict(last=-1), dict(n=99),
                                        dict(n=-1), dict(page_table=table.long()), dict(page_table=torch.cat((table, table))), dict(bounds=bounds.float()),
                                        dict(out=torch.empty(1, 1, 2, 7, device="cuda")), dict(block=1 << 31),
                                        dict(out=torch.empty(1, 1, 2, 2 * table.shape[1], device="cuda").double())]),
            (tks.block_attention, good_a, [dict(blocks=lists.long()), dict(blocks=lists[0]), dict(blocks=lists[:, :, :1].contiguous()), dict(block=0),
                                           dict(block=12), dict(block=1 << 24), dict(kv_len=end), dict(scales=None), dict(q=q.float()),
                                           dict(blocks=lists.cpu()), dict(softmax_scale=float("inf")), dict(out=q.float())])):
        for bad in bads:
            with pytest.raises((ValueError, tks.TksError)):
                call(**{**good, **bad})
    for bad in (dict(block="8"), dict(first=1.5), dict(n=2.0)):
        with pytest.raises(TypeError):
            tks.block_scores(**{**good_s, **bad})


# ---------------------------------------------------------------------------
# More blocks than the device scores at once (decode steps of batches)
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens, q_heads, kv_heads", [(1, 8, 1), (1, 32, 2), (1, 17, 1), (3, 10, 2), (16, 2, 2), (2, 16, 2)])
def test_scores_of_ragged_batches(tokens, q_heads, kv_heads, dim):
    g = gen(tokens + dim)
    batch, of_page, width = 70, 4, 300
    bounds = torch.randn(500, of_page, kv_heads, 2, dim, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(batch, tokens, q_heads, dim, device="cuda", generator=g).to(torch.bfloat16)
    table = torch.randint(500, (batch, width), device="cuda", generator=g).to(torch.int32)
    lens = torch.randint(0, width * of_page * 8 + 1, (batch, tokens), device="cuda", generator=g)
    lens[3], lens[4], lens[5], lens[-1] = 0, 1, width * of_page * 8, 64
    lens = lens.to(torch.int32)
    for first, last, n in ((0, 0, None), (2, 1, 1001)):
        cut = lens if n is None else lens.clamp(max=8 * n)
        scores, seen = tks.block_scores(q, bounds, table, cut, 8, first=first, last=last, n=n)
        columns = width * of_page if n is None else n
        count = (cut + 7) // 8
        assert torch.equal(seen, count.unsqueeze(-1).expand(-1, -1, kv_heads))
        group = q_heads // kv_heads
        j = torch.arange(columns, device="cuda")
        for b in (0, 3, 4, 5, 33, 69):
            mine = bounds[table[b][j // of_page].long(), j % of_page].double()
            for h in range(kv_heads):
                x = q[b, :, h * group : (h + 1) * group].double()
                lo, hi = mine[:, h, 0], mine[:, h, 1]
                want = (x.clamp(min=0) @ hi.T + x.clamp(max=0) @ lo.T).amax(1)
                size = (x.abs() @ torch.maximum(lo.abs(), hi.abs()).T).amax(1)
                vis = j < count[b].unsqueeze(1)
                forced = vis & ((j < first) | (j >= count[b].unsqueeze(1) - last))
                got = scores[b, :, h]
                assert (got[~vis] == -math.inf).all() and (got[forced] == math.inf).all()
                plain = vis & ~forced
                assert ((got.double() - want).abs() <= 2 * dim * 2.0 ** -23 * size)[plain].all()


def test_scores_of_more_sequences_than_are_counted():
    g = gen(21)
    bounds = torch.randn(90, 2, 1, 2, 64, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(1500, 1, 4, 64, device="cuda", generator=g).to(torch.bfloat16)
    table = torch.randint(90, (1500, 60), device="cuda", generator=g).to(torch.int32)
    lens = torch.randint(0, 961, (1500, 1), device="cuda", generator=g).to(torch.int32)
    many, seen = tks.block_scores(q, bounds, table, lens, 8)
    for at in range(0, 1500, 20):  # a few at a time, by the other kernel
        few, n = tks.block_scores(q[at : at + 20], bounds, table[at : at + 20], lens[at : at + 20], 8)
        assert torch.equal(seen[at : at + 20], n)
        a, b = many[at : at + 20], few
        assert torch.equal(a == -math.inf, b == -math.inf) and ((a - b).abs() <= 1e-4)[a != -math.inf].all()


def test_wrong_pages_and_numbers_among_many():
    g = gen(22)
    bounds = torch.randn(100, 2, 2, 2, 64, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(40, 1, 8, 64, device="cuda", generator=g).to(torch.bfloat16)
    table = torch.randint(1, 100, (40, 900), device="cuda", generator=g).to(torch.int32)
    lens = torch.full((40, 1), 14400, dtype=torch.int32, device="cuda")
    good, _ = tks.block_scores(q, bounds, table, lens, 8)
    wrong = table.clone()
    wrong[7, 450], wrong[9, 0], wrong[11, 899] = 100, -1, 2 ** 31 - 1
    got, _ = tks.block_scores(q, bounds, wrong, lens, 8)
    assert tks.device_status() == tks.TKS_E_INDEX
    bad = torch.zeros(40, 900, dtype=torch.bool, device="cuda")
    bad[7, 450] = bad[9, 0] = bad[11, 899] = True
    bad = bad.repeat_interleave(2, 1)[:, None, None].expand_as(good)
    assert (got[bad] == -math.inf).all() and torch.equal(got[~bad], good[~bad])
    bounds[0, 1, 1, 0, 5] = math.nan
    wrong[7, 450] = 0
    wrong[9, 0], wrong[11, 899] = table[9, 0], table[11, 899]
    got, _ = tks.block_scores(q, bounds, wrong, lens, 8)
    assert got[7, 0, 1, 901] == math.inf and got.isinf().sum() == 1
    many = lens.clone()
    many[3] = 14401
    got, seen = tks.block_scores(q, bounds, table, many, 8)
    assert tks.device_status() == tks.TKS_E_ROW_LEN and torch.equal(got, good) and (seen == 1800).all()


def test_scores_of_more_tiles_than_are_counted():
    g = gen(31)
    bounds = torch.randn(60, 1, 1, 2, 64, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(110, 330, 8, 64, device="cuda", generator=g).to(torch.bfloat16)
    table = torch.randint(60, (110, 150), device="cuda", generator=g).to(torch.int32)
    lens = torch.randint(0, 1201, (110, 330), device="cuda", generator=g).to(torch.int32)
    many, seen = tks.block_scores(q, bounds, table, lens, 8, first=1)
    for at in (0, 37, 100):
        few, n = tks.block_scores(q[at : at + 10], bounds, table[at : at + 10], lens[at : at + 10], 8, first=1)
        assert torch.equal(seen[at : at + 10], n) and torch.equal(many[at : at + 10], few)


def test_offsets_beyond_32_bits():
    """Pages at the far end of a cache, and of bounds, of more than 2^31 elements."""
    pages, page, heads, dim, block = 20_000, 64, 16, 128, 4
    k, v = (torch.empty((pages, page, heads, dim), dtype=torch.int8, device="cuda") for _ in range(2))
    scales = torch.empty((pages, page, heads, 2), device="cuda")
    bounds = torch.empty((pages, page // block, heads, 2, dim), dtype=torch.bfloat16, device="cuda")
    assert k.numel() > 2 ** 31 and bounds.numel() > 2 ** 30 and bounds.numel() * 2 > 2 ** 31
    g = gen(41)
    far = [pages - 1, pages - 2, pages - 3]
    for pg in far[:2] + [0, 1]:
        for c in (k, v):
            c[pg] = torch.randint(-127, 128, c.shape[1:], dtype=torch.int8, device="cuda", generator=g)
        scales[pg] = torch.rand(scales.shape[1:], device="cuda", generator=g) + 0.01
    table, lens = ints([far[:2], [0, 1]]), ints([100, 128])
    tks.cache_bounds(k, table, lens, bounds, scales=scales)
    values = lambda c, plane, pgs: c[pgs].flatten(0, 1).float() * scales[pgs].flatten(0, 1)[..., plane, None]  # noqa: E731
    for b, pgs in enumerate((far[:2], [0, 1])):
        n = int(lens[b])
        got = bounds[pgs].flatten(0, 1)[: n // block]
        assert torch.equal(got, bounds_of(values(k, 0, pgs)[:n], block))
    for tokens in (1, 20):  # few rows, and many
        q = torch.randn(2, tokens, 32, dim, device="cuda", generator=g).to(torch.bfloat16)
        kv = lens.unsqueeze(1).expand(2, tokens).contiguous()
        scores, seen = tks.block_scores(q, bounds, table, kv, block)
        picked = tks.topk_indices(scores.flatten(0, 2), 9, row_len=seen.flatten()).view(*seen.shape, 9)
        out, lse = tks.block_attention(q, k, v, table, picked, block, kv_len=kv, scales=scales, return_lse=True)
        for b, pgs in enumerate((far[:2], [0, 1])):
            for h in (0, 15):
                mine = bounds[pgs].flatten(0, 1)[: int(lens[b]) // block, h]
                want, size = scores_of(q[b, 0, 2 * h : 2 * h + 2], mine)
                assert ((scores[b, 0, h, : len(want)].double() - want).abs() <= 2 * dim * 2.0 ** -23 * size).all()
                pos = (picked[b, 0, h].long().unsqueeze(1) * block + torch.arange(block, device="cuda")).flatten()
                kk, vv = (values(c, plane, pgs)[pos, h].double() for c, plane in ((k, 0), (v, 1)))
                check_rows(out[b, 0, 2 * h : 2 * h + 2], lse[b, 0, 2 * h : 2 * h + 2], q[b, 0, 2 * h : 2 * h + 2].double(), kk, vv,
                           torch.ones(2, len(pos), dtype=torch.bool, device="cuda"), dim ** -0.5, "int8")
    tks.cache_copy(ints([far[0], 1]), ints([2, far[2]]), k, v, scales=scales, bounds=bounds)
    for c in (k, v, scales, bounds):
        assert torch.equal(c[2], c[far[0]]) and torch.equal(c[far[2]], c[1])

"""Forking, compacting and copying pages, against page tables made one entry at a time."""

import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402
from tests.attention_plain import PagedCache  # noqa: E402
from tests.blocks_plain import compact, fork  # noqa: E402

STATUS = {"row_len": tks.TKS_E_ROW_LEN, "index": tks.TKS_E_INDEX, "no_page": tks.TKS_E_NO_PAGE}


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert tks.device_status() == tks.TKS_OK


def ints(x, shape=None):
    t = torch.tensor(x, dtype=torch.int32, device="cuda")
    return t if shape is None else t.view(shape)


def expected(status):
    for name in ("no_page", "index", "row_len"):
        if name in status:
            return STATUS[name]
    return tks.TKS_OK


def check_fork(table, lens, parents, new_lens, pages, page, keep=None, table_dev=None, width=None):
    width = len(table[0]) if table else width or 0
    want = fork(table if table else [], lens, parents, new_lens, pages, page, keep)
    if not table:
        want = fork_from_nothing(parents, new_lens, pages, page, width, keep)
    dev = ints(table, (len(lens), width)) if table_dev is None else table_dev
    got = tks.cache_fork(dev, ints(lens, (len(lens),)), ints(parents, (len(parents),)), ints(new_lens, (len(parents),)), pages, page,
                         keep=None if keep is None else torch.tensor(keep, dtype=torch.bool, device="cuda"))
    assert got[0].tolist() == want[0]
    assert got[1].tolist() == want[1] and got[2].tolist() == want[2]
    assert tks.device_status() == expected(want[3])
    return want


def fork_from_nothing(parents, new_lens, pages, page, width, keep):
    """fork() for no sequences: a row of no entries stands in, and every parent is none."""
    want = fork([[-1] * width], [0], [p if p < 0 else 1 for p in parents], new_lens, pages, page, keep)
    return want


def pool(rng, sequences, width, pages, page, share=0.5):
    """A page table of sequences that share some of their first pages, as forks leave them; no page is partly filled by two."""
    order = list(range(pages))
    rng.shuffle(order)
    table, lens = [], []
    for s in range(sequences):
        n = rng.choice((0, 1, page, rng.randint(0, width * page), rng.randint(0, width * page)))
        row = []
        if table and rng.random() < share:
            other = rng.randrange(s)
            row = table[other][: rng.randint(0, min(lens[other], n) // page)]
        need = -(-n // page) - len(row)
        if need > len(order):
            n, need = len(row) * page, 0
        row = row + [order.pop() for _ in range(need)]
        table.append(row + [-1] * (width - len(row)))
        lens.append(n)
    return table, lens


@pytest.mark.parametrize("seed", range(30))
def test_random_forks(seed):
    rng = random.Random(seed)
    page, width = rng.choice((1, 2, 16, 64)), rng.choice((1, 5, 40, 300, 700))
    sequences, children = rng.choice((1, 3, 17, 90)), rng.choice((1, 4, 33, 150))
    pages = rng.choice((sequences * width // 4 + 3, sequences * width + children * width + 50))
    table, lens = pool(rng, sequences, width, pages, page)
    parents = [rng.choice((-1, rng.randrange(sequences), rng.randrange(sequences))) for _ in range(children)]
    new = []
    for p in parents:
        n = lens[p] if p >= 0 else 0
        new.append(min(width * page, rng.choice((n, n + 1, n + rng.randint(0, 3 * page), max(0, n - rng.randint(0, 3 * page)), rng.randint(0, width * page)))))
    keep = [rng.random() < 0.1 for _ in range(pages)] if seed % 3 == 0 else None
    check_fork(table, lens, parents, new, pages, page, keep)


def test_beams_share_what_is_full_and_copy_what_they_write_to():
    table, src, dst, status = check_fork([[5, 2, 9, -1], [7, 1, -1, -1]], [10, 8], [0, 0, 1, 0, 1], [11, 11, 9, 10, 9], 12, 4)
    # child 3 only reads page 9, so children 0 and 1 both copy it; a full page is shared
    assert table == [[5, 2, 0, -1], [5, 2, 3, -1], [7, 1, 4, -1], [5, 2, 9, -1], [7, 1, 6, -1]]
    assert src == [9, 9, -1, -1, -1] and dst == [0, 3, -1, -1, -1] and not status
    table, src, dst, _ = check_fork([[5, 2, 9, -1]], [10], [0, 0, 0], [11, 11, 11], 12, 4)
    assert table[0] == [5, 2, 9, -1] and src == [-1, 9, 9] and dst == [-1, 0, 1]


def test_ends_frees_and_starts():
    # sequence 1 has no child: its pages are the first to be handed out
    table, *_ = check_fork([[4, 5, -1], [0, 1, 2], [3, -1, -1]], [8, 12, 3], [2, 0, -1], [5, 9, 9], 7, 4)
    assert table == [[3, 0, -1], [4, 5, 1], [2, 6, -1]]


def test_cut_sequences_give_pages_back_and_do_not_write_to_what_is_shared():
    # two continue from one sequence: the first is cut in the middle of page 1, which the second has in full, and grows
    table, src, dst, _ = check_fork([[0, 1, 2, -1]], [12], [0, 0], [6, 16], 8, 4)
    assert table == [[0, 1, -1, -1], [0, 1, 2, 3]] and src == [-1, -1]
    table, src, dst, _ = check_fork([[0, 1, 2, -1]], [6], [0, 0], [7, 6], 8, 4)  # (the second does not write)
    assert src == [1, -1] and dst == [2, -1] and table == [[0, 2, -1, -1], [0, 1, -1, -1]]


def test_kept_pages_are_neither_given_nor_written_to():
    table, src, dst, _ = check_fork([[1, 3, -1]], [6], [0], [9], 8, 4, keep=[True, False, False, True, False, True, False, False])
    assert table == [[1, 2, 4]] and src == [3] and dst == [2]
    check_fork([[1, 3, -1]], [6], [0, 0], [9, 9], 8, 4, keep=[True] * 8)


def test_no_page_left():
    table, src, dst, status = check_fork([[0, 1, -1, -1]], [6], [0, 0, -1], [7, 16, 3], 4, 4)
    assert "no_page" in status and table == [[0, 1, -1, -1], [0, 2, 3, -1], [-1, -1, -1, -1]] and src == [-1, 1, -1]
    table, src, dst, status = check_fork([[0, 1]], [6], [0, 0], [7, 7], 2, 4)
    assert table == [[0, 1], [0, -1]] and src == dst == [-1, -1] and "no_page" in status
    check_fork([[0, 1]], [8], [0, 0], [8, 8], 2, 4)  # (none is wanted)


def test_wrong_lengths_parents_and_entries():
    check_fork([[0, 1], [2, 3]], [99, -3], [0, 1, 0], [9, 5, -7], 9, 4)
    check_fork([[0, 1], [2, 3]], [5, 7], [2, 0, 2 ** 31 - 1, -2 ** 31], [8, 6, 3, 8], 9, 4)
    check_fork([[0, 9], [-1, 3], [4, -5]], [5, 7, 8], [0, 0, 1, 2], [8, 6, 8, 8], 9, 4)


@pytest.mark.parametrize("children, width", [(1, 0), (5, 0), (3, 7)])
def test_no_sequences_or_no_entries(children, width):
    check_fork([], [], [-1] * children, [0] * children, 5, 4, width=width)
    if width:
        check_fork([], [], [-1, -1, 3], [9, 28, 3], 12, 4, width=width)


def test_many_children_and_pages():
    rng = random.Random(1)
    pages, width = 50_000, 30
    table, lens = pool(rng, 1200, width, pages, 4)
    parents = [rng.randrange(1200) for _ in range(3000)]
    check_fork(table, lens, parents, [min(width * 4, lens[p] + 1) for p in parents], pages, 4)


def test_tables_with_a_stride_and_given_outputs():
    rng = random.Random(2)
    table, lens = pool(rng, 9, 11, 200, 8)
    wide = torch.full((9, 20), -9, dtype=torch.int32, device="cuda")
    wide[:, 4:15] = ints(table)
    parents = [rng.randrange(9) for _ in range(14)]
    check_fork(table, lens, parents, [min(88, lens[p] + 1) for p in parents], 200, 8, table_dev=wide[:, 4:15])
    out = torch.empty(14, 11, dtype=torch.int32, device="cuda")
    got = tks.cache_fork(wide[:, 4:15], ints(lens), ints(parents), ints([lens[p] for p in parents]), 200, 8, out=out)
    assert got[0] is out and out.tolist() == fork(table, lens, parents, [lens[p] for p in parents], 200, 8)[0]
    with pytest.raises(tks.TksError):
        tks.cache_fork(out, ints([0] * 14), ints([0] * 14), ints([0] * 14), 200, 8, out=out)


# ---------------------------------------------------------------------------
# Compacting
# ---------------------------------------------------------------------------


def check_compact(table, lens, pages, page, keep=None, table_dev=None, out=None, width=None):
    width = len(table[0]) if table else width or 0
    want = compact(table, lens, pages, page, keep)
    dev = ints(table, (len(lens), width)) if table_dev is None else table_dev
    got = tks.cache_compact(dev, ints(lens, (len(lens),)), pages, page, keep=None if keep is None else torch.tensor(keep, dtype=torch.uint8, device="cuda"),
                            out=dev if out == "same" else None)
    assert [x.tolist() for x in got] == list(want[:4])
    assert tks.device_status() == expected(want[4])
    return want


@pytest.mark.parametrize("seed", range(30))
def test_random_compactions(seed):
    rng = random.Random(seed)
    page, width, sequences = rng.choice((1, 2, 16, 64)), rng.choice((1, 5, 40, 300, 700)), rng.choice((1, 3, 17, 90))
    pages = rng.choice((1, 2, sequences * width // 4 + 3, sequences * width * 2 + 50))
    table, lens = pool(rng, sequences, width, pages, page)
    keep = [rng.random() < 0.2 for _ in range(pages)] if seed % 3 == 0 else None
    check_compact(table, lens, pages, page, keep, out="same" if seed % 2 else None)


def test_a_compaction_by_hand():
    table, src, dst, count, _ = check_compact([[7, 2, -1], [7, 9, 4]], [6, 12], 10, 4)
    # four pages are held, of which 4, 7 and 9 lie beyond the first four, where 0, 1 and 3 are free
    assert src == [4, 7, 9, -1, -1] and dst == [0, 1, 3, -1, -1] and count == [3, 4]
    assert table == [[1, 2, -1], [1, 3, 0]]
    # kept pages stay, and count
    table, src, dst, count, _ = check_compact([[7, 2, -1]], [6], 10, 4, keep=[False] * 7 + [True, False, True])
    assert count == [0, 3] and table == [[7, 2, -1]]


def test_wrong_lengths_and_entries_of_a_compaction():
    check_compact([[5, 1], [2, 3]], [99, -3], 9, 4)
    check_compact([[5, 9], [-1, 3]], [8, 7], 9, 4)
    check_compact([], [], 7, 4, keep=[False, True] * 3 + [True], width=3)
    check_compact([[8, 8, 8]], [9], 9, 4)


def test_a_large_pool():
    rng = random.Random(3)
    table, lens = pool(rng, 700, 60, 60_001, 16, share=0.2)
    check_compact(table, lens, 60_001, 16)


@pytest.mark.parametrize("pages", [100, 9000, 9013])
@pytest.mark.parametrize("offset", [1, 2, 4, 7])
def test_kept_pages_at_any_alignment(offset, pages):
    rng = random.Random(offset)
    table, lens = pool(rng, 50, 60, pages, 2, share=0.9)
    keep = torch.tensor([rng.random() < 0.3 for _ in range(pages)], device="cuda")
    other = torch.ones(pages + 16, dtype=torch.uint8, device="cuda")[offset : offset + pages].copy_(keep.to(torch.uint8) * 128)
    parents = [rng.randrange(-1, 50) for _ in range(50)]
    args = (ints(table, (50, 60)), ints(lens, (50,)))
    more = (ints(parents, (50,)), ints([min(120, lens[p] + 3) for p in parents], (50,)), pages, 2)
    for call in (lambda k: tks.cache_fork(*args, *more, keep=k), lambda k: tks.cache_compact(*args, pages, 2, keep=k)):
        assert all(torch.equal(x, y) for x, y in zip(call(keep), call(other)))
        tks.device_status()


@pytest.mark.parametrize("pages", [360_447, 360_448, 360_449, 500_001])
def test_very_large_pools(pages):
    rng = random.Random(pages)
    table, lens = pool(rng, 40, 3000, pages, 2, share=0.3)
    keep = [rng.random() < 0.1 for _ in range(pages)] if pages % 2 else None
    check_compact(table, lens, pages, 2, keep)
    parents = [rng.randrange(-1, 40) for _ in range(60)]
    check_fork(table, lens, parents, [min(6000, max(0, lens[p] + rng.randrange(-4, 400))) for p in parents], pages, 2, keep)


@pytest.mark.parametrize("children", [2047, 2048, 2049])
def test_about_as_many_children_as_are_held(children):
    rng = random.Random(children)
    table, lens = pool(rng, 300, 40, 9001, 4, share=0.5)
    keep = [rng.random() < 0.1 for _ in range(9001)]
    parents = [rng.randrange(-1, 300) for _ in range(children)]
    check_fork(table, lens, parents, [min(160, max(0, lens[p] + rng.randrange(-4, 3))) for p in parents], 9001, 4, keep)


@pytest.mark.parametrize("pages", [1023, 1024, 1025, 8191, 8192, 8193])
@pytest.mark.parametrize("sequences, width", [(1, 2048), (1, 4096), (1, 4097), (8, 512), (8, 513), (16, 129), (32, 64), (32, 65), (32, 128), (33, 16)])
def test_small_tables_and_pools_of_both_ways(sequences, width, pages):
    rng = random.Random(sequences * width + pages)
    keep = [rng.random() < 0.05 for _ in range(pages)] if pages % 2 else None
    table, lens = pool(rng, sequences, width, pages, 2, share=0.5)
    check_compact(table, lens, pages, 2, keep)
    parents = [rng.randrange(-1, sequences) for _ in range(sequences)]
    check_fork(table, lens, parents, [min(width * 2, max(0, lens[p] + rng.randrange(-4, 6))) for p in parents], pages, 2, keep)


@pytest.mark.parametrize("pages", [4095, 4096, 4097])
@pytest.mark.parametrize("sequences, width", [(1, 8192), (1, 8193), (2, 4096), (31, 256), (32, 256), (33, 256), (32, 257), (16, 512)])
def test_tables_about_as_large_as_one_thread_block_makes(sequences, width, pages):
    rng = random.Random(sequences * width)
    keep = [rng.random() < 0.05 for _ in range(pages)]
    for share in (0.1, 0.9):
        table, lens = pool(rng, sequences, width, pages, 2, share=share)
        check_compact(table, lens, pages, 2, keep)
        parents = [rng.randrange(-1, sequences) for _ in range(sequences)]
        check_fork(table, lens, parents, [min(width * 2, max(0, lens[p] + rng.randrange(-4, 6))) for p in parents], pages, 2, keep)


# ---------------------------------------------------------------------------
# Copies
# ---------------------------------------------------------------------------


def random_cache(pages, page, heads, dim, held, layout="tokens", seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    cache = PagedCache(pages, page, heads, dim, held, layout, seed)
    if held == "bf16":
        for c in (cache.k, cache.v):
            c.copy_(torch.randn(c.shape, device="cuda", generator=g))
    else:
        cache.scales.copy_(torch.rand(cache.scales.shape, device="cuda", generator=g))
    bounds = torch.randn(pages, max(1, page // 8), heads, 2, dim, device="cuda", generator=g).to(torch.bfloat16)
    return cache, bounds


def planes(cache, bounds):
    return [x for x in (cache.k, cache.v, cache.scales, bounds) if x is not None]


def check_copy(cache, bounds, src, dst, count=None, with_bounds=True):
    before = [x.clone() for x in planes(cache, bounds)]
    tks.cache_copy(ints(src, (len(src),)), ints(dst, (len(src),)), cache.k, cache.v, scales=cache.scales, bounds=bounds if with_bounds else None,
                   count=None if count is None else ints([count]))
    pages = cache.k.shape[0]
    for a, b in list(zip(src, dst))[:count]:
        if 0 <= a < pages and 0 <= b < pages:
            for x in before[: None if with_bounds else -1]:
                x[b] = x[a]
    for x, y in zip(planes(cache, bounds), before):
        assert torch.equal(x, y)


@pytest.mark.parametrize("held", ["int8", "bf16"])
@pytest.mark.parametrize("layout", ["tokens", "heads", "side by side"])
@pytest.mark.parametrize("page, heads, dim", [(1, 1, 64), (16, 3, 64), (64, 8, 128), (256, 2, 128), (2, 5, 64)])
def test_copies(page, heads, dim, layout, held):
    cache, bounds = random_cache(20, page, heads, dim, held, layout)
    check_copy(cache, bounds, [3, -1, 3, 19, 5, 17, 7], [0, 1, 2, 4, -7, 18, 6])  # (no page is in both lists)
    check_copy(cache, bounds, [9, 8, 11, 12], [10, 13, 14, 15], with_bounds=False)


@pytest.mark.parametrize("count", [-5, 0, 1, 3, 4, 2 ** 31 - 1])
def test_copies_of_some_pairs(count):
    cache, bounds = random_cache(12, 16, 2, 64, "int8")
    src, dst = [1, 2, 3, 4], [5, 6, 7, 8]
    check_copy(cache, bounds, src, dst, count if count >= 0 else 0)
    if count < 0:
        check_copy(cache, bounds, [], [])
        before = [x.clone() for x in planes(cache, bounds)]
        tks.cache_copy(ints(src), ints(dst), cache.k, cache.v, scales=cache.scales, bounds=bounds, count=ints([count]))
        assert all(torch.equal(x, y) for x, y in zip(planes(cache, bounds), before))


def test_wrong_pages_of_a_copy():
    cache, bounds = random_cache(12, 16, 2, 64, "bf16")
    check_copy(cache, bounds, [1, 12, 3, 2 ** 31 - 1, -2 ** 31], [5, 6, 12, 7, 8])
    assert tks.device_status() == tks.TKS_E_INDEX


def test_many_copies():
    cache, bounds = random_cache(6000, 16, 2, 64, "int8")
    order = torch.randperm(6000).tolist()
    check_copy(cache, bounds, order[:3000], order[3000:])


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("held", ["int8", "bf16"])
def test_beams_decode_as_if_each_had_a_cache_of_its_own(held):
    """Beam search for some steps, with compactions between: attention equals that over caches that nothing is shared in."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rng = random.Random(4)
    beams, page, heads, dim, width, pages, block = 4, 8, 2, 64, 9, 30, 4
    cache, bounds = PagedCache(pages, page, heads, dim, held), torch.zeros(pages, page // block, heads, 2, dim, dtype=torch.bfloat16, device="cuda")
    rows = lambda n: torch.randn(n, heads, dim, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    # one prompt of 21 tokens, of which all beams come
    table, src, dst = tks.cache_fork(torch.full((0, width), -1, dtype=torch.int32, device="cuda"), ints([], (0,)), ints([-1]), ints([21]), pages, page)
    history = [(rows(21), rows(21))]
    lens = ints([21])
    pos = torch.arange(21, device="cuda")
    tks.cache_write(*history[0], cache.k, cache.v, (table[0][pos // page] * page + pos % page).to(torch.int32), scales=cache.scales)
    tks.cache_bounds(cache.k, table, lens, bounds, scales=cache.scales)
    for step in range(14):
        parents = [rng.randrange(len(history)) for _ in range(beams)]
        grown = lens[parents] + 1
        table, src, dst = tks.cache_fork(table, lens, ints(parents), grown, pages, page)
        tks.cache_copy(src, dst, cache.k, cache.v, scales=cache.scales, bounds=bounds)
        lens = grown
        k, v = rows(beams), rows(beams)
        history = [(torch.cat((history[p][0], k[i : i + 1])), torch.cat((history[p][1], v[i : i + 1]))) for i, p in enumerate(parents)]
        at = (lens - 1).long()
        tks.cache_write(k, v, cache.k, cache.v, (table.gather(1, (at // page).unsqueeze(1)).squeeze(1) * page + at % page).to(torch.int32), scales=cache.scales)
        tks.cache_bounds(cache.k, table, lens, bounds, start=lens - 1, scales=cache.scales)
        if step % 4 == 3:
            table, src, dst, count = tks.cache_compact(table, lens, pages, page, out=table)
            tks.cache_copy(src, dst, cache.k, cache.v, scales=cache.scales, bounds=bounds, count=count)
            assert table.max() < count[1]
        q = torch.randn(beams, 1, 4, dim, device="cuda", generator=g).to(torch.bfloat16)
        out = tks.tree_attention(q, cache.k, cache.v, table, lens - 1, scales=cache.scales)
        scores, seen = tks.block_scores(q, bounds, table, lens.unsqueeze(1), block)
        # the same from caches that hold each beam alone
        own, own_table = PagedCache(beams * width, page, heads, dim, held), []
        for k, v in history:
            own_table.append(own.fill(k, v, width)[0])
        own_table = torch.stack(own_table)
        own_bounds = torch.zeros(beams * width, page // block, heads, 2, dim, dtype=torch.bfloat16, device="cuda")
        tks.cache_bounds(own.k, own_table, lens, own_bounds, scales=own.scales)
        assert torch.equal(out, tks.tree_attention(q, own.k, own.v, own_table, lens - 1, scales=own.scales))
        want, _ = tks.block_scores(q, own_bounds, own_table, lens.unsqueeze(1), block)
        assert torch.equal(scores, want)
    assert tks.device_status() == tks.TKS_OK


def test_streams_graphs_and_two_calls_at_once():
    rng = random.Random(6)
    cases = []
    for i in range(2):
        table, lens = pool(rng, 40, 50, 1500, 8)
        parents = [rng.randrange(40) for _ in range(60)]
        new = [min(400, lens[p] + 1) for p in parents]
        cases.append((ints(table), ints(lens), ints(parents), ints(new), [torch.tensor(x, dtype=torch.int32) for x in fork(table, lens, parents, new, 1500, 8)[:3]]))
    streams = [torch.cuda.Stream() for _ in cases]
    graphs, held = [], []
    for s, (table, lens, parents, new, _) in zip(streams, cases):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            tks.cache_fork(table, lens, parents, new, 1500, 8)
        s.synchronize()
    for (table, lens, parents, new, _) in cases:  # both graphs of one stream: they share nothing
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            held.append(tks.cache_fork(table, lens, parents, new, 1500, 8))
        graphs.append(graph)
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for got, case in zip(held, cases):
        assert all(torch.equal(a.cpu(), b) for a, b in zip(got, case[4]))
    with torch.cuda.stream(streams[1]):
        got = tks.cache_fork(*cases[0][:4], 1500, 8, stream=streams[0])
    streams[0].synchronize()
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, cases[0][4]))
    assert all(tks.device_status(s) == tks.TKS_OK for s in streams)


def test_refusals():
    cache, bounds = random_cache(6, 16, 2, 64, "int8")
    table, lens = ints([[0, 1], [2, -1]]), ints([20, 3])
    one = ints([0])
    good_f = dict(page_table=table, lens=lens, parents=ints([0, 0]), new_lens=ints([21, 21]), pages=6, page_size=16)
    good_c = dict(page_table=table, lens=lens, pages=6, page_size=16)
    good_p = dict(src=one, dst=ints([1]), k_cache=cache.k, v_cache=cache.v, scales=cache.scales, bounds=bounds)
    tks.cache_fork(**good_f), tks.cache_compact(**good_c), tks.cache_copy(**good_p)
    tables = [dict(page_table=table.long()), dict(page_table=table[0]), dict(page_table=table.cpu()), dict(page_table=table.repeat(1, 2)[:, ::2]),
              dict(lens=lens.long()), dict(lens=lens[:1]), dict(pages=0), dict(pages=-1), dict(page_size=0), dict(page_size=12), dict(pages=1 << 28),
              dict(keep=torch.zeros(5, dtype=torch.bool, device="cuda")), dict(keep=torch.zeros(6, device="cuda")), dict(keep=torch.zeros(6, dtype=torch.bool)),
              dict(out=torch.empty(2, 3, dtype=torch.int32, device="cuda")), dict(out=torch.empty(2, 2, device="cuda"))]
    for call, good, bads in (
            (tks.cache_fork, good_f, tables + [dict(parents=lens.long()), dict(new_lens=one), dict(new_lens=None), dict(out=table)]),
            (tks.cache_compact, good_c, tables),
            (tks.cache_copy, good_p, [dict(src=one.long()), dict(dst=ints([1, 2])), dict(scales=None), dict(bounds=bounds[1:]), dict(count=lens.long()),
                                      dict(count=ints([], (0,))), dict(src=one.cpu(), dst=one.cpu()), dict(bounds=bounds.float())])):
        for bad in bads:
            with pytest.raises((ValueError, tks.TksError)):
                call(**{**good, **bad})

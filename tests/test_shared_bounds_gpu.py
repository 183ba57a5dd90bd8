"""Bounds of blocks in pages that sequences of different lengths hold: up to the furthest of their ends."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402
from tests.attention_plain import PagedCache  # noqa: E402
from tests.blocks_plain import bounds_of  # noqa: E402


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert tks.device_status() == tks.TKS_OK


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(lens, page, heads, dim, held, seed=3):
    """One long sequence's cache and pages; every row of the table begins with them, as far as it is long."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = max(lens)
    cache = PagedCache(-(-n // page) + 2, page, heads, dim, held, "tokens", seed)
    k, v = (torch.randn(n, heads, dim, device="cuda", generator=g) for _ in range(2))
    row = cache.fill(k, v, -(-n // page) + 1)[0]
    table = row.expand(len(lens), -1).clone()
    for b, x in enumerate(lens):
        table[b, -(-x // page):] = -1
    pos = torch.arange(n, device="cuda")
    pg, tok = row[pos // page].long(), pos % page
    keys = cache.k[pg, tok].float()
    return cache, row, table, keys if cache.scales is None else keys * cache.scales[pg, tok, :, 0].unsqueeze(-1)


def check(cache, row, table, keys, lens, starts, page, block):
    of_page = page // block
    bounds = torch.full((cache.k.shape[0], of_page, cache.k.shape[2], 2, cache.k.shape[3]), 7.0, dtype=torch.bfloat16, device="cuda")
    want = bounds.clone()
    for a, n in zip(starts, lens):
        for j in range(a // block, -(-n // block) if a < n else 0):
            # who holds the block's page: all that reach into it
            last = max(x for x in lens if x > j * block // page * page)
            want[row[j // of_page].long(), j % of_page] = bounds_of(keys[j * block : min(last, (j + 1) * block)], block)[0]
    for _ in range(3):
        bounds.fill_(7.0)
        tks.cache_bounds(cache.k, table, ints(lens), bounds, start=ints(starts), scales=cache.scales)
        assert torch.equal(bounds.float(), want.float())


@pytest.mark.parametrize("held", ["int8", "bf16"])
@pytest.mark.parametrize("page, block", [(64, 64), (64, 16), (16, 16), (32, 32)])
@pytest.mark.parametrize("lens", [[90, 130], [130, 90], [70, 71, 200, 77, 1, 130, 128], [0, 5, 0, 9, 60]], ids=str)
def test_the_furthest_end_counts(lens, page, block, held):
    cache, row, table, keys = pool(lens, page, 3, 64 if page == 16 else 128, held)
    check(cache, row, table, keys, lens, [0] * len(lens), page, block)
    # the longest has nothing new, a shorter one is filled: its blocks hold for the longer one too
    check(cache, row, table, keys, lens, [n if n == max(lens) else 0 for n in lens], page, block)
    check(cache, row, table, keys, lens, [max(0, n - 1) for n in lens], page, block)


@pytest.mark.parametrize("sequences", [33, 129, 300, 700])
def test_many_sequences(sequences):
    """(Sequences are looked at 128 at once: the furthest may be among any of them.)"""
    lens = [(37 * i) % 250 + 1 for i in range(sequences)]
    cache, row, table, keys = pool(lens, 64, 2, 64, "int8")
    check(cache, row, table, keys, lens, [0] * sequences, 64, 32)
    check(cache, row, table, keys, lens, [max(0, n - 3) for n in lens], 64, 32)


def test_ends_beyond_the_row_are_held_to_it():
    cache, row, table, keys = pool([70, 128], 64, 1, 64, "bf16")
    table = table[:, :2].contiguous()
    table[0, 1] = table[1, 1] = row[1]
    bounds = torch.zeros(cache.k.shape[0], 1, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = cache.k[row[1].long()].float()  # all of the page: the second's end is held to 128
    tks.cache_bounds(cache.k, table, ints([70, 10 ** 9]), bounds, start=ints([64, 2 ** 31 - 1]))
    assert tks.device_status() == tks.TKS_E_ROW_LEN
    assert torch.equal(bounds[row[1].long()].float(), bounds_of(slots, 64).float())


def test_pages_that_are_not_shared_are_as_before():
    """The same pages at the same places, but of rows that end before: nothing beyond a sequence's own end counts."""
    cache, row, _, keys = pool([128], 64, 2, 64, "int8")
    table = torch.stack((row, row.flip(0)))[:, :2].contiguous()
    table[1, 0] = table[1, 1] = -1
    bounds = torch.zeros(cache.k.shape[0], 2, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    tks.cache_bounds(cache.k, table, ints([100, 0]), bounds, scales=cache.scales)
    got = torch.cat([bounds[row[i].long()] for i in range(2)])
    assert torch.equal(got.float(), bounds_of(keys[:100], 32).float())


@pytest.mark.parametrize("held", ["int8", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sequences", [607, 608, 609])
def test_about_as_many_sequences_as_take_all_heads_of_a_block_at_once(sequences, dim, held):
    lens = [(53 * i) % 180 for i in range(sequences)]
    cache, row, table, keys = pool(lens, 64, 5, dim, held)
    check(cache, row, table, keys, lens, [0] * sequences, 64, 64)
    check(cache, row, table, keys, lens, [max(0, n - 1) for n in lens], 64, 16)

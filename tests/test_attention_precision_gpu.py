"""What the range and the rounding of queries and weights may do to a result, and what they may not.

The bounds are derived beside each test, from the formats: a half keeps 11 bits of values from 2^-14
up and steps of 2^-24 below; a bfloat16 keeps 8.
"""

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402
from tests.attention_cancelling import cancelling  # noqa: E402
from tests.attention_plain import PagedCache, check_rows  # noqa: E402
from tests.test_attention_gpu import HELD, ancestors, gen, rand_rows, random_parents  # noqa: E402


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert tks.device_status() == tks.TKS_OK


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# Queries: each row's result is its own
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("what", [2.0 ** 40, 1e30, 3e38, math.inf, math.nan])
@pytest.mark.parametrize("drafts, count, heads", [(4, 3, 4), (9, 1, 1), (40, 7, 2)])
def test_queries_beyond_the_drafts_have_no_influence(drafts, count, heads, what, held):
    """A padded query row may hold anything."""
    g = gen(11)
    ctx = 150
    cache = PagedCache(16, 16, 1, 64, held)
    table, _, _ = cache.fill(rand_rows(ctx + count, 1, 64, g), rand_rows(ctx + count, 1, 64, g))
    q = torch.randn(1, drafts, heads, 64, device="cuda", generator=g).to(torch.bfloat16)
    call = lambda x: tks.tree_attention(x, cache.k, cache.v, table[None], ints(ctx), draft_len=ints(count), scales=cache.scales, return_lse=True)  # noqa: E731
    q[:, count:] = 0
    want, want_lse = call(q)
    q[:, count:] = what
    out, lse = call(q)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("apart", [2.0 ** 20, 2.0 ** 40, 2.0 ** 80])
@pytest.mark.parametrize("heads", [2, 16, 48])
@pytest.mark.parametrize("dim", [64, 128])
def test_rows_of_very_different_queries(dim, heads, apart, held):
    """Query rows far apart in size, over keys that make the small ones' scores ordinary: those rows as if they were alone.

    check_rows' bounds hold for each row by itself: a score is off by dim * 2^-23 of the sum of its products'
    magnitudes, which leaves room for the 2^-25 of its largest element by which a half may miss the rest of a row.
    """
    g = gen(12)
    n = 200
    cache = PagedCache(16, 16, 1, dim, held)
    k = rand_rows(n, 1, dim, g) * apart ** 0.5
    table, kh, vh = cache.fill(k, rand_rows(n, 1, dim, g))
    q = torch.randn(1, 1, heads, dim, device="cuda", generator=g) * apart ** -0.5
    q[:, :, 1::2] *= apart  # (their softmax has one key)
    q = q.to(torch.bfloat16)
    out, lse = tks.tree_attention(q, cache.k, cache.v, table[None], ints(n - 1), scales=cache.scales, return_lse=True)
    ones = torch.ones(heads, n, dtype=torch.bool, device="cuda")
    check_rows(out[0, 0, ::2], lse[0, 0, ::2], q[0, 0, ::2].double(), kh[:, 0], vh[:, 0], ones[::2], dim ** -0.5, held)
    assert out.isfinite().all() and lse.isfinite().all()


# ---------------------------------------------------------------------------
# Weights
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("heads", [1, 16, 20, 80])
def test_scores_so_large_that_they_differ_in_steps(heads, held):
    """Scores near 2^28 (of powers of two), where 32 bits go in steps of 16, and each a step above the one before.

    Such scores tell only which key is the largest, but a weight must not leave the range of its type: the result
    is a mean of values, nearly those of the last keys.
    """
    n, dim, group = 12800, 64, 128
    k = torch.zeros(n, 1, dim, device="cuda")
    k[:, 0, 0] = 127.0
    k[:, 0, 1] = torch.arange(n, device="cuda") // group  # 0 .. 99, a step each
    v = torch.where(torch.arange(n, device="cuda") < n - group, 1.0, 2.0)[:, None, None].expand(n, 1, dim)
    many = 320  # (sequences enough that a row's keys are not split over blocks)
    q = torch.zeros(many, 1, heads, dim, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    q[..., 1] = 2.0 ** -17
    cache = PagedCache(n // 16 + 1, 16, 1, dim, held)
    table, _, _ = cache.fill(k, v)
    for scale in (2.0 ** 20, 2.0 ** 21, 2.0 ** 22, 2.0 ** 30):
        out, lse = tks.tree_attention(q, cache.k, cache.v, table[None].expand(many, -1), torch.full((many,), n - 1, dtype=torch.int32, device="cuda"),
                                      scales=cache.scales, softmax_scale=scale * math.log(2.0), return_lse=True)
        assert out.isfinite().all() and lse.isfinite().all()
        assert out.min() >= 1.0 - 2.0 ** -7 and out.max() <= 2.0 + 2.0 ** -6


def dominant_key_case(sequences, heads, held):
    """One key 25.2 doublings above 2^20 equal ones: together they are 2.7 % of the row.

    As many sequences as the device takes at once, all in the same pages, so that a row's keys are not split over
    blocks. A weight is held to 2^-11 of itself (a bfloat16 cache: 2^-15) or, small, to 2^-32 of the largest, so
    the output to n * 2^-32 of the largest value beside its own rounding. Sums of weights are held in 32 bits by
    lanes that take every eighth key or fewer: the lane of the dominant one may lose its share of the tail. (A tail
    that counts for nothing in the output would be 0.027.)
    """
    n, page, dim, below = 1 << 20, 64, 64, 25.2
    shape = (n // page + 1, page, 1, dim)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    k, v = torch.zeros(n, 1, dim, device="cuda"), torch.ones(n, 1, dim, device="cuda")
    k[0, 0, 0] = 1.0
    v[0, 0, dim // 2 :] = 0.0
    if held == "int8":
        kc, vc, scales = torch.zeros(shape, dtype=torch.int8, device="cuda"), torch.zeros(shape, dtype=torch.int8, device="cuda"), torch.zeros(*shape[:3], 2, device="cuda")
    else:
        kc, vc, scales = torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), None
    tks.cache_write(k, v, kc, vc, slots, scales=scales)
    q = torch.zeros(sequences, 1, heads, dim, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = below * math.log(2.0)
    table = torch.arange(shape[0], dtype=torch.int32, device="cuda")[None].expand(sequences, -1)
    out, lse = tks.tree_attention(q, kc, vc, table, torch.full((sequences,), n - 1, dtype=torch.int32, device="cuda"), scales=scales,
                                  softmax_scale=scale, return_lse=True)
    tail = (n - 1) * 2.0 ** -below
    want = torch.ones(dim, dtype=torch.float64, device="cuda")
    want[dim // 2 :] = tail / (1 + tail)
    bound = 2.0 ** -8 * want + (2.0 ** -11 if held == "int8" else 2.0 ** -15) * want + want * tail / 8 + n * 2.0 ** -32 + 2.0 ** -18
    assert (lse.double() - (scale + math.log1p(tail))).abs().max().item() <= tail / 8 + 2.0 ** -22 * scale + 2.0 ** -18
    return (out.double() - want).abs() / bound


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("sequences, heads", [(304, 4), (152, 24), (152, 70)])
def test_a_long_flat_tail_behind_a_dominant_key(sequences, heads, held):
    """Where the dominant key has a value of zero, the tail is all there is."""
    assert dominant_key_case(sequences, heads, held)[..., 32:].max().item() <= 1.0


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("sequences, heads", [(304, 4), (152, 24), (152, 70)])
def test_a_dominant_key_before_a_long_flat_tail(sequences, heads, held):
    """Where the dominant key has a value, the tail's are added to it, each less than 2^-24 of it."""
    assert dominant_key_case(sequences, heads, held).max().item() <= 1.0


@pytest.mark.parametrize("held", HELD)
@pytest.mark.parametrize("heads, dim", [(3, 64), (3, 128), (9, 64), (24, 128)])
def test_runs_of_several_pieces(heads, dim, held):
    """Sequences of one cache, cut at many lengths around the pieces' ends, that fill the device several times."""
    g = gen(13)
    n, page, drafts, many = 70000, 64, 5, 340
    cache = PagedCache(n // page + 2, page, 1, dim, held)
    table, kh, vh = cache.fill(rand_rows(n, 1, dim, g), rand_rows(n, 1, dim, g))
    lens = [69990, 1, 32768, 32763, 65536, 0, 65540, 32769, 50001, 40000, 69000]
    ctx = [lens[i % len(lens)] for i in range(many)]
    counts = [i % (drafts + 1) for i in range(many)]
    q = torch.randn(many, drafts, heads, dim, device="cuda", generator=g).to(torch.bfloat16)
    parents = random_parents(many, drafts, g)
    out, lse = tks.tree_attention(q, cache.k, cache.v, table[None].expand(many, -1), ints(*ctx), tree=tks.tree_mask(parents), draft_len=ints(*counts),
                                  scales=cache.scales, return_lse=True)
    assert tks.device_status() == tks.TKS_OK
    for b in range(0, many, 9):
        seen = torch.zeros(drafts, ctx[b] + counts[b], dtype=torch.bool)
        seen[:, : ctx[b]] = True
        seen[:, ctx[b] :] = ancestors(parents[b].tolist())[:, : counts[b]]
        seen[counts[b] :] = False
        end = ctx[b] + counts[b]
        check_rows(out[b].reshape(-1, dim), lse[b].reshape(-1), q[b].reshape(-1, dim).double(), kh[:end, 0], vh[:end, 0],
                   seen.cuda().repeat_interleave(heads, 0), dim ** -0.5, held)


@pytest.mark.parametrize("heads", [4, 40])
def test_infinite_values_in_a_later_piece(heads):
    """Values of drafts that lie in the second piece of a run reach the rows that attend, as they do in the first."""
    g = gen(14)
    n, many, dim = 40004, 320, 64
    cache = PagedCache(n // 64 + 2, 64, 1, dim, "bf16")
    table, _, _ = cache.fill(rand_rows(n, 1, dim, g), rand_rows(n, 1, dim, g))
    for pos, d, x in ((10, 3, math.inf), (40002, 5, -math.inf), (40003, 6, math.nan)):  # one in the context, two among the drafts
        cache.v[table[pos // 64], pos % 64, 0, d] = x
    q = 0.1 * torch.randn(many, 4, heads, dim, device="cuda", generator=g)
    out = tks.tree_attention(q.to(torch.bfloat16), cache.k, cache.v, table[None].expand(many, -1), torch.full((many,), n - 4, dtype=torch.int32, device="cuda"))
    assert (out[..., 3] == math.inf).all()
    assert (out[:, 2:, :, 5] == -math.inf).all() and out[:, :2, :, 5].isfinite().all()
    assert out[:, 3, :, 6].isnan().all() and out[:, :3, :, 6].isfinite().all()


@pytest.mark.parametrize("q_heads", [4, 16, 40, 130])
@pytest.mark.parametrize("dim", [64, 128])
def test_weights_over_a_bfloat16_cache_are_held_to_sixteen_bits(dim, q_heads):
    """Values that cancel, but for what the weights are off by."""
    case = cancelling(dim, device="cuda")
    n = case["k"].shape[0]
    cache = PagedCache(-(-n // 16) + 1, 16, 1, dim, "bf16")
    table, kh, vh = cache.fill(case["k"][:, None], case["v"][:, None])
    q = case["q"].expand(1, 1, q_heads, dim).contiguous()
    out, lse = tks.tree_attention(q, cache.k, cache.v, table[None], ints(n - 1), softmax_scale=case["scale"], return_lse=True)
    err = (out[0, 0].double() - case["want"]).abs()
    assert (err / case["bound"]).max().item() <= 1.0
    sel, _ = tks.selected_attention(q, cache.k, cache.v, table[None], torch.randperm(n, device="cuda").to(torch.int32).view(1, 1, -1),
                                    softmax_scale=case["scale"], return_lse=True)
    assert ((sel[0, 0].double() - case["want"]).abs() / case["bound"]).max().item() <= 1.0

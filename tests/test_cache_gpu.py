"""Writing rows into the paged cache and reading them back, against the definition."""

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402
from tests.attention_plain import PagedCache, quantise  # noqa: E402


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert tks.device_status() == tks.TKS_OK


def rows(n, heads, dim, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(n, heads, dim, device="cuda", generator=g) * torch.exp(3 * torch.randn(n, heads, 1, device="cuda", generator=g))
    return x.to(dtype)


def check(cache, k, v, slots):
    """The cache holds rows k, v at slots exactly as the definition says, and reads back as it."""
    pg, tok = slots.long() // cache.page, slots.long() % cache.page
    for dtype in (torch.float32, torch.bfloat16):
        back = tks.cache_read(cache.k, cache.v, slots, scales=cache.scales, dtype=dtype)
        for x, c, plane, got in ((k, cache.k, 0, back[0]), (v, cache.v, 1, back[1])):
            if cache.held == "int8":
                codes, scale = quantise(x)
                assert torch.equal(c[pg, tok], codes)
                assert torch.equal(cache.scales[pg, tok, :, plane], scale)
                assert torch.equal(got, (codes.float() * scale.unsqueeze(-1)).to(dtype))
            else:
                assert torch.equal(c[pg, tok], x.to(torch.bfloat16))
                assert torch.equal(got, x.to(torch.bfloat16).to(dtype))


@pytest.mark.parametrize("held", ["int8", "bf16"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n, heads", [(1, 1), (1, 8), (3, 5), (33, 2), (1000, 3)])
def test_round_trip(n, heads, dim, dtype, held):
    k, v = rows(n, heads, dim, dtype, 1), rows(n, heads, dim, dtype, 2)
    cache = PagedCache(n // 16 + 3, 16, heads, dim, held)
    slots = torch.randperm((n // 16 + 3) * 16, device="cuda")[:n].to(torch.int32)
    tks.cache_write(k, v, cache.k, cache.v, slots, scales=cache.scales)
    check(cache, k, v, slots)


@pytest.mark.parametrize("held", ["int8", "bf16"])
@pytest.mark.parametrize("layout", ["tokens", "heads", "side by side"])
@pytest.mark.parametrize("page", [1, 4, 128])
def test_layouts(page, layout, held):
    n = 50
    k, v = rows(n, 3, 128, torch.bfloat16, 3), rows(n, 3, 128, torch.bfloat16, 4)
    cache = PagedCache(256 // page, page, 3, 128, held, layout)
    before = cache.k.clone()
    slots = torch.randperm(256 // page * page, device="cuda")[:n].to(torch.int32)
    tks.cache_write(k, v, cache.k, cache.v, slots, scales=cache.scales)
    check(cache, k, v, slots)
    rest = torch.ones(256 // page * page, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    rest = rest.nonzero()[:, 0]
    untouched = lambda c: torch.nan_to_num(c[rest // page, rest % page].float())  # noqa: E731
    assert torch.equal(untouched(cache.k), untouched(before))
    if held == "int8":
        assert cache.scales[rest // page, rest % page].isnan().all()


def test_views_of_a_fused_projection():
    n, heads = 21, 2
    fused = rows(n, 3 * heads, 64, torch.bfloat16, 5)
    k, v = fused[:, heads : 2 * heads], fused[:, 2 * heads :]
    cache = PagedCache(4, 16, heads, 64, "int8")
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    tks.cache_write(k, v, cache.k, cache.v, slots, scales=cache.scales)
    check(cache, k, v, slots)
    odd = torch.zeros(n, heads, 67, device="cuda")
    odd[..., 1:65] = v.float()
    tks.cache_write(odd[..., 1:65], odd[..., 1:65], cache.k, cache.v, slots, scales=cache.scales)
    check(cache, v.float(), v.float(), slots)
    once = rows(1, heads, 64, torch.bfloat16, 6).expand(n, heads, 64)  # one row for all tokens
    tks.cache_write(once, once, cache.k, cache.v, slots, scales=cache.scales)
    check(cache, once, once, slots)


def test_zeros_tiny_and_huge_rows():
    x = torch.zeros(8, 1, 64, device="cuda")
    x[1] = 1e-30
    x[2] = 2.0 ** -40
    x[3, 0, 5] = 3e38
    x[4] = 2.0 ** 80
    x[5, 0, :3] = torch.tensor([math.inf, -math.inf, 1.0])
    x[6] = torch.linspace(-1, 1, 64)
    x[7, 0, 0] = 1e-45
    cache = PagedCache(1, 16, 1, 64, "int8")
    slots = torch.arange(8, dtype=torch.int32, device="cuda")
    tks.cache_write(x, -x, cache.k, cache.v, slots, scales=cache.scales)
    check(cache, x, -x, slots)
    assert cache.k[0, 5, 0, :2].tolist() == [127, -127]
    assert cache.scales[0, :8].isfinite().all() and (cache.scales[0, :8] >= 2.0 ** -47).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_nan_row_has_a_nan_scale_and_no_other_row_does(dtype):
    x = rows(40, 2, 128, dtype, 7)
    x[5, 1, 77] = math.nan
    x[39, 0, 0] = -math.nan
    cache = PagedCache(4, 16, 2, 128, "int8")
    slots = torch.arange(40, dtype=torch.int32, device="cuda")
    tks.cache_write(x, x, cache.k, cache.v, slots, scales=cache.scales)
    k, _ = tks.cache_read(cache.k, cache.v, slots, scales=cache.scales)
    bad = k.isnan().any(-1)
    assert bad.nonzero().tolist() == [[5, 1], [39, 0]] and k[5, 1].isnan().all()


def test_skipped_and_wrong_slots():
    x = rows(6, 1, 64, torch.bfloat16, 8)
    cache = PagedCache(2, 4, 1, 64, "int8")
    slots = torch.tensor([3, -1, 7, -2 ** 31, 0, -5], dtype=torch.int32, device="cuda")
    tks.cache_write(x, x, cache.k, cache.v, slots, scales=cache.scales)
    assert tks.device_status() == tks.TKS_OK
    check(cache, x[[0, 2, 4]], x[[0, 2, 4]], slots[[0, 2, 4]])
    k, v = tks.cache_read(cache.k, cache.v, slots, scales=cache.scales)
    assert (k[[1, 3, 5]] == 0).all() and (v[[1, 3, 5]] == 0).all() and (k[[0, 2, 4]] != 0).any(-1).all()
    wrong = torch.tensor([8, 1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    tks.cache_write(x[:3], x[:3], cache.k, cache.v, wrong, scales=cache.scales)
    assert tks.device_status() == tks.TKS_E_INDEX
    check(cache, x[1:2], x[1:2], wrong[1:2])
    k, _ = tks.cache_read(cache.k, cache.v, wrong, scales=cache.scales)
    assert tks.device_status() == tks.TKS_E_INDEX
    assert (k[[0, 2]] == 0).all()


def test_nothing_to_do():
    cache = PagedCache(2, 4, 1, 64, "bf16")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    tks.cache_write(x, x, cache.k, cache.v, none)
    assert tks.cache_read(cache.k, cache.v, none)[0].shape == (0, 1, 64)


def test_on_another_stream():
    x = rows(500, 2, 64, torch.bfloat16, 9)
    cache = PagedCache(40, 16, 2, 64, "int8")
    slots = torch.randperm(640, device="cuda")[:500].to(torch.int32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tks.cache_write(x, x, cache.k, cache.v, slots, scales=cache.scales, stream=s)
    k, v = tks.cache_read(cache.k, cache.v, slots, scales=cache.scales, stream=s)
    torch.cuda.synchronize()
    check(cache, x, x, slots)
    assert torch.equal(k, v)


def test_refusals():
    x = rows(4, 2, 64, torch.bfloat16, 10)
    cache = PagedCache(2, 4, 2, 64, "int8")
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    write = lambda **k: tks.cache_write(**{**dict(k=x, v=x, k_cache=cache.k, v_cache=cache.v, slots=slots, scales=cache.scales), **k})  # noqa: E731
    read = lambda **k: tks.cache_read(**{**dict(k_cache=cache.k, v_cache=cache.v, slots=slots, scales=cache.scales), **k})  # noqa: E731
    write(), read()
    for bad in (dict(scales=None), dict(slots=slots.long()), dict(slots=slots.cpu()), dict(slots=slots[::2]), dict(k_cache=cache.k[0]),
                dict(k_cache=cache.k.half(), v_cache=cache.v.half()), dict(k_cache=cache.k[:, :3], v_cache=cache.v[:, :3])):
        for call in (write, read):
            with pytest.raises(ValueError):
                call(**bad)
    for bad in (dict(k=x[:3]), dict(v=x.float()), dict(k=x.half(), v=x.half()), dict(k=x.cpu(), v=x.cpu()), dict(k=x[:, :1], v=x[:, :1])):
        with pytest.raises(ValueError):
            write(**bad)
    for bad in (dict(dtype=torch.float16), dict(out=(x, x[:3])), dict(out=(x.float(), x))):
        with pytest.raises(ValueError):
            read(**bad)
    assert torch.equal(read(out=(torch.empty_like(x), torch.empty_like(x)))[0], read()[0])

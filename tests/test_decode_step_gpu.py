"""The example of a decode step, with its operators together, against the definitions in 64 bits."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402
from tests.attention_plain import check_rows  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def held(layer, b, n):
    """The first n positions' keys and values of sequence b as the cache holds them, [n, heads, dim] in 64 bits."""
    pos = torch.arange(n, device="cuda")
    pg, tok = layer.table[b, pos // layer.page_size].long(), pos % layer.page_size
    s = layer.scales[pg, tok].double()
    return layer.k_cache[pg, tok].double() * s[..., :1], layer.v_cache[pg, tok].double() * s[..., 1:]


@pytest.mark.parametrize("context,tokens,q_heads,kv_heads,dim,k", [
    ([700, 33, 0, 1500], 8, 8, 2, 64, 96),
    ([260, 3000], 8, 40, 2, 128, 512),
])
def test_decode_step(context, tokens, q_heads, kv_heads, dim, k):
    m = example()
    layer = m.Layer(context, 64, kv_heads, dim, page_size=16, seed=3)
    layer.prompt()
    parents = [-1, 0, 0, 1, 1, 2, 3, 6]
    bits = tks.tree_mask(torch.tensor([parents] * len(context), device="cuda"))
    logits = torch.randn(len(context), tokens, 2 * max(context), device="cuda", generator=layer.gen)
    group = q_heads // kv_heads
    for _ in range(2):
        layer.draft(tokens)
        q = layer.random(len(context), tokens, q_heads, dim)
        dense, (idx, sparse) = layer.dense(q, bits), layer.sparse(q, logits, k)
        paths = [m.path_to(parents, 7 if b % 2 else 5) for b in range(len(context))]
        lens = layer.ctx_len.tolist()
        for b, n in enumerate(lens):
            keys, values = held(layer, b, n + tokens)
            tree = torch.zeros(tokens, n + tokens, dtype=torch.bool, device="cuda")
            few = torch.zeros_like(tree)
            for t in range(tokens):
                tree[t, :n] = True
                tree[t, [n + j for j in m.path_to(parents, t)]] = True
                few[t, torch.topk(logits[b, t, :n], min(k, n)).indices] = True
            rows = q[b].double()
            for h in range(kv_heads):
                mine = slice(h * group, (h + 1) * group)
                qr = rows[:, mine].reshape(-1, dim)
                for out, seen in ((dense, tree), (sparse, few)):
                    check_rows(out[b][:, mine].reshape(-1, dim), None, qr, keys[:, h], values[:, h],
                               seen.repeat_interleave(group, 0), dim ** -0.5, "int8")
        before = [held(layer, b, n + tokens) for b, n in enumerate(lens)]
        layer.accept(paths)
        for b, n in enumerate(lens):
            assert layer.ctx_len[b].item() == n + len(paths[b])
            rows = list(range(n)) + [n + d for d in paths[b]]
            # The codes stay; the scale passes two products in 32 bits (127 s, and by 1/127, itself
            # rounded), each to 2^-24 of it.
            for old, new in zip(before[b], held(layer, b, len(rows))):
                assert torch.all((old[rows] - new).abs() <= 4 * 2.0 ** -24 * old[rows].abs())
    assert tks.device_status() == tks.TKS_OK


def test_threads_on_one_stream():
    """Calls of several host threads on one stream, each of two kernels that share a workspace."""
    import ctypes
    import threading

    lib = tks.load()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    n, page, heads, dim, calls = 20000, 64, 2, 64, 24
    pages = -(-(n + 1) // page)
    k, v = (torch.randn(pages, page, heads, dim, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
    qs = torch.randn(4, calls, 1, 1, heads, dim, device="cuda", generator=g).to(torch.bfloat16)
    want = torch.stack([torch.stack([tks.tree_attention(q, k, v, table, ctx) for q in row]) for row in qs])
    out = torch.zeros_like(qs)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    cache = tks.Cache(k.data_ptr(), v.data_ptr(), None, tks.TKS_BF16, pages, page, heads, dim, *k.stride()[:3])
    rcs = [[] for _ in range(4)]

    def run(i):
        for j in range(calls):
            q = tks.Queries(qs[i, j].data_ptr(), heads * dim, heads * dim, dim, out[i, j].data_ptr(), None, 1, 1, heads,
                            table.data_ptr(), pages, pages, dim ** -0.5)
            rcs[i].append(lib.tks_tree_attention(ctypes.byref(cache), ctypes.byref(q), ctx.data_ptr(), None, None, stream.cuda_stream))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert rcs == [[tks.TKS_OK] * calls] * 4
    assert tks.device_status(stream) == tks.TKS_OK
    assert torch.equal(out, want)

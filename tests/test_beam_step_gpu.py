"""The example of beam search over selected blocks, with its operators together, against the definitions in 64 bits."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_attention_topk_gb300 as tks  # noqa: E402
from tests.attention_plain import check_rows  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("beam_step", os.path.join(ROOT, "examples", "beam_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("prompts, beams, q_heads, kv_heads, dim, page, block, selected", [
    ([200, 33, 1], 3, 8, 2, 64, 16, 8, 5),
    ([700, 64], 4, 40, 2, 128, 64, 32, 7),
])
def test_beam_step(prompts, beams, q_heads, kv_heads, dim, page, block, selected):
    layer = example().Beams(prompts, beams, 40, 400, kv_heads, dim, page, block, seed=5)
    group = beams * torch.arange(len(prompts), device="cuda").repeat_interleave(beams)
    n = len(group)
    for step in range(2 * page // 8 + 3):
        parents = (group + torch.randint(beams, (n,), device="cuda", generator=layer.gen)).to(torch.int32)
        # the keys that each beam comes from, by the tables as they are
        def rows(b, length):
            pos = torch.arange(length, device="cuda")
            pg, tok = layer.table[b][pos // page].long(), pos % page
            s = layer.scales[pg, tok].double()
            return layer.k_cache[pg, tok].double() * s[..., :1], layer.v_cache[pg, tok].double() * s[..., 1:]
        before = [rows(p, int(layer.lens[p])) for p in parents.tolist()]
        q = layer.random(n, 1, q_heads, dim)
        blocks, out = layer.step(parents, q, selected)
        assert tks.device_status() == tks.TKS_OK
        for b in range(n):
            length = int(layer.lens[b])
            k, v = rows(b, length)
            assert torch.equal(k[:-1], before[b][0]) and torch.equal(v[:-1], before[b][1])  # nothing of another beam's token
            for h in range(kv_heads):
                mine = blocks[b, 0, h]
                mine = mine[mine >= 0].long()
                count = -(-length // block)
                assert len(mine) == min(selected, count) and 0 in mine and count - 1 in mine
                pos = (mine.unsqueeze(1) * block + torch.arange(block, device="cuda")).flatten()
                pos = pos[pos < length]
                hs = slice(h * (q_heads // kv_heads), (h + 1) * (q_heads // kv_heads))
                check_rows(out[b, 0, hs], None, q[b, 0, hs].double(), k[pos, h], v[pos, h],
                           torch.ones(q_heads // kv_heads, len(pos), dtype=torch.bool, device="cuda"), dim ** -0.5, "int8")
        if step % 3 == 2:
            used = layer.compact()
            assert used == len({e for b in range(n) for e in layer.table[b][: -(-int(layer.lens[b]) // page)].tolist()}) and layer.table.max() < used
    assert tks.device_status() == tks.TKS_OK


def test_the_example_runs(capsys):
    example().main()
    assert "step 4" in capsys.readouterr().out

"""Plain implementations of the cache and attention operators in 64 bits, and
the bounds their 32- and 16-bit counterparts have to keep.

Written from the definitions, one query row at a time, without the package.
"""

import math

import torch

LOW, HIGH = 2.0 ** -40, 2.0 ** 80


def quantise(x):
    """Codes and scales of rows x, in the 32-bit arithmetic of the definition."""
    x = x.float()
    amax = x.abs().amax(-1).clamp(LOW, HIGH)
    scale = amax * torch.tensor(1.0 / 127.0, dtype=torch.float32, device=x.device)
    codes = torch.round(x * scale.reciprocal().unsqueeze(-1)).clamp(-127, 127)
    return codes.to(torch.int8), scale


class PagedCache:
    """A cache of given layout with every slot unwritten: what it holds there is NaN (bfloat16), or codes with NaN scales."""

    def __init__(self, pages, page, heads, dim, held, layout="tokens", seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.page, self.heads, self.dim, self.held = page, heads, dim, held
        dt = torch.int8 if held == "int8" else torch.bfloat16
        if layout == "tokens":  # [pages, page, heads, dim]
            k, v = (torch.empty((pages, page, heads, dim), dtype=dt, device=device) for _ in range(2))
        elif layout == "heads":  # heads outside tokens
            k, v = (torch.empty((pages, heads, page, dim), dtype=dt, device=device).transpose(1, 2) for _ in range(2))
        else:  # keys and values of a page side by side, with a gap after each row
            both = torch.empty((pages, 2, page, heads, dim + 16), dtype=dt, device=device)
            k, v = both[:, 0, :, :, :dim], both[:, 1, :, :, :dim]
        for c in (k, v):
            if held == "int8":
                c.copy_(torch.randint(-127, 128, c.shape, dtype=torch.int8, device=device, generator=g))
            else:
                c.fill_(math.nan)
        self.k, self.v = k, v
        self.scales = torch.full((pages, page, heads, 2), math.nan, device=device) if held == "int8" else None
        self.free = torch.randperm(pages, generator=g, device=device).tolist()

    def fill(self, k, v, width=None):
        """Puts one sequence's rows [n, heads, dim] into fresh pages; returns its page table row and the values held."""
        n = k.shape[0]
        need = -(-n // self.page)
        mine = [self.free.pop() for _ in range(need)]
        table = torch.full((max(width or need, 1),), -1, dtype=torch.int32, device=k.device)
        table[:need] = torch.tensor(mine, dtype=torch.int32, device=k.device)
        pos = torch.arange(n, device=k.device)
        pg, tok = table[pos // self.page].long(), pos % self.page
        out = []
        for x, c, plane in ((k, self.k, 0), (v, self.v, 1)):
            if self.held == "int8":
                codes, scale = quantise(x)
                c[pg, tok] = codes
                self.scales[pg, tok, :, plane] = scale
                out.append(codes.double() * scale.double().unsqueeze(-1))
            else:
                c[pg, tok] = x.to(torch.bfloat16)
                out.append(x.to(torch.bfloat16).double())
        return table, out[0], out[1]


def attend(q, k, v, scale):
    """One row: q [dim], k and v [n, dim] of the keys it attends to -> (out, lse, bound on |out - got|, bound on |lse - got|)
    without the weights' rounding, and sum w |v|, which that is relative to."""
    if k.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, -math.inf, z
    x = (k @ q) * scale
    lse = torch.logsumexp(x, 0)
    w = torch.exp(x - lse)
    return w @ v, lse.item(), w @ v.abs()


def check_rows(got_out, got_lse, q, keys, values, seen, scale, held):
    """Every query row against the definition.

    q [rows, dim] in 64 bits, keys and values [n, dim] as held, seen bool [rows, n].
    Bounds, before any run: the output's rounding to bfloat16 is 2^-8 of it; a weight's
    rounding is 2^-8 (bfloat16) or 2^-11 (half, with 2^-25 of the largest weight for
    subnormal ones) of the weight, so of sum w |v|; scores are sums of dim products in 32
    bits, off by at most dim * 2^-23 of sum |q k|, which moves each weight by that much,
    and exponentials, logarithms and reciprocals are good to 2^-20.
    """
    rows, dim = q.shape
    n = keys.shape[0]
    a = (q @ keys.T) * scale
    a = a.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(a, -1) if n else torch.full((rows,), -math.inf, dtype=q.dtype, device=q.device)
    w = torch.exp(a - torch.where(lse == -math.inf, 0.0, lse).unsqueeze(-1))
    clean = torch.where(seen.any(0).unsqueeze(-1), values, 0.0) if n else values
    want = w @ clean
    size = w @ clean.abs()
    most = (q.abs() @ keys.abs().T * seen).amax(-1) * abs(scale) if n else torch.zeros(rows, dtype=q.dtype, device=q.device)
    score = dim * 2.0 ** -23 * most + 2.0 ** -20
    weight = 2.0 ** -8 if held == "bf16" else 2.0 ** -11
    top = clean.abs().amax() if n else 0.0
    bound = 2.0 ** -8 * want.abs() + (weight + 2 * score).unsqueeze(-1) * size + (n * 2.0 ** -25 * top if held == "int8" else 0.0) + 1e-30
    empty = ~seen.any(-1)
    assert torch.equal(got_out[empty].double(), torch.zeros_like(want[empty])), "rows that see nothing give zeros"
    err = (got_out.double() - want).abs()
    assert not got_out.isnan().any(), "NaN in the output"
    worst = (err / bound).max().item()
    assert worst <= 1.0, f"output off by {worst:.2f} of its bound"
    if got_lse is not None:
        assert torch.equal(got_lse[empty], torch.full_like(got_lse[empty], -math.inf))
        if (~empty).any():
            worst = ((got_lse.double() - lse).abs()[~empty] / (2 * score + 2.0 ** -22 * lse.abs() + 2.0 ** -20)[~empty]).max().item()
            assert worst <= 1.0, f"log-sum-exp off by {worst:.2f} of its bound"

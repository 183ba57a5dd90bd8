"""A row of attention over a bfloat16 cache whose values cancel, so that its output shows how exactly
the weights are held."""

import torch


def first_part(w):
    """The larger of a weight's two parts: cut to 8 bits, a little below the weight."""
    return ((w.float() * 0.99609375).view(torch.int32) & -65536).view(torch.float32).double()


def cancelling(dim, n=1024, seed=0, device="cpu"):
    """q [dim], k and v [n, dim] (bfloat16), scale, and what is wanted in 64 bits with its bound.

    Every fourth key has the largest score and a value of zero, so that weights are relative to 1. The others,
    in order of their weights, are pairs of almost the same weight with values of opposite sign: in the first half
    of the elements the sign follows what rounding to one bfloat16 does to the weight, in the second what is left
    out with the smaller of two parts.

    Bound: the output's rounding is 2^-8 of it; a weight that is the sum of two bfloat16 is off by at most
    2^-15 of it, a score by dim * 2^-23 of itself (it has one product), an exponential by 2^-20.
    """
    g = torch.Generator()
    g.manual_seed(seed)
    scale = 0.125
    k = torch.zeros(n, dim)
    k[:, 0] = torch.rand(n, generator=g) * 8 - 8
    k[::4, 0] = 0
    k = k.to(torch.bfloat16)
    q = torch.zeros(dim)
    q[0] = 1
    w = torch.exp(k[:, 0].double() * scale)
    v = torch.zeros(n, dim)
    at = torch.arange(n)[torch.arange(n) % 4 != 0]
    at = at[w[at].argsort()].view(-1, 2)
    for half, error in ((0, w.to(torch.bfloat16).double() - w), (1, first_part(w) - w)):
        sign = torch.where(error[at[:, 0]] >= error[at[:, 1]], 1.0, -1.0)
        cols = slice(half * dim // 2, (half + 1) * dim // 2)
        v[at[:, 0], cols] = sign[:, None]
        v[at[:, 1], cols] = -sign[:, None]
    v = v.to(torch.bfloat16)
    total = w.sum()
    want, size = (w @ v.double()) / total, (w @ v.double().abs()) / total
    score = dim * 2.0 ** -23 * 1.0 + 2.0 ** -20
    bound = 2.0 ** -8 * want.abs() + (2.0 ** -15 + 2 * score) * size
    return {"q": q.to(torch.bfloat16).to(device), "k": k.to(device), "v": v.to(device), "scale": scale, "weights": w,
            "want": want.to(device), "bound": bound.to(device)}

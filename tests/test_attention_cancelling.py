"""The cancelling case tells weights of 16 bits from weights of 8, by mistakes planted in a plain computation."""

import pytest

torch = pytest.importorskip("torch")

from tests.attention_cancelling import cancelling, first_part  # noqa: E402


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("held", ["one bfloat16", "the first part alone", "two parts"])
def test_weights(held, dim):
    case = cancelling(dim)
    w, v = case["weights"], case["v"].double()
    if held == "one bfloat16":
        parts = w.to(torch.bfloat16).double()
    else:
        parts = first_part(w)
        if held == "two parts":
            parts = parts + (w - parts).to(torch.bfloat16).double()
    out = ((parts @ v) / w.sum()).to(torch.bfloat16).double()
    worst = ((out - case["want"]).abs() / case["bound"]).max().item()
    assert worst <= 1.0 if held == "two parts" else worst > 4.0

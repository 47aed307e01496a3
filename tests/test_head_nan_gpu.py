"""The output head's alternatives where logits are NaN, -Inf or both."""

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_head_gpu import Head, batch  # noqa: E402


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 50, 300, 1100])
@pytest.mark.parametrize("k,finite", [(5, 2), (24, 10), (64, 0)])
def test_alternatives_beside_parts_of_nan(k, finite, n, kind):
    """A NaN is never among the alternatives and takes no place of a logit of -Inf, which comes last."""
    rows, cols, first = 5000, 64, 4800
    h = Head(rows, cols, kind)
    x = batch(n, cols, kind, rows=rows)[0].abs()
    h.w[:first] = math.nan  # whole parts, more of them than alternatives
    h.w[first:rows - finite] = -math.inf
    h.view(h.params, h.offs[0], rows).copy_(h.w)
    out = h.logprob(x, torch.full((n,), rows - 1, device="cuda"), top_k=k)
    assert torch.isnan(out["logp"]).all() and torch.isnan(out["entropy"]).all()
    assert torch.equal(out["top_ids"][:, :finite].sort(1).values, torch.arange(rows - finite, rows, device="cuda").expand(n, finite))
    if kind == "bf16":  # in fp32 an infinite weight may make a NaN
        assert torch.equal(out["top_ids"][:, finite:], torch.arange(first, first + k - finite, device="cuda").expand(n, k - finite))
    h.w[:] = math.nan
    h.view(h.params, h.offs[0], rows).copy_(h.w)
    out = h.logprob(x, None, top_k=k)
    assert (out["top_ids"] == -1).all() and torch.isnan(out["entropy"]).all()

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


@pytest.mark.parametrize("table,x", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("n", [20, 300])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, 3e38, math.nan])
def test_gradients_that_are_not_finite(n, table, x, bad):
    """An infinite, huge or NaN gradient of one row's log probability spoils that row of dx alone."""
    rows, cols = 700, 96
    h = Head(rows, cols, table)
    data, ids = batch(n, cols, x, rows=rows)
    out = h.logprob(data, ids)
    dlogp = torch.ones(n, device="cuda")
    dlogp[3] = 0.0
    want, _ = h.grad(data, out["records"], dlogp, None, ids)
    dlogp[3] = bad
    for dent in (None, torch.full((n,), 0.0, device="cuda")):
        dx, dw = h.grad(data, out["records"], dlogp, dent, ids)
        others = torch.arange(n, device="cuda") != 3
        assert torch.equal(dx[others], want[others])
        assert not torch.isfinite(dx[3]).all() or bad == 3e38
        assert not torch.isfinite(dw).all() or bad == 3e38

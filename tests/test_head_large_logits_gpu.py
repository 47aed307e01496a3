"""The output head over logits of any finite size: differences from the largest
are never above 0.  Bounds as in tests/head_ref.py."""

import math

import pytest

from tests.head_ref import LN2, U

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_head_gpu import TYPES, Head  # noqa: E402


@pytest.mark.parametrize("weight", [3.1e3, -7.7e10, 1.3e30, -1.1e38, 2.1e38])
@pytest.mark.parametrize("table,x", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_large_equal_logits(n, table, x, weight):
    """Every row's logit is one product, the same for all: uniform probabilities."""
    rows, cols = 2000, 64
    values = torch.zeros(rows, cols, device="cuda")
    values[:, 7] = weight
    h = Head(rows, cols, table, values=values)
    data = torch.zeros(n, cols, dtype=TYPES[x][0], device="cuda")
    data[:, 7] = 1.0
    ids = torch.arange(n, device="cuda")
    out = h.logprob(data, ids, top_k=3)
    tol = 4 * U * math.log(rows)
    assert ((out["logp"].double() + math.log(rows)).abs() <= tol).all()
    assert ((out["entropy"].double() - math.log(rows)).abs() <= tol).all()
    assert (out["top_ids"] == torch.arange(3, device="cuda")).all()
    # p is 1 / rows to the roundings of lp = (y - max) - log2(sum), at most log2(rows) in size, and of 2^lp; dz of the table's
    # column 0 (x there 0 but in this row) is read off dw
    data[:, 0] = 1.0
    out = h.logprob(data, ids)
    dlogp = torch.zeros(n, device="cuda")
    dlogp[0] = -1.0
    dx, dw = h.grad(data, out["records"], dlogp, None, ids)
    want = torch.full((rows,), 1.0 / rows, dtype=torch.float64, device="cuda")
    want[0] -= 1.0
    half = 2.0 ** -8 if table == x == "bf16" else 0.0  # dz in bf16
    half += 2.0 ** -8 if table == "bf16" else 0.0      # dw's own type
    assert ((dw[:, 0].double() - want).abs() <= want.abs() * (1.01 * half + LN2 * U * 2 * math.log2(rows) + 8 * U)).all()
    assert torch.isfinite(dx).all() and not dx[1:].any()


@pytest.mark.parametrize("size", [1e7, 1e12, 1e30])
@pytest.mark.parametrize("table,x", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_probabilities_of_logits_formed_again(n, table, x, size):
    """The gradient's logits are summed in another order than the forward call's of few tokens: what that moves them by is
    many powers of 2 here, and a probability is at most 1 all the same."""
    rows, cols = 2000, 200
    gen = torch.Generator(device="cuda").manual_seed(n)
    h = Head(rows, cols, table, values=torch.randn(rows, cols, generator=gen, device="cuda") * size)
    data = torch.randn(n, cols, generator=gen, device="cuda").to(TYPES[x][0])
    ids = torch.randint(0, rows, (n,), generator=gen, device="cuda")
    out = h.logprob(data, ids)
    assert torch.isfinite(out["logp"]).all() and (out["logp"] <= 0).all() and (out["entropy"] >= 0).all()
    dlogp = torch.randn(n, generator=gen, device="cuda")
    dx, dw = h.grad(data, out["records"], dlogp, None, ids)
    a = dlogp.double().abs()[:, None]
    # |dz| is at most |a| for a row's target (1 - p) and for the others (p) together twice that; bf16 steps and sums on top
    assert (dw.double().abs() <= 1.02 * (a * data.double().abs()).sum(0)).all()
    top = h.w.double().abs().amax(0)
    spread = 1.02 * (a * top * 2)
    assert (dx.double().abs() <= spread).all()

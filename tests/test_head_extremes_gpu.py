"""The output head at the ends of the fp32 range: finite logits far below the
largest.  Bounds as in tests/head_ref.py."""

import math

import pytest

from matrix_optimizer_owner_amd import binding as B
from tests.head_ref import U, Reference, close

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_head_gpu import Head, batch, stream  # noqa: E402


def masked_head(rows, weight, kind, shards=1):
    """A table whose rows but the first and last 10 hold `weight` in column 3."""
    cols = 64
    gen = torch.Generator(device="cuda").manual_seed(6)
    values = torch.randn(rows, cols, generator=gen, device="cuda") * (2 / math.sqrt(cols))
    values[10:rows - 10, 3] = weight
    keep = torch.cat([torch.arange(10), torch.arange(rows - 10, rows)]).cuda()
    return Head(rows, cols, kind, values=values, shards=shards), keep


# A part of 32 or more rows with y = log2(e) * weight has sum * y past the fp32 range from 1e37 on; 40000 rows joined from
# 1e34 on.  Every logit is finite.
@pytest.mark.parametrize("rows,weight", [(300, -1e37), (300, -1e38), (40000, -1e34), (40000, -2e38)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 50, 700])
def test_finite_logits_far_below_the_largest(rows, weight, kind, n):
    """They have probability 0 and no part in entropy and gradients, as -Inf has; a target there has their log probability."""
    h, keep = masked_head(rows, weight, kind)
    x, _ = batch(n, 64, kind, rows=rows)
    x[:, 3] = 1.0
    ids = torch.arange(n, device="cuda") % 10
    small = Reference(x, h.w[keep], ids, ids >= 0, 1.0)
    for top_k in (0, 4):
        out = h.logprob(x, ids, top_k=top_k)
        small.check_forward(out["logp"], out["entropy"])
    sorted_y, best = small.y.sort(dim=1, descending=True, stable=True)
    best = best[:, :4]
    near = (sorted_y[:, :5].diff(dim=1).abs() <= 2 * small.ey.amax(1, keepdim=True)).any(1)  # order not decided
    assert torch.equal(out["top_ids"][~near], keep[best][~near])
    far = h.logprob(x, torch.full_like(ids, 100))
    # y, its difference from the largest and the product with ln 2 are rounded, and the weight itself is `h.w`
    want = x[:, 3].double() * h.w[100, 3].double()
    assert ((far["logp"].double() - want).abs() <= 8 * U * want.abs()).all()
    assert ((far["entropy"].double() - small.entropy[:, 0]).abs() <= small.entropy_tol[:, 0]).all()
    gen = torch.Generator(device="cuda").manual_seed(n)
    dlogp, dent = (torch.randn(n, generator=gen, device="cuda") for _ in range(2))
    for d in (None, dent):
        dx, dw = h.grad(x, out["records"], dlogp, d, ids)
        rx, ex, rw, ew = small.grads(dlogp, d, torch.bfloat16 if kind == "bf16" else torch.float32)
        close(dx, rx, ex)
        close(dw[keep], rw, ew)
        rest = torch.ones(rows, dtype=torch.bool, device="cuda")
        rest[keep] = False
        assert not dw[rest].any()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_parts_far_below_the_largest_are_joined(kind):
    """Shards of nothing but such logits, first, between and last."""
    rows, n, shards = 4000, 30, 5
    h, _ = masked_head(rows, -1e37, kind, shards=shards)
    x, _ = batch(n, 64, kind, rows=rows)
    x[:, 3] = 1.0
    x[0, 3] = -1.0  # all but the first and last rows' logits are far above instead
    ids = torch.zeros(n, dtype=torch.int64, device="cuda")
    parts = [h.logprob(x, ids, entry=e)["records"] for e in range(shards)]
    ends = torch.cat([torch.arange(10), torch.arange(rows - 10, rows)]).cuda()
    small = Reference(x, h.w[ends], ids, ids >= 0, 1.0)
    for order in ([0, 1, 2, 3, 4], [1, 2, 0, 4, 3], [3, 2, 1, 4, 0]):
        records = torch.cat([parts[e].reshape(-1) for e in order])
        logp, entropy = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        out = torch.empty(n, 6, device="cuda")
        B.head_total(records.data_ptr(), shards, n, out.data_ptr(), logp=logp.data_ptr(), entropy=entropy.data_ptr(),
                     stream=stream())
        assert ((logp.double() - small.logp()).abs()[1:] <= small.logp_tol[1:, 0]).all()
        assert ((entropy.double() - small.entropy[:, 0]).abs()[1:] <= small.entropy_tol[1:, 0]).all()
        # 3980 logits of 1e37 whose differences, steps of their fp32 sums, are far apart or 0: it is finite, and not negative
        assert torch.isfinite(logp[0]) and torch.isfinite(entropy[0]) and entropy[0] >= 0

"""The output head's 256-edge tiles at ragged sizes, and its few-token kernels over
tables of many rows: sizes that the kernels' choice by size sends there.  Bounds
as in tests/head_ref.py."""


import pytest

from tests.head_ref import LN2, U, close

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_head_gpu import Head, batch, reference  # noqa: E402


# logits, dx, dW in 256-tiles: all three; logits and dW of a table read in place; dx alone, whose contraction is not cut
SIZES = [(19990, 1498, 1490, "bf16", "bf16"), (10100, 1024, 1010, "bf16", "bf16"), (700, 4000, 2100, "bf16", "bf16"),
         (7690, 1030, 1490, "f32", "f32"), (7690, 1030, 1490, "f32", "bf16"), (7690, 1498, 1490, "bf16", "f32")]


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("rows,cols,n,table,x", SIZES)
def test_forward_and_gradients(rows, cols, n, table, x, add):
    h = Head(rows, cols, table)
    data, ids = batch(n, cols, x, rows=rows, padded=0.1, outside=0.1)
    # a third of the targets on group and tile borders and in the last rows, some of them many times
    border = torch.tensor([0, 127, 128, 255, 256, 383, 384, rows - 130, rows - 2, rows - 1], device="cuda")
    at = torch.arange(0, n, 3, device="cuda")
    ids[at] = torch.where(ids[at] >= 0, border[at % 10], ids[at])
    scale = 1.2
    out = h.logprob(data, ids, scale=scale)
    ref = reference(h, data, ids, scale)
    ref.check_forward(out["logp"], out["entropy"])
    gen = torch.Generator(device="cuda").manual_seed(9)
    dlogp, dent = (torch.randn(n, generator=gen, device="cuda") for _ in range(2))
    before = torch.randn(rows, cols, generator=gen, device="cuda").to(h.dtype) if add else None
    dx, dw = h.grad(data, out["records"], dlogp, dent, ids, scale, add=before)
    rx, ex, rw, ew = ref.grads(dlogp, dent, torch.bfloat16 if table == x == "bf16" else torch.float32)
    spread = 4e-3 if "bf16" in (table, x) else 2e-5
    close(dx, rx, ex, spread)
    if add:
        rw = rw + before.double()
        ew = ew + U * rw.abs()
    close(dw, rw, ew, None if add else spread)
    assert not dx[ids < 0].any()


@pytest.mark.parametrize("n,top_k", [(300, 20), (300, 64), (1100, 5)])
def test_alternatives(n, top_k):
    """Whole-number logits, exact in fp32: which ids, and in which order, is decided."""
    rows, cols = (32690, 1030) if n == 300 else (16200, 1030)
    gen = torch.Generator(device="cuda").manual_seed(n)
    h = Head(rows, cols, values=torch.randint(-9, 10, (rows, cols), generator=gen, device="cuda").float())
    x = torch.randint(-9, 10, (n, cols), generator=gen, device="cuda").to(torch.bfloat16)
    out = h.logprob(x, None, scale=2.0 ** -8, top_k=top_k)
    z = x.double() @ h.w.double().t()
    want, at = torch.sort(z, dim=1, descending=True, stable=True)
    assert torch.equal(out["top_ids"], at[:, :top_k])
    ref = reference(h, x, None, 2.0 ** -8, exact=True)
    ref.check_forward(out["logp"], out["entropy"])
    lp = ref.lp.gather(1, at[:, :top_k]) * LN2
    assert ((out["top_logp"].double() - lp).abs() <= ref.logp_tol).all()


def few(rows, cols, n, table, x, lead):
    h = Head(rows, cols, table, lead=lead)
    data, ids = batch(n, cols, x, rows=rows, padded=0.1 if n > 4 else 0.0)
    ids[-1] = rows - 1
    data[-1] = torch.nan_to_num(data[-1], 1.0)
    out = h.logprob(data, ids, scale=0.9, top_k=3)
    ref = reference(h, data, ids, 0.9)
    ref.check_forward(out["logp"], out["entropy"])
    best = ref.y.sort(dim=1, descending=True, stable=True)
    near = (best.values[:, :4].diff(dim=1).abs() <= 2 * ref.ey.amax(1, keepdim=True)).any(1)  # order not decided
    decided = ~near & ref.live
    assert torch.equal(out["top_ids"][decided], best.indices[decided, :3])


@pytest.mark.parametrize("n", [1, 5, 32, 33, 64])
@pytest.mark.parametrize("rows", [98304, 98381, 98400])
def test_few_tokens_over_many_rows_of_whole_lines(rows, n):
    few(rows, 128, n, "bf16", "bf16", 128)


@pytest.mark.parametrize("n", [1, 32])
@pytest.mark.parametrize("table,x", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,cols", [(32768, 64), (32801, 131), (32833, 520)])
def test_few_tokens_over_many_rows(rows, cols, table, x, n):
    few(rows, cols, n, table, x, 48)

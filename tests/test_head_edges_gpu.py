"""The output head where its parts meet: equal logits, alternatives of batches
of every size class, targets that many rows share, few tokens over whole and
ragged tables, padding's gradients, other streams.  Bounds as in
tests/head_ref.py."""

import math

import pytest

from matrix_optimizer_owner_amd import binding as B
from tests.head_ref import LN2, U, Reference, close

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_head_gpu import Head, batch, reference, stream  # noqa: E402


@pytest.mark.parametrize("n", [1, 40, 64, 65, 300, 1024, 1025])
@pytest.mark.parametrize("rows", [70, 20000, 40000])
def test_equal_logits(rows, n):
    """Nothing but ties, more of them than any list in shared memory holds: the lowest ids, uniform probabilities."""
    h = Head(rows, 40)
    x, ids = batch(n, 40, rows=rows)
    out = h.logprob(x, ids, scale=0.0, top_k=64)
    assert (out["top_ids"] == torch.arange(64, device="cuda")).all()
    # a sum of `rows` ones is exact; its logarithm and the product with ln 2 are rounded
    tol = 4 * U * math.log(rows)
    assert ((out["logp"].double() + math.log(rows)).abs() <= tol).all()
    assert ((out["top_logp"].double() + math.log(rows)).abs() <= tol).all()
    assert ((out["entropy"].double() - math.log(rows)).abs() <= tol).all()


@pytest.mark.parametrize("n", [33, 64, 65, 182, 1023, 1024, 1025])
@pytest.mark.parametrize("rows,top_k", [(9291, 20), (20000, 64), (700, 3)])
def test_alternatives_of_any_batch(rows, top_k, n):
    """Whole-number logits of a wide range, exact in fp32: which ids, and in which order, is decided."""
    cols = 33
    gen = torch.Generator(device="cuda").manual_seed(rows + n)
    h = Head(rows, cols, values=torch.randint(-60, 61, (rows, cols), generator=gen, device="cuda").float())
    x = torch.randint(-60, 61, (n, cols), generator=gen, device="cuda").to(torch.bfloat16)
    out = h.logprob(x, None, scale=2.0 ** -10, top_k=top_k, logits=True)
    z = x.double() @ h.w.double().t()
    z, at = torch.sort(z, dim=1, descending=True, stable=True)
    assert torch.equal(out["top_ids"], at[:, :top_k])
    ref = reference(h, x, None, 2.0 ** -10, exact=True)
    want = ref.lp.gather(1, at[:, :top_k]) * LN2
    assert ((out["top_logp"].double() - want).abs() <= ref.logp_tol).all()


@pytest.mark.parametrize("k", [0.0, 1.0, -1.0])
@pytest.mark.parametrize("n", [1, 50, 700])
def test_logits_of_minus_infinity(n, k):
    """A weight of -Inf against x of one sign: such rows have probability 0, are no target's neighbours, and come last
    among the alternatives; a target there has log probability -Inf."""
    rows, cols = 300, 64
    h = Head(rows, cols)
    x, _ = batch(n, cols, rows=rows)
    x[:, 3] = 1.0
    h.w[10:290, 3] = -math.inf
    h.view(h.params, h.offs[0], rows).copy_(h.w)
    ids = torch.full((n,), 5 if k == 0 else 100, device="cuda")
    if k < 0:
        ids[:] = -1
    out = h.logprob(x, ids, top_k=24)
    keep = torch.cat([torch.arange(10), torch.arange(290, 300)]).cuda()
    small = Reference(x, h.w[keep], ids.clamp(0, 9), ids >= 0, 1.0)
    if k < 0:
        assert not out["logp"].any() and not out["entropy"].any() and (out["top_ids"] == -1).all()
        return
    if k == 0:
        small.check_forward(out["logp"], out["entropy"])
    else:
        assert (out["logp"] == -math.inf).all()
        assert ((out["entropy"].double() - small.entropy[:, 0]).abs() <= small.entropy_tol[:, 0]).all()
    assert torch.equal(out["top_ids"][:, :20].sort(1).values, keep.expand(n, 20))


@pytest.mark.parametrize("table,x", [("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("spread", ["one", "last", "borders", "skewed"])
@pytest.mark.parametrize("n", [40, 1500])
def test_gradients_of_shared_targets(n, spread, table, x):
    rows, cols = 1003, 200
    h = Head(rows, cols, table)
    data, _ = batch(n, cols, x, rows=rows)
    gen = torch.Generator(device="cuda").manual_seed(n)
    if spread == "one":
        ids = torch.full((n,), 128, device="cuda")
    elif spread == "last":
        ids = torch.full((n,), rows - 1, device="cuda")
    elif spread == "borders":
        ids = torch.tensor([0, 127, 128, 255, 256, 895, 896, rows - 1, rows, -1], device="cuda")[
            torch.randint(0, 10, (n,), generator=gen, device="cuda")]
    else:
        ids = (rows ** torch.rand(n, generator=gen, device="cuda")).long().clamp_max(rows) - 1
    out = h.logprob(data, ids)
    ref = reference(h, data, ids, 1.0)
    ref.check_forward(out["logp"], out["entropy"])
    dlogp, dent = (torch.randn(n, generator=gen, device="cuda") for _ in range(2))
    dx, dw = h.grad(data, out["records"], dlogp, dent, ids)
    dz_type = torch.bfloat16 if table == x == "bf16" else torch.float32
    rx, ex, rw, ew = ref.grads(dlogp, dent, dz_type)
    close(dx, rx, ex, 4e-3)
    close(dw, rw, ew, 4e-3)


@pytest.mark.parametrize("n", [1, 16, 32, 33, 47, 64])
@pytest.mark.parametrize("rows", [1, 31, 33, 1000, 8195])
@pytest.mark.parametrize("cols", [64, 256, 1088])
def test_few_tokens_over_whole_lines(rows, cols, n):
    h = Head(rows, cols, lead=128)
    x, ids = batch(n, cols, rows=rows, padded=0.2, outside=0.1)
    out = h.logprob(x, ids, scale=0.9)
    reference(h, x, ids, 0.9).check_forward(out["logp"], out["entropy"])


@pytest.mark.parametrize("n", [1, 33, 64])
@pytest.mark.parametrize("table,x", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("cols", [1, 7, 9, 63, 131, 513])
def test_few_tokens_over_odd_rows(cols, n, table, x):
    rows = 517
    h = Head(rows, cols, table, lead=48)
    data, ids = batch(n, cols, x, rows=rows, padded=0.1)
    wide = torch.full((n * (cols + 3) + 8,), float("nan"), dtype=data.dtype, device="cuda")
    at = wide[1:1 + n * (cols + 3)].view(n, cols + 3)
    at[:, :cols] = data
    out = h.logprob(at, ids, x_stride=cols + 3)
    reference(h, data, ids, 1.0).check_forward(out["logp"], out["entropy"])


@pytest.mark.parametrize("n", [30, 300])
def test_padding_and_outside_rows_give_no_gradient(n):
    """Non-finite gradients, records and x at padding reach nothing; an id outside the table has no part in dlogp."""
    rows, cols = 400, 72
    h = Head(rows, cols)
    x, ids = batch(n, cols, rows=rows, padded=0.3, outside=0.2)
    out = h.logprob(x, ids)
    gen = torch.Generator(device="cuda").manual_seed(3)
    dlogp, dent = (torch.randn(n, generator=gen, device="cuda") for _ in range(2))
    ref = reference(h, x, ids, 1.0)
    rx, ex, rw, ew = ref.grads(dlogp, dent, torch.bfloat16)
    dlogp[ids < 0] = math.nan
    dent[ids < 0] = math.inf
    dlogp[ids >= rows] = 1e30
    dx, dw = h.grad(x, out["records"], dlogp, dent, ids)
    close(dx, rx, ex, 4e-3)
    close(dw, rw, ew, 4e-3)
    assert not dx[ids < 0].any()
    # all rows padding: zeros, or what was there
    none = torch.full_like(ids, -3)
    out = h.logprob(x, none)
    assert not out["records"].any() and not out["logp"].any()
    dx, dw = h.grad(x, out["records"], dlogp, dent, none)
    assert not dx.any() and not dw.any()
    keep = torch.randn(rows, cols, generator=gen, device="cuda").to(torch.bfloat16)
    _, dw = h.grad(x, out["records"], dlogp, dent, none, add=keep)
    assert torch.equal(dw, keep)


def test_gradients_on_another_stream():
    rows, cols, n = 900, 128, 200
    h = Head(rows, cols)
    x, ids = batch(n, cols, rows=rows)
    dlogp = torch.ones(n, device="cuda")
    out = h.logprob(x, ids)
    want = h.grad(x, out["records"], dlogp, None, ids)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = h.logprob(x, ids)
        grads = h.grad(x, got["records"], dlogp, None, ids)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got["records"], out["records"])
    assert torch.equal(grads[0], want[0]) and torch.equal(grads[1], want[1])


def test_two_captured_graphs_share_a_workspace():
    """Replayed in turn on one stream, each call's results depend on nothing that the other left in the workspace."""
    rows, cols = 2100, 192
    h = Head(rows, cols)
    calls, graphs, wants, kept = [], [], [], []  # a graph's tensors outlive it
    ws = h.space(300, B.BF16, 8, grad=True)
    for n in (30, 300):
        x, ids = batch(n, cols, rows=rows, seed=n, padded=0.1)
        rec, logp = torch.empty(n, 6, device="cuda"), torch.empty(n, device="cuda")
        top = torch.empty(n, 8, dtype=torch.int64, device="cuda")
        dlogp = torch.randn(n, device="cuda")
        dx, grads = torch.empty_like(x), torch.zeros(h.nbytes, dtype=torch.uint8, device="cuda")

        def call(n=n, x=x, ids=ids, rec=rec, logp=logp, top=top, dlogp=dlogp, dx=dx, grads=grads):
            h.plan.head_logprob(0, h.params.data_ptr(), x.data_ptr(), n, rec.data_ptr(), ws.data_ptr(), ws.numel(),
                                ids=ids.data_ptr(), logp=logp.data_ptr(), top_k=8, top_ids=top.data_ptr(), stream=stream())
            h.plan.head_grad(0, h.params.data_ptr(), grads.data_ptr(), x.data_ptr(), n, rec.data_ptr(), dlogp.data_ptr(),
                             ws.data_ptr(), ws.numel(), dx=dx.data_ptr(), ids=ids.data_ptr(), stream=stream())

        call()
        torch.cuda.synchronize()
        outs = (rec.view(torch.int32), logp, top, dx, grads)
        wants.append([o.clone() for o in outs])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)
        kept.append(call)
        calls.append(outs)
    for turn in range(3):
        for k in (0, 1, 0):
            for o in calls[k]:
                o.zero_()
            graphs[k].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(calls[k], wants[k])), (turn, k)

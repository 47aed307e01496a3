"""The output head over a table of the owner buffer against a 64-bit
reference: log probabilities, entropy, alternatives, joined tables, gradients.
Bounds are derived in tests/head_ref.py."""

import math

import pytest

from matrix_optimizer_owner_amd import binding as B
from tests.head_ref import LN2, U, Reference, close

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, B.BF16), "f32": (torch.float32, B.F32)}


def stream():
    return torch.cuda.current_stream().cuda_stream


def canary(shape, dtype, fill=7.0):
    """A tensor of `shape` with 64 elements of a known value before and after it."""
    n = math.prod(shape)
    whole = torch.full((n + 128,), fill, dtype=dtype, device="cuda")
    return whole, whole[64:64 + n].view(shape)


def intact(whole, fill=7.0):
    assert (whole[:64] == fill).all() and (whole[-64:] == fill).all()


class Head:
    """A table cut into `shards` entries of one buffer whose other bytes are NaN."""

    def __init__(self, rows, cols, table="bf16", shards=1, seed=1, values=None, role=B.ROLE_ADAMW8, lead=16):
        self.rows, self.cols = rows, cols
        self.dtype, kind = TYPES[table]
        gen = torch.Generator(device="cuda").manual_seed(seed)
        values = torch.randn(rows, cols, generator=gen, device="cuda") * (2 / math.sqrt(cols)) if values is None else values
        self.w = values.to(self.dtype)
        cut = [rows * k // shards for k in range(shards + 1)]
        self.firsts = cut[:-1]
        es = self.dtype.itemsize
        offs, at = [], lead
        for a, b in zip(cut, cut[1:]):
            offs.append(at)
            at += -(-(b - a) * cols * es // 16) * 16 + 32
        self.params = torch.full((at + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        for o, a, b in zip(offs, cut, cut[1:]):
            self.view(self.params, o, b - a).copy_(self.w[a:b])
        self.offs, self.sizes, self.nbytes = offs, [b - a for a, b in zip(cut, cut[1:])], at + 64
        self.plan = B.OwnerPlan([B.TableEntry(o, r, cols, kind, role) for o, r in zip(offs, self.sizes)], self.nbytes,
                                B.make_hparams())

    def view(self, buf, off, rows):
        return buf[off:off + rows * self.cols * self.dtype.itemsize].view(self.dtype).view(rows, self.cols)

    def space(self, n, x_type, top_k=0, grad=False, entry=0):
        need = self.plan.head_workspace_bytes(entry, n, x_type=x_type, top_k=top_k, grad=grad)
        return torch.full((max(need, 256),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten

    def logprob(self, x, ids=None, scale=1.0, top_k=0, x_stride=0, entry=0, logits=False):
        n = x.shape[0]
        xt = B.BF16 if x.dtype == torch.bfloat16 else B.F32
        ws = self.space(n, xt, top_k, entry=entry)
        rw, records = canary((n, 6), torch.float32)
        lw, logp = canary((n,), torch.float32)
        ew, entropy = canary((n,), torch.float32)
        iw, top_ids = canary((n, top_k), torch.int64, 7)
        tw, top = canary((n, top_k), torch.float32)
        gw, tlog = canary((n, top_k), torch.float32)
        self.plan.head_logprob(entry, self.params.data_ptr(), x.data_ptr(), n, records.data_ptr(), ws.data_ptr(), ws.numel(),
                               ids=0 if ids is None else ids.data_ptr(),
                               id_type=B.I32 if ids is not None and ids.dtype == torch.int32 else B.I64, x_type=xt,
                               x_stride=x_stride, first_id=self.firsts[entry], scale=scale, logp=logp.data_ptr(),
                               entropy=entropy.data_ptr(), top_k=top_k, top_ids=top_ids.data_ptr() if top_k else 0,
                               top_logp=top.data_ptr() if top_k else 0, top_logits=tlog.data_ptr() if top_k else 0,
                               stream=stream())
        for w in (rw, lw, ew, tw, gw):
            intact(w)
        intact(iw, 7)
        return dict(records=records, logp=logp, entropy=entropy, top_ids=top_ids, top_logp=top, top_logits=tlog)

    def grad(self, x, records, dlogp, dentropy=None, ids=None, scale=1.0, x_stride=0, dx_stride=0, entry=0, add=None,
             want_dx=True, want_dw=True):
        n = x.shape[0]
        xt = B.BF16 if x.dtype == torch.bfloat16 else B.F32
        ws = self.space(n, xt, grad=True, entry=entry)
        width = dx_stride or self.cols
        dw_whole, dx = canary((n, width), x.dtype)
        grads = torch.full((self.nbytes,), 0x5A, dtype=torch.uint8, device="cuda")
        mine = self.view(grads, self.offs[entry], self.sizes[entry])
        if add is not None:
            mine.copy_(add)
        before = grads.clone()
        self.plan.head_grad(entry, self.params.data_ptr(), grads.data_ptr() if want_dw else 0, x.data_ptr(), n,
                            records.data_ptr(), dlogp.data_ptr(), ws.data_ptr(), ws.numel(),
                            dentropy=0 if dentropy is None else dentropy.data_ptr(), dx=dx.data_ptr() if want_dx else 0,
                            ids=0 if ids is None else ids.data_ptr(),
                            id_type=B.I32 if ids is not None and ids.dtype == torch.int32 else B.I64, x_type=xt,
                            x_stride=x_stride, dx_stride=dx_stride, first_id=self.firsts[entry], scale=scale,
                            accumulate=add is not None, stream=stream())
        intact(dw_whole)
        if width > self.cols:
            assert (dx[:, self.cols:] == 7).all()
        same = torch.ones(self.nbytes, dtype=torch.bool, device="cuda")
        if want_dw:
            o = self.offs[entry]
            same[o:o + self.sizes[entry] * self.cols * self.dtype.itemsize] = False
        assert torch.equal(before[same], grads[same])
        if not want_dx:
            assert (dx == 7).all()
        return dx[:, :self.cols], mine


def batch(n, cols, x="bf16", seed=2, rows=None, ids="i64", padded=0.0, outside=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    data = torch.randn(n, cols, generator=gen, device="cuda").to(TYPES[x][0])
    t = torch.randint(0, rows, (n,), generator=gen, device="cuda")
    u = torch.rand(n, generator=gen, device="cuda")
    t = torch.where(u < outside, t + rows, t)
    t = torch.where(u > 1 - padded, -1 - t, t)
    data[t < 0] = float("nan")  # what padding holds is not read into a result
    return data, t.to(torch.int32 if ids == "i32" else torch.int64)


def reference(h, x, ids, scale, entry=None, exact=False):
    live = torch.ones(len(x), dtype=torch.bool, device="cuda") if ids is None else ids >= 0
    t = torch.full((len(x),), -1, device="cuda") if ids is None else ids.long()
    t = torch.where((t >= 0) & (t < h.rows), t, -1)
    return Reference(x, h.w, t, live, scale, exact=exact)


SHAPES = [(1, 1, 1), (7, 3, 5), (64, 64, 3), (127, 65, 33), (128, 64, 64), (129, 192, 65), (300, 100, 128), (513, 128, 129),
          (1000, 515, 257), (2500, 72, 600), (777, 1001, 40)]
PAIRS = [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("table,x", PAIRS)
@pytest.mark.parametrize("rows,cols,n", SHAPES)
def test_forward_and_gradients(rows, cols, n, table, x):
    h = Head(rows, cols, table)
    data, ids = batch(n, cols, x, rows=rows, padded=0.15 if n > 4 else 0.0, outside=0.1 if n > 4 else 0.0)
    scale = 1.3
    out = h.logprob(data, ids, scale=scale)
    ref = reference(h, data, ids, scale)
    ref.check_forward(out["logp"], out["entropy"])
    gen = torch.Generator(device="cuda").manual_seed(9)
    dlogp, dent = (torch.randn(n, generator=gen, device="cuda") for _ in range(2))
    add = torch.randn(rows, cols, generator=gen, device="cuda").to(h.dtype) if n % 2 else None
    dx, dw = h.grad(data, out["records"], dlogp, dent, ids, scale, add=add)
    dz_type = torch.bfloat16 if table == x == "bf16" else torch.float32
    rx, ex, rw, ew = ref.grads(dlogp, dent, dz_type)
    # rounding errors of dz and of the outputs are independent from element to element: 2^-8 / sqrt(3) each at most
    spread = 4e-3 if "bf16" in (table, x) else 2e-5
    close(dx, rx, ex, spread)
    if add is not None:
        rw = rw + add.double()
        ew = ew + U * rw.abs()
    close(dw, rw, ew, spread if add is None else None)
    assert not dx[ids < 0].any()


@pytest.mark.parametrize("n", [1, 31, 64, 65, 200])
@pytest.mark.parametrize("table,x", PAIRS)
@pytest.mark.parametrize("rows,top_k", [(3, 5), (64, 64), (129, 1), (1000, 20), (5003, 8)])
def test_alternatives_with_ties(rows, top_k, n, table, x):
    """Whole-number logits, exact in fp32 in any order: ranks and ties are decided, to the lower id."""
    cols = 96
    gen = torch.Generator(device="cuda").manual_seed(rows + n)
    h = Head(rows, cols, table, values=torch.randint(-3, 4, (rows, cols), generator=gen, device="cuda").float())
    data = torch.randint(-2, 3, (n, cols), generator=gen, device="cuda").to(TYPES[x][0])
    ids = torch.randint(0, rows, (n,), generator=gen, device="cuda")
    if n > 3:
        ids[2] = -1
    out = h.logprob(data, ids, scale=0.25, top_k=top_k)
    ref = reference(h, data, ids, 0.25, exact=True)
    ref.check_forward(out["logp"], out["entropy"])
    z = (data.double() @ h.w.double().t()).cpu()
    z, at = torch.sort(z, dim=1, descending=True, stable=True)
    k = min(top_k, rows)
    want = torch.full((n, top_k), -1)
    want[:, :k] = at[:, :k]
    live = ref.live.cpu()
    want[~live] = -1
    assert torch.equal(out["top_ids"].cpu(), want)
    lp = torch.full((n, top_k), -math.inf, dtype=torch.float64)
    lp[:, :k] = ref.lp.cpu().gather(1, at[:, :k]) * LN2
    lp[~live] = -math.inf
    got = out["top_logp"].double().cpu()
    assert torch.equal(torch.isinf(got), torch.isinf(lp))
    fine = ~torch.isinf(lp)
    assert ((got - lp).abs()[fine] <= ref.logp_tol.cpu().expand_as(lp)[fine]).all()


@pytest.mark.parametrize("shards", [1, 2, 5])
@pytest.mark.parametrize("n", [40, 300])
def test_joined_tables(shards, n):
    """A table cut into entries gives the whole table's results, alternatives and ties among them included."""
    rows, cols, k = 1003, 64, 12
    gen = torch.Generator(device="cuda").manual_seed(5)
    values = torch.randint(-3, 4, (rows, cols), generator=gen, device="cuda").float()
    whole, cut = Head(rows, cols, values=values), Head(rows, cols, values=values, shards=shards)
    data = torch.randint(-2, 3, (n, cols), generator=gen, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, rows, (n,), generator=gen, device="cuda")
    ids[3], ids[4] = -5, rows + 7
    one = whole.logprob(data, ids, scale=0.5, top_k=k)
    parts = [cut.logprob(data, ids, scale=0.5, top_k=k, entry=e) for e in range(shards)]
    records = torch.cat([p["records"].reshape(-1) for p in parts])
    pid = torch.cat([p["top_ids"].reshape(-1) for p in parts])
    plog = torch.cat([p["top_logits"].reshape(-1) for p in parts])
    logp, entropy = (torch.empty(n, device="cuda") for _ in range(2))
    tid, tlp, tlog = torch.empty(n, k, dtype=torch.int64, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(n, k, device="cuda")
    B.head_total(records.data_ptr(), shards, n, records.data_ptr(), logp=logp.data_ptr(), entropy=entropy.data_ptr(), top_k=k,
                 part_top_ids=pid.data_ptr(), part_top_logits=plog.data_ptr(), top_ids=tid.data_ptr(),
                 top_logp=tlp.data_ptr(), top_logits=tlog.data_ptr(), stream=stream())
    ref = reference(whole, data, ids, 0.5, exact=True)
    ref.check_forward(logp, entropy)
    assert torch.equal(tid, one["top_ids"]) and torch.equal(tlog, one["top_logits"])
    fine = tid >= 0
    assert ((tlp - one["top_logp"]).abs()[fine] <= 2 * ref.logp_tol.expand_as(tlp)[fine]).all()
    assert torch.equal(tlp == -math.inf, ~fine)
    # gradients of the cut table from the joined records: dx adds up, the tables' gradients are its rows
    joined = records[:6 * n]
    dlogp = torch.randn(n, generator=gen, device="cuda")
    dent = torch.randn(n, generator=gen, device="cuda") * 0.1
    rx, ex, rw, ew = ref.grads(dlogp, dent, torch.bfloat16)
    got = [cut.grad(data, joined, dlogp, dent, ids, 0.5, entry=e) for e in range(shards)]
    dx = torch.stack([g[0].double() for g in got])
    tol = ex + 2.0 ** -8 * dx.abs().sum(0) * 1.01
    assert ((dx.sum(0) - rx).abs() <= tol).all()
    close(torch.cat([g[1] for g in got]), rw, ew, 4e-3)


def test_empty_tables_and_batches():
    h = Head(0, 8)
    x = torch.ones(3, 8, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([2, -1, 0], device="cuda")
    out = h.logprob(x, ids, top_k=2)
    assert not out["logp"].any() and not out["entropy"].any() and (out["top_ids"] == -1).all()
    assert (out["top_logp"] == -math.inf).all()
    rec = out["records"]
    assert rec[0].tolist()[:4] == [-math.inf, 0, 0, 0] and not rec[1].any()
    dx, _ = h.grad(x, rec, torch.ones(3, device="cuda"), ids=ids)
    assert not dx.any()
    h = Head(5, 8)
    none = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    h.logprob(none)
    dl = torch.ones(1, device="cuda")
    _, dw = h.grad(none, rec, dl)
    assert not dw.any()
    keep = torch.ones(5, 8, device="cuda")
    _, dw = h.grad(none, rec, dl, add=keep)
    assert (dw == 1).all()
    # an empty part beside a full one changes nothing
    full = h.logprob(x, ids)
    both = torch.cat([full["records"].reshape(-1), Head(0, 8).logprob(x, ids)["records"].reshape(-1)])
    out = torch.empty(3, 6, device="cuda")
    B.head_total(both.data_ptr(), 2, 3, out.data_ptr(), stream=stream())
    assert torch.equal(out, full["records"])


@pytest.mark.parametrize("scale", [-0.7, 0.0, 30.0])
def test_scales(scale):
    h = Head(700, 80, "f32")
    x, ids = batch(90, 80, "f32", rows=700)
    out = h.logprob(x, ids, scale=scale, top_k=3)
    ref = reference(h, x, ids, scale)
    ref.check_forward(out["logp"], out["entropy"])
    if scale == 0:
        assert (out["top_ids"] == torch.arange(3, device="cuda")).all()
        assert ((out["logp"].double() + math.log(700)).abs() <= ref.logp_tol[:, 0]).all()
    dlogp = torch.ones(90, device="cuda")
    dx, dw = h.grad(x, out["records"], dlogp, dlogp * 0.1, ids, scale)
    rx, ex, rw, ew = ref.grads(dlogp, dlogp * 0.1, torch.float32)
    close(dx, rx, ex)
    close(dw, rw, ew)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("shift,stride", [(0, 131), (1, 128), (3, 200), (0, 136)])
def test_strides_and_alignment(shift, stride, x):
    n, cols, rows = 150, 128, 400
    h = Head(rows, cols, "f32" if x == "f32" else "bf16", lead=16 * 3)
    data, ids = batch(n, cols, x, rows=rows, ids="i32", padded=0.1)
    wide = torch.full((n * stride + 8,), float("nan"), dtype=data.dtype, device="cuda")
    rows_ = wide[shift:shift + n * stride].view(n, stride)
    rows_[:, :cols] = data
    out = h.logprob(rows_, ids, x_stride=stride)
    ref = reference(h, data, ids, 1.0)
    ref.check_forward(out["logp"], out["entropy"])
    dlogp = torch.ones(n, device="cuda")
    dx, dw = h.grad(rows_, out["records"], dlogp, None, ids, x_stride=stride, dx_stride=stride + 1)
    rx, ex, rw, ew = ref.grads(dlogp, None, data.dtype)
    close(dx, rx, ex)
    close(dw, rw, ew)


def test_one_output_at_a_time_and_no_ids():
    h = Head(300, 64)
    x, ids = batch(100, 64, rows=300)
    out = h.logprob(x, None, top_k=4)
    ref = reference(h, x, None, 1.0)
    assert not out["logp"].any()
    ref.check_forward(out["logp"], out["entropy"])
    both = h.grad(x, out["records"], torch.ones(100, device="cuda"), torch.ones(100, device="cuda"))
    rx, ex, rw, ew = ref.grads(torch.ones(100, device="cuda"), torch.ones(100, device="cuda"), torch.bfloat16)
    close(both[0], rx, ex, 4e-3)
    close(both[1], rw, ew, 4e-3)
    alone = h.grad(x, out["records"], torch.ones(100, device="cuda"), torch.ones(100, device="cuda"), want_dw=False)[0]
    assert torch.equal(alone, both[0])
    alone = h.grad(x, out["records"], torch.ones(100, device="cuda"), torch.ones(100, device="cuda"), want_dx=False)[1]
    assert torch.equal(alone, both[1])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n", [20, 200])
def test_non_finite_values(n, kind):
    """A NaN in one row of x spoils that row alone.  An infinite weight spoils the rows whose logit it makes +Inf or NaN,
    and may spoil (fp32) or leave finite (bf16) those where it is -Inf; padding stays zero."""
    h = Head(500, 64, kind)
    x, _ = batch(n, 64, kind, rows=500)
    ids = torch.arange(n, device="cuda")
    x[3, 5] = float("nan")
    out = h.logprob(x, ids, top_k=2)
    bad = torch.isnan(out["logp"])
    assert bad[3] and int(bad.sum()) == 1 and torch.isnan(out["entropy"][3])
    assert (out["top_ids"][3] == -1).all()
    h.w[77, 2] = float("inf")
    h.view(h.params, h.offs[0], 500).copy_(h.w)
    ids[4] = -1
    out = h.logprob(x, ids, top_k=2)
    z = x[:, 2]
    up = torch.isnan(z) | (z > 0) | torch.isnan(x).any(1)
    up[4] = False
    got = torch.isnan(out["logp"])
    assert got[up].all() and out["logp"][4] == 0 and out["entropy"][4] == 0
    if kind == "bf16":
        assert torch.equal(got, up)
        best = out["top_ids"][:, 0]
        assert (best[(z > 0) & ~torch.isnan(x).any(1) & (ids >= 0)] == 77).all()
    dx, _ = h.grad(x, out["records"], torch.ones(n, device="cuda"), None, ids)
    assert not dx[4].any()


def test_gradients_against_differences():
    """Directional derivatives of sum(a logp + b H), from the operator's own outputs half a step apart either way."""
    rows, cols, n = 900, 96, 70
    gen = torch.Generator(device="cuda").manual_seed(8)
    h = Head(rows, cols, "f32")
    x, ids = batch(n, cols, "f32", rows=rows)
    a, b = torch.randn(n, generator=gen, device="cuda"), torch.randn(n, generator=gen, device="cuda")
    out = h.logprob(x, ids)
    dx, dw = h.grad(x, out["records"], a, b, ids)
    table = h.view(h.params, h.offs[0], rows)
    w0 = table.clone()

    def f(xs):
        o = h.logprob(xs, ids)
        return float((a.double() * o["logp"].double() + b.double() * o["entropy"].double()).sum())

    ux = torch.randn(n, cols, generator=gen, device="cuda") / math.sqrt(cols)
    uw = torch.randn(rows, cols, generator=gen, device="cuda") / math.sqrt(cols)
    # Central differences at steps s and 2s, extrapolated: what is left is of the fifth order in a step, over logits that
    # move by at most about 4 s; and the outputs' own error, 2e-6 each at most here, over s: 70 * 3 * 2e-6 * 1.7 / s.
    s = 1 / 32

    def slope(step, base):
        return (base(step) - base(-step)) / (2 * step)

    def at_w(step):
        table.copy_(w0 + step * uw)
        return f(x)

    for base, want in ((lambda t: f(x + t * ux), (dx.double() * ux.double()).sum()),
                       (at_w, (dw.double() * uw.double()).sum())):
        got = (4 * slope(s, base) - slope(2 * s, base)) / 3
        assert abs(got - float(want)) <= 0.03 + 1e-3 * abs(float(want)), (got, float(want))
    table.copy_(w0)


@pytest.mark.parametrize("n,top_k", [(12, 3), (150, 0)])
def test_captured_replayed_and_repeated(n, top_k):
    rows, cols = 3000, 256
    h = Head(rows, cols)
    x, ids = batch(n, cols, rows=rows, padded=0.1)
    ws = h.space(n, B.BF16, top_k, grad=True)
    rec, logp, ent = torch.empty(n, 6, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    tid, tlp = torch.empty(n, max(top_k, 1), dtype=torch.int64, device="cuda"), torch.empty(n, max(top_k, 1), device="cuda")
    dlogp = torch.randn(n, device="cuda")
    dx = torch.empty(n, cols, dtype=torch.bfloat16, device="cuda")
    grads = torch.zeros(h.nbytes, dtype=torch.uint8, device="cuda")

    def call():
        h.plan.head_logprob(0, h.params.data_ptr(), x.data_ptr(), n, rec.data_ptr(), ws.data_ptr(), ws.numel(),
                            ids=ids.data_ptr(), logp=logp.data_ptr(), entropy=ent.data_ptr(), top_k=top_k,
                            top_ids=tid.data_ptr(), top_logp=tlp.data_ptr(), stream=stream())
        h.plan.head_grad(0, h.params.data_ptr(), grads.data_ptr(), x.data_ptr(), n, rec.data_ptr(), dlogp.data_ptr(),
                         ws.data_ptr(), ws.numel(), dx=dx.data_ptr(), ids=ids.data_ptr(), stream=stream())

    def outputs():
        torch.cuda.synchronize()
        return [t.clone() for t in (rec.view(torch.int32), logp, ent, dx, grads) + ((tid, tlp) if top_k else ())]

    call()
    first = outputs()
    call()
    assert all(torch.equal(a, b) for a, b in zip(first, outputs()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        x.copy_(batch(n, cols, seed=20 + k, rows=rows)[0])
        x[ids < 0] = float("nan")
        call()
        want = outputs()
        for t in (rec, logp, ent, dx):
            t.zero_()
        ws.fill_(0xFF)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, outputs()))


def test_two_streams_with_a_workspace_each():
    h = Head(5000, 512)
    x1, i1 = batch(300, 512, rows=5000, seed=3)
    x2, i2 = batch(40, 512, rows=5000, seed=4)
    want = h.logprob(x1, i1), h.logprob(x2, i2, top_k=3)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = h.logprob(x1, i1)
        with torch.cuda.stream(s2):
            b = h.logprob(x2, i2, top_k=3)
        torch.cuda.synchronize()
        assert torch.equal(a["logp"], want[0]["logp"]) and torch.equal(a["entropy"], want[0]["entropy"])
        assert torch.equal(b["logp"], want[1]["logp"]) and torch.equal(b["top_ids"], want[1]["top_ids"])


def test_a_table_past_32_bits():
    """4194304 x 600 bf16: 5 GB, the most rows an entry may have; each row's logits are its number's, by construction."""
    rows, cols, n = 1 << 22, 600, 3
    plan = B.OwnerPlan([B.TableEntry(0, rows, cols, B.BF16, B.ROLE_ADAMW)], rows * cols * 2, B.make_hparams())
    w = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(rows, device="cuda")
    digits = [(at >> (4 * k)) & 15 for k in range(6)]  # of the row's number, each exact
    for k, d in enumerate(digits):
        w[:, cols - 1 - k] = d.to(torch.bfloat16)
    x = torch.zeros(n, cols, dtype=torch.bfloat16, device="cuda")
    x[0, cols - 6] = 1.0       # largest where the top digit is: rows 0x300000 on (the top digit has two bits)
    x[1, cols - 1] = -1.0      # least where the lowest digit is 0
    x[2, cols - 1], x[2, cols - 6] = 1.0, 2.0
    ids = torch.tensor([rows - 1, 16, rows - 2], device="cuda")
    for count in (n, 70):      # few rows, and a batch of tiles
        xs, is_ = x.repeat(-(-count // n), 1)[:count].contiguous(), ids.repeat(-(-count // n))[:count].contiguous()
        ws = torch.empty(plan.head_workspace_bytes(0, count, top_k=3), dtype=torch.uint8, device="cuda")
        rec, logp, ent = torch.empty(count, 6, device="cuda"), torch.empty(count, device="cuda"), torch.empty(count, device="cuda")
        tid, tlp = torch.empty(count, 3, dtype=torch.int64, device="cuda"), torch.empty(count, 3, device="cuda")
        plan.head_logprob(0, w.data_ptr(), xs.data_ptr(), count, rec.data_ptr(), ws.data_ptr(), ws.numel(), ids=is_.data_ptr(),
                          logp=logp.data_ptr(), entropy=ent.data_ptr(), top_k=3, top_ids=tid.data_ptr(),
                          top_logp=tlp.data_ptr(), stream=stream())
        for i in range(count):
            j = i % n
            z = (digits[5].double(), -digits[0].double(), digits[0].double() + 2 * digits[5].double())[j]
            lse = torch.logsumexp(z, 0)
            p = torch.exp(z - lse)
            # y is exact but for one rounding of 33 at most; sums of exponentials: joins of 32768 to 131072 parts
            tol = 4 * U * 50 + 4096 * U
            assert abs(float(logp[i]) - float(z[is_[i]] - lse)) <= tol
            assert abs(float(ent[i]) + float((p * (z - lse)).sum())) <= 20 * tol
            first = (0x300000, 0, 0x30000F)[j]
            step = (1, 16, 16)[j]
            assert tid[i].tolist() == [first, first + step, first + 2 * step]


def test_gradient_of_a_batch_past_32_bits():
    """20000 rows over 128256: dz alone is 5 GB.  Spot rows of dx and of the table's gradient against 64 bits."""
    rows, cols, n = 128256, 64, 20000
    h = Head(rows, cols)
    x, ids = batch(n, cols, rows=rows)
    out = h.logprob(x, ids)
    dlogp = torch.randn(n, device="cuda")
    dx, dw = h.grad(x, out["records"], dlogp, None, ids)
    spots = [0, 1, 12345, 16777, n - 1]
    ref = Reference(x[spots], h.w, ids[spots], torch.ones(len(spots), dtype=torch.bool, device="cuda"), 1.0)
    rx, ex, _, _ = ref.grads(dlogp[spots], None, torch.bfloat16)
    close(dx[spots], rx, ex)
    assert ((out["logp"][spots].double() - ref.logp()).abs() <= ref.logp_tol[:, 0]).all()
    # some rows of the table's gradient, the batch in pieces
    some = [0, 77, 65536, rows - 1]
    want = torch.zeros(len(some), cols, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for a in range(0, n, 1000):
        r = Reference(x[a:a + 1000], h.w, ids[a:a + 1000], torch.ones(1000, dtype=torch.bool, device="cuda"), 1.0)
        hot = (ids[a:a + 1000, None] == torch.tensor(some, device="cuda")).double()
        dz = dlogp[a:a + 1000].double()[:, None] * (hot - r.p[:, some])
        want += dz.t() @ x[a:a + 1000].double()
        size += dz.abs().t() @ x[a:a + 1000].double().abs()
    # dz within half a bf16 step and 1e-4 of p (its exponent within 1e-4), sums of 20000 terms
    close(dw[some], want, size * (2.0 ** -8 + 2e-4 + n * U))

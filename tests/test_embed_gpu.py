"""Embedding lookup and the table's gradient against plain 64-bit forms.

Tolerances, fixed by arithmetic (u = 2^-24, half a step of fp32; h = half a
step of the stored type, 2^-8 for bf16, u for fp32):

* lookup: one fp32 product, one rounding to the type: bitwise equal to the
  same on the host;
* gradient: a sum of L fp32 terms in any order is off by at most
  (L - 1) u sum|x|; the product and the addition to what is there add one
  rounding each of their results; the stored value one of h.
"""

import numpy as np
import pytest

from matrix_optimizer_owner_amd import binding as B
from tests.test_grad_ops_gpu import _bf16_bits

pytestmark = pytest.mark.gpu

BF, F = B.BF16, B.F32
U = 2.0 ** -24
CANARY = 0xFF


def _torch_type(dt):
    import torch

    return torch.bfloat16 if dt == BF else torch.float32


def _f32(t):
    return t.float().cpu().numpy()


class Table:
    """A gain, the table, and a bias in one owner buffer; every other byte is a canary."""

    def __init__(self, rows, cols, dt, seed=0, gap=16):
        import torch

        self.torch, self.rows, self.cols, self.dt = torch, rows, cols, dt
        es = 2 if dt == BF else 4
        at = gap + 16
        after = at + -(-rows * cols * es // 16) * 16 + gap
        nbytes = after + 64
        self.plan = B.OwnerPlan([B.TableEntry(0, 1, 4, F), B.TableEntry(at, rows, cols, dt, B.ROLE_ADAMW),
                                 B.TableEntry(after, 1, 9, F)], nbytes, B.make_hparams())
        self.buf = torch.full((nbytes,), CANARY, dtype=torch.uint8, device="cuda")
        self.span = (at, at + rows * cols * es)
        self.w = self.buf[self.span[0]:self.span[1]].view(_torch_type(dt)).view(rows, cols)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w.copy_(torch.randn(rows, cols, generator=gen, device="cuda"))

    def outside_untouched(self):
        h = self.buf.cpu().numpy()
        return (h[:self.span[0]] == CANARY).all() and (h[self.span[1]:] == CANARY).all()


def _ids(kind, n, rows, first, rng):
    if kind == "same":
        r = np.full(n, rows // 2)
    elif kind == "spread":
        r = (np.arange(n) * 7919 + 13) % rows
    elif kind == "zipf":
        r = np.minimum(np.exp(rng.random(n) * np.log(rows + 1)).astype(np.int64) - 1, rows - 1)
    elif kind == "ends":
        r = rng.choice([0, rows - 1], n)
    elif kind == "falling":
        r = (np.arange(n)[::-1] * rows) // max(n, 1)
    elif kind == "lengths":  # row k has k % 40 + 1 positions, anywhere
        r = np.repeat(np.arange(rows), np.arange(rows) % 40 + 1)
        r = rng.permutation(np.resize(r, n))
    elif kind == "outside":
        return rng.choice([first - 1, first + rows, -1, -(1 << 31), (1 << 31) - 1], n)
    else:
        r = rng.integers(0, rows, n)
    ids = r.astype(np.int64) + first
    if kind == "mixed" and n:
        away = rng.random(n) < 0.4
        ids[away] = rng.choice([first - 1, first + rows, -5, first + rows + 1000], int(away.sum()))
    return ids


def _device_ids(ids, id_type):
    import torch

    return torch.from_numpy(ids.astype(np.int64 if id_type == B.I64 else np.int32)).cuda()


def _rows(n, cols, dt, stride, shift, fill, values=None):
    """An activation matrix of n rows at the given stride whose first element is `shift` elements off the
    allocation's 16-byte boundary; returns (storage, address, view)."""
    import torch

    stride = stride or cols
    flat = torch.full((max(1, n) * stride + shift + 64,), fill, dtype=_torch_type(dt), device="cuda")
    view = torch.as_strided(flat, (n, cols), (stride, 1), shift)
    if values is not None:
        view.copy_(values)
    return flat, flat.data_ptr() + shift * flat.element_size(), view


LOOKUPS = [  # rows, cols, n, table, out, ids, kind, scale, stride pad, shift
    (1, 1, 1, BF, BF, B.I64, "any", 1.0, 0, 0),
    (5, 3, 2, F, BF, B.I32, "mixed", 0.3, 2, 1),
    (300, 64, 65, BF, BF, B.I64, "mixed", 8.0, 0, 0),
    (300, 8, 1000, F, F, B.I32, "zipf", 0.7, 0, 0),
    (5003, 515, 257, BF, F, B.I64, "mixed", 22.6, 3, 1),
    (1000, 1001, 300, F, BF, B.I32, "mixed", 0.5, 0, 0),
    (1000, 1001, 300, BF, BF, B.I32, "any", 1.0, 7, 3),
    (70000, 40, 5000, BF, BF, B.I64, "zipf", 1.0, 8, 0),
    (4097, 4096, 33, BF, BF, B.I64, "ends", 64.0, 0, 0),
    (4097, 4104, 1, F, F, B.I64, "any", 1.0, 0, 0),
    (40, 16000, 700, BF, F, B.I64, "any", 0.1, 0, 0),
    (100, 24, 20, BF, BF, B.I64, "outside", 2.0, 0, 0),
    (100, 24, 20, F, F, B.I32, "outside", 2.0, 1, 0),
    (3, 2, 70000, BF, F, B.I32, "any", 1.0, 0, 0),
]


@pytest.mark.parametrize("rows,cols,n,dt,ot,it,kind,scale,pad,shift", LOOKUPS)
@pytest.mark.parametrize("first", [0, 12345])
def test_lookup(rows, cols, n, dt, ot, it, kind, scale, pad, shift, first):
    t = Table(rows, cols, dt)
    ids = _ids(kind, n, rows, first, np.random.default_rng(n))
    dev = _device_ids(ids, it)
    flat, addr, view = _rows(n, cols, ot, cols + pad, shift, 7.0)
    before = t.buf.clone()
    t.plan.embed_lookup(1, t.buf.data_ptr(), dev.data_ptr(), n, addr, id_type=it, out_type=ot, first_id=first,
                        out_stride=cols + pad if pad else 0, scale=scale, stream=t.torch.cuda.current_stream().cuda_stream)
    t.torch.cuda.synchronize()
    w = _f32(t.w)
    r = ids - first
    inside = (r >= 0) & (r < rows)
    want = np.where(inside[:, None], np.float32(scale) * w[np.clip(r, 0, rows - 1)], np.float32(0))
    if ot == BF:
        want = (_bf16_bits(want).astype(np.uint32) << np.uint32(16)).view(np.float32)
    got = _f32(view)
    assert (got == want).all()
    touched = t.torch.zeros_like(flat, dtype=t.torch.bool)
    t.torch.as_strided(touched, (n, cols), (cols + pad, 1), shift).fill_(True)
    assert bool((flat[~touched] == 7.0).all())
    assert t.torch.equal(before, t.buf)


def test_lookup_keeps_non_finite_rows_and_ignores_far_ids():
    t = Table(50, 20, F)
    t.w[3] = float("nan")
    t.w[4] = float("inf")
    ids = np.array([3, 4, 5, -(1 << 63), (1 << 63) - 1, 50, -1], np.int64)
    dev = _device_ids(ids, B.I64)
    flat, addr, view = _rows(7, 20, F, 20, 0, 7.0)
    t.plan.embed_lookup(1, t.buf.data_ptr(), dev.data_ptr(), 7, addr, out_type=F, scale=2.0)
    t.torch.cuda.synchronize()
    got = _f32(view)
    assert np.isnan(got[0]).all() and np.isinf(got[1]).all() and np.isfinite(got[2]).all() and (got[3:] == 0).all()


def test_lookup_of_an_empty_vocabulary_piece():
    """A table without rows holds no id: every row of the result is zero."""
    import torch

    plan = B.OwnerPlan([B.TableEntry(0, 0, 12, F)], 256, B.make_hparams())
    buf = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dev = torch.arange(5, device="cuda")
    out = torch.full((5, 12), 7.0, device="cuda")
    plan.embed_lookup(0, buf.data_ptr(), dev.data_ptr(), 5, out.data_ptr(), out_type=F)
    torch.cuda.synchronize()
    assert bool((out == 0).all())


GRADS = [  # rows, cols, n, table, dout, ids, kind, scale, stride pad, shift
    (1, 1, 1, BF, BF, B.I64, "any", 1.0, 0, 0),
    (1, 7, 0, F, F, B.I64, "any", 1.0, 0, 0),
    (5, 3, 2, F, BF, B.I32, "mixed", 0.3, 2, 1),
    (1, 64, 5000, BF, BF, B.I64, "same", 0.5, 0, 0),
    (300, 64, 63, BF, BF, B.I64, "mixed", 1.0, 0, 0),
    (300, 8, 1000, F, F, B.I32, "zipf", 0.7, 0, 0),
    (5003, 515, 129, F, F, B.I32, "mixed", 1.0, 0, 0),
    (5003, 515, 257, BF, F, B.I64, "zipf", 22.6, 3, 1),
    (1000, 1001, 2000, BF, BF, B.I64, "mixed", 1.0, 1, 3),
    (1000, 1001, 4097, F, BF, B.I32, "zipf", 0.5, 0, 0),
    (70000, 40, 5000, BF, BF, B.I64, "zipf", 1.0, 8, 0),
    (70000, 40, 20000, F, BF, B.I32, "spread", 1.0, 0, 0),
    (300000, 16, 9000, BF, F, B.I64, "falling", 1.0, 0, 0),
    (4097, 4096, 777, BF, BF, B.I64, "ends", 1.0, 0, 0),
    (2000, 768, 30000, F, BF, B.I64, "zipf", 1.0, 0, 0),
    (2000, 768, 30011, BF, BF, B.I32, "same", 1.0, 0, 0),
    (257, 2304, 16384, F, F, B.I64, "any", 2.0, 0, 0),
    (100, 24, 2000, BF, BF, B.I64, "outside", 2.0, 0, 0),
    (100, 24, 9000, F, F, B.I32, "outside", 2.0, 1, 0),
    (3, 2, 70000, F, BF, B.I32, "any", 1.0, 0, 0),
    (129, 9, 131073, F, F, B.I64, "mixed", 1.0, 0, 0),
    (1 << 21, 1, 12000, F, F, B.I64, "any", 1.0, 0, 0),
    (1 << 22, 2, 40000, BF, BF, B.I32, "zipf", 1.0, 0, 0),
    (500, 515, 512, BF, BF, B.I64, "zipf", 1.0, 0, 0),
    (500, 515, 513, BF, BF, B.I64, "zipf", 1.0, 0, 0),
    (90, 12, 511, F, F, B.I32, "mixed", 1.0, 0, 0),
    (9000, 5, 300, F, BF, B.I64, "any", 1.0, 0, 0),
    (40000, 2051, 100, BF, BF, B.I64, "any", 1.0, 0, 0),
    (5000, 100, 2048, BF, F, B.I64, "zipf", 1.0, 0, 0),
    (5000, 100, 2049, F, F, B.I64, "zipf", 1.0, 0, 0),
    (700, 768, 3000, BF, BF, B.I32, "lengths", 1.0, 0, 0),
    (200000, 24, 4096, F, BF, B.I64, "mixed", 1.0, 3, 1),
    (3, 33, 4096, BF, BF, B.I64, "any", 1.0, 0, 0),
    (262143, 8, 4000, F, F, B.I64, "any", 1.0, 0, 0),
    (262144, 8, 4000, F, F, B.I64, "any", 1.0, 0, 0),
    (900, 200, 18000, F, BF, B.I64, "lengths", 1.0, 0, 0),
    (3000, 1024, 61000, BF, BF, B.I32, "lengths", 1.0, 0, 0),
    (1000, 8, 300001, F, BF, B.I64, "zipf", 1.0, 0, 0),
    (1 << 21, 9, 140000, BF, BF, B.I32, "zipf", 1.0, 0, 0),
    (900, 96, 16384, BF, F, B.I64, "zipf", 1.0, 0, 0),
    (900, 96, 16385, BF, F, B.I64, "zipf", 1.0, 0, 0),
    (1000, 128, 16384, F, BF, B.I32, "lengths", 0.5, 0, 0),
    (1, 130, 10240, F, F, B.I32, "mixed", 1.0, 0, 0),
    (500, 64, 999, BF, BF, B.I64, "any", 1.0, 0, 0),
    (500, 64, 1000, BF, BF, B.I64, "any", 1.0, 0, 0),
    (7, 21, 13, F, BF, B.I64, "any", 1.0, 0, 0),
    (7, 21, 14, F, BF, B.I64, "mixed", 1.0, 2, 1),
    (1, 1, 2, BF, F, B.I32, "same", 1.0, 0, 0),
    (1000, 4100, 2000, BF, BF, B.I64, "zipf", 1.0, 0, 0),
]


def _grad_reference(ids, first, rows, dout, scale, old):
    """(gradient, bound on the fp32 sums' error before the last rounding), 64 bits."""
    cols = dout.shape[1]
    r = ids - first
    inside = np.nonzero((r >= 0) & (r < rows))[0]
    s, a, count = np.zeros((rows, cols)), np.zeros((rows, cols)), np.zeros(rows)
    order = inside[np.argsort(r[inside], kind="stable")]
    keys = r[order]
    starts = np.nonzero(np.append(True, keys[1:] != keys[:-1]))[0] if len(keys) else np.array([], int)
    if len(keys):
        d = dout[order].astype(np.float64)
        s[keys[starts]] = np.add.reduceat(d, starts, axis=0)
        a[keys[starts]] = np.add.reduceat(np.abs(d), starts, axis=0)
        count[keys[starts]] = np.diff(np.append(starts, len(keys)))
    f = float(np.float32(scale))
    want = f * s + (old if old is not None else 0.0)
    err = abs(f) * np.maximum(count - 1, 0)[:, None] * U * a * 1.01
    err += U * np.abs(f * s) * (count > 0)[:, None] + U * np.abs(want) * (count > 0)[:, None]
    return want, err, count > 0


@pytest.mark.parametrize("rows,cols,n,dt,ot,it,kind,scale,pad,shift", GRADS)
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient(rows, cols, n, dt, ot, it, kind, scale, pad, shift, accumulate):
    first = 1000 if n % 2 else 0
    t = Table(rows, cols, dt, seed=1)
    rng = np.random.default_rng(n + rows)
    ids = _ids(kind, n, rows, first, rng)
    dev = _device_ids(ids, it)
    gen = t.torch.Generator(device="cuda").manual_seed(2)
    vals = t.torch.randn(n, cols, generator=gen, device="cuda")
    r = ids - first
    # a position whose id is not in the table holds NaN, and so does every element between two rows
    vals[t.torch.from_numpy((r < 0) | (r >= rows)).cuda()] = float("nan")
    flat, addr, view = _rows(n, cols, ot, cols + pad, shift, float("nan"), vals)
    old = _f32(t.w) if accumulate else None
    ws = t.plan.embed_workspace_bytes(1, n)
    space = t.torch.full((ws + 256,), CANARY, dtype=t.torch.uint8, device="cuda")
    stream = t.torch.cuda.current_stream().cuda_stream

    def call():
        t.plan.embed_grad(1, t.buf.data_ptr(), dev.data_ptr(), n, addr, space.data_ptr() if ws else 0, ws, id_type=it,
                          dout_type=ot, first_id=first, dout_stride=cols + pad if pad else 0, scale=scale,
                          accumulate=accumulate, stream=stream)

    keep = t.w.clone()
    call()
    t.torch.cuda.synchronize()
    got = _f32(t.w).astype(np.float64)
    want, err, hit = _grad_reference(ids, first, rows, np.nan_to_num(_f32(view)), scale,
                                     None if old is None else old.astype(np.float64))
    h = 2.0 ** -8 if dt == BF else U
    bound = err + h * (np.abs(want) + err)
    assert (np.abs(got - want) <= bound).all(), float(np.nanmax(np.abs(got - want) - bound))
    if accumulate:
        assert (got[~hit] == old[~hit]).all()
    else:
        assert (got[~hit] == 0).all()
    assert t.outside_untouched()
    assert bool((space[ws:] == CANARY).all())
    # bitwise the same a second time, with the workspace as the first call left it and as noise
    result = t.w.clone()
    for noise in (None, 0x00, 0x7F):
        t.w.copy_(keep)
        if noise is not None:
            space.fill_(noise)
        call()
        t.torch.cuda.synchronize()
        assert t.torch.equal(result.view(t.torch.uint8), t.w.view(t.torch.uint8))


@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_wide_rows(accumulate):
    """14001 positions of 20000 columns on 50 rows (chunks at their longest), against sums in 64 bits on the device."""
    import torch

    rows, cols, n = 50, 20000, 14001
    t = Table(rows, cols, F, seed=8)
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(-2, rows + 1, (n,), generator=gen, device="cuda")
    dout = torch.randn(n, cols, generator=gen, device="cuda").to(torch.bfloat16)
    old = t.w.double()
    ws = t.plan.embed_workspace_bytes(1, n)
    space = torch.full((ws,), CANARY, dtype=torch.uint8, device="cuda")
    t.plan.embed_grad(1, t.buf.data_ptr(), ids.data_ptr(), n, dout.data_ptr(), space.data_ptr(), ws, scale=0.5,
                      accumulate=accumulate)
    keep = (ids >= 0) & (ids < rows)
    x, at = dout[keep].double(), ids[keep]
    sums = torch.zeros(rows, cols, dtype=torch.float64, device="cuda").index_add_(0, at, x)
    size = torch.zeros(rows, cols, dtype=torch.float64, device="cuda").index_add_(0, at, x.abs_())
    count = torch.bincount(at, minlength=rows)[:, None]
    want = 0.5 * sums + (old if accumulate else 0.0)
    bound = 1.01 * (0.5 * (count - 1) * U * size + U * (0.5 * sums).abs() + 2 * U * want.abs())
    assert bool(((t.w.double() - want).abs() <= bound).all())
    assert t.outside_untouched()


def test_a_workspace_serves_smaller_batches():
    """One workspace sized for the largest batch, for batches of every way of grouping, in turn."""
    import torch

    rows, cols, most = 6000, 64, 70000
    t = Table(rows, cols, F)
    ws = t.plan.embed_workspace_bytes(1, most)
    space = torch.full((ws + 256,), CANARY, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(1)
    for n in (70000, 100, 3000, 33000, 2048, 16500, 5000, 70000):
        ids = _ids("zipf", n, rows, 0, rng)
        dout = rng.standard_normal((n, cols)).astype(np.float32)
        dev, d = _device_ids(ids, B.I64), torch.from_numpy(dout).cuda()
        t.plan.embed_grad(1, t.buf.data_ptr(), dev.data_ptr(), n, d.data_ptr(), space.data_ptr(), ws, dout_type=F)
        torch.cuda.synchronize()
        want, err, _ = _grad_reference(ids, 0, rows, dout, 1.0, None)
        assert (np.abs(_f32(t.w) - want) <= err + U * (np.abs(want) + err)).all(), n
        assert bool((space[ws:] == CANARY).all())


@pytest.mark.parametrize("n", [300, 3000, 9000])
def test_table_past_32_bits(n):
    """A table of 4.6 G elements (9.2 GB): offsets of rows, words and bytes pass 32 bits."""
    import torch

    rows, cols = 1 << 22, 1100
    at = 256
    plan = B.OwnerPlan([B.TableEntry(0, 1, 4, F), B.TableEntry(at, rows, cols, BF, B.ROLE_ADAMW)], at + rows * cols * 2,
                       B.make_hparams())
    buf = torch.full((at + rows * cols * 2,), 0x11, dtype=torch.uint8, device="cuda")
    w = buf[at:].view(torch.bfloat16).view(rows, cols)
    gen = torch.Generator(device="cuda").manual_seed(n)
    ids = torch.randint(0, rows, (n,), generator=gen, device="cuda")
    ids[:6] = torch.tensor([rows - 1, 0, rows - 1, rows // 2, rows - 2, 3904516], device="cuda")
    dout = torch.randn(n, cols, generator=gen, device="cuda").to(torch.bfloat16)
    ws = plan.embed_workspace_bytes(1, n)
    space = torch.empty(ws + 256, dtype=torch.uint8, device="cuda")
    plan.embed_grad(1, buf.data_ptr(), ids.data_ptr(), n, dout.data_ptr(), space.data_ptr(), ws)
    out = torch.empty(n, cols, dtype=torch.float32, device="cuda")
    plan.embed_lookup(1, buf.data_ptr(), ids.data_ptr(), n, out.data_ptr(), out_type=F)
    uniq, inv = torch.unique(ids, return_inverse=True)
    sums = torch.zeros(len(uniq), cols, dtype=torch.float64, device="cuda").index_add_(0, inv, dout.double())
    # one rounding to bf16, and the fp32 sum of at most 4 terms below 7: 3 * 2^-24 * 28 = 5e-6
    got = w[uniq].double()
    assert int(torch.bincount(inv).max()) <= 4 and float(dout.abs().max()) < 7
    assert bool(((got - sums).abs() <= 2.0 ** -8 * (sums.abs() + 5.1e-6) + 5.1e-6).all())
    assert torch.equal(out, w[ids].float())
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[uniq] = False
    for k in range(0, rows, 1 << 19):  # every other row is zero
        part = w[k:k + (1 << 19)][rest[k:k + (1 << 19)]]
        assert not bool(part.view(torch.int16).any()), k
    # the norm and clipping of the same buffer
    gws = torch.empty(plan.grad_workspace_bytes, dtype=torch.uint8, device="cuda")
    stats = torch.zeros(4, device="cuda")
    buf[:at] = 0
    plan.grad_norm(buf.data_ptr(), gws.data_ptr(), gws.numel(), stats.data_ptr(), 1.0)
    total = float(got.square().sum()) ** 0.5
    assert abs(float(stats[2]) - total) <= 2.0 ** -23 * total
    plan.grad_clip(buf.data_ptr(), buf.data_ptr(), stats.data_ptr() + 12, gws.data_ptr(), gws.numel(),
                   flags=B.STEP_DESCRIPTORS_RESIDENT)
    assert torch.equal(w[uniq], (got.float() * stats[3]).to(torch.bfloat16))


@pytest.mark.parametrize("n", [5, 700, 1100])
@pytest.mark.parametrize("accumulate", [False, True])
def test_widest_rows(n, accumulate):
    """Rows of 2^22 columns, the widest an entry can have; activations past 2^32 elements.  Whole numbers below 2^24:
    every sum is exact."""
    import torch

    rows, cols = 3, 1 << 22
    plan = B.OwnerPlan([B.TableEntry(0, rows, cols, F, B.ROLE_ADAMW)], rows * cols * 4, B.make_hparams())
    w = torch.full((rows, cols), 3.0, device="cuda")
    i, c = torch.arange(n, device="cuda"), (torch.arange(cols, device="cuda") % 5).float()
    ids = torch.where(i % 11 == 10, -1, i % (rows - 1))  # the last row has none
    dout = (i[:, None] % 7).to(torch.bfloat16) + c.to(torch.bfloat16)
    ws = plan.embed_workspace_bytes(0, n)
    space = torch.empty(ws + 256, dtype=torch.uint8, device="cuda")
    plan.embed_grad(0, w.data_ptr(), ids.data_ptr(), n, dout.data_ptr(), space.data_ptr(), ws, accumulate=accumulate)
    for r in range(rows):
        mine = ids == r
        want = c * int(mine.sum()) + float((i % 7)[mine].sum()) + (3.0 if accumulate else 0.0)
        assert torch.equal(w[r], want), r
    for ot in (BF, F):
        out = torch.empty(5, cols, dtype=_torch_type(ot), device="cuda")
        plan.embed_lookup(0, w.data_ptr(), ids.data_ptr(), 5, out.data_ptr(), out_type=ot, scale=0.5)
        assert torch.equal(out, (0.5 * w[ids[:5]]).to(_torch_type(ot)))


def test_gradient_matches_differences():
    """loss = sum(dout * lookup(W)): (loss(W + d) - loss(W - d)) / 2 = <grad, d>.

    The loss is linear in W, so the difference is exact but for the roundings: each of the two losses is a 64-bit
    sum of fp32 products scale * w with relative error u, the gradient's entries are off by at most their bound."""
    rows, cols, n, scale = 60, 17, 400, 1.5
    t = Table(rows, cols, F, seed=3)
    g = Table(rows, cols, F, seed=4)
    rng = np.random.default_rng(5)
    ids = _ids("mixed", n, rows, 7, rng)
    dev = _device_ids(ids, B.I64)
    dout = t.torch.from_numpy(rng.standard_normal((n, cols)).astype(np.float32)).cuda()
    ws = g.plan.embed_workspace_bytes(1, n)
    space = t.torch.empty(ws + 256, dtype=t.torch.uint8, device="cuda")
    g.plan.embed_grad(1, g.buf.data_ptr(), dev.data_ptr(), n, dout.data_ptr(), space.data_ptr(), ws, dout_type=F, first_id=7,
                      scale=scale)
    base, d = t.w.clone(), t.torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).cuda()
    out = t.torch.empty(n, cols, device="cuda")
    loss, size = [], 0.0
    for sign in (1.0, -1.0):
        t.w.copy_(base + sign * d)
        t.plan.embed_lookup(1, t.buf.data_ptr(), dev.data_ptr(), n, out.data_ptr(), out_type=F, first_id=7, scale=scale)
        t.torch.cuda.synchronize()
        loss.append(float((out.double() * dout.double()).sum()))
        size += float((out.double() * dout.double()).abs().sum())
    got = float((g.w.double() * d.double()).sum())
    # W + d and W - d are rounded to fp32 (u each), the product too; the gradient's own bound is the reference's
    want, err, _ = _grad_reference(ids, 7, rows, _f32(dout), scale, None)
    e = err + U * (np.abs(want) + err)
    bound = 3 * U * size + float((e * np.abs(_f32(d).astype(np.float64))).sum())
    assert abs((loss[0] - loss[1]) / 2 - got) <= bound
    assert bound < 1e-3 * abs(got)


def test_non_finite_gradients_stay_in_their_rows():
    rows, cols, n = 200, 33, 5000
    t = Table(rows, cols, F)
    rng = np.random.default_rng(9)
    ids = rng.integers(0, rows, n)
    dout = rng.standard_normal((n, cols)).astype(np.float32)
    hit = {17: np.nan, 90: np.inf}
    for v, x in hit.items():
        ids[v * 3] = v
        dout[v * 3, 5] = x
    dev, d = _device_ids(ids, B.I32), t.torch.from_numpy(dout).cuda()
    ws = t.plan.embed_workspace_bytes(1, n)
    space = t.torch.empty(ws + 256, dtype=t.torch.uint8, device="cuda")
    t.plan.embed_grad(1, t.buf.data_ptr(), dev.data_ptr(), n, d.data_ptr(), space.data_ptr(), ws, id_type=B.I32, dout_type=F)
    t.torch.cuda.synchronize()
    got = _f32(t.w)
    bad = ~np.isfinite(got)
    assert bad[17, 5] and bad[90, 5] and bad.sum() == 2


@pytest.mark.parametrize("rows,cols,n", [(300, 64, 200), (5000, 96, 20000)])
def test_graph_of_gradient_norm_step_and_lookup(rows, cols, n):
    """The operators together: gradient into the buffer, norm, scaled AdamW step, lookup of the new table; captured
    once, replayed with new ids and output gradients, each replay bitwise equal to the eager run."""
    import torch

    def make():
        t = Table(rows, cols, F, seed=6)
        t.params = torch.zeros_like(t.buf)
        t.params[t.span[0]:t.span[1]].view(torch.float32).normal_(generator=torch.Generator(device="cuda").manual_seed(1))
        t.buf.zero_()
        t.state = torch.zeros(t.plan.state_bytes, dtype=torch.uint8, device="cuda")
        t.ws = torch.empty(t.plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        t.gws = torch.empty(t.plan.grad_workspace_bytes, dtype=torch.uint8, device="cuda")
        t.ews = torch.empty(t.plan.embed_workspace_bytes(1, n) + 256, dtype=torch.uint8, device="cuda")
        t.stats = torch.zeros(4, device="cuda")
        t.ids = torch.zeros(n, dtype=torch.int64, device="cuda")
        t.dout = torch.zeros(n, cols, dtype=torch.bfloat16, device="cuda")
        t.out = torch.zeros(n, cols, dtype=torch.bfloat16, device="cuda")
        return t

    def whole(t, flags):
        st = torch.cuda.current_stream().cuda_stream
        t.plan.embed_grad(1, t.buf.data_ptr(), t.ids.data_ptr(), n, t.dout.data_ptr(), t.ews.data_ptr(), t.ews.numel(),
                          stream=st)
        t.plan.grad_norm(t.buf.data_ptr(), t.gws.data_ptr(), t.gws.numel(), t.stats.data_ptr(), 0.5, stream=st, flags=flags)
        t.plan.step_scaled(t.params.data_ptr(), t.buf.data_ptr(), t.state.data_ptr(), t.ws.data_ptr(), t.ws.numel(), 3,
                           t.stats.data_ptr() + 12, stream=st, flags=flags)
        t.plan.embed_lookup(1, t.params.data_ptr(), t.ids.data_ptr(), n, t.out.data_ptr(), scale=8.0, stream=st)

    def feed(t, k):
        gen = torch.Generator(device="cuda").manual_seed(k)
        u = torch.rand(n, generator=gen, device="cuda")
        t.ids.copy_((torch.exp(u * np.log(rows + 40)) - 1).long())  # a few ids past the table
        t.dout.copy_(torch.randn(n, cols, generator=gen, device="cuda") * 0.1)

    a, b = make(), make()
    for t in (a, b):
        feed(t, 0)
        whole(t, 0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        whole(b, B.STEP_DESCRIPTORS_RESIDENT)
    for k in range(1, 6):
        for t in (a, b):
            feed(t, k)
        whole(a, B.STEP_DESCRIPTORS_RESIDENT)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("buf", "params", "state", "stats", "out"):
            x, y = getattr(a, name), getattr(b, name)
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (k, name)
    assert 0 < float(a.stats[3]) < 1
    graph.reset()


def test_gradients_on_two_streams():
    """Two calls at once, each with a workspace of its own."""
    import torch

    rows, cols, n = 3000, 128, 30000
    ts = [Table(rows, cols, F, seed=k) for k in range(2)]
    rng = np.random.default_rng(3)
    ids = [_device_ids(_ids("zipf", n, rows, 0, rng), B.I64) for _ in range(2)]
    dout = [torch.randn(n, cols, device="cuda") for _ in range(2)]
    ws = ts[0].plan.embed_workspace_bytes(1, n)
    space = [torch.empty(ws + 256, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]

    def call(k, stream):
        ts[k].plan.embed_grad(1, ts[k].buf.data_ptr(), ids[k].data_ptr(), n, dout[k].data_ptr(), space[k].data_ptr(), ws,
                              dout_type=F, stream=stream)

    want = []
    for k in range(2):
        call(k, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        want.append(ts[k].w.clone())
        ts[k].w.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for k in range(2):
            call(k, streams[k].cuda_stream)
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(want[k], ts[k].w)

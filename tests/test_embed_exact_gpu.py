"""The embedding table's gradient on data whose every sum is exact, by each way
of grouping positions.

Output gradients are whole numbers 1 .. 8 and no sum, with what it is added to,
reaches 2^24, so fp32 sums are exact in any order: an fp32 gradient has to be
equal, a bf16 one equal to the exact value rounded once.  A position that is
lost or counted twice, alone or with a whole piece of a long run, shows.
"""

import numpy as np
import pytest

from matrix_optimizer_owner_amd import binding as B
from tests.test_embed_gpu import CANARY, Table, _device_ids, _ids, _torch_type
from tests.test_embed_zero_rows_gpu import _call, _whole

pytestmark = pytest.mark.gpu

BF, F = B.BF16, B.F32


def _sums(ids, x, rows):
    """(exact sums of the rows in 64 bits, which rows have a position), from running sums over the sorted positions."""
    import torch

    r = torch.from_numpy(ids).cuda()
    keep = ((r >= 0) & (r < rows)).nonzero().flatten()
    key, order = r[keep].sort()
    last = (key != torch.cat([key[1:], key.new_tensor([-1])])).nonzero().flatten()
    upto = x[keep[order]].double().cumsum(0)[last]
    s = torch.zeros(rows, x.shape[1], dtype=torch.float64, device="cuda")
    s[key[last]] = torch.diff(upto, dim=0, prepend=torch.zeros_like(upto[:1]))
    return s, torch.bincount(r[keep], minlength=rows) > 0


# rows, cols, n, kind: more ids than the searches take, unless their counts of rows send them to a sort
SORTED = [
    (5000, 64, 30011, "same"),       # runs of hundreds of pieces, 8 lanes a row
    (6000, 8, 300001, "same"),       # 4688 pieces of one run
    (2000, 768, 30011, "same"),
    (3, 2, 70000, "any"),            # three runs of about 23000
    (3, 33, 70001, "any"),
    (1, 300, 20000, "same"),
    (900, 4104, 17000, "ends"),      # two runs, nine groups of columns
    (129, 9, 131073, "mixed"),
    (1000, 8, 300001, "zipf"),
    (3000, 96, 61000, "lengths"),    # runs of 13 to 21 pieces' borders everywhere
    (50257, 768, 40000, "zipf"),
    (1 << 22, 3, 40000, "zipf"),     # a digit of 12 bits
    (4096, 72, 8191, "zipf"),        # one block sorts up to 8192 ids of up to 2^18 - 1 rows
    (4096, 72, 8192, "same"),
    (4096, 72, 8192, "lengths"),
    (4096, 72, 8193, "zipf"),
    (1 << 17, 24, 8192, "mixed"),
    (1 << 17, 24, 8193, "mixed"),
    ((1 << 18) - 1, 16, 8192, "zipf"),
    (1 << 18, 16, 8192, "zipf"),
    (128256, 515, 4096, "zipf"),
]
SEARCHED = [  # by counts, without a sort
    (7, 21, 5, "any"), (300, 64, 500, "zipf"), (300, 64, 512, "same"), (5000, 100, 2048, "same"),
    (5000, 1536, 2048, "same"), (5000, 1537, 1024, "same"),  # by position
    (2, 768, 8192, "same"), (2, 768, 8192, "any"), (1000, 512, 10240, "same"), (154, 2764, 4144, "zipf"),
    (900, 96, 16384, "same"), (90, 12, 511, "mixed"),  # by row
]


@pytest.mark.parametrize("rows,cols,n,kind", SORTED + SEARCHED)
@pytest.mark.parametrize("dt,ot,accumulate", [(F, BF, False), (F, F, True), (BF, BF, True)])
def test_exact_sums(rows, cols, n, kind, dt, ot, accumulate):
    t = Table(rows, cols, dt, seed=1)
    t.w.copy_(t.torch.arange(rows, device="cuda")[:, None] % 100 - 50)
    old = t.w.clone()
    ids = _ids(kind, n, rows, 0, np.random.default_rng(n + rows))
    x = _whole(n, cols)
    _call(t, _device_ids(ids, B.I64), x.to(_torch_type(ot)), ot, 0.5, accumulate)
    s, hit = _sums(ids, x, rows)
    want = 0.5 * s + (old.double() if accumulate else 0.0)
    assert float(s.max()) < 2 ** 24 and t.torch.equal(want.float().double(), want)
    want = want.to(t.torch.float32).to(_torch_type(dt))
    if accumulate:
        want[~hit] = old[~hit]
    bad = (t.w != want).any(1)
    assert not bool(bad.any()), bad.nonzero().flatten()[:10].tolist()
    assert t.outside_untouched()


@pytest.mark.parametrize("rows,n", [(5000, 8000), (5000, 40000), (300, 40000)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_non_finite_values_stay_in_their_rows_when_sorted(rows, n, accumulate):
    """A NaN inside a run of 3000 positions that is joined from pieces, an Inf at a lone position, NaN at padding."""
    cols = 33
    t = Table(rows, cols, F)
    rng = np.random.default_rng(9)
    ids = rng.integers(100, rows, n)
    ids[rng.choice(n, 3000, replace=False)] = 17
    ids[rng.choice(n, 50, replace=False)] = -1
    ids[ids == 90] = 100
    ids[n // 2] = 90
    dout = rng.standard_normal((n, cols)).astype(np.float32)
    run = np.nonzero(ids == 17)[0]
    assert len(run) > 2500
    dout[run[len(run) // 2], 5] = np.nan
    dout[n // 2, 7] = np.inf
    dout[ids == -1] = np.nan
    _call(t, _device_ids(ids, B.I32).long(), t.torch.from_numpy(dout).cuda(), F, 1.0, accumulate)
    bad = ~t.w.isfinite()
    assert bool(bad[17, 5]) and bool(bad[90, 7]) and int(bad.sum()) == 2


@pytest.mark.parametrize("accumulate", [False, True])
def test_most_ids(accumulate):
    """2^30 ids, the largest batch, of one column: 256 positions of each of 2^22 rows, far apart."""
    import torch

    rows, each = 1 << 22, 256
    t = Table(rows, 1, F)
    t.w.fill_(3.0)
    ids = torch.arange(rows, dtype=torch.int32, device="cuda").repeat(each)
    x = ((torch.arange(each, device="cuda")[:, None] * 3 + torch.arange(rows, device="cuda")) % 8 + 1).to(torch.bfloat16)
    want = x.float().sum(0) + (3.0 if accumulate else 0.0)
    ws = t.plan.embed_workspace_bytes(1, len(ids))
    space = torch.full((ws + 256,), CANARY, dtype=torch.uint8, device="cuda")
    t.plan.embed_grad(1, t.buf.data_ptr(), ids.data_ptr(), len(ids), x.data_ptr(), space.data_ptr(), ws, id_type=B.I32,
                      accumulate=accumulate)
    assert torch.equal(t.w[:, 0], want)
    assert bool((space[ws:] == CANARY).all()) and t.outside_untouched()
    out = torch.empty(len(ids), dtype=torch.float32, device="cuda")
    t.plan.embed_lookup(1, t.buf.data_ptr(), ids.data_ptr(), len(ids), out.data_ptr(), id_type=B.I32, out_type=F, scale=2.0)
    assert bool((out.view(each, rows) == 2.0 * want).all())

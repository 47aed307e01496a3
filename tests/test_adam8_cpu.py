"""Host-side checks of AdamW entries with moments in 8 bits: state layout,
refusals, the owner planner and checkpoint copies.  No GPU is needed."""

import ctypes

import numpy as np
import pytest

from matrix_optimizer_owner_amd import binding as B
from tests import adam8_ref as ref

E = B.TableEntry
A8 = B.ROLE_ADAMW8
ADDR = 1 << 20
INVALID, UNSUPPORTED = 1, 4


def _status(fn, *a, **kw):
    try:
        fn(*a, **kw)
        return 0
    except B.MfsdpError as e:
        assert e.message
        return e.status


def _plan(**hp):
    return B.OwnerPlan([E(0, 40, 50), E(1 << 16, 1, 77, B.F32), E(1 << 17, 0, 5, B.F32, A8), E(1 << 18, 100, 13, B.F32, A8),
                        E(1 << 19, 1, 1, B.BF16, A8)], 1 << 24, B.make_hparams(**hp))


def test_moments_args_layout():
    """Five fields in the header's order, as a C compiler lays them out."""
    want = [("state", 0), ("first", 8), ("second", 16), ("type", 24), ("stream", 32)]
    assert [(n, getattr(B.MomentsArgs, n).offset) for n, _ in B.MomentsArgs._fields_] == want
    assert ctypes.sizeof(B.MomentsArgs) == 40


@pytest.mark.parametrize("guard", [0, 300])
def test_state_layout(guard):
    p = _plan(guard_bytes=guard)
    roles = [p.entry_info(i).role for i in range(5)]
    assert roles == [B.ROLE_MUON, B.ROLE_ADAMW, -1, A8, A8]
    gap = -(-guard // 256) * 256
    at = 0
    want = [(0, 40 * 50 * 4), (1, 77 * 4), (1, 77 * 4), (3, ref.code_bytes(1300)), (3, ref.code_bytes(1300)),
            (4, ref.code_bytes(1)), (4, ref.code_bytes(1))]
    regions = [r for r in p.regions() if r.buffer == B.BUFFER_STATE]
    assert [(r.entry, r.bytes) for r in regions] == want
    for r in regions:
        assert r.offset == at
        at = -(-(at + r.bytes) // 256) * 256 + gap
    assert p.state_bytes == at
    for i in (3, 4):
        info = p.entry_info(i)
        assert [info.state_offset, info.state_offset2] == [r.offset for r in regions if r.entry == i]


def test_tables_without_such_entries_keep_their_layout():
    """The two forms of one table differ in their state and descriptors only by what the 8-bit entries need."""
    rows = [E(0, 40, 50), E(1 << 16, 1, 77, B.F32)]
    a = B.OwnerPlan(rows, 1 << 24, B.make_hparams())
    b = B.OwnerPlan(rows + [E(1 << 18, 100, 13, B.F32, A8)], 1 << 24, B.make_hparams())
    assert b.state_bytes - a.state_bytes == 2 * -(-ref.code_bytes(1300) // 256) * 256
    assert b.workspace_bytes - a.workspace_bytes == 512  # a descriptor and two chunk counts, 256 bytes each


def test_refusals():
    p = _plan()
    ok = dict(state=ADDR, first=ADDR, second=ADDR)
    for call in (p.moments_read, p.moments_write):
        for bad in (dict(state=0), dict(state=ADDR + 128), dict(first=0), dict(first=ADDR + 8), dict(second=None),
                    dict(second=ADDR + 4)):
            assert _status(call, 3, **dict(ok, **bad)) == INVALID
        for entry in (-1, 5):
            assert _status(call, entry, **ok) == INVALID
        for kind in (-1, 2):
            assert _status(call, 3, **ok, type=kind) == UNSUPPORTED
        assert _status(call, 0, **ok) == UNSUPPORTED  # a Muon entry
        assert _status(call, 2, 0, 0, 0) == 0  # an empty shard: nothing is read
    lib = B.load()
    assert lib.mfsdp_moments_read(None, 0, None) == INVALID and lib.mfsdp_moments_write(p._h, 0, None) == INVALID
    # the step's own checks hold for a table of such entries alone
    q = B.OwnerPlan([E(0, 3, 5, B.F32, A8)], 1 << 12, B.make_hparams())
    assert _status(q.step, ADDR, ADDR, ADDR, ADDR, q.workspace_bytes, 0) == INVALID  # step count
    assert _status(q.step, ADDR, ADDR, 0, ADDR, q.workspace_bytes, 1) == INVALID


def test_planner_places_them_by_their_cost_and_memory():
    shapes, rate = [(1000, 1000), (1000, 1000), (3, 5)], 1e12
    p = B.owner_partition(shapes, [B.F32, B.BF16, B.F32], 2, roles=[A8, A8, A8], byte_rate=rate)
    assert p.role == [A8] * 3
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    for i, ((r, c), es) in enumerate(zip(shapes, (4, 2, 4))):
        n = r * c
        assert p.cost[i] == pytest.approx((n * (3 * es + 4) + -(-n // 128) * 16) / rate, rel=1e-12)
        assert p.mem_bytes[i] == 2 * up(n * es) + 2 * up(ref.code_bytes(n))
    # a table of the plan's own making, and its state within the memory that was counted
    t = p.table(0, [B.F32, B.BF16, B.F32], shapes)
    assert B.OwnerPlan(t, p.owner_param_bytes[0], B.make_hparams()).state_bytes <= p.owner_mem_bytes[0]


def test_checkpoint_copies_codes_and_scales():
    p = _plan()
    rng = np.random.default_rng(4)
    state = rng.integers(0, 256, p.state_bytes, dtype=np.uint8)
    sizes = [(8000, 0), (308, 308), (0, 0), (ref.code_bytes(1300),) * 2, (ref.code_bytes(1),) * 2]
    parts = [[np.zeros(max(n, 1), np.uint8) for n in s] for s in sizes]
    addr = lambda k: [x[k].ctypes.data for x in parts]  # noqa: E731
    p.gather(0, 0, state.ctypes.data, state.size, None, addr(0), addr(1))
    for i in (3, 4):
        info = p.entry_info(i)
        for k, off in enumerate((info.state_offset, info.state_offset2)):
            assert (parts[i][k] == state[off:off + sizes[i][k]]).all()
    back = np.zeros_like(state)
    p.scatter(None, addr(0), addr(1), 0, 0, back.ctypes.data, back.size)
    for r in p.regions():
        if r.buffer == B.BUFFER_STATE:
            assert (back[r.offset:r.offset + r.bytes] == state[r.offset:r.offset + r.bytes]).all()

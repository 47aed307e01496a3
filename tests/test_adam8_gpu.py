"""The AdamW step with moments in 8 bits against a 64-bit reference, and the
moments as values.  Every step is checked from the state the GPU held before
it; tolerances count the kernel's roundings (tests/adam8_ref.py)."""

import numpy as np
import pytest

from matrix_optimizer_owner_amd import binding as B
from tests import adam8_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HP = dict(adam_lr=0.01, adam_beta1=0.9, adam_beta2=0.95, adam_eps=1e-8, adam_weight_decay=0.1)
A8, A32 = B.ROLE_ADAMW8, B.ROLE_ADAMW


def stream():
    return torch.cuda.current_stream().cuda_stream


class Owner:
    """Tensors (rows, cols, dtype, role) in one buffer, gaps between them filled with a pattern."""

    def __init__(self, tensors, hp=HP, guard=0, seed=1, grad_std=1e-3):
        self.tensors, self.hp = tensors, hp
        offs, at = [], 32
        for r, c, dt, _ in tensors:
            offs.append(at)
            at += -(-r * c * (2 if dt == B.BF16 else 4) // 16) * 16 + 48
        self.offs, self.nbytes = offs, at
        self.plan = B.OwnerPlan([B.TableEntry(o, *t) for o, t in zip(offs, tensors)], at,
                                B.make_hparams(ns_steps=1, guard_bytes=guard, **hp))
        self.info = [self.plan.entry_info(i) for i in range(len(tensors))]
        self.params = torch.full((at,), 0x5A, dtype=torch.uint8, device="cuda")
        self.grads = torch.full((at,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN between the tensors
        self.state = torch.zeros(self.plan.state_bytes, dtype=torch.uint8, device="cuda")
        self.space = torch.empty(max(256, self.plan.workspace_bytes), dtype=torch.uint8, device="cuda")
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        for i in range(len(tensors)):
            v = self.view(self.params, i)
            v.copy_(torch.randn(v.shape, generator=self.gen, device="cuda") * 0.05)
        self.new_grads(grad_std)

    def view(self, buf, i):
        r, c, dt, _ = self.tensors[i]
        n = r * c * (2 if dt == B.BF16 else 4)
        return buf[self.offs[i]:self.offs[i] + n].view(torch.bfloat16 if dt == B.BF16 else torch.float32)

    def new_grads(self, std):
        for i in range(len(self.tensors)):
            v = self.view(self.grads, i)
            size = 10.0 ** (torch.rand(v.shape, generator=self.gen, device="cuda") * 3 - 3)
            v.copy_(torch.randn(v.shape, generator=self.gen, device="cuda") * std * size)

    def step(self, t, factor=None, static=False, flags=0):
        a = (self.params.data_ptr(), self.grads.data_ptr(), self.state.data_ptr())
        if static:
            self.plan.step_static(*a, t, stream=stream(), flags=flags)
        elif factor is None:
            self.plan.step(*a, self.space.data_ptr(), self.space.numel(), t, stream=stream(), flags=flags)
        else:
            self.plan.step_scaled(*a, self.space.data_ptr(), self.space.numel(), t, factor.data_ptr(), stream=stream(),
                                  flags=flags)

    def regions(self, state, i):
        r, c, _, _ = self.tensors[i]
        n = ref.code_bytes(r * c)
        o1, o2 = self.info[i].state_offset, self.info[i].state_offset2
        return state[o1:o1 + n], state[o2:o2 + n]

    def snapshot(self):
        return self.params.clone(), self.state.cpu().numpy()


def half_step(x, dt):
    """Half a step of the parameter's type at x, 0 for fp32 (counted in the tolerance)."""
    return np.abs(x) * 2.0 ** -8 if dt == B.BF16 else 0.0


def check(owner, before, t, factor=1.0):
    """Every 8-bit entry after one step against the reference from the state before it."""
    params, state = before
    after = owner.state.cpu().numpy()
    for i, (r, c, dt, role) in enumerate(owner.tensors):
        if role != A8 or r * c == 0:
            continue
        n = r * c
        wide = lambda buf: owner.view(buf, i).double().cpu().numpy()  # noqa: E731
        m1, r1 = owner.regions(state, i)
        w, tol, m, em, root, er = ref.step(wide(params), wide(owner.grads) * factor, ref.first_values(m1, n),
                                           ref.root_values(r1, n), owner.hp, t, i)
        got = wide(owner.params)
        bad = np.abs(got - w) > tol + half_step(np.abs(w) + tol, dt)
        assert not bad.any(), (i, n, int(bad.sum()), got[bad][:3], w[bad][:3])
        um, ur = ref.dither(t, i, np.arange(n))
        for x, ex, region, u, count, least in ((m, em, 0, um, 127, 0), (root, er, 1, ur, 255, 1)):
            codes, scales = ref.split(owner.regions(after, i)[region], n)
            most, emost = ref.group_max(np.abs(x)), ref.group_max(ex)
            assert (np.abs(scales - most) <= emost + ref.U * most).all(), (i, n, region)
            lo, hi = ref.code_range(x, ex, np.repeat(most, 128)[:n], np.repeat(emost, 128)[:n], count, u)
            if least:
                lo, hi = np.where(x > 0, np.maximum(lo, 1), lo), np.where(x > 0, np.maximum(hi, 1), hi)
                c_ = codes.astype(np.float64)
            else:
                c_ = codes.view(np.int8).astype(np.float64)
                assert ((np.sign(c_) == np.sign(x)) | (c_ == 0) | (np.abs(x) <= ex)).all(), (i, n)
            bad = (np.abs(c_) < lo) | (np.abs(c_) > hi)
            assert not bad.any(), (i, n, region, int(bad.sum()), c_[bad][:3], lo[bad][:3], hi[bad][:3])
            # codes behind the tensor's end, up to the scales
            assert (owner.regions(after, i)[region][n:-(-n // 8) * 8] == 0).all()


TABLES = {
    "sizes-f32": [(1, n, B.F32, A8) for n in (1, 7, 8, 9, 127, 128, 129, 1000, 2047, 2048, 2049, 4097)],
    "sizes-bf16": [(1, n, B.BF16, A8) for n in (1, 7, 8, 9, 127, 128, 129, 1000, 2047, 2048, 2049, 4097)],
    "matrices": [(33, 45, B.F32, A8), (0, 5, B.F32, A8), (515, 203, B.BF16, A8), (1, 1, B.F32, A8), (777, 1001, B.BF16, A8)],
    "mixed-roles": [(96, 160, B.F32, A8), (40, 50, B.BF16, B.ROLE_AUTO), (1, 333, B.F32, A32), (64, 100, B.BF16, A8),
                    (1, 50, B.BF16, A32)],
}


@pytest.mark.parametrize("name", sorted(TABLES))
@pytest.mark.parametrize("form", ["plain", "scaled", "static"])
def test_steps_against_reference(name, form):
    o = Owner(TABLES[name])
    factor = torch.full((1,), 0.37, device="cuda") if form == "scaled" else None
    for t in range(1, 5):
        before = o.snapshot()
        o.step(t, factor=factor, static=form == "static", flags=B.STEP_DESCRIPTORS_RESIDENT if t > 2 else 0)
        check(o, before, t, ref.f32(0.37) if factor is not None else 1.0)
        o.new_grads(10.0 ** (-t))


def test_first_step_from_zero_state_and_zero_gradients():
    o = Owner([(3, 100, B.F32, A8), (5, 128, B.BF16, A8)])
    o.grads.zero_()
    before = o.snapshot()
    o.step(1)
    check(o, before, 1)
    assert not o.state.any()


@pytest.mark.parametrize("std", [1e-17, 1e-12, 1.0, 1e12, 1e17])
def test_gradient_sizes(std):
    o = Owner([(9, 300, B.F32, A8), (7, 130, B.BF16, A8)], grad_std=std, hp=dict(HP, adam_eps=1e-30))
    for t in (1, 2, 3):
        before = o.snapshot()
        o.step(t)
        check(o, before, t)
        o.new_grads(std)


def test_the_32_bit_entries_of_a_mixed_table_are_untouched_by_the_others():
    """A table with 8-bit entries beside it steps its other entries to the same bits."""
    tensors = TABLES["mixed-roles"]
    a = Owner(tensors)
    keep = [i for i, t in enumerate(tensors) if t[3] != A8]
    alone = B.OwnerPlan([B.TableEntry(a.offs[i], *tensors[i]) for i in keep], a.nbytes, B.make_hparams(ns_steps=1, **HP))
    p, st = a.params.clone(), torch.zeros(alone.state_bytes, dtype=torch.uint8, device="cuda")
    ws = torch.empty(alone.workspace_bytes, dtype=torch.uint8, device="cuda")
    for t in (1, 2):
        alone.step(p.data_ptr(), a.grads.data_ptr(), st.data_ptr(), ws.data_ptr(), ws.numel(), t, stream=stream())
        a.step(t)
    for i in keep:
        assert torch.equal(a.view(a.params, i), a.view(p, i))


def test_nothing_outside_the_regions_is_written():
    o = Owner(TABLES["matrices"], guard=512)
    regions = [r for r in o.plan.regions() if r.buffer == B.BUFFER_STATE]
    mask = torch.ones(o.state.numel(), dtype=torch.bool)
    for r in regions:
        mask[r.offset:r.offset + r.bytes] = False
    mask = mask.cuda()
    o.state[mask] = 0xA5
    owned = torch.zeros(o.nbytes, dtype=torch.bool)
    for off, (r, c, dt, _) in zip(o.offs, o.tensors):
        owned[off:off + r * c * (2 if dt == B.BF16 else 4)] = True
    owned = owned.cuda()
    grads = o.grads.clone()
    for t in (1, 2):
        o.step(t)
    assert (o.state[mask] == 0xA5).all() and (o.params[~owned] == 0x5A).all() and torch.equal(grads, o.grads)


def test_rows_without_gradient_keep_their_codes():
    """Groups whose gradients are all zero keep every code while their scales decay: 200 steps."""
    o = Owner([(40, 128, B.F32, A8)])
    o.step(1)
    m0, r0 = (x.copy() for x in o.regions(o.state.cpu().numpy(), 0))
    o.grads.zero_()
    for t in range(2, 202):
        o.step(t)
    m1, r1 = o.regions(o.state.cpu().numpy(), 0)
    n = 40 * 128
    assert (m0[:n] == m1[:n]).all() and (r0[:n] == r1[:n]).all()
    # 200 roundings of a scale: unit, value, product with beta (m; r twice, with the root between)
    for a, b, decay in ((m0, m1, ref.f32(0.9) ** 200), (r0, r1, ref.f32(0.95) ** 100)):
        sa, sb = ref.split(a, n)[1], ref.split(b, n)[1]
        assert (np.abs(sb / (sa * decay) - 1) < 200 * 8 * ref.U).all()


def test_slow_second_moment_moves():
    """beta2 = 0.999 and gradients of a new size: the mean of v follows b2 v + (1-b2) g^2.  A step moves v by at most 0.4%
    of itself here, half a code step or less, so codes rounded to nearest would mostly stay."""
    o = Owner([(64, 128, B.F32, A8)], hp=dict(HP, adam_beta2=0.999))
    g = o.view(o.grads, 0)
    level = torch.rand(64, 128, device="cuda", generator=o.gen) * 0.5 + 0.5
    level[:, 0] = 1.5  # each group's largest, at a steady value: its code stays 255
    v = (level * level).contiguous()
    m = torch.zeros_like(v)
    o.plan.moments_write(0, o.state.data_ptr(), m.data_ptr(), v.data_ptr(), type=B.F32, stream=stream())
    level[:, 1:] *= 0.6
    g.copy_(level.view(-1))
    got = torch.empty_like(v)
    o.plan.moments_read(0, o.state.data_ptr(), m.data_ptr(), got.data_ptr(), type=B.F32, stream=stream())
    want = got.double()
    b2 = ref.f32(0.999)
    for t in range(1, 301):
        o.step(t)
        want = b2 * want + (1 - b2) * g.view(64, 128).double() ** 2
    o.plan.moments_read(0, o.state.data_ptr(), m.data_ptr(), got.data_ptr(), type=B.F32, stream=stream())
    ratio = (got.double() / want)[:, 1:]
    # The dither's noise: a code takes at most 1/4 a step of variance, 300 steps 75, so at codes of 145 or more at most
    # 8.7/145 = 6% of r and 12% of v for one element; the mean over 64 x 127 of them is within 5 of 12% / 90 = 0.7%.
    # Its bias: c^2 is off by at most 1/4 a step, 300 / 4 / 145^2 = 0.4% of r, 0.8% of v.  Standing still would be 18% off.
    assert abs(float(ratio.mean()) - 1) < 0.015, float(ratio.mean())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_a_non_finite_gradient_stays_in_its_group(bad):
    o = Owner([(4, 256, B.F32, A8)])
    o.step(1)
    o.view(o.grads, 0)[300] = bad
    o.step(2)
    w = o.view(o.params, 0)
    assert torch.isfinite(torch.cat([w[:300], w[301:]])).all()
    if bad != 3e38:
        assert torch.isnan(w[300])
    o.new_grads(1e-3)
    o.step(3)
    # 3e38 overflows in v only: its update is 0, its group's second moment is not a number from then on
    poisoned = torch.isnan(o.view(o.params, 0))
    assert poisoned[256:384].all() and not poisoned[:256].any() and not poisoned[384:].any()


@pytest.mark.parametrize("role", [A8, A32])
@pytest.mark.parametrize("kind", [B.F32, B.BF16])
@pytest.mark.parametrize("n", [1, 8, 127, 128, 129, 2049, 100_003])
def test_moments_into_the_state_and_back(role, kind, n):
    o = Owner([(1, 5, B.F32, A8), (1, n, B.BF16, role)], guard=256)
    tt = torch.float32 if kind == B.F32 else torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(n)
    m = (torch.randn(n, generator=gen, device="cuda") * 10.0 ** (torch.rand(n, generator=gen, device="cuda") * 8 - 8)).to(tt)
    v = (torch.randn(n, generator=gen, device="cuda") * 10.0 ** (torch.rand(n, generator=gen, device="cuda") * 6 - 8)).square().to(tt)
    pad = lambda x: torch.cat([x, torch.full((64,), 7.0, device="cuda", dtype=tt)])  # noqa: E731
    m_in, v_in, m_out, v_out = pad(m), pad(v), pad(torch.zeros_like(m)), pad(torch.zeros_like(v))
    o.state.fill_(0xA5)
    o.plan.moments_write(1, o.state.data_ptr(), m_in.data_ptr(), v_in.data_ptr(), type=kind, stream=stream())
    kept = o.state.clone()
    o.plan.moments_read(1, o.state.data_ptr(), m_out.data_ptr(), v_out.data_ptr(), type=kind, stream=stream())
    assert torch.equal(kept, o.state)
    assert (m_out[n:] == 7).all() and (v_out[n:] == 7).all()
    # bytes of the state that are not the entry's
    mine = torch.zeros(o.state.numel(), dtype=torch.bool)
    for r in o.plan.regions():
        if r.buffer == B.BUFFER_STATE and r.entry == 1:
            mine[r.offset:r.offset + r.bytes] = True
    assert (kept[~mine.cuda()] == 0xA5).all()
    if role == A32:
        assert torch.equal(m_out[:n], m) and torch.equal(v_out[:n], v)
        return
    # half a code step either way, (c +- 1/2)^2 of the scale, then the fp32 roundings and the type's own
    half = 0.0 if kind == B.F32 else 2.0 ** -8
    for x, got, count, root in ((m, m_out, 127, False), (v, v_out, 255, True)):
        x, got = x.double().cpu().numpy(), got[:n].double().cpu().numpy()
        y = np.sqrt(x) if root else np.abs(x)
        most = np.repeat(ref.group_max(y), 128)[:n]
        with np.errstate(invalid="ignore", divide="ignore"):
            c = np.where(most > 0, count * np.sqrt(y / most), 0.0)
        lo, hi = np.maximum(c - 0.5001, 0), np.minimum(c + 0.5001, count)
        if root:
            hi = np.where(y > 0, np.maximum(hi, 1), hi)
        lo, hi = most * (lo / count) ** 2, most * (hi / count) ** 2
        if root:
            lo, hi = lo ** 2, hi ** 2
        spare = half + 16 * ref.U
        assert ((np.abs(got) >= lo * (1 - spare)) & (np.abs(got) <= hi * (1 + spare))).all()
        if not root:
            assert ((np.sign(got) == np.sign(x)) | (got == 0)).all()
    # what the state holds comes back to the same bytes (fp32: bf16 values are other values)
    if kind == B.F32:
        o.plan.moments_write(1, o.state.data_ptr(), m_out.data_ptr(), v_out.data_ptr(), type=kind, stream=stream())
        assert torch.equal(kept, o.state)


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e30, 3e38])
def test_moments_of_the_types_whole_range(scale):
    o = Owner([(1, 256, B.F32, A8)])
    m = torch.linspace(-1, 1, 256, device="cuda") * scale
    v = torch.linspace(0, 1, 256, device="cuda") * scale
    got_m, got_v = torch.empty_like(m), torch.empty_like(v)
    o.plan.moments_write(0, o.state.data_ptr(), m.data_ptr(), v.data_ptr(), stream=stream())
    o.plan.moments_read(0, o.state.data_ptr(), got_m.data_ptr(), got_v.data_ptr(), stream=stream())
    # (c + 1/2)^2 - c^2 over 127^2 is at most 1/127 of the group's largest value; v: twice 1/255 of r, squared.  Values
    # below the smallest normal number, 1.2e-38, may be lost.
    for x, got, off in ((m, got_m, 1 / 127), (v, got_v, 2 / 255 + 1 / 255 ** 2)):
        most = x.double().view(2, 128).abs().amax(1, keepdim=True)
        err = (x.double() - got.double()).view(2, 128).abs()
        assert (err <= most * off * 1.0001 + 1.2e-38).all()


def test_captured_and_replayed_on_another_stream():
    o = Owner(TABLES["matrices"])
    o.step(1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    p0, s0 = o.params.clone(), o.state.clone()
    o.step(7, flags=B.STEP_DESCRIPTORS_RESIDENT)
    want = o.params.clone(), o.state.clone()
    o.params.copy_(p0)
    o.state.copy_(s0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    m, v = (torch.empty(777 * 1001, device="cuda") for _ in range(2))
    with torch.cuda.graph(graph, stream=side):
        o.step(7, flags=B.STEP_DESCRIPTORS_RESIDENT)
        o.plan.moments_read(4, o.state.data_ptr(), m.data_ptr(), v.data_ptr(), stream=stream())
    for _ in range(3):
        o.params.copy_(p0)
        o.state.copy_(s0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.params, want[0]) and torch.equal(o.state, want[1])
        m2, v2 = torch.empty_like(m), torch.empty_like(v)
        o.plan.moments_read(4, o.state.data_ptr(), m2.data_ptr(), v2.data_ptr(), stream=stream())
        assert torch.equal(m, m2) and torch.equal(v, v2)


def test_a_tensor_past_2_to_the_31_elements():
    """4194304 x 520 bf16 elements: groups at the front, across 2^31 and at the end against the reference."""
    rows, cols = 4194304, 520
    n = rows * cols
    plan = B.OwnerPlan([B.TableEntry(0, rows, cols, B.BF16, A8)], 2 * n, B.make_hparams(**HP))
    params = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    grads = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    state = torch.zeros(plan.state_bytes, dtype=torch.uint8, device="cuda")
    space = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    spots = [0, 2 ** 31 - 640, 2 ** 31 + 128, n - 1024]
    gen = torch.Generator(device="cuda").manual_seed(3)
    for a in spots:
        grads[a:a + 1024] = (torch.randn(1024, generator=gen, device="cuda") * 1e-3).bfloat16()
    plan.step(params.data_ptr(), grads.data_ptr(), state.data_ptr(), space.data_ptr(), space.numel(), 1, stream=stream())
    info = plan.entry_info(0)
    at = -(-n // 256) * 256
    for a in spots:
        g = grads[a:a + 1024].double().cpu().numpy()
        zero = np.zeros(1024)
        w, tol, m, em, r, er = ref.step(zero + 0.5, g, zero, zero, HP, 1, 0)
        got = params[a:a + 1024].double().cpu().numpy()
        assert (np.abs(got - w) <= tol + 2.0 ** -8 * (np.abs(w) + tol)).all()
        um, ur = ref.dither(1, 0, np.arange(a, a + 1024))
        for off, x, ex, u, count in ((info.state_offset, m, em, um, 127), (info.state_offset2, r, er, ur, 255)):
            codes = state[off + a:off + a + 1024].cpu().numpy()
            c = np.abs(codes.view(np.int8).astype(float)) if count == 127 else codes.astype(float)
            scales = state[off + at + a // 32:off + at + a // 32 + 32].view(torch.float32).double().cpu().numpy()
            most, emost = ref.group_max(np.abs(x)), ref.group_max(ex)
            assert (np.abs(scales - most) <= emost + ref.U * most).all()
            lo, hi = ref.code_range(x, ex, np.repeat(most, 128), np.repeat(emost, 128), count, u)
            if count == 255:
                lo, hi = np.where(x > 0, np.maximum(lo, 1), lo), np.where(x > 0, np.maximum(hi, 1), hi)
            assert ((c >= lo) & (c <= hi)).all()
    # the groups between kept their zero moments, their parameters only decayed
    untouched = float(torch.tensor(0.5 * (1 - ref.f32(0.01) * ref.f32(0.1))).bfloat16())
    assert (params[4096:2 ** 31 - 4096] == untouched).all()

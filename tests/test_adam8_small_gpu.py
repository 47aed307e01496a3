"""Moments in 8 bits down to the fp32 range's end: what a step reads out of the
state, and groups of tiny gradients.  Tolerances count the kernel's roundings
(tests/adam8_ref.py), and where values are below the smallest normal number
half of 2^-149 for each of them."""

import numpy as np
import pytest

from matrix_optimizer_owner_amd import binding as B
from tests import adam8_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_adam8_gpu import A8, HP, Owner  # noqa: E402

TINY = 2.0 ** -149
SCALES = [1e18, 3.7, 1.0, 1e-3, 7e-11, 1.3e-20, 1e-30, 2.9e-33, 1e-34, 8e-36, 1.7e-37, 1e-38, 2.3e-39, 5e-41, 1.1e-43]


def set_state(o, i, first, first_scales, root, root_scales):
    """Codes (uint8, rows * cols) and scales (fp32, one a group) of entry i."""
    n = len(first)
    at = -(-n // 256) * 256
    for off, codes, scales in ((o.info[i].state_offset, first, first_scales), (o.info[i].state_offset2, root, root_scales)):
        o.state[off:off + n].copy_(torch.from_numpy(codes.view(np.uint8)))
        o.state[off + at:off + at + 4 * len(scales)].copy_(torch.from_numpy(scales.astype(np.float32).view(np.uint8)))


@pytest.mark.parametrize("form", ["plain", "scaled"])
def test_a_groups_largest_value_is_its_scale(form):
    """With zero gradients a step multiplies both moments by their betas: the first moment's scale by beta1, bit for bit."""
    o = Owner([(len(SCALES), 128, B.F32, A8)])
    rng = np.random.default_rng(1)
    n = len(SCALES) * 128
    c = rng.integers(-126, 127, n).astype(np.int8)
    d = rng.integers(0, 255, n).astype(np.uint8)
    c[::128], d[::128] = np.where(np.arange(len(SCALES)) % 2, -127, 127), 255
    s = np.array(SCALES, dtype=np.float32)
    set_state(o, 0, c, s, d, s)
    o.grads.zero_()
    want = s
    for t in range(2, 12):
        held = ref.split(o.regions(o.state.cpu().numpy(), 0)[1], n)[1]
        o.step(t, factor=torch.ones(1, device="cuda") if form == "scaled" else None)
        want = want * np.float32(HP["adam_beta1"])  # rounded once, subnormal or not
        m, r = o.regions(o.state.cpu().numpy(), 0)
        assert np.array_equal(ref.split(m, n)[1], want.astype(np.float64))
        # the square, its product, the root (2) and half a step of 2^-149
        after = ref.split(r, n)[1]
        assert (np.abs(after - held * np.sqrt(ref.f32(HP["adam_beta2"]))) <= 5 * ref.U * held + TINY / 2).all()


def wide(x):
    return x.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("beta2", [0.95, 0.999])
@pytest.mark.parametrize("std", [1e-38, 1e-37, 1e-36, 1e-34, 1e-32, 1e-28, 1e-20])
def test_gradients_of_the_ranges_end(std, beta2):
    """Gradients 0.001 to 1 times `std`: every step from the values the state holds."""
    hp = dict(HP, adam_eps=1e-30, adam_beta2=beta2)
    o = Owner([(9, 300, B.F32, A8), (7, 130, B.BF16, A8)], hp=hp, grad_std=std)
    for t in range(1, 5):
        params, state = o.snapshot()
        o.step(t)
        after = o.state.cpu().numpy()
        for i, (rows, cols, dt, _) in enumerate(o.tensors):
            n = rows * cols
            m0, r0 = o.regions(state, i)
            w, tol, m, em, r, er = ref.step(wide(o.view(params, i)), wide(o.view(o.grads, i)), ref.first_values(m0, n),
                                            ref.root_values(r0, n), hp, t, i)
            # the value held, its product and (1 - beta1) g: half of 2^-149 each; the root: the value held, itself
            em, er = em + 1.5 * TINY, er + TINY
            tol = tol + hp["adam_lr"] / (1 - hp["adam_beta1"] ** t) * (np.abs(m) + em) / hp["adam_eps"] * (
                ref.U + 1.5 * TINY / np.maximum(np.abs(m) + em, TINY) + er / hp["adam_eps"])
            got = wide(o.view(o.params, i))
            half = 2.0 ** -8 if dt == B.BF16 else 0.0
            assert (np.abs(got - w) <= tol + half * (np.abs(w) + tol)).all()
            um, ur = ref.dither(t, i, np.arange(n))
            for x, ex, region, u, count in ((m, em, 0, um, 127), (r, er, 1, ur, 255)):
                codes, scales = ref.split(o.regions(after, i)[region], n)
                most, emost = ref.group_max(np.abs(x)), ref.group_max(ex)
                assert (np.abs(scales - most) <= emost + ref.U * most).all(), (i, region)
                lo, hi = ref.code_range(x, ex, np.repeat(most, 128)[:n], np.repeat(emost, 128)[:n], count, u)
                if region:
                    lo, hi = np.where(x - ex > 0, np.maximum(lo, 1), lo), np.maximum(hi, 1)
                c = np.abs(codes.astype(np.float64) if region else codes.view(np.int8).astype(np.float64))
                bad = (c < lo) | (c > hi)
                assert not bad.any(), (i, region, int(bad.sum()), c[bad][:3], lo[bad][:3], hi[bad][:3])
        o.new_grads(std)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_codes_of_a_group_that_is_nan(bad):
    """No element of it has a code but 0 in the first moment, and 0 or 1 in the root; other groups are as without it."""
    a, b = Owner([(4, 256, B.F32, A8)]), Owner([(4, 256, B.F32, A8)])
    a.view(a.grads, 0)[300] = bad
    for o in (a, b):
        o.step(1)
    got, want = a.state.cpu().numpy(), b.state.cpu().numpy()
    for region in (0, 1):
        (c, s), (c0, s0) = (ref.split(o.regions(st, 0)[region], 1024) for o, st in ((a, got), (b, want)))
        hit = np.zeros(1024, dtype=bool)
        hit[256:384] = np.isnan(s[2])
        assert np.isnan(s[2]) or (region == 0 and bad == 3e38)
        assert (c[hit] <= region).all() and np.array_equal(np.delete(s, 2), np.delete(s0, 2))
        assert np.array_equal(np.delete(c, np.arange(256, 384)), np.delete(c0, np.arange(256, 384)))

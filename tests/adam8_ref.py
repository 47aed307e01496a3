"""64-bit NumPy reference of the AdamW step with moments in 8 bits, with the
interval each fp32 value may lie in."""

import numpy as np

GROUP = 128
U = 2.0 ** -24  # half a step of fp32, relative


def f32(x):
    return float(np.float32(x))


def code_bytes(numel):
    return -(-numel // 256) * 256 + 4 * -(-numel // GROUP)


def split(region, numel):
    """(codes, scale of each element) of one moment's region bytes; uint8 codes."""
    at = -(-numel // 256) * 256
    scales = region[at:at + 4 * -(-numel // GROUP)].view(np.float32)
    return region[:numel], scales.astype(np.float64)


def first_values(region, numel):
    codes, scales = split(region, numel)
    c = codes.view(np.int8).astype(np.float64)
    return c * np.abs(c) / 16129.0 * np.repeat(scales, GROUP)[:numel]


def root_values(region, numel):
    codes, scales = split(region, numel)
    return (codes.astype(np.float64) / 255.0) ** 2 * np.repeat(scales, GROUP)[:numel]


def _mix(h):
    h = (h ^ (h >> np.uint32(16))) * np.uint32(0x85EBCA6B)
    h = (h ^ (h >> np.uint32(13))) * np.uint32(0xC2B2AE35)
    return h ^ (h >> np.uint32(16))


def dither(step, entry, index):
    """(of the first moment, of the second's root) of elements `index` (int64)."""
    with np.errstate(over="ignore"):
        key = _mix(np.array([(step + 0x9E3779B9 * (entry + 1)) & 0xFFFFFFFF], dtype=np.uint32))
        low = ((index >> 1) & 0xFFFFFFFF).astype(np.uint32)
        high = (index >> 33).astype(np.uint32)
        word = _mix(low + high * np.uint32(0x9E3779B9) + key)
    shift = np.where(index & 1, 16, 0).astype(np.uint32)
    take = lambda k: (((word >> (shift + np.uint32(k))) & np.uint32(255)).astype(np.float64) + 0.5) / 256  # noqa: E731
    return take(0), take(8)


def group_max(x):
    pad = np.zeros(-len(x) % GROUP)
    return np.concatenate([x, pad]).reshape(-1, GROUP).max(1)


def step(w, g, m, r, hp, t, entry, start=0):
    """One step in 64 bits from the values held.  Returns (w, tolerance of w, m, its error bound, r, its error bound).

    The kernel's roundings, in units of U = 2^-24 relative: a held value takes 3 (scale * fp32 constant, its own
    rounding, the product); omb * g 3 with the scaled gradient; one for each fused sum.  r is an approximate root
    (2 U) of v; the update's reciprocal takes 2, the fused denominator 1, its constants 1 each."""
    b1, b2 = f32(hp["adam_beta1"]), f32(hp["adam_beta2"])
    lr, eps, wd = f32(hp["adam_lr"]), f32(hp["adam_eps"]), f32(hp["adam_weight_decay"])
    m2 = b1 * m + (1 - b1) * g
    em = 5 * U * (b1 * np.abs(m) + (1 - b1) * np.abs(g))
    v2 = b2 * r * r + (1 - b2) * g * g
    r2 = np.sqrt(v2)
    er = (9 / 2 + 3) * U * r2  # v: 7 for r^2 or 5 for omb g^2, one for the sum, one spare
    bc1, bc2 = 1 - b1 ** t, 1 - b2 ** t
    den = r2 / np.sqrt(bc2) + eps
    upd = lr / bc1 * m2 / den
    w2 = w * (1 - lr * wd) - upd
    tol = U * (2.5 * np.abs(w) + 1.1 * np.abs(w2)) + lr / bc1 / den * em + 16 * U * np.abs(upd)
    return w2, tol, m2, em, r2, er


def code_range(x, ex, scale, escale, count, u):
    """Smallest and largest code that fp32 may give for magnitudes |x| (+- ex) under the group scale (+- escale)."""
    with np.errstate(divide="ignore", invalid="ignore"):
        lo = np.maximum(np.abs(x) - ex, 0) / (scale + escale)
        hi = (np.abs(x) + ex) / np.maximum(scale - escale, 1e-300)
    # share: 3 roundings and an approximate reciprocal (2 U); its root 2 U; the fused sum 1
    lo = np.floor(count * np.sqrt(lo * (1 - 6 * U)) * (1 - 4 * U) + u - 2 * U * count)
    hi = np.floor(count * np.sqrt(hi * (1 + 6 * U)) * (1 + 4 * U) + u + 2 * U * count)
    zero = scale == 0
    return np.where(zero, 0, np.clip(lo, 0, count)), np.where(zero, 0, np.clip(hi, 0, count))

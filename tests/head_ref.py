"""64-bit reference of the output head's log probabilities and gradients, with
error bounds that count the kernels' roundings.

U = 2^-24 is half a step of fp32, relative.  A logit y (base 2) is a sum of K
products, each addition rounded at most once: (K + 4) U of the sum of the
products' magnitudes, the product with log2(e) scale among them.  Differences
from the largest, sums of at most 128 terms in a lane's and its part's order,
joins of parts in a tree and chains of at most 600 together, and 2 U for each
exp2 follow from there."""

import math

import torch

U = 2.0 ** -24
TINY = 2.0 ** -126
LN2 = math.log(2.0)
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
CHAIN = 800  # roundings of a sum of exponentials at most: terms of a part, joins of parts


class Reference:
    """x [n, d], w [v, d] of any type on one device; target rows (-1: none), live rows."""

    def __init__(self, x, w, target, live, scale, exact=False):
        self.x, self.w, self.target, self.live, self.scale = x.double(), w.double(), target, live, scale
        self.x = torch.where(live[:, None], self.x, 0.0)
        self.c = scale / LN2
        self.y = self.x @ self.w.t() * self.c
        size = self.x.abs() @ self.w.abs().t() * abs(self.c)
        terms = 4 if exact else x.shape[1] + 4
        self.ey = U * terms * (self.y.abs() if exact else size)  # error of each y
        self.m = self.y.amax(1, keepdim=True)
        # one bound a row for the difference of two y, rounded
        self.dy = 2 * self.ey.amax(1, keepdim=True) + U * (self.y - self.m).abs().amax(1, keepdim=True)
        e = torch.exp2(self.y - self.m)
        s = e.sum(1, keepdim=True)
        self.p = e / s
        self.lp = self.y - self.m - torch.log2(s)
        self.lse = self.m + torch.log2(s)
        mean = (self.p * (self.y - self.m).abs()).sum(1, keepdim=True)
        self.entropy = -(self.p * self.lp).sum(1, keepdim=True) * LN2
        rel = LN2 * self.dy + (CHAIN + 8) * U  # of a sum of exponentials
        self.logp_tol = LN2 * (self.dy + rel / LN2) + 4 * U * self.lp.abs().amax(1, keepdim=True) * LN2
        self.entropy_tol = LN2 * (rel / LN2 + self.dy + 3 * rel * mean) + 4 * U * (1 + self.entropy)
        self.rel = rel

    def logp(self):
        at = self.target.clamp_min(0)[:, None]
        v = self.lp.gather(1, at)[:, 0] * LN2
        return torch.where(self.target >= 0, v, 0.0)

    def check_forward(self, logp, entropy):
        want = self.logp()
        err = (logp.double() - want).abs()
        assert (err <= self.logp_tol[:, 0]).all(), (float(err.max()), float(self.logp_tol.max()))
        h = torch.where(self.live, self.entropy[:, 0], 0.0)
        err = (entropy.double() - h).abs()
        assert (err <= self.entropy_tol[:, 0]).all(), (float(err.max()), float(self.entropy_tol.max()))

    def grads(self, dlogp, dentropy, dz_type, found=None):
        """(dx, its bound, dw, its bound) from the formula; bounds before the outputs' own rounding."""
        n = len(self.target)
        found = (self.target >= 0) if found is None else found
        a = torch.where(found & self.live, dlogp.double(), 0.0)[:, None]
        b = (dentropy.double() if dentropy is not None else torch.zeros(n, device=a.device, dtype=torch.float64))[:, None]
        b = torch.where(self.live[:, None], b, 0.0)
        lp = self.lp * LN2
        h = self.entropy
        hot = torch.zeros_like(self.p)
        here = (self.target >= 0) & self.live
        hot[here, self.target[here]] = 1.0
        dz = self.scale * (a * (hot - self.p) - b * self.p * (lp + h))
        size = abs(self.scale) * self.p * (a.abs() + b.abs() * (lp.abs() + h.abs()))
        ez = (self.rel + 2 * LN2 * self.dy + 12 * U) * size + abs(self.scale) * b.abs() * self.p * (
            self.entropy_tol + LN2 * 2 * self.dy) + 4 * U * abs(self.scale) * hot * a.abs()
        # a p below the smallest normal number, 2^-126, is 0 to the exponential: that much is lost of it, times its factor
        ez = ez + TINY * abs(self.scale) * (a.abs() + b.abs() * (lp.abs() + h.abs()))
        ez = ez + HALF[dz_type] * (dz.abs() + ez)
        ez = torch.where(self.live[:, None], ez, 0.0)
        dz = torch.where(self.live[:, None], dz, 0.0)
        aw, ax, az = self.w.abs(), self.x.abs(), dz.abs() + ez
        v = self.w.shape[0]
        # and so is each product or sum of the matrix instructions below it
        return (dz @ self.w, ez @ aw + U * (v + 4) * (az @ aw) + 2 * v * TINY, dz.t() @ self.x,
                ez.t() @ ax + U * (n + 4) * (az.t() @ ax) + 2 * n * TINY)


def close(got, want, bound, spread=None):
    """Within the bound and half a step of got's type; and, over all elements, within `spread` in the 2-norm."""
    g = got.double()
    tol = bound + HALF[got.dtype] * (want.abs() + bound)
    bad = ~((g - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), g[bad][:3], want[bad][:3], tol[bad][:3])
    if spread is not None and want.numel() > 1000:
        off = float((g - want).norm() / want.norm())
        assert off <= spread, off

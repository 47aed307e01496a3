"""Gradient norm, clipping and the scaled step against plain 64-bit forms.

Tolerances, fixed by arithmetic:

* norms: sums and root in fp64 (relative error below 1e-10 here), one rounding
  to fp32: half a step, 2^-24 of the value, or 2^-150 below the normal range;
* clipping: the fp32 product rounded once to the type, so bitwise equal to
  the same two roundings on the host;
* the scaled step: bitwise equal to clipping and stepping where both round
  alike (fp32 gradients), and to the unscaled step at a scale of 1.
"""

import math

import numpy as np
import pytest

from matrix_optimizer_owner_amd import binding as B
from matrix_optimizer_owner_amd import workloads as W
from tests.harness import DeviceRun

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -150
CANARY = 0xFF  # NaN in both types


def _table(spec, gap=16):
    """[(rows, cols, dtype)] -> entries packed at 16-byte multiples, and the buffer's size."""
    out, at = [], gap
    for r, c, dt in spec:
        out.append(B.TableEntry(at, r, c, dt))
        at += -(-r * c * (2 if dt == B.BF16 else 4) // 16) * 16 + gap
    return out, at


def _to_f32(u8, e):
    n = e.rows * e.cols
    if e.dtype == B.BF16:
        return (u8[e.offset:e.offset + 2 * n].view(np.uint16).astype(np.uint32) << np.uint32(16)).view(np.float32)
    return u8[e.offset:e.offset + 4 * n].view(np.float32)


def _bf16_bits(x):
    """fp32 -> bf16 bits, nearest even (NaN stays NaN)."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> np.uint64(16)) & np.uint64(1))) >> np.uint64(16)).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def _fill(entries, nbytes, seed, std=1e-2):
    """Gradients N(0, std) in every entry, canary bytes everywhere else."""
    rng = np.random.default_rng(seed)
    u8 = np.full(nbytes, CANARY, np.uint8)
    for e in entries:
        n = e.rows * e.cols
        x = (rng.standard_normal(n) * std).astype(np.float32)
        _put(u8, e, x)
    return u8


def _put(u8, e, x):
    if e.dtype == B.BF16:
        u8[e.offset:e.offset + 2 * len(x)] = _bf16_bits(x).view(np.uint8)
    else:
        u8[e.offset:e.offset + 4 * len(x)] = np.ascontiguousarray(x, np.float32).view(np.uint8)


class Grads:
    def __init__(self, entries, u8):
        import torch

        self.torch, self.entries = torch, entries
        self.plan = B.OwnerPlan(entries, len(u8), B.make_hparams())
        self.g = torch.from_numpy(u8.copy()).cuda()
        self.ws_bytes = self.plan.grad_workspace_bytes
        self.ws = torch.full((self.ws_bytes,), CANARY, dtype=torch.uint8, device="cuda")
        self.stats = torch.full((4,), -7.0, dtype=torch.float32, device="cuda")
        self.norms = torch.full((max(1, len(entries)) + 8,), -7.0, dtype=torch.float32, device="cuda")

    @property
    def stream(self):
        return self.torch.cuda.current_stream().cuda_stream

    def norm(self, max_norm=math.inf, eps=1e-6, flags=0, entries=True):
        self.plan.grad_norm(self.g.data_ptr(), self.ws.data_ptr(), self.ws_bytes, self.stats.data_ptr(), max_norm, eps,
                            entry_norms=self.norms.data_ptr() if entries else 0, stream=self.stream, flags=flags)

    def clip(self, out, scale_ptr, flags=0):
        self.plan.grad_clip(self.g.data_ptr(), out.data_ptr(), scale_ptr, self.ws.data_ptr(), self.ws_bytes,
                            stream=self.stream, flags=flags)

    @property
    def scale_ptr(self):
        return self.stats.data_ptr() + B.GradStats.SCALE_OFFSET

    def read(self):
        self.torch.cuda.synchronize()
        h = self.stats.cpu().numpy()
        return float(h.view(np.float64)[0]), float(h[2]), float(h[3]), self.norms.cpu().numpy()


def _check(entries, u8, sumsq, norm, scale, norms, max_norm, eps):
    sq = [float(np.sum(_to_f32(u8, e).astype(np.float64) ** 2)) for e in entries]
    total = math.fsum(sq)
    assert abs(sumsq - total) <= 1e-10 * total
    want = math.sqrt(total)
    assert abs(norm - want) <= 2.0 ** -24 * want * 1.001 + TINY
    f = 1.0 if math.isinf(max_norm) else min(1.0, max_norm / (want + eps) if want + eps > 0 else 1.0)
    assert abs(scale - f) <= 2.0 ** -24 * f * 1.001 + TINY
    for k, s in enumerate(sq):
        assert abs(norms[k] - math.sqrt(s)) <= 2.0 ** -24 * math.sqrt(s) * 1.001 + TINY, k
    assert (norms[len(entries):] == -7.0).all()


BF, F = B.BF16, B.F32
TABLES = {
    "one": [(1, 1, BF)],
    "one-f32": [(1, 1, F)],
    "lengths": [(1, n, BF) for n in (1, 2, 7, 8, 9, 15, 16, 17, 63, 255, 2047, 2048, 2049)]
               + [(1, n, F) for n in (1, 3, 4, 5, 1023, 1024, 1025)],
    "empties": [(0, 64, BF), (5, 0, F), (3, 3, BF), (0, 0, BF), (2, 2, F), (7, 0, BF)],
    "chunk-edges": [(1, n, d) for d in (BF, F) for n in (4095, 4096, 4097, 8191, 8192, 8193, 16384, 16385)],
    "many": [(1 + i % 7, 1 + 13 * i % 101, BF if i % 3 else F) for i in range(700)],
    "ragged": [(777, 1001, BF), (520, 130, BF), (1, 333, F), (77, 5, F), (1300, 2003, F)],
    "large": [(4096, 4096, BF), (5000, 4097, BF), (3001, 4095, F), (1, 4096, F)],
}


@pytest.mark.parametrize("name", list(TABLES))
def test_norm(name):
    entries, nbytes = _table(TABLES[name])
    u8 = _fill(entries, nbytes, 1)
    run = Grads(entries, u8)
    for k, (max_norm, eps) in enumerate([(math.inf, 1e-6), (0.05, 1e-6), (1e9, 0.0), (1.0, 0.5)]):
        run.norm(max_norm, eps, flags=B.STEP_DESCRIPTORS_RESIDENT if k else 0)
        _check(entries, u8, *run.read(), max_norm, eps)
    assert (run.g.cpu().numpy() == u8).all()


def test_norm_of_empty_tables():
    for entries in ([], [B.TableEntry(0, 0, 5), B.TableEntry(0, 3, 0, F)]):
        run = Grads(entries, np.zeros(256, np.uint8))
        run.norm(1.0)
        sumsq, norm, scale, norms = run.read()
        assert (sumsq, norm, scale) == (0.0, 0.0, 1.0)
        assert (norms[:len(entries)] == 0).all() and (norms[len(entries):] == -7.0).all()
        run.clip(run.g, run.scale_ptr)
        run.torch.cuda.synchronize()


@pytest.mark.parametrize("value,dt", [(0.0, BF), (-0.0, F), (3e38, BF), (3e38, F), (1e-38, BF), (1e-44, F), (1e-25, BF),
                                      (2.0 ** 64, F)])
def test_norm_over_the_types_range(value, dt):
    """Squares that fp32 cannot hold, at both ends."""
    entries, nbytes = _table([(300, 50, dt), (1, 3, dt)])
    u8 = _fill(entries, nbytes, 2)
    for e in entries:
        _put(u8, e, np.full(e.rows * e.cols, value, np.float32))
    run = Grads(entries, u8)
    run.norm(1.0)
    sumsq, norm, scale, norms = run.read()
    x = float(_to_f32(u8, entries[0])[0])
    want = abs(x) * math.sqrt(15003)
    if want > float(np.finfo(np.float32).max):
        assert math.isinf(norm)
    else:
        assert abs(norm - want) <= 2.0 ** -24 * want * 1.001 + TINY
    f = min(1.0, 1.0 / (want + 1e-6))
    assert abs(scale - f) <= 2.0 ** -24 * f * 1.001 + TINY
    assert abs(sumsq - 15003 * x * x) <= 1e-10 * 15003 * x * x


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dt", [BF, F])
def test_non_finite_gradients_propagate(bad, dt):
    entries, nbytes = _table([(40, 70, BF), (33, 9, dt), (5, 5, F)])
    u8 = _fill(entries, nbytes, 3)
    x = _to_f32(u8, entries[1]).copy()
    x[-1] = bad
    _put(u8, entries[1], x)
    run = Grads(entries, u8)
    run.norm(1.0)
    sumsq, norm, scale, norms = run.read()
    if math.isnan(bad):
        assert math.isnan(sumsq) and math.isnan(norm) and math.isnan(scale) and math.isnan(norms[1])
    else:
        assert sumsq == norm == norms[1] == math.inf and scale == 0.0
    assert math.isfinite(norms[0]) and math.isfinite(norms[2])
    run.clip(run.g, run.scale_ptr, flags=B.STEP_DESCRIPTORS_RESIDENT)
    run.torch.cuda.synchronize()
    got = run.g.cpu().numpy()
    for k, e in enumerate(entries):
        y = _to_f32(got, e)
        if math.isnan(bad):
            assert np.isnan(y).all()
        else:
            assert (y[:-1] == 0).all() and (np.isnan(y[-1]) if k == 1 else y[-1] == 0)
    run.norm(math.inf)
    assert run.read()[2] == 1.0  # no limit, no scale, whatever the norm


@pytest.mark.parametrize("name", ["lengths", "empties", "chunk-edges", "ragged"])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("scale", [0.37, 1.0, 0.0, 1.0 + 2.0 ** -23, 3e-39])
def test_clip(name, in_place, scale):
    """Any device float is a scale; bytes that belong to no entry stay as they were."""
    entries, nbytes = _table(TABLES[name])
    u8 = _fill(entries, nbytes, 4)
    run = Grads(entries, u8)
    out = run.g if in_place else run.torch.full((nbytes,), 0x5A, dtype=run.torch.uint8, device="cuda")
    f = run.torch.tensor([scale], dtype=run.torch.float32, device="cuda")
    run.clip(out, f.data_ptr())
    run.torch.cuda.synchronize()
    want = u8.copy() if in_place else np.full(nbytes, 0x5A, np.uint8)
    for e in entries:
        x = _to_f32(u8, e)
        _put(want, e, x if scale == 1.0 else np.float32(scale) * x)
    assert (out.cpu().numpy() == want).all()
    assert in_place or (run.g.cpu().numpy() == u8).all()


def test_clipped_norm_is_the_limit():
    """Together: after clipping, the norm is max_norm up to the roundings of the elements."""
    entries, nbytes = _table(TABLES["large"])
    u8 = _fill(entries, nbytes, 5)
    run = Grads(entries, u8)
    run.norm(1.0)
    before = run.read()
    assert before[1] > 10 and before[2] < 0.1
    run.clip(run.g, run.scale_ptr, flags=B.STEP_DESCRIPTORS_RESIDENT)
    run.norm(math.inf, flags=B.STEP_DESCRIPTORS_RESIDENT)
    after = run.read()
    # every element moves by at most 2^-8 (bf16) of itself, so the norm does too; eps takes 1e-7 more
    assert abs(after[1] - 1.0) <= 2.0 ** -8 + 2e-6
    got = run.g.cpu().numpy()
    _check(entries, got, *after, math.inf, 1e-6)


def test_total_over_owners():
    """Records of several owners joined in order, also into one of them."""
    import torch

    rng = np.random.default_rng(6)
    sq = rng.random(9) * 10.0 ** rng.integers(-6, 6, 9)
    parts = torch.zeros(9, 2, dtype=torch.float64, device="cuda")
    parts[:, 0] = torch.from_numpy(sq).cuda()
    for count in (1, 2, 9):
        total = 0.0
        for x in sq[:count]:
            total += float(x)
        stats = torch.zeros(4, dtype=torch.float32, device="cuda")
        same = parts.clone()
        B.grad_total(parts.data_ptr(), count, stats.data_ptr(), 0.5, 1e-6, torch.cuda.current_stream().cuda_stream)
        B.grad_total(same.data_ptr(), count, same.data_ptr(), 0.5, 1e-6, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        h = stats.cpu().numpy()
        assert float(h.view(np.float64)[0]) == total
        assert abs(h[2] - math.sqrt(total)) <= 2.0 ** -24 * math.sqrt(total) * 1.001
        f = min(1.0, 0.5 / (math.sqrt(total) + 1e-6))
        assert abs(h[3] - f) <= 2.0 ** -24 * f * 1.001
        assert (same[0].cpu().numpy().view(np.uint8) == h.view(np.uint8)).all()


def test_norm_is_bitwise_repeatable_and_streams_are_independent():
    import torch

    entries, nbytes = _table(TABLES["ragged"])
    u8 = _fill(entries, nbytes, 7)
    a, b = Grads(entries, u8), Grads(entries, u8)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(20):
        for run, s in ((a, s1), (b, s2)):
            with torch.cuda.stream(s):
                run.norm(0.1, flags=B.STEP_DESCRIPTORS_RESIDENT if k else 0)
        torch.cuda.synchronize()
        got = [(x.stats.cpu().numpy().tobytes(), x.norms.cpu().numpy().tobytes()) for x in (a, b)]
        assert got[0] == got[1]
        if k == 0:
            first = got[0]
        assert got[0] == first


def _run_pair(wl, hp=None):
    runs = [DeviceRun(wl, hp) for _ in range(2)]
    for r in runs:
        r.fill(1, params_too=True)
    return runs


def _step_scaled(r, t, ptr, flags=0):
    r.plan.step_scaled(r.params.data_ptr(), r.grads.data_ptr(), r.state.data_ptr(), r.ws.data_ptr(), r.ws_bytes, t,
                       ptr, stream=r.torch.cuda.current_stream().cuda_stream, ns_out=r.ns_out.data_ptr(), flags=flags)


def _same(a, b):
    a.torch.cuda.synchronize()
    return all(bool(a.torch.equal(getattr(a, k), getattr(b, k))) for k in ("params", "state", "ns_out"))


@pytest.mark.parametrize("precision,hp", [(0, {}), (1, {}), (0, {"momentum_dtype": 1}), (0, {"nesterov": 0}),
                                          (0, {"ns_steps": 0}), (1, {"momentum_dtype": 1})])
def test_scale_of_one_is_the_plain_step(precision, hp):
    wl = W.small_ragged(precision=precision)
    a, b = _run_pair(wl, hp)
    one = a.torch.ones(1, device="cuda")
    for t in (1, 2, 3):
        for r in (a, b):
            r.fill(t, params_too=False)
        a.run(t)
        _step_scaled(b, t, one.data_ptr())
        assert _same(a, b), t


def _f32_workload():
    sp = [W.TensorSpec(f"m{i}", r, c, "f32", grad_std=1e-2) for i, (r, c) in enumerate([(100, 300), (257, 130), (64, 64)])]
    sp += [W.TensorSpec(f"v{i}", 1, n, "f32", "zeros", grad_std=1e-2) for i, n in enumerate([1, 333, 4096, 5001])]
    return W.Workload("f32-table", sp, seed=11, hparams=dict(W.MUON_DEFAULTS, ns_precision=1))


def test_scaled_step_is_clip_then_step_for_f32():
    """norm -> clip -> step and norm -> scaled step, three steps: bitwise equal."""
    a, b = _run_pair(_f32_workload())
    torch = a.torch
    ws = [torch.empty(r.plan.grad_workspace_bytes, dtype=torch.uint8, device="cuda") for r in (a, b)]
    stats = [torch.zeros(4, dtype=torch.float32, device="cuda") for _ in range(2)]
    st = torch.cuda.current_stream().cuda_stream
    for t in (1, 2, 3):
        for r, w, s in zip((a, b), ws, stats):
            r.fill(t, params_too=False)
            r.plan.grad_norm(r.grads.data_ptr(), w.data_ptr(), w.numel(), s.data_ptr(), 0.25, stream=st)
        a.plan.grad_clip(a.grads.data_ptr(), a.grads.data_ptr(), stats[0].data_ptr() + 12, ws[0].data_ptr(),
                         ws[0].numel(), stream=st, flags=B.STEP_DESCRIPTORS_RESIDENT)
        a.run(t)
        _step_scaled(b, t, stats[1].data_ptr() + 12)
        assert _same(a, b), t
        assert float(stats[0][3]) < 0.2  # the limit binds


@pytest.mark.parametrize("precision", [0, 1])
def test_scaled_momentum_and_moments(precision):
    """From zero state the momentum is scale * g and AdamW's moments are (1-b) times it and its square."""
    wl = W.small_ragged(precision=precision)
    r = DeviceRun(wl)
    r.fill(1, params_too=True)
    f = np.float32(0.3)
    ptr = r.torch.tensor([f], device="cuda")
    _step_scaled(r, 1, ptr.data_ptr())
    for i, s in enumerate(wl.specs):
        if s.numel == 0:
            continue
        g = (f * r.dev_entry(i, "grad").astype(np.float32)).astype(np.float64)
        if r.info[i].role == B.ROLE_MUON:
            assert (r.dev_entry(i, "state") == g).all(), s.name  # beta * 0 + g, exact
        else:
            # one or two fp32 roundings of each product: three half steps at most
            o1, o2 = 1.0 - float(np.float32(0.9)), 1.0 - float(np.float32(0.95))
            for got, want in ((r.dev_entry(i, "state"), o1 * g), (r.dev_entry(i, "state2"), o2 * g * g)):
                assert (np.abs(got - want) <= 3 * 2.0 ** -24 * np.abs(want) + 2.0 ** -149).all(), s.name


def test_graph_of_norm_clip_and_scaled_step():
    """Captured once with resident descriptors and replayed with fresh gradients between other eager work of the
    same program: every replay bitwise equal to the eager run."""
    sp = [s for s in W.small_ragged().specs if s.rows > 1 and s.cols > 1]
    wl = W.Workload("matrices", sp, seed=5, hparams=dict(W.MUON_DEFAULTS, ns_precision=0))
    a, b = _run_pair(wl)
    torch = a.torch
    ws = [torch.empty(r.plan.grad_workspace_bytes, dtype=torch.uint8, device="cuda") for r in (a, b)]
    stats = [torch.zeros(4, dtype=torch.float32, device="cuda") for _ in range(2)]
    clipped = [torch.zeros_like(r.grads) for r in (a, b)]

    def whole(k, r, t, flags):
        st = torch.cuda.current_stream().cuda_stream
        r.plan.grad_norm(r.grads.data_ptr(), ws[k].data_ptr(), ws[k].numel(), stats[k].data_ptr(), 0.5, stream=st,
                         flags=flags)
        r.plan.grad_clip(r.grads.data_ptr(), clipped[k].data_ptr(), stats[k].data_ptr() + 12, ws[k].data_ptr(),
                         ws[k].numel(), stream=st, flags=flags)
        _step_scaled(r, t, stats[k].data_ptr() + 12, flags)

    whole(0, a, 1, 0)
    whole(1, b, 1, 0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        whole(1, b, 2, B.STEP_DESCRIPTORS_RESIDENT)
    for t in range(2, 7):
        a.fill(t, params_too=False)
        whole(0, a, t, B.STEP_DESCRIPTORS_RESIDENT)
        b.fill(t, params_too=False)
        graph.replay()
        assert _same(a, b), t
        assert torch.equal(clipped[0], clipped[1]) and torch.equal(stats[0], stats[1]), t
    graph.reset()

"""One training step of an owner that holds a tied vocabulary table: lookup,
log probabilities, their gradient, the lookup's gradient added to it, norm and
factor, and the scaled step with moments in 8 bits, eager and captured."""

import pytest

from matrix_optimizer_owner_amd import binding as B
from tests import adam8_ref as aref
from tests.head_ref import Reference, close

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HP = dict(adam_lr=1e-3, adam_beta1=0.9, adam_beta2=0.95, adam_eps=1e-8, adam_weight_decay=0.1)
ROWS, COLS, N = 1500, 192, 210


class Run:
    def __init__(self):
        gen = torch.Generator(device="cuda").manual_seed(3)
        self.gen = gen
        entries = [B.TableEntry(0, 1, 100, B.F32, B.ROLE_ADAMW), B.TableEntry(512, ROWS, COLS, B.BF16, B.ROLE_ADAMW8)]
        size = 512 + ROWS * COLS * 2
        self.plan = p = B.OwnerPlan(entries, size, B.make_hparams(**HP))
        new = lambda n: torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")  # noqa: E731
        self.params, self.grads, self.state = new(size), new(size), new(p.state_bytes)
        self.table = self.params[512:].view(torch.bfloat16).view(ROWS, COLS)
        self.dtable = self.grads[512:].view(torch.bfloat16).view(ROWS, COLS)
        self.table.copy_(torch.randn(ROWS, COLS, generator=gen, device="cuda") * 0.1)
        self.grads[:400].view(torch.float32).copy_(torch.randn(100, generator=gen, device="cuda") * 1e-3)
        self.step_ws, self.norm_ws = new(p.workspace_bytes), new(p.grad_workspace_bytes)
        self.head_ws = new(p.head_workspace_bytes(1, N, grad=True))
        self.embed_ws = new(p.embed_workspace_bytes(1, N))
        self.ids = torch.zeros(N, dtype=torch.int64, device="cuda")
        self.targets = torch.zeros(N, dtype=torch.int64, device="cuda")
        self.x = torch.zeros(N, COLS, dtype=torch.bfloat16, device="cuda")
        self.dx = torch.zeros_like(self.x)
        self.records = torch.zeros(N, 6, device="cuda")
        self.logp = torch.zeros(N, device="cuda")
        self.dlogp = torch.zeros(N, device="cuda")
        self.stats = torch.zeros(4, device="cuda")
        self.fresh()

    def fresh(self):
        self.ids.copy_(torch.randint(0, ROWS, (N,), generator=self.gen, device="cuda"))
        self.targets.copy_(torch.randint(0, ROWS, (N,), generator=self.gen, device="cuda"))
        self.targets[5] = -1
        self.dlogp.copy_(-torch.rand(N, generator=self.gen, device="cuda") / N)

    def call(self, step, flags):
        p, s = self.plan, torch.cuda.current_stream().cuda_stream
        args = (self.params.data_ptr(), self.grads.data_ptr())
        p.embed_lookup(1, args[0], self.ids.data_ptr(), N, self.x.data_ptr(), scale=4.0, stream=s)
        ws = (self.head_ws.data_ptr(), self.head_ws.numel())
        p.head_logprob(1, args[0], self.x.data_ptr(), N, self.records.data_ptr(), *ws, ids=self.targets.data_ptr(),
                       logp=self.logp.data_ptr(), stream=s)
        p.head_grad(1, *args, self.x.data_ptr(), N, self.records.data_ptr(), self.dlogp.data_ptr(), *ws,
                    dx=self.dx.data_ptr(), ids=self.targets.data_ptr(), stream=s)
        p.embed_grad(1, args[1], self.ids.data_ptr(), N, self.dx.data_ptr(), self.embed_ws.data_ptr(), self.embed_ws.numel(),
                     scale=4.0, accumulate=True, stream=s)
        p.grad_norm(args[1], self.norm_ws.data_ptr(), self.norm_ws.numel(), self.stats.data_ptr(), max_norm=0.01, stream=s,
                    flags=flags)
        p.step_scaled(*args, self.state.data_ptr(), self.step_ws.data_ptr(), self.step_ws.numel(), step,
                      self.stats.data_ptr() + B.GradStats.SCALE_OFFSET, stream=s, flags=flags)


def test_eager_step_against_the_formulas():
    r = Run()
    for step in (1, 2):
        before, state = r.table.double().clone(), r.state.cpu().numpy()
        r.call(step, B.STEP_DESCRIPTORS_RESIDENT if step > 1 else 0)
        # the lookup, exact: products with 4
        assert torch.equal(r.x, (before[r.ids] * 4).bfloat16())
        t = r.targets
        ref = Reference(r.x, before, torch.where(t >= 0, t, -1), t >= 0, 1.0)
        assert ((r.logp.double() - ref.logp()).abs() <= ref.logp_tol[:, 0]).all()
        rx, ex, rw, ew = ref.grads(r.dlogp, None, torch.bfloat16)
        close(r.dx, rx, ex, 4e-3)
        # the head's gradient is rounded to bf16, the lookup's added to it in fp32 and rounded again
        want = rw.index_add(0, r.ids, 4 * r.dx.double())
        size = rw.abs().index_add(0, r.ids, 4 * r.dx.double().abs())
        close(r.dtable, want, ew + 2.0 ** -8 * (rw.abs() + ew) + N * 2.0 ** -24 * size)
        g = torch.cat([r.grads[:400].view(torch.float32).double(), r.dtable.double().view(-1)])
        norm = float(g.norm())
        assert abs(float(r.stats[2]) / norm - 1) < 1e-6
        factor = float(r.stats[3])
        assert abs(factor / min(1.0, 0.01 / (norm + 1e-6)) - 1) < 1e-6
        info, n = r.plan.entry_info(1), ROWS * COLS
        m, root = (state[o:o + aref.code_bytes(n)] for o in (info.state_offset, info.state_offset2))
        w, tol, *_ = aref.step(before.view(-1).cpu().numpy(), r.dtable.double().view(-1).cpu().numpy() * factor,
                               aref.first_values(m, n), aref.root_values(root, n), HP, step, 1)
        got = r.table.double().view(-1).cpu().numpy()
        assert (abs(got - w) <= tol + 2.0 ** -8 * (abs(w) + tol)).all()
        r.fresh()


def test_captured_step_replayed_with_fresh_inputs():
    r = Run()
    r.call(1, 0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = r.params.clone(), r.state.clone()
    with torch.cuda.graph(graph):
        r.call(2, B.STEP_DESCRIPTORS_RESIDENT)
    for _ in range(3):
        r.fresh()
        r.params.copy_(keep[0])
        r.state.copy_(keep[1])
        r.call(2, B.STEP_DESCRIPTORS_RESIDENT)
        torch.cuda.synchronize()
        want = [t.clone() for t in (r.params, r.state, r.grads, r.logp, r.dx, r.stats)]
        r.params.copy_(keep[0])
        r.state.copy_(keep[1])
        for t in (r.grads[512:], r.logp, r.dx, r.stats):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (r.params, r.state, r.grads, r.logp, r.dx, r.stats)))

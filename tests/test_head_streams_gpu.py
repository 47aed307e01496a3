"""Calls of the output head that are on their way at the same time: two streams,
a workspace each, no wait of the host between them."""

import pytest

from matrix_optimizer_owner_amd import binding as B

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_head_gpu import Head, batch  # noqa: E402


def test_calls_on_two_streams_overlap():
    h = Head(30000, 512)
    calls = []
    for n, top_k, seed in ((600, 0, 3), (40, 3, 4)):
        x, ids = batch(n, 512, rows=30000, seed=seed)
        dlogp = torch.randn(n, device="cuda")
        ws = h.space(n, B.BF16, top_k, grad=True)
        outs = dict(records=torch.empty(n, 6, device="cuda"), logp=torch.empty(n, device="cuda"),
                    entropy=torch.empty(n, device="cuda"), top=torch.empty(n, max(top_k, 1), dtype=torch.int64, device="cuda"),
                    dx=torch.empty_like(x), grads=torch.zeros(h.nbytes, dtype=torch.uint8, device="cuda"))

        def call(stream, n=n, top_k=top_k, x=x, ids=ids, dlogp=dlogp, ws=ws, o=outs):
            s = stream.cuda_stream
            h.plan.head_logprob(0, h.params.data_ptr(), x.data_ptr(), n, o["records"].data_ptr(), ws.data_ptr(), ws.numel(),
                                ids=ids.data_ptr(), logp=o["logp"].data_ptr(), entropy=o["entropy"].data_ptr(), top_k=top_k,
                                top_ids=o["top"].data_ptr(), stream=s)
            h.plan.head_grad(0, h.params.data_ptr(), o["grads"].data_ptr(), x.data_ptr(), n, o["records"].data_ptr(),
                             dlogp.data_ptr(), ws.data_ptr(), ws.numel(), dx=o["dx"].data_ptr(), ids=ids.data_ptr(), stream=s)

        call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        o = {k: v.clone() for k, v in outs.items()}
        for v in outs.values():
            v.zero_()
        calls.append((call, outs, o))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):  # nothing here waits: each stream's queue fills while the other's runs
        for (call, _, _), s in zip(calls, streams):
            call(s)
    torch.cuda.synchronize()
    for _, outs, want in calls:
        for k in want:
            if k != "top" or want[k].shape[1] > 1:
                assert torch.equal(outs[k].view(torch.uint8), want[k].view(torch.uint8)), k

"""AdamW on the longest tail that a GPU of 288 GB holds: more 2048-element
chunks than one launch has blocks for."""

import pytest

from matrix_optimizer_owner_amd import binding as B

pytestmark = [pytest.mark.gpu, pytest.mark.slow]


@pytest.mark.parametrize("scaled", [False, True])
def test_tail_of_more_than_2_to_34_elements(scaled):
    """2^22 x 4097 bf16 elements (206 GB with gradients and moments), all of the same values: every element comes out
    as those of a small table do, the first and the last ones among them."""
    import gc

    import torch

    gc.collect()
    torch.cuda.empty_cache()
    rows, cols = 1 << 22, 4097
    n = rows * cols
    if torch.cuda.mem_get_info()[0] < 12 * n + (4 << 30):
        pytest.skip("not enough free device memory")
    stream = torch.cuda.current_stream().cuda_stream
    scale = torch.full((1,), 0.5, device="cuda")

    def step(rows):
        n = rows * cols
        plan = B.OwnerPlan([B.TableEntry(0, rows, cols, B.BF16, B.ROLE_ADAMW)], 2 * n, B.make_hparams())
        params = torch.full((n,), 1.0, dtype=torch.bfloat16, device="cuda")
        grads = torch.full((n,), 0.25, dtype=torch.bfloat16, device="cuda")
        state = torch.zeros(plan.state_bytes // 4, dtype=torch.float32, device="cuda")
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        args = (params.data_ptr(), grads.data_ptr(), state.data_ptr(), ws.data_ptr(), ws.numel(), 1)
        if scaled:
            plan.step_scaled(*args, scale.data_ptr(), stream=stream)
        else:
            plan.step(*args, stream=stream)
        torch.cuda.synchronize()
        info = plan.entry_info(0)
        m, v = info.state_offset // 4, info.state_offset2 // 4
        return params, state[m:m + n], state[v:v + n]

    want = [float(x[0]) for x in step(3)]
    assert want[0] != 1.0 and want[1] != 0.0 and want[2] != 0.0
    got = step(rows)
    for x, w in zip(got, want):
        for k in range(0, n, 1 << 30):
            part = x[k:k + (1 << 30)]
            assert bool(part.amin() == w) and bool(part.amax() == w), (k, float(part.amin()), float(part.amax()), w)
    del got
    torch.cuda.empty_cache()

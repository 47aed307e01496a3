"""Norm and clipping of a table of 20000 small tensors beside a large one (more
tensors than the clipping list has chunks for a table of large ones)."""

import numpy as np
import pytest

from matrix_optimizer_owner_amd import binding as B
from tests.test_grad_ops_gpu import BF, F, Grads, _check, _fill, _put, _table, _to_f32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("large", [False, True])
def test_many_tensors(large):
    spec = [(1 + i % 5, 1 + i % 61, BF if i % 2 else F) for i in range(20000)]
    if large:
        spec.insert(7000, (9001, 4099, BF))
    entries, nbytes = _table(spec)
    u8 = _fill(entries, nbytes, 1)
    run = Grads(entries, u8)
    run.norm(0.5)
    got = run.read()
    _check(entries, u8, *got, 0.5, 1e-6)
    scale = np.float32(got[2])
    assert scale < 1
    run.clip(run.g, run.scale_ptr, flags=B.STEP_DESCRIPTORS_RESIDENT)
    run.torch.cuda.synchronize()
    want = u8.copy()
    for e in entries:
        _put(want, e, scale * _to_f32(u8, e))
    assert (run.g.cpu().numpy() == want).all()

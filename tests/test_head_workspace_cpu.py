"""Device workspace of the output head's forward call on few tokens."""

import pytest

from matrix_optimizer_owner_amd import binding as B


@pytest.mark.parametrize("rows,cols,kind", [(128256, 4096, B.F32), (128256, 4100, B.BF16), (128256, 4096, B.BF16), (50257, 768, B.F32),
                                            (700, 33, B.F32), (1, 1, B.BF16)])
@pytest.mark.parametrize("x_type", [B.F32, B.BF16])
def test_few_tokens_need_no_copy_of_the_table(rows, cols, kind, x_type):
    """Up to 64 tokens: 16 bytes a token and part of 32 rows (or two of each 128, as larger batches have them), 4 a token and
    row for alternatives, targets."""
    plan = B.OwnerPlan([B.TableEntry(0, rows, cols, kind, B.ROLE_ADAMW)], 1 << 34, B.make_hparams())
    for n in (1, 2, 31, 32, 33, 63, 64):
        for top_k in (0, 5):
            need = plan.head_workspace_bytes(0, n, x_type=x_type, top_k=top_k)
            parts = 16 * n * max(-(-rows // 32), 2 * -(-rows // 128))
            logits = 4 * n * -(-rows // 256) * 256 if top_k else 0
            assert need <= parts + logits + 4 * 256 + 4 * 256, (n, top_k, need)
    # a batch has the packed operands in it, and is never below
    assert plan.head_workspace_bytes(0, 65, x_type=x_type) >= plan.head_workspace_bytes(0, 64, x_type=x_type)

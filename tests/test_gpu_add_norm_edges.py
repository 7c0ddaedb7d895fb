"""mla_add_norm and mla_add_norm_bwd with rows that stand for all rows."""
import pytest
import torch

from tests.test_gpu_add_norm import EPS, _rows, smla  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [None, 128, 0])
def test_broadcast_rows_beside_given_outputs(smla, group):  # noqa: F811
    x, r, w = _rows(21, 700, 520)
    pool = torch.zeros(701, 520, dtype=x.dtype, device=x.device)
    pool[0] = r[0]
    row, z = pool[:1].expand(700, 520), pool[1:]
    want = smla.mla_add_norm(x, w, row.contiguous(), eps=EPS, group=group)
    got = smla.mla_add_norm(x, w, row, eps=EPS, group=group, residual_out=z)
    assert got[2] is z and torch.equal(pool[0], r[0])
    for a, b in zip(got, want):
        assert a is b is None or torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    grads = smla.mla_add_norm_bwd(want[2], w, row.contiguous(), row.contiguous(), eps=EPS)
    same = smla.mla_add_norm_bwd(want[2], w, row, row, eps=EPS, dx=z)
    assert same[0] is z and all(torch.equal(a, b) for a, b in zip(same, grads))

"""Sizes and extents of the residual norm's and the dense attention's calls that
the binding alone sees (no GPU): counts past what the library takes, and outputs
beside broadcast rows."""
import pytest
import torch

from tests.test_binding_checks import _ok, _refused, b  # noqa: F401  (the recorder fixture)

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
BIG = 2 ** 32 + 8   # 8 in 32 bits


def _meta(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("n,d", [(BIG, 64), (8, BIG), (2 ** 31, 8)])
def test_norms_refuse_counts_past_32_bits(b, n, d):  # noqa: F811
    x, w = _meta(n, d), _meta(d)
    _refused(b, b.mla_add_norm, x, w, x, match="2\\^31")
    _refused(b, b.mla_add_norm, x, w, group=128, match="2\\^31")
    _refused(b, b.mla_add_norm_bwd, x, w, x, match="2\\^31")
    with pytest.raises(ValueError, match="2\\^31"):
        b.add_norm_bwd_workspace_size(n, d)


@pytest.mark.parametrize("nq,nk,h,hk,d,dv", [(BIG, 8, 1, 1, 128, 128), (8, BIG, 1, 1, 128, 128), (8, 8, 1, 1, 2 ** 32 + 192, 128),
                                             (8, 8, 1, 1, 192, 2 ** 32 + 128), (1, 1, BIG, 1, 128, 128)])
def test_attention_refuses_counts_past_32_bits(b, nq, nk, h, hk, d, dv):  # noqa: F811
    q, k, v = _meta(nq, h, d), _meta(nk, hk, d), _meta(nk, hk, dv)
    _refused(b, b.dense_mha_fwd, q, k, v, 0.1, match="2\\^31")
    _refused(b, b.dense_mha_bwd, q, k, v, 0.1, _meta(nq, h, dv), _meta(nq, h, dtype=F32), _meta(nq, h, dv), match="2\\^31")
    with pytest.raises(ValueError, match="2\\^31"):
        b.dense_mha_bwd_workspace_size(nq, nk, 1, h, hk, d, dv)


def test_attention_refuses_more_offsets_than_32_bits_count(b):  # noqa: F811
    q, k, v, cu = _meta(8, 1, 128), _meta(8, 1, 128), _meta(8, 1, 128), _meta(2 ** 32 + 2, dtype=I32)
    _refused(b, b.dense_mha_fwd, q, k, v, 0.1, cu, cu, match="2\\^31")


def test_an_output_behind_a_broadcast_row_is_apart_from_it(b):  # noqa: F811
    """A row that stands for all of them takes up one row of memory."""
    pool, w = torch.zeros(11, 64, dtype=BF), torch.zeros(64, dtype=BF)
    row, x, out = pool[:1].expand(5, 64), pool[6:], pool[1:6]
    for kw in (dict(x=row, out=out), dict(x=x, residual=row, residual_out=out),
               dict(x=x, residual=row, group=0, scales=out.view(-1)[:10].view(F32))):
        _ok(b, "mla_add_norm", b.mla_add_norm, weight=w, **kw)
    _ok(b, "mla_add_norm_bwd", b.mla_add_norm_bwd, z=row, weight=w, dout=x, dx=out)
    _ok(b, "mla_add_norm_bwd", b.mla_add_norm_bwd, z=x, weight=w, dout=row, dresidual=row, dx=out)
    # the row itself, and rows that meet it
    _refused(b, b.mla_add_norm, row, w, out=pool[:5])
    _refused(b, b.mla_add_norm, x, w, row, residual_out=pool[:5])
    _refused(b, b.mla_add_norm_bwd, x, w, row, dx=pool[:5])

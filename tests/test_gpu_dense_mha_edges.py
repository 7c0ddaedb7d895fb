"""dense_mha_fwd and dense_mha_bwd where their formulas have an edge: orders of a
CTA's stages, values that are not finite, rows that see one key, tiles that take
long, and sizes past what a product of two counters holds.  Helpers and the derivation of the
tolerances are test_gpu_dense_mha's."""
import pytest
import torch

from tests.test_gpu_dense_mha import _inputs, smla  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,h,hk", [(192, 4, 4), (128, 8, 1)])
def test_gradients_repeat_bit_for_bit(smla, d, h, hk):  # noqa: F811
    """Many blocks through every stage of the ring, beside another call that shifts the CTAs' timing: a number that
    a stage's reader takes before its writer has put it there shows as other bits."""
    q, k, v, do, cq, ck = _inputs(30, [700, 1, 1900, 65], [1000, 1, 1900, 65], h, hk, d)
    out, lse = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
    want = smla.dense_mha_bwd(q, k, v, 0.1, out, lse, do, cq, ck)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(30):
        with torch.cuda.stream(side):
            smla.dense_mha_fwd(q[:700 - 20 * i], k[:700], v[:700], 0.1)
        got = smla.dense_mha_bwd(q, k, v, 0.1, out, lse, do, cq, ck)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
    torch.cuda.synchronize()


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_two_tiles_that_end_in_one_block(smla, what):  # noqa: F811
    """All heads of a token side by side, two tokens to a CTA: both tiles look over the same last block of values,
    and what either takes out is put back in the rows of both that see it."""
    n, h = 900, 128
    q, k, v, *_ = _inputs(31, [n], [n], h, 1, 128)
    want = smla.dense_mha_fwd(q, k, v, 0.1)
    cols = torch.zeros(128, dtype=torch.bool, device=v.device)
    cols[3::50] = True
    for at in (0, 127, 128, 300, 301, 640, 898, 899):
        v2 = v.clone()
        v2[at, :, cols] = what
        for _ in range(5):
            out, lse = smla.dense_mha_fwd(q, k, v2, 0.1)
            assert torch.equal(lse, want[1]) and torch.equal(out[:at], want[0][:at])
            assert torch.equal(out[..., ~cols], want[0][..., ~cols]) and not out[at:][..., cols].isfinite().any()

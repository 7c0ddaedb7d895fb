"""mla_norm_rope and mla_norm_rope_bwd: cache factors that are not powers of
two, byte by byte; rows at the ends of the norm's range; padding rows of
outputs that the call allocates; more rows than the backward's warps."""
import numpy as np
import pytest
import torch

import mla_inputs as mi
from oracle import fp4_kv_oracle as f4
from oracle import norm_rope_oracle as nro
from tests import test_gpu_norm_rope as base

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def smla(cuda_lib):
    import serving_sparse_mla_gb300 as pkg
    pkg.clear_device_error()
    yield pkg
    assert pkg.get_device_error() == 0


@pytest.mark.parametrize("normed", [True, False])
@pytest.mark.parametrize("ks", [0.3, 0.1, 0.7, 1.7, 0.01, 1 / 3, 12345.678, 3e-19, 1.7e19])
def test_cache_bytes_with_any_factor(smla, ks, normed):
    """Scales and codes where the factor rounds: unnormed rows have few bits, so
    that many quotients lie at a border."""
    base._run_and_check(smla, 91, 700, 1, "fp4", True, q_norm=False, kv_norm=normed, kv_scale=ks, page=64)


@pytest.mark.parametrize("ks", [1.0, 0.25, 0.3, 0.7])
def test_kv_out_and_the_slots(smla, ks):
    """kv_out is the slot's row rounded to bf16: the same where the factor is a
    power of two, else within half a step of it (and not always the same)."""
    n = 200
    q, kv, _, kw = (t.to(DEV) for t in mi.norm_rows(92, n, 1))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    cache = torch.zeros(4, 64, 416, dtype=torch.uint8, device=DEV)
    _, ko = smla.mla_norm_rope(q, kv, pos, mi.rope_table(n).to(DEV), kv_weight=kw, kv_cache=cache, slots=pos, kv_scale=ks)
    row = f4.dequantize_slots(cache.view(-1, 416)[:n], ks)
    d = np.abs(ko.double().cpu().numpy() - row)
    # half a step, and one fp32 rounding before it (scale * factor; the product)
    assert np.all(d <= (2.0 ** -8 + 2.0 ** -22) * np.abs(row))
    assert (d.max() == 0) == (ks in (1.0, 0.25))


@pytest.mark.parametrize("ks", [0.3, 0.7, 2.0 ** -3])
def test_serving_chain_with_a_factor(smla, ks):
    """Rows written with a factor, then the decode with it, against the oracle
    over the slots themselves: an engine's two calls of a step."""
    n, h, page, topk, sn = 150, 8, 16, 96, 3
    q, kv, qw, kw = (t.to(DEV) for t in mi.norm_rows(33, n, h))
    table = torch.randperm(14, generator=torch.Generator().manual_seed(1))[:10].int().view(1, 10)
    pos = torch.arange(n, dtype=torch.int32)
    slots = table[0][(pos // page).long()] * page + pos % page
    cache = torch.full((14, page, 416), 0x7F, dtype=torch.uint8, device=DEV)   # NaN scales wherever nothing is written
    qo, _ = smla.mla_norm_rope(q, kv, pos.to(DEV), mi.rope_table(n).to(DEV), qw, kw, kv_cache=cache,
                               slots=slots.to(DEV), kv_scale=ks)
    idx = mi.prefill_indices(4, n, n, topk)[n - sn:].view(1, sn, topk)
    qd, lens = qo[n - sn:].view(1, sn, h, 576), torch.tensor([n], dtype=torch.int32)
    o, l = smla.sparse_mla_decode_fp4(qd, cache, table.to(DEV), lens.to(DEV), idx.to(DEV), 576 ** -0.5, kv_scale=ks)
    ro, rl = f4.sparse_mla_decode_fp4(qd.cpu(), cache.cpu(), table, lens, idx, 576 ** -0.5, page, ks)
    got = o.double().cpu().numpy().reshape(ro.shape)
    assert np.all(np.abs(got - ro) <= 2.0 ** -8 * np.abs(ro) + 2e-3)
    assert np.all(np.abs(l.double().cpu().numpy().reshape(rl.shape) - rl) <= 1e-4)


@pytest.mark.parametrize("given", ["", "q", "kv", "both"])
def test_padding_rows_of_fresh_outputs(smla, given):
    """Outputs that the call allocates are zeros in padding tokens' rows; those
    it is given keep what they hold."""
    n, h = 40, 4
    q, kv, qw, kw = (t.to(DEV) for t in mi.norm_rows(93, n, h))
    pos = torch.arange(n, dtype=torch.int32)
    pos[5], pos[30:] = n, -1
    live = (pos >= 0) & (pos < n)
    cs = mi.rope_table(n).to(DEV)
    out = dict(q_out=torch.full((n, h, 576), 3.0, dtype=torch.bfloat16, device=DEV) if given in ("q", "both") else None,
               kv_out=torch.full((n, 576), 3.0, dtype=torch.bfloat16, device=DEV) if given in ("kv", "both") else None)
    for _ in range(3):
        # blocks of the outputs' sizes, freed full of NaN, are what the call gets
        dirty = [torch.full_like(q, float("nan")) for _ in range(4)] + [torch.full_like(kv, float("nan")) for _ in range(4)]
        del dirty
        qo, ko = smla.mla_norm_rope(q, kv, pos.to(DEV), cs, qw, kw, **out)
        assert bool((qo[~live] == (3 if given in ("q", "both") else 0)).all())
        assert bool((ko[~live] == (3 if given in ("kv", "both") else 0)).all())
        want = smla.mla_norm_rope(q[live], kv[live], pos[live].to(DEV), cs, qw, kw)
        assert torch.equal(qo[live], want[0]) and torch.equal(ko[live], want[1])


@pytest.mark.parametrize("size,eps", [(2.0 ** 59, 1e-6), (2.0 ** -50, 0.0), (2.0 ** 40, 0.0), (2.0 ** -40, 1e-30)])
def test_rows_at_the_ends_of_the_range(smla, size, eps):
    """Mean squares up to 2^118 and down to 2^-100."""
    n, h = 6, 3
    g = torch.Generator().manual_seed(7)
    q, kv = torch.randn(n, h, 576, generator=g), torch.randn(n, 576, generator=g)
    q[..., :512] *= size
    kv[..., :512] *= size
    q, kv = q.bfloat16(), kv.bfloat16()
    qw, kw = (1 + 0.2 * torch.randn(2, 512, generator=g)).bfloat16()
    pos, cs = torch.arange(n, dtype=torch.int32), mi.rope_table(n)
    d = lambda t: t.to(DEV)  # noqa: E731
    qo, ko = smla.mla_norm_rope(d(q), d(kv), d(pos), d(cs), d(qw), d(kw), eps=eps)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    ref = nro.rms_norm(f64(q)[..., :512], f64(qw), eps)
    assert np.all(np.abs(f64(qo)[..., :512] - ref) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(ref))
    assert np.array_equal(f64(ko)[:, :512], nro.round_bf16(nro.rms_norm(f64(kv)[:, :512], f64(kw), eps)))
    dq, dkv = torch.randn(n, h, 576, generator=g), torch.randn(n, 576, generator=g)
    got = smla.mla_norm_rope_bwd(d(q), d(kv), d(pos), d(cs), d(dq), d(dkv), d(qw), d(kw), eps=eps)
    ang = f64(cs)
    for k, x, dy, w, a in ((0, q, dq, qw, ang[:, None]), (1, kv, dkv, kw, ang)):
        dx, dw = nro.norm_rope_bwd(f64(x), f64(dy), a, f64(w), eps, True)
        x64 = f64(x)[..., :512]
        r = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + eps)
        gw, xh = np.abs(f64(dy)[..., :512] * f64(w)), np.abs(x64) * r
        terms = r * (gw + xh * (gw * xh).mean(-1, keepdims=True))
        # 2^-133: half of bf16's smallest step, which gradients of rows of 2^59 come near to
        tol = 2.0 ** -8 * np.abs(dx[..., :512]) + 2.0 ** -18 * terms + 2.0 ** -133
        assert np.all(np.abs(f64(got[k])[..., :512] - dx[..., :512]) <= tol)
        tw = (np.abs(f64(dy)[..., :512]) * xh).reshape(-1, 512).sum(0)
        assert np.all(np.abs(f64(got[2 + k]) - dw) <= 2.0 ** -18 * tw)


@pytest.mark.parametrize("n,h,norms", [(5200, 1, "qk"), (6001, 2, "k"), (5200, 1, "q")])
def test_backward_of_more_rows_than_warps(smla, n, h, norms):
    """Over 2 x 2432 tokens: every warp takes several latent rows."""
    base.test_backward(smla, True, n, h, norms, 7)

"""The 4-bit decode where sizes differ: a cache factor far from 1 with queries
that make up for it, large scores, lists much longer than usual.

Bounds.  A score is a sum of 576 exact products in two chains of 18 MMAs; an
MMA's sum may be cut off instead of rounded, 2^-22 of the sizes at hand, and
four more roundings follow: e = 22 * 2^-22 sum |q x| sm_scale.  The latent
query is f16 after a power of two: elements below 2^-14 of the head's largest
one lose at most 2^-25 of that, e += 2^-25 max |q| sum |x| sm_scale.  LSE: e
and 2^-21 of the largest score (base-2 scores, the logarithm).  Outputs: half
a bf16 step 2^-8 |out|, and for P's rounding to f16 (2^-11), the scores' error
in either sum (2 e) and the fp32 sums (2^-14): (2^-11 + 2 e + 2^-14) sum p |x|.
f16's steps end at 2^-24: P, 2^7 for a weight as large as the running maximum,
is off by up to 2^-25 however small it is, that is by 2^-32 of the largest
weight p <= 1, and the output by 2^-32 sum |x|."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import mla_inputs as mi
from oracle import fp4_kv_oracle as f4
from oracle import sparse_mla_oracle as orc

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def smla(cuda_lib):
    import serving_sparse_mla_gb300 as pkg
    pkg.clear_device_error()
    yield pkg
    assert pkg.get_device_error() == 0


def _check(smla, c, u, ks):
    """The decode of case c over slots u with the factor ks, head by head."""
    d = lambda t: t.to(DEV)  # noqa: E731
    out, lse = smla.sparse_mla_decode_fp4(d(c.q), d(u), d(c.block_table), d(c.cache_seqlens), d(c.indices), c.sm_scale,
                                          c.page_size, kv_scale=ks)
    n = c.batch * c.s_next
    o, l = out.double().cpu().numpy().reshape(n, c.h_q, 512), lse.double().cpu().numpy().reshape(n, c.h_q)
    X = f4.dequantize_slots(u, ks).reshape(-1, 576)
    idx, tab, lens = c.indices.numpy().astype(np.int64), c.block_table.numpy().astype(np.int64), c.cache_seqlens.numpy()
    for t in range(n):
        b, j = divmod(t, c.s_next)
        x = X[orc.rows_paged(idx[b, j], tab[b], int(lens[b]), c.page_size, u.shape[0])]
        q = c.q[b, j].double().numpy().reshape(c.h_q, 576)
        s = c.sm_scale * (q @ x.T)
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        want = (top + np.log(p.sum(1, keepdims=True)))[:, 0]
        p /= p.sum(1, keepdims=True)
        e = 22 * 2.0 ** -22 * c.sm_scale * (np.abs(q) @ np.abs(x).T)
        e += 2.0 ** -25 * c.sm_scale * np.abs(q[:, :512]).max(1, keepdims=True) * np.abs(x[:, :512]).sum(1)
        # only rows that weigh something count: the others' share is below 2^-40 whatever their error below 2
        e = np.where(p > 2.0 ** -50, e, 0).max(1)
        assert np.all(e < 2), "the case says nothing"
        bad = np.abs(l[t] - want) > e + 2.0 ** -21 * np.abs(s).max(1)
        assert not bad.any(), f"lse off by {np.abs(l[t] - want).max():.3e}, allowed {e.max():.3e}"
        ref, size = p @ x[:, :512], p @ np.abs(x[:, :512])
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * e[:, None] + 2.0 ** -14) * size
        tol += 2.0 ** -32 * np.abs(x[:, :512]).sum(0)
        bad = np.abs(o[t] - ref) > tol
        assert not bad.any(), f"{int(bad.sum())} outputs off, worst {(np.abs(o[t] - ref) / tol).max():.2f} of the bound"


@pytest.mark.parametrize("h_q", [8, 12, 24, 64])
@pytest.mark.parametrize("ks", [2.0 ** 16, 2.0 ** 20, 2.0 ** 24, 2.0 ** -24, 2.0 ** 60, 2.0 ** -60])
def test_latent_queries_that_make_up_for_the_factor(smla, h_q, ks):
    """Latent rows of size ks, latent queries of size 1 / ks, rotated parts of
    size 1: scores as ever.  The latent part's exponent is its own."""
    c, u = mi.decode_case_fp4(1500 + h_q, batch=3, s_next=2, h_q=h_q, lo=100, hi=400, topk=200, page=64, spare_pages=2)
    q = c.q.float()
    q[..., :512] /= ks
    c.q = q.bfloat16()
    _check(smla, c, u, ks)


@pytest.mark.parametrize("h_q", [8, 24])
@pytest.mark.parametrize("latent,rotated", [(0.0, 1.0), (1.0, 0.0), (2.0 ** -30, 1.0), (1.0, 2.0 ** -30), (1.0, 2.0 ** 6)])
def test_parts_of_unequal_size(smla, h_q, latent, rotated):
    c, u = mi.decode_case_fp4(1520 + h_q, batch=2, s_next=2, h_q=h_q, lo=100, hi=400, topk=200, page=64, spare_pages=2)
    q = c.q.float()
    q[..., :512] *= latent
    q[..., 512:] *= rotated
    c.q = q.bfloat16()
    _check(smla, c, u, 1.0)


@pytest.mark.parametrize("h_q", [8, 16, 24, 64])
@pytest.mark.parametrize("ks", [0.3, 2.0 ** 8, 2.0 ** 12])
def test_large_scores(smla, h_q, ks):
    """Scores up to some 10^4, where one row or a few take all: each head's LSE
    against its own bound."""
    c, u = mi.decode_case_fp4(1540 + h_q, batch=2, s_next=2, h_q=h_q, lo=300, hi=600, topk=256, page=64, spare_pages=2)
    _check(smla, c, u, ks)


@pytest.mark.parametrize("h_q", [8, 16, 24])
def test_small_weights_of_a_long_list(smla, h_q):
    """One row far above 262143 others, whose weights are 2^-26 of its own: they
    add up to 0.4 %.  Enough tokens that a CTA has a whole list.  P's steps
    cost at most 2^-32 a row (n 2^-32 of the largest value), the sums over
    16384 MMAs 2^-9 (each cut off by 2^-23 of what is there)."""
    n, topk, h = 456, 1 << 18, h_q
    u = np.zeros((16, 416), dtype=np.uint8)
    u[:, 256:288] = 0x38                      # scales of 1
    u[0, 0], u[0, 256] = 0x07, 0x44           # row 0: column 0 is 6 * 3
    u[1, 8] = 0x07                            # row 1: column 16 is 6
    cache = torch.from_numpy(u).view(1, 16, 416).to(DEV)
    q = torch.zeros(1, n, h, 576)
    q[..., 0] = 1
    lists = torch.ones(topk, dtype=torch.int32, device=DEV)
    lists[0] = 0
    z = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    out, lse = smla.sparse_mla_decode_fp4(q.bfloat16().to(DEV), cache, z([[0]]), z([16]),
                                          lists.expand(1, n, topk).contiguous(), 1.0)
    a, b = math.exp(18.0), topk - 1.0
    want = np.zeros(512)
    want[0], want[16] = 18 * a / (a + b), 6 * b / (a + b)
    got = out.double().cpu().numpy().reshape(-1, 512)
    tol = (2.0 ** -8 + 2.0 ** -9) * want + 6 * topk * 2.0 ** -32
    assert tol[16] < want[16] / 16
    assert np.all(np.abs(got - want) <= tol), np.abs(got - want).max(0)[[0, 16]]
    # fp32 sums of topk / 32 weights a lane: the lane that holds the large one loses its share of the small ones
    assert np.all(np.abs(lse.double().cpu().numpy() - math.log(a + b)) <= b / a / 16 + 2.0 ** -20 * 18)


@pytest.mark.parametrize("h_q", [8, 16, 24])
@pytest.mark.parametrize("step", [1, 2, 3, 4, 5, 6])
def test_scores_past_the_steps_of_one(smla, h_q, step):
    """Scores near 2^27 in powers of two, 16 apart (one step of fp32 there), the
    higher ones in later blocks: P stays finite, the output lies between the
    rows and the LSE is the higher score's to fp32's steps."""
    n, topk = 456, 1024
    u = np.zeros((16, 416), dtype=np.uint8)
    u[:, 256:288] = 0x38                      # scales of 1
    u[:2, 0], u[:2, 256] = 0x06, 0x40         # column 0 is 4 * 2 = 8
    u[0, 8], u[1, 8] = 0x02, 0x07             # column 16 is 1 and 6
    rope = torch.tensor([step, step + 1]) * 2.0 ** -20
    u[:2, 288:290] = rope.bfloat16().view(torch.uint8).numpy().reshape(2, 2)
    cache = torch.from_numpy(u).view(1, 16, 416).to(DEV)
    q = torch.zeros(1, n, h_q, 576)
    q[..., 0] = q[..., 512] = 1
    z = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    lists = (torch.arange(topk, device=DEV, dtype=torch.int32) // 128) % 2
    out, lse = smla.sparse_mla_decode_fp4(q.bfloat16().to(DEV), cache, z([[0]]), z([16]),
                                          lists.expand(1, n, topk).contiguous(), math.log(2) * 2.0 ** 24)
    o = out.double().cpu().numpy().reshape(-1, 512)
    assert np.all(np.isfinite(o)) and bool(torch.isfinite(lse).all())
    assert np.all(np.abs(o[:, 0] - 8) <= 2.0 ** -8 * 8) and np.all((o[:, 16] >= 1 - 2.0 ** -8) & (o[:, 16] <= 6 + 6 * 2.0 ** -8))
    want = math.log(2) * 2.0 ** 24 * (8 + float(rope[1]))
    assert np.all(np.abs(lse.double().cpu().numpy() - want) <= 2.0 ** -21 * want)


def test_the_first_call_of_a_process_may_be_captured():
    """A process whose first call of the library is a captured 4-bit decode: the
    kernels' set-up takes place during the capture."""
    code = """
import torch
import mla_inputs as mi
import serving_sparse_mla_gb300 as smla
d = lambda t: t.to("cuda:0")
cases = [mi.decode_case_fp4(60 + k, batch=2, s_next=2, h_q=h, lo=300, hi=400, topk=256, spare_pages=2) for k, h in enumerate((8, 24))]
args = [([d(t) for t in (c.q, u, c.block_table, c.cache_seqlens, c.indices)], c.sm_scale) for c, u in cases]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = [smla.sparse_mla_decode_fp4(*a, s) for a, s in args]
g.replay()
torch.cuda.synchronize()
for (a, s), r in zip(args, got):
    want = smla.sparse_mla_decode_fp4(*a, s)
    torch.cuda.synchronize()
    assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1]) and bool((r[0] != 0).any())
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, r.stdout + r.stderr

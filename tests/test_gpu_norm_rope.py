"""mla_norm_rope and mla_norm_rope_bwd against the float64 oracle.

Tolerances.  A bf16 output is within half a step of its exact value, 2^-8 of
it (8 significant bits: the step is at most 2^-7 of the value, half of it
2^-8), plus the fp32 arithmetic before the rounding: the norm is a few
roundings and a reciprocal square root (2 ulp), under 2^-20 relative; a
rotated value is a sum of two products, under 2^-22 (|x| + |y|).  The latent
row's values are rounded once from 46 bits: equal to the oracle's, and so are
the codes."""
import numpy as np
import pytest
import torch

import mla_inputs as mi
from oracle import fp4_kv_oracle as f4
from oracle import fp8_kv_oracle as f8
from oracle import norm_rope_oracle as nro
from oracle import sparse_mla_oracle as orc
from tests.parity import GRAD_ATOL_RMS, GRAD_RTOL, grad_term_bounds, record

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 1e-6
WIDTH = {"bf16": 576, "fp8": 656, "fp4": 416}


@pytest.fixture(scope="module")
def smla(cuda_lib):
    import serving_sparse_mla_gb300 as pkg
    pkg.clear_device_error()
    yield pkg
    assert pkg.get_device_error() == 0


def _f64(t):
    return t.double().cpu().numpy()


def _pair_size(r, interleaved):
    a, b = nro.planes(interleaved)
    out = np.empty_like(r)
    out[..., a] = out[..., b] = np.abs(r[..., a]) + np.abs(r[..., b])
    return out


def _check_rows(got, x, cs, w, interleaved, what):
    ref = nro.norm_rope(x, cs, w, EPS, interleaved)
    tol = (2.0 ** -8 + 2.0 ** -20) * np.abs(ref) + 1e-38
    tol[..., 512:] += 2.0 ** -22 * _pair_size(x[..., 512:], interleaved)
    bad = np.abs(_f64(got) - ref) > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} values off"


def _cache(form, blocks, page, fill):
    if form == "bf16":
        return torch.full((blocks, page, 576), float(fill), dtype=torch.bfloat16, device=DEV)
    return torch.full((blocks, page, WIDTH[form]), fill, dtype=torch.uint8, device=DEV)


def _slot_bytes(cache):
    c = cache.cpu()
    return c.view(-1, c.shape[-1]).contiguous().view(torch.uint8).numpy().reshape(-1, c.shape[-1] * c.element_size())


def _want_latent(y, form, kv_scale):
    """What the slot stands for, and its bytes before the rope values."""
    y = nro.round_bf16(y)
    if form == "bf16":
        return y, torch.from_numpy(y).bfloat16().view(torch.uint8).numpy().reshape(len(y), 1024)
    if form == "fp8":
        code, scale, val = nro.quantize_fp8(y)
        return val, np.concatenate([code, scale.astype("<f4").view(np.uint8).reshape(len(y), 16)], 1)
    code, scale, val = nro.quantize_fp4(y, kv_scale)
    return val, np.concatenate([code, scale], 1)


def _run_and_check(smla, seed, n, h, form, interleaved, q_norm, kv_norm, pad=0, kv_scale=1.0, page=16, n_pos=300):
    q, kv, qw, kw = mi.norm_rows(seed, n, h)
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, n_pos, (n,), generator=g).int()
    blocks = n // page + 2
    slots = torch.randperm(blocks * page, generator=g)[:n].int()
    if pad:
        pos[n - pad:] = torch.tensor([-1, n_pos, 2 ** 31 - 1, -2 ** 31]).repeat(pad)[:pad].int()
        slots[0] = -1                        # a token without a slot
        slots[1] = blocks * page             # and one past the cache
    cs = mi.rope_table(n_pos)
    cache = _cache(form, blocks, page, 7)
    before = _slot_bytes(cache).copy()
    qo = torch.full((n, h, 576), 3.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((n, 576), 3.0, dtype=torch.bfloat16, device=DEV)
    w = dict(q_weight=qw.to(DEV) if q_norm else None, kv_weight=kw.to(DEV) if kv_norm else None)
    r = smla.mla_norm_rope(q.to(DEV), kv.to(DEV), pos.to(DEV), cs.to(DEV), eps=EPS, interleaved=interleaved,
                           kv_cache=cache, slots=slots.to(DEV), kv_scale=kv_scale, q_out=qo, kv_out=ko, **w)
    torch.cuda.synchronize()
    assert r[0] is qo and r[1] is ko
    live = ((pos >= 0) & (pos < n_pos)).numpy()
    ang = cs.double().numpy()[np.where(live, pos.numpy(), 0)]
    what = f"{form} n={n} h={h}"
    _check_rows(qo[live], _f64(q)[live], ang[live][:, None], _f64(qw) if q_norm else None, interleaved, what + " q")
    assert bool((qo[~torch.from_numpy(live)] == 3).all()) and bool((ko[~torch.from_numpy(live)] == 3).all())
    y = nro.rms_norm(_f64(kv)[live][:, :512], _f64(kw) if kv_norm else None, EPS)
    val, lat = _want_latent(y, form, kv_scale)
    val = torch.from_numpy(val).to(torch.float32).bfloat16().double().numpy()
    got = _f64(ko[live])
    assert np.array_equal(got[:, :512], val), f"{what}: {(got[:, :512] != val).sum()} latent values differ"
    _check_rows(ko[live], np.concatenate([val, _f64(kv)[live][:, 512:]], 1), ang[live], None, interleaved, what + " kv")
    # the cache: the slots of the live tokens hold those bytes, all others are as they were
    want = before
    rope = ko[live][:, 512:].contiguous().cpu().view(torch.uint8).numpy().reshape(-1, 128)
    keep = (slots >= 0).numpy() & (slots < blocks * page).numpy() & live
    want[slots.numpy()[keep]] = np.concatenate([lat, rope], 1)[keep[live]]
    assert np.array_equal(_slot_bytes(cache), want), f"{what}: cache bytes"


@pytest.mark.parametrize("form", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,h,pad", [(1, 1, 0), (5, 3, 1), (37, 8, 4), (130, 20, 3)])
def test_forward(smla, form, interleaved, n, h, pad):
    _run_and_check(smla, 10 * n + h, n, h, form, interleaved, q_norm=h != 3, kv_norm=True, pad=pad)


@pytest.mark.parametrize("form,ks", [("fp4", 0.5), ("fp4", 2.0 ** -6), ("fp4", 64.0), ("fp8", 1.0), ("bf16", 1.0)])
def test_forward_without_the_latent_norm_and_cache_factors(smla, form, ks):
    _run_and_check(smla, 77, 64, 2, form, True, q_norm=False, kv_norm=False, pad=2, kv_scale=ks, page=64)


def test_forward_many_rows(smla):
    """More rows than the grid takes at once."""
    _run_and_check(smla, 5, 3001, 33, "fp4", True, q_norm=True, kv_norm=True, pad=2)


def test_strided_rows_and_no_cache(smla):
    """Rows inside wider projections; without a cache kv_out is the bf16 row."""
    n, h = 19, 5
    q, kv, qw, kw = mi.norm_rows(3, n, h)
    wide_q = torch.zeros(n, h + 2, 648, dtype=torch.bfloat16, device=DEV)
    wide_q[:, 1:-1, 8:584] = q.to(DEV)
    wide_kv = torch.zeros(n, 2120, dtype=torch.bfloat16, device=DEV)
    wide_kv[:, 1536:2112] = kv.to(DEV)
    pos, cs = torch.arange(n, dtype=torch.int32, device=DEV), mi.rope_table(n).to(DEV)
    w = dict(q_weight=qw.to(DEV), kv_weight=kw.to(DEV), interleaved=False)
    a = smla.mla_norm_rope(q.to(DEV), kv.to(DEV), pos, cs, **w)
    s = smla.mla_norm_rope(wide_q[:, 1:-1, 8:584], wide_kv[:, 1536:2112], pos, cs, **w)
    assert torch.equal(a[0], s[0]) and torch.equal(a[1], s[1])
    y = nro.round_bf16(nro.rms_norm(_f64(kv)[:, :512], _f64(kw), EPS))
    assert np.array_equal(_f64(a[1])[:, :512], y)
    # in place
    qd, kd = q.to(DEV), kv.to(DEV)
    smla.mla_norm_rope(qd, kd, pos, cs, q_out=qd, kv_out=kd, **w)
    assert torch.equal(qd, a[0]) and torch.equal(kd, a[1])
    # the gradients take the same strides
    dq, dkv = torch.randn(n, h, 576, device=DEV), torch.randn(n, 576, device=DEV)
    ga = smla.mla_norm_rope_bwd(q.to(DEV), kv.to(DEV), pos, cs, dq, dkv, **w)
    gs = smla.mla_norm_rope_bwd(wide_q[:, 1:-1, 8:584], wide_kv[:, 1536:2112], pos, cs, dq, dkv, **w)
    assert all(torch.equal(x, y) for x, y in zip(ga, gs))


@pytest.mark.parametrize("form", ["bf16", "fp8", "fp4"])
def test_rows_of_zeros_extremes_and_non_finite_values(smla, form):
    """Zero rows, values whose scales meet their limits (no norm), a NaN and an
    infinity: their tile or group reads as NaN, every other as it would."""
    n = 9
    _, kv, _, kw = mi.norm_rows(8, n, 1)
    kv[0, :] = 0
    kv[1] *= 2.0 ** -60
    kv[2] *= 2.0 ** 40
    kv[3, 300] = float("nan")
    kv[4, 17] = float("inf")
    kv[5] = 448.0
    kv[6, :512] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 64)
    kv[7] *= 2.0 ** -110
    kv[8, :512] = -0.0
    pos, cs = torch.arange(n, dtype=torch.int32, device=DEV), mi.rope_table(n).to(DEV)
    cache = _cache(form, 1, 16, 0)
    q = kv.view(n, 1, 576).to(DEV)
    _, ko = smla.mla_norm_rope(q, kv.to(DEV), pos, cs, kv_cache=cache, slots=pos)
    y = _f64(kv)[:, :512]
    val, lat = _want_latent(y, form, 1.0)
    if form == "bf16":
        val = y
    with np.errstate(over="ignore"):
        val = torch.from_numpy(val).to(torch.float32).bfloat16().double().numpy()
    assert np.array_equal(_f64(ko)[:, :512], val, equal_nan=True)
    read = {"bf16": lambda c: _f64(c), "fp8": f8.dequantize_slots, "fp4": f4.dequantize_slots}[form](cache.cpu())
    read = np.asarray(read).reshape(16, 576)[:n, :512]
    assert np.array_equal(torch.from_numpy(read).float().bfloat16().double().numpy(), val, equal_nan=True)
    # normed: a row of zeros stays zero
    _, ko = smla.mla_norm_rope(q, kv.to(DEV), pos, cs, kv_weight=kw.to(DEV), kv_cache=cache, slots=pos)
    assert bool((ko[0] == 0).all()) and bool((ko[8, :512] == 0).all())
    assert bool(torch.isfinite(ko[[1, 2, 5, 6]]).all())


@pytest.mark.parametrize("ks", [2.0 ** -64, 2.0 ** -20, 2.0 ** 20, 2.0 ** 64])
def test_values_far_past_the_largest_scale(smla, ks):
    """Groups whose values pass 448 * 6 factors many times over keep code 6 and
    their signs; factors at the ends of their range."""
    n = 6
    _, kv, _, _ = mi.norm_rows(18, n, 1)
    size = torch.tensor([2.0 ** 120, 2.0 ** 60, 1.0, 2.0 ** -60, ks, ks * 2.0 ** 12], dtype=torch.float64)
    kv[:, :512] = (kv[:, :512].double() * size[:, None]).bfloat16()
    kv[0, :16] = 2.0 ** -70
    kv[0, 3] = -2.0 ** 127
    pos, cs = torch.arange(n, dtype=torch.int32, device=DEV), mi.rope_table(n).to(DEV)
    cache = _cache("fp4", 1, 16, 0)
    q = kv.view(n, 1, 576).to(DEV)
    _, ko = smla.mla_norm_rope(q, kv.to(DEV), pos, cs, kv_cache=cache, slots=pos, kv_scale=ks)
    val, lat = _want_latent(_f64(kv)[:, :512], "fp4", ks)
    assert np.array_equal(_slot_bytes(cache)[:n, :288], lat)
    assert np.array_equal(_f64(ko)[:, :512], torch.from_numpy(val).to(torch.float32).bfloat16().double().numpy())


def _bwd_reference(q, kv, qw, kw, ang, live, dq, dkv, il):
    rq, rwq = nro.norm_rope_bwd(q, dq * live[:, None, None], ang[:, None], qw, EPS, il)
    rk, rwk = nro.norm_rope_bwd(kv, dkv * live[:, None], ang, kw, EPS, il)
    return rq, rk, rwq, rwk


def _row_size(x, dy, w, il):
    """Size of the terms of a row's gradient: what fp32 rounding scales with."""
    a, g = x[..., :512], np.abs(dy[..., :512])
    out = np.empty_like(x)
    if w is None:
        out[..., :512] = 0
    else:
        r = 1 / np.sqrt((a * a).mean(-1, keepdims=True) + EPS)
        xh = np.abs(a) * r
        g = g * np.abs(w)
        out[..., :512] = r * (g + xh * (g * xh).mean(-1, keepdims=True))
    out[..., 512:] = _pair_size(dy[..., 512:], il)
    return out


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,h,norms,pad", [(1, 1, "qk", 0), (3, 5, "k", 1), (40, 8, "qk", 3), (40, 8, "q", 0),
                                          (33, 2, "", 2), (257, 20, "qk", 9)])
def test_backward(smla, interleaved, n, h, norms, pad):
    """dx in bf16: half a step, and the fp32 terms' rounding (under 2^-18 of
    their size: sums of 512 products taken as 16 in a lane and 5 levels).  dw: a
    sum of rows, the error of each term under 2^-20, of the partial sums under
    (rows / warps + 20) 2^-24."""
    q, kv, qw, kw = mi.norm_rows(n + h, n, h)
    g = torch.Generator().manual_seed(n)
    pos = torch.randint(0, 500, (n,), generator=g).int()
    if pad:
        pos[n - pad:] = -1
    cs = mi.rope_table(500)
    dq, dkv = torch.randn(n, h, 576, generator=g) * 0.1, torch.randn(n, 576, generator=g)
    w = dict(q_weight=qw if "q" in norms else None, kv_weight=kw if "k" in norms else None)
    dev = {k: None if t is None else t.to(DEV) for k, t in w.items()}
    args = [t.to(DEV) for t in (q, kv, pos, cs, dq, dkv)]
    got = smla.mla_norm_rope_bwd(*args, eps=EPS, interleaved=interleaved, **dev)
    again = smla.mla_norm_rope_bwd(*args, eps=EPS, interleaved=interleaved, **dev)
    for x, y in zip(got, again):
        assert (x is None and y is None) or torch.equal(x, y)
    live = (pos >= 0).double().numpy()
    ang = cs.double().numpy()[pos.clamp(min=0).numpy()]
    w64 = {k: None if t is None else _f64(t) for k, t in w.items()}
    ref = _bwd_reference(_f64(q), _f64(kv), w64["q_weight"], w64["kv_weight"], ang, live, _f64(dq), _f64(dkv),
                         interleaved)
    size = (_row_size(_f64(q), _f64(dq), w64["q_weight"], interleaved),
            _row_size(_f64(kv), _f64(dkv), w64["kv_weight"], interleaved))
    for k, name in ((0, "dq_in"), (1, "dkv_in")):
        bad = np.abs(_f64(got[k]) - ref[k]) > 2.0 ** -8 * np.abs(ref[k]) + 2.0 ** -18 * size[k]
        assert not bad.any(), f"{name}: {int(bad.sum())} values off"
        assert np.all(_f64(got[k])[live == 0] == 0)
    for k, x, dy, wt in ((2, q, dq, w64["q_weight"]), (3, kv, dkv, w64["kv_weight"])):
        if wt is None:
            assert got[k] is None
            continue
        a = _f64(x)[..., :512]
        xh = np.abs(a) / np.sqrt((a * a).mean(-1, keepdims=True) + EPS)
        lv = live.reshape((n,) + (1,) * (a.ndim - 1))
        terms = (np.abs(_f64(dy)[..., :512]) * xh * lv).reshape(-1, 512).sum(0)
        assert np.all(np.abs(_f64(got[k]) - ref[k]) <= 2.0 ** -18 * terms), ("dq_weight", "dkv_weight")[k - 2]


def test_empty_batch(smla):
    q, kv, qw, kw = (t.to(DEV) for t in mi.norm_rows(1, 4, 2))
    pos, cs = torch.zeros(0, dtype=torch.int32, device=DEV), mi.rope_table(4).to(DEV)
    a, b = smla.mla_norm_rope(q[:0], kv[:0], pos, cs, qw, kw)
    assert a.shape == (0, 2, 576) and b.shape == (0, 576)
    dw = torch.ones(512, device=DEV)
    r = smla.mla_norm_rope_bwd(q[:0], kv[:0], pos, cs, q[:0].float(), kv[:0].float(), qw, kw, dkv_weight=dw)
    assert bool((r[2] == 0).all()) and r[3] is dw and bool((dw == 0).all())
    # a table without positions: every token is padding
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    out = torch.ones_like(q)
    smla.mla_norm_rope(q, kv, pos, cs[:0], qw, kw, q_out=out)
    assert bool((out == 1).all())


def test_slots_past_four_gigabytes(smla):
    """The last slot of a cache whose byte offsets pass 32 bits."""
    page, blocks = 64, 2 ** 32 // (64 * 416) + 40
    cache = torch.zeros(blocks, page, 416, dtype=torch.uint8, device=DEV)
    q, kv, _, kw = (t.to(DEV) for t in mi.norm_rows(2, 2, 1))
    last = blocks * page - 1
    pos = torch.tensor([3, 4], dtype=torch.int32, device=DEV)
    slots = torch.tensor([last, 0], dtype=torch.int32, device=DEV)
    _, ko = smla.mla_norm_rope(q, kv, pos, mi.rope_table(8).to(DEV), kv_weight=kw, kv_cache=cache, slots=slots)
    rows = torch.stack([cache[-1, -1], cache[0, 0]]).cpu()
    assert np.array_equal(f4.dequantize_slots(rows), _f64(ko))
    # and the decode reads it there
    table = torch.tensor([[blocks - 1]], dtype=torch.int32, device=DEV)
    qd = torch.randn(1, 1, 8, 576, device=DEV).bfloat16()
    idx = torch.tensor([[[63, -1]]], dtype=torch.int32, device=DEV)
    o, _ = smla.sparse_mla_decode_fp4(qd, cache, table, torch.tensor([64], dtype=torch.int32, device=DEV), idx, 0.04)
    assert torch.equal(o[0, 0, 0], ko[0, :512])


def test_captured_and_replayed_on_another_stream(smla):
    n, h = 50, 8
    q, kv, qw, kw = (t.to(DEV) for t in mi.norm_rows(21, n, h))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    cs = mi.rope_table(64).to(DEV)
    cache = _cache("fp4", 2, 64, 0)
    dq, dkv = torch.randn(n, h, 576, device=DEV), torch.randn(n, 576, device=DEV)

    def step():
        a = smla.mla_norm_rope(q, kv, pos, cs, qw, kw, kv_cache=cache, slots=pos)
        return a + smla.mla_norm_rope_bwd(q, kv, pos, cs, dq, dkv, qw, kw)

    want = [t.clone() for t in step()] + [cache.clone()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for _ in range(2):
        cache.zero_()
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got + (cache,), want))


def test_serving_chain(smla):
    """Prefill and one decode step as an engine runs them: rows normed, rotated
    and written to a 4-bit cache, then attention over that cache through its
    block table, against the oracle over the rows that kv_out says are held."""
    n, h, page, topk = 150, 8, 16, 96
    q, kv, qw, kw = (t.to(DEV) for t in mi.norm_rows(31, n, h))
    blocks = 14
    table = torch.randperm(blocks, generator=torch.Generator().manual_seed(1))[:10].int().view(1, 10)
    pos = torch.arange(n, dtype=torch.int32)
    slots = table[0][(pos // page).long()] * page + pos % page
    cache = _cache("fp4", blocks, page, 0x7F)     # NaN scales wherever nothing is written
    cs = mi.rope_table(n)
    qo, ko = smla.mla_norm_rope(q, kv, pos.to(DEV), cs.to(DEV), qw, kw, kv_cache=cache, slots=slots.to(DEV))
    lists = mi.prefill_indices(4, n, n, topk)
    sn = 3
    idx = lists[n - sn:].view(1, sn, topk)
    o, l = smla.sparse_mla_decode_fp4(qo[n - sn:].view(1, sn, h, 576), cache, table.to(DEV),
                                      torch.tensor([n], dtype=torch.int32, device=DEV), idx.to(DEV), 576 ** -0.5)
    ro, rl = orc.sparse_mla_fwd(qo[n - sn:].cpu(), ko.cpu(), lists[n - sn:], 576 ** -0.5)
    assert np.all(np.abs(_f64(o[0]) - ro) <= 2.0 ** -8 * np.abs(ro) + 2e-3)
    assert np.all(np.abs(_f64(l[0]) - rl) <= 1e-4)


def test_training_chain(smla):
    """Norm and rotation, sparse attention, its backward, and back through the
    rotation and the norm: the gradients of the inputs against the float64
    chain, within the attention backward's own bounds taken through the
    absolute values of the norm's Jacobian."""
    n, h, topk = 40, 8, 24
    q, kv, qw, kw = mi.norm_rows(41, n, h)
    cs, pos = mi.rope_table(n), torch.arange(n, dtype=torch.int32)
    idx = mi.prefill_indices(6, n, n, topk)
    sc = 576 ** -0.5
    d = lambda t: t.to(DEV)  # noqa: E731
    qo, ko = smla.mla_norm_rope(d(q), d(kv), d(pos), d(cs), d(qw), d(kw))
    out, lse = smla.sparse_mla_fwd(qo, ko, d(idx), sc)
    dout = torch.randn(n, h, 512, generator=torch.Generator().manual_seed(2)).bfloat16()
    dq, dkv = smla.sparse_mla_bwd(qo, ko, d(idx), sc, out, lse, d(dout))
    got = smla.mla_norm_rope_bwd(d(q), d(kv), d(pos), d(cs), dq, dkv, d(qw), d(kw))
    qf, kf = qo.cpu(), ko.cpu()
    rdq, rdkv = orc.sparse_mla_bwd(qf, kf, idx, sc, dout)
    # the forward output that the backward took, token by token: its actual error
    given = iter(_f64(out))
    bq, bkv = grad_term_bounds(qf, kf, idx, sc, dout, lambda O: np.abs(next(given) - O))
    # what sparse_mla_bwd is held to besides (tests/parity.py, compare_grad): the term bounds leave out the fp32
    # rounding of P, dP and D, which is all that is left where dP - D cancels (a token with one key: dS = 0)
    bq, bkv = (b + GRAD_ATOL_RMS * np.sqrt((r * r).mean()) + GRAD_RTOL * np.abs(r) for b, r in ((bq, rdq), (bkv, rdkv)))
    ang = cs.double().numpy()
    for k, x, w, r, bd, a in ((0, q, qw, rdq, bq, ang[:, None]), (1, kv, kw, rdkv, bkv, ang)):
        x, w = _f64(x), _f64(w)
        ref, dw = nro.norm_rope_bwd(x, r, a, w, EPS, True)
        spread = _row_size(x, bd, w, True)
        tol = 2.0 ** -8 * np.abs(ref) + spread + 2.0 ** -18 * _row_size(x, r, w, True)
        bad = np.abs(_f64(got[k]) - ref) > tol
        assert not bad.any(), f"{int(bad.sum())} gradients off"
        # the bound says something: it is well under the gradients' own size
        assert np.median(tol) < 0.5 * np.sqrt((ref ** 2).mean())
        xh = np.abs(x[..., :512]) / np.sqrt((x[..., :512] ** 2).mean(-1, keepdims=True) + EPS)
        tw = ((bd[..., :512] + 2.0 ** -18 * np.abs(r[..., :512])) * xh).reshape(-1, 512).sum(0)
        assert np.all(np.abs(_f64(got[2 + k]) - dw) <= tw)
        record(f"training chain {'q' if k == 0 else 'kv'}", max_d=float(np.abs(_f64(got[k]) - ref).max()))

"""dense_mha_fwd and dense_mha_bwd against the float64 oracle.

Tolerances.  A bf16 output is within half a step, 2^-8, of its exact value.
The weights P (and dS) are rounded to bf16 for the tensor cores, 2^-8 of each,
so an output is off by at most 2^-8 of the sum of its terms' magnitudes more.
Sums of up to 192 products in fp32, in any order and with truncating adders,
are within 2^-16 of their terms' magnitudes; a score off by e moves its weight
by e of itself and, through the sum, all others: 2 e.  Beside this bound on
each value, the 2-norm of the error is held to 2^-8 of the result's: either
rounding is spread over its step (2^-8 / sqrt(3) of a value at most, in the
mean square), and the rows' terms are independent in sign."""
import math

import pytest
import torch

from oracle import dense_mha_oracle as dmo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U, S = 2.0 ** -8, 2.0 ** -16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def smla(cuda_lib):
    import serving_sparse_mla_gb300 as pkg
    pkg.clear_device_error()
    yield pkg
    assert pkg.get_device_error() == 0


def _offsets(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)


def _inputs(seed, lq, lk, h, hk, d, tail=0, size=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    nq, nk = sum(lq) + tail, sum(lk) + tail
    q, k = (randn(nq, h, d) * size).bfloat16(), (randn(nk, hk, d) * torch.exp(0.3 * randn(d))).bfloat16()
    v, do = randn(nk, hk, 128).bfloat16(), (randn(nq, h, 128) * 0.1).bfloat16()
    if tail:
        for t in (q[-tail:], k[-tail:], v[-tail:], do[-tail:]):
            t.fill_(NAN)
    return q, k, v, do, _offsets(lq), _offsets(lk)


def _near(got, ref, bound, what, rel=U):
    got = got.double()
    off = (got - ref).abs()
    bad = ~(off <= bound + 1e-30)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values off, by up to {off[bad].max():.3e} " \
                          f"({(off / bound)[bad].max():.1f} times the bound); first at {bad.nonzero()[0].tolist()}"
    if ref.norm() > 0:
        assert (got - ref).norm() <= rel * ref.norm(), f"{what}: 2-norm off by {(got - ref).norm() / ref.norm():.2e}"


def _check_fwd(out, lse, q, k, v, scale, cq=None, ck=None, what=""):
    ro, rl, size, terms = dmo.fwd(q, k, v, scale, cq, ck)
    none = rl == -math.inf
    assert torch.equal(lse == -math.inf, none), what + " rows without keys"
    assert (out[none] == 0).all()
    _near(out, ro, U * ro.abs() + (U + 2 * S * (terms + 1))[..., None] * size, what + " out")
    _near(lse[~none], rl[~none], (S * (terms + 1))[~none] + 2.0 ** -22 * rl[~none].abs(), what + " lse", rel=1.0)


def _check_bwd(grads, q, k, v, scale, out, lse, do, cq=None, ck=None, what=""):
    clean = [torch.nan_to_num(t) for t in (q, k, v, out, lse, do)]
    clean[4] = torch.where(lse == -math.inf, lse, clean[4])
    ref, bounds = dmo.bwd(*clean[:3], scale, *clean[3:], cq, ck, U, S)
    for g, r, e, n in zip(grads, ref, bounds, ("dq", "dk", "dv")):
        _near(g, r, e, f"{what} {n}", rel=1.5 * U)


def _run(smla, seed, lq, lk, h, hk, d, tail=0, size=1.0, dense=False):
    q, k, v, do, cq, ck = _inputs(seed, lq, lk, h, hk, d, tail, size)
    scale = d ** -0.5
    seqs = () if dense else (cq, ck)
    out, lse = smla.dense_mha_fwd(q, k, v, scale, *seqs)
    _check_fwd(out, lse, q, k, v, scale, *seqs)
    if tail:
        assert (out[-tail:] == 0).all() and (lse[-tail:] == -INF).all()
    grads = smla.dense_mha_bwd(q, k, v, scale, out, lse, do, *seqs)
    _check_bwd(grads, q, k, v, scale, out, lse, do, *seqs)
    if tail:
        assert all((g[-tail:] == 0).all() for g in grads)
    for a, b in zip((out, lse) + grads, smla.dense_mha_fwd(q, k, v, scale, *seqs) +
                    smla.dense_mha_bwd(q, k, v, scale, out, lse, do, *seqs)):
        assert torch.equal(a, b)   # the same call gives the same bits


@pytest.mark.parametrize("d", [192, 128])
@pytest.mark.parametrize("n", [1, 2, 16, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 640, 1025])
def test_one_sequence(smla, n, d):
    _run(smla, n, [n], [n], 2, 2, d, dense=True)


@pytest.mark.parametrize("d", [192, 128])
@pytest.mark.parametrize("h,hk", [(1, 1), (8, 8), (8, 1), (6, 2), (12, 4), (5, 1), (14, 2), (9, 1), (11, 1), (48, 2), (40, 1),
                                  (130, 1), (128, 1), (64, 4)])
def test_groups_of_heads(smla, h, hk, d):
    _run(smla, h, [37, 150, 5], [37, 150, 9], h, hk, d)


PACKED = [([1], [500]), ([1, 1, 1, 1], [3, 700, 129, 128]), ([3, 5], [1000, 2]), ([100], [40]), ([300], [1]), ([64], [0]),
          ([0, 70, 0, 0, 200, 1], [5, 70, 0, 9, 210, 1]), ([17] * 30, [17] * 30), ([129, 300, 7], [900, 300, 500]),
          ([2, 250], [2000, 128]), ([1] * 150, [20] * 150), ([0], [0]), ([0, 0], [4, 3])]


@pytest.mark.parametrize("d,h,hk", [(192, 4, 4), (128, 8, 2)])
@pytest.mark.parametrize("lq,lk", PACKED)
def test_packed(smla, lq, lk, d, h, hk):
    _run(smla, sum(lk), lq, lk, h, hk, d, tail=3)


@pytest.mark.parametrize("size", [0.0, 6.0, 60.0])
def test_even_and_single_key_rows(smla, size):
    """Scores all alike, and so far apart that one key has the row (sums far below the maximum's)."""
    _run(smla, 77, [300], [420], 3, 3, 192, size=size)


def test_rising_scores(smla):
    """Each key scores above all before it by far more than the softmax keeps: every block moves the maximum."""
    n, d = 700, 128
    q = torch.zeros(n, 1, d, device=DEV).bfloat16()
    k = torch.zeros(n, 1, d, device=DEV).bfloat16()
    q[..., 0] = 8.0
    k[:, 0, 0] = torch.arange(n, device=DEV).bfloat16()
    for sign in (1, -1):
        kk = k * sign
        v = _inputs(1, [n], [n], 1, 1, d)[2]
        out, lse = smla.dense_mha_fwd(q, kk, v, 0.5)
        ro, rl, sz, _ = dmo.fwd(q, kk, v, 0.5)   # products of few bits: the scores are exact
        _near(out, ro, U * ro.abs() + 2 * U * sz, "out")
        _near(lse, rl, 2.0 ** -20 * rl.abs() + 1e-6, "lse", rel=1.0)


@pytest.mark.parametrize("d", [192, 128])
def test_strided_rows(smla, d):
    """Heads before tokens; keys and values of one projection; a gradient in a wider tensor."""
    lq, lk, h, hk = [70, 130], [70, 200], 6, 3
    q, k, v, do, cq, ck = _inputs(3, lq, lk, h, hk, d)
    want = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
    grads = smla.dense_mha_bwd(q, k, v, 0.1, *want, do, cq, ck)
    q2 = q.transpose(0, 1).contiguous().transpose(0, 1)
    kv = torch.full((sum(lk), hk, d + 8 + 128), NAN, dtype=q.dtype, device=DEV)
    kv[..., :d], kv[..., d + 8:] = k, v
    wide = torch.full((sum(lq), h + 1, 256), NAN, dtype=q.dtype, device=DEV)
    wide[:, 1:, 64:192] = do
    got = smla.dense_mha_fwd(q2, kv[..., :d], kv[..., d + 8:], 0.1, cq, ck)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = smla.dense_mha_bwd(q2, kv[..., :d], kv[..., d + 8:], 0.1, *want, wide[:, 1:, 64:192], cq, ck)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))


def test_given_outputs_keep_the_rows_behind_the_last_sequence(smla):
    q, k, v, do, cq, ck = _inputs(4, [50, 90], [60, 90], 4, 2, 192, tail=37)
    out = torch.full((177, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((177, 4), 7.0, device=DEV)
    got = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    want = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
    assert torch.equal(out[:140], want[0][:140]) and (out[140:] == 7).all()
    assert torch.equal(lse[:140], want[1][:140]) and (lse[140:] == 7).all()
    o2, l2 = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck, out=out.fill_(7.0))
    assert (o2[140:] == 7).all() and (l2[140:] == -INF).all()
    grads = [torch.full(t.shape, 7.0, dtype=t.dtype, device=DEV) for t in (q, k, v)]
    back = smla.dense_mha_bwd(q, k, v, 0.1, *want, do, cq, ck, dq=grads[0], dk=grads[1], dv=grads[2])
    assert all(a is b for a, b in zip(back, grads))
    assert all((g[n:] == 0).all() for g, n in zip(back, (140, 150, 150)))


@pytest.mark.parametrize("what", [NAN, INF, -INF])
@pytest.mark.parametrize("at", [100, 127, 128, 300, 449])
def test_hidden_values_that_are_not_finite(smla, at, what):
    """A row that is not finite reaches no row that does not see it: the rows
    before it and the other sequences have the results of finite inputs."""
    lens = [80, 450, 130]
    q, k, v, do, cq, _ = _inputs(5, lens, lens, 4, 2, 192)
    want = smla.dense_mha_fwd(q, k, v, 0.1, cq, cq)
    grads = smla.dense_mha_bwd(q, k, v, 0.1, *want, do, cq, cq)
    k2, v2, q2, do2 = k.clone(), v.clone(), q.clone(), do.clone()
    for t in (k2, v2, q2, do2):
        t[80 + at, :, 5::60] = what
    sees = torch.zeros(660, dtype=torch.bool, device=DEV)
    sees[80 + at:530] = True
    got = smla.dense_mha_fwd(q, k2, v2, 0.1, cq, cq)
    assert torch.equal(got[0][~sees], want[0][~sees]) and torch.equal(got[1][~sees], want[1][~sees])
    only_v = smla.dense_mha_fwd(q, k, v2, 0.1, cq, cq)[0]
    assert torch.equal(only_v[~sees], want[0][~sees])
    cols = torch.zeros(128, dtype=torch.bool, device=DEV)
    cols[5::60] = True
    assert not only_v[sees][..., cols].isfinite().any()
    assert torch.equal(only_v[..., ~cols], want[0][..., ~cols])
    # keys and values: the gradients of the queries that do not see them
    dq, _, _ = smla.dense_mha_bwd(q, k2, v2, 0.1, *want, do, cq, cq)
    assert torch.equal(dq[~sees], grads[0][~sees])
    # a query's row: the gradients of the keys that it does not see
    _, dk, dv = smla.dense_mha_bwd(q2, k, v, 0.1, *want, do2, cq, cq)
    seen = torch.zeros(660, dtype=torch.bool, device=DEV)
    seen[80:80 + at + 1] = True
    assert torch.equal(dk[~seen], grads[1][~seen]) and torch.equal(dv[~seen], grads[2][~seen])
    assert not dk[seen].isfinite().any() and not dv[seen][..., cols].isfinite().any()


def test_no_rows_and_no_keys(smla):
    q, k, v, do, *_ = _inputs(6, [40], [50], 2, 2, 192)
    out, lse = smla.dense_mha_fwd(q, k[:0], v[:0], 0.1)
    assert (out == 0).all() and (lse == -INF).all()
    dq, dk, dv = smla.dense_mha_bwd(q, k[:0], v[:0], 0.1, out, lse, do)
    assert (dq == 0).all() and dk.shape == (0, 2, 192) and dv.shape == (0, 2, 128)
    out, lse = smla.dense_mha_fwd(q[:0], k, v, 0.1)
    assert out.shape == (0, 2, 128) and lse.shape == (0, 2)
    dq, dk, dv = smla.dense_mha_bwd(q[:0], k, v, 0.1, out, lse, do[:0])
    assert dq.shape == (0, 2, 192) and (dk == 0).all() and (dv == 0).all()


def test_offsets_outside_of_the_tensors_are_cut(smla):
    q, k, v, do, *_ = _inputs(7, [90], [90], 2, 1, 128)
    cq = torch.tensor([0, 60, 500, 10], dtype=torch.int32, device=DEV)
    ck = torch.tensor([-4, 60, 1000, 2000], dtype=torch.int32, device=DEV)
    out, lse = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
    good = _offsets([60, 30])
    want = smla.dense_mha_fwd(q, k, v, 0.1, good, good)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    smla.dense_mha_bwd(q, k, v, 0.1, out, lse, do, cq, ck)
    torch.cuda.synchronize()


def test_gradients_are_differences(smla):
    """The loss sum(out dout) along random directions of q, k and v, from the oracle's unrounded forward."""
    q, k, v, do, cq, ck = _inputs(8, [40, 150], [60, 150], 4, 2, 192)
    out, lse = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
    grads = smla.dense_mha_bwd(q, k, v, 0.1, out, lse, do, cq, ck)
    g = torch.Generator(device=DEV).manual_seed(9)
    f = lambda *x: (dmo.fwd(*x, 0.1, cq, ck)[0] * do.double()).sum()  # noqa: E731
    ins = [t.double() for t in (q, k, v)]
    for i in range(3):
        u = torch.randn(ins[i].shape, generator=g, device=DEV, dtype=torch.float64)
        moved = lambda e: [t + e * u if j == i else t for j, t in enumerate(ins)]  # noqa: E731
        diff = (f(*moved(1e-6)) - f(*moved(-1e-6))) / 2e-6
        got = grads[i].double()
        # each value is off by a few 2^-8 of itself, with signs of their own: 4 standard deviations
        assert (got * u).sum().sub(diff).abs() <= 4 * 2 * U * (got * u).norm() + 1e-6


def test_streams_and_graphs(smla):
    lq, lk = [130, 1, 60], [400, 1, 60]
    q, k, v, do, cq, ck = _inputs(10, lq, lk, 8, 2, 192)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck, stream=side)
    a += smla.dense_mha_bwd(q, k, v, 0.1, *a, do, cq, ck, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
    b += smla.dense_mha_bwd(q, k, v, 0.1, *b, do, cq, ck)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
        c += smla.dense_mha_bwd(q, k, v, 0.1, *c, do, cq, ck)
    # other values and other lengths of the same sums
    q2, k2, v2, do2, cq2, ck2 = _inputs(11, [60, 61, 70], [60, 1, 400], 8, 2, 192)
    for x, y in zip((q, k, v, do, cq, ck), (q2, k2, v2, do2, cq2, ck2)):
        x.copy_(y)
    graph.replay()
    d = smla.dense_mha_fwd(q2, k2, v2, 0.1, cq2, ck2)
    d += smla.dense_mha_bwd(q2, k2, v2, 0.1, *d, do2, cq2, ck2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(c, d))


def test_agrees_with_the_absorbed_form(smla):
    """Keys and values up-projected from latent rows, against sparse_mla_fwd_causal over the rows themselves:
    one head's query is its latent part times the up-projection, the other part as it is."""
    n, h = 200, 4
    g = torch.Generator(device=DEV).manual_seed(12)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    lat = randn(n, 576).bfloat16()
    uk, uv = randn(h, 128, 512) / 22, randn(h, 128, 512) / 22
    q = randn(n, h, 192).bfloat16()
    k = torch.cat([torch.einsum("nl,hdl->nhd", lat[:, :512].float(), uk), lat[:, None, 512:].float().expand(n, h, 64)], 2)
    v = torch.einsum("nl,hdl->nhd", lat[:, :512].float(), uv)
    out, lse = smla.dense_mha_fwd(q, k.bfloat16(), v.bfloat16(), 0.07)
    qa = torch.cat([torch.einsum("nhd,hdl->nhl", q[..., :128].float(), uk), q[..., 128:].float()], 2).bfloat16()
    oa, la = smla.sparse_mla_fwd_causal(qa, lat, 0.07)
    want = torch.einsum("nhl,hdl->nhd", oa.float(), uv)
    # either side rounds its operands to bf16: a few 2^-9 of scores of size 2 and of values of size 1
    assert (lse - la).abs().max() < 0.1 and (out.float() - want).norm() < 0.02 * want.norm()


def test_keys_past_32_bit_offsets(smla):
    """A key tensor of more than 2^31 elements; a sequence at its end."""
    n, hk = (1 << 31) // (64 * 192) + 300, 64
    q, k, v, do, cq, _ = _inputs(13, [150], [150], hk, hk, 192)
    kl = torch.zeros(n, hk, 192, dtype=torch.bfloat16, device=DEV)
    vl = torch.zeros(n, hk, 128, dtype=torch.bfloat16, device=DEV)
    kl[-150:], vl[-150:] = k, v
    ck = torch.tensor([0, n - 150, n], dtype=torch.int32, device=DEV)
    cq = torch.tensor([0, 0, 150], dtype=torch.int32, device=DEV)
    out, lse = smla.dense_mha_fwd(q, kl, vl, 0.1, cq, ck)
    want = smla.dense_mha_fwd(q, k, v, 0.1)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    dq, dk, dv = smla.dense_mha_bwd(q, kl, vl, 0.1, out, lse, do, cq, ck)
    for a, b in zip((dq, dk[-150:], dv[-150:]), smla.dense_mha_bwd(q, k, v, 0.1, *want, do)):
        assert torch.equal(a, b)
    assert (dk[:-150] == 0).all() and (dv[:-150] == 0).all()


def test_a_layer(smla):
    """The run of them: a norm with 8-bit rows, its projections, attention, the next norm, and back."""
    lens, h, d = [100, 37, 260], 4, 512
    n = sum(lens)
    cu = _offsets(lens)
    g = torch.Generator(device=DEV).manual_seed(14)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x, res = randn(n, d).bfloat16(), randn(n, d).bfloat16()
    w1, w2 = (1 + 0.1 * randn(d)).bfloat16(), (1 + 0.1 * randn(h * 128)).bfloat16()
    wq, wk, wv = (randn(d, h * m) / d ** 0.5 for m in (192, 192, 128))
    codes, scales, z = smla.mla_add_norm(x, w1, res, group=128)
    rows = (codes.float().view(n, -1, 128) * scales[..., None]).view(n, d)
    q, k, v = ((rows @ m).bfloat16().view(n, h, -1) for m in (wq, wk, wv))
    out, lse = smla.dense_mha_fwd(q, k, v, 192 ** -0.5, cu, cu)
    y, _, z2 = smla.mla_add_norm(out.view(n, -1), w2, z)
    dy, dz = randn(n, h * 128).bfloat16(), randn(n, h * 128).bfloat16()
    dz2, dw2 = smla.mla_add_norm_bwd(z2, w2, dy, dz)
    grads = smla.dense_mha_bwd(q, k, v, 192 ** -0.5, out, lse, dz2.view(n, h, 128), cu, cu)
    drows = sum(a.float().reshape(n, -1) @ m.T for a, m in zip(grads, (wq, wk, wv)))
    dx, dw1 = smla.mla_add_norm_bwd(z, w1, drows.bfloat16(), dz2)

    # the same in 64 bits, rounding passed through
    t = [a.double().requires_grad_() for a in (x, res, w1, w2)]
    zz = t[0] + t[1]
    nrm = lambda a, b: a * torch.rsqrt((a * a).mean(-1, keepdim=True) + 1e-6) * b  # noqa: E731
    r = nrm(zz, t[2])
    qq, kk, vv = ((r @ m.double()).view(n, h, -1) for m in (wq, wk, wv))
    parts = []
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        s = torch.einsum("ihd,jhd->hij", qq[a:b], kk[a:b]) * 192 ** -0.5
        s = s.masked_fill(torch.ones(b - a, b - a, device=DEV).triu(1).bool(), -INF)
        parts.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), vv[a:b]))
    zz2 = torch.cat(parts).reshape(n, -1) + zz
    ((nrm(zz2, t[3]) * dy.double()).sum() + (zz2 * dz.double()).sum()).backward()
    # e4m3 rows are off by up to 2^-4 of each value, 2^-4 / sqrt(3) / 2 in the mean; scores and values by as much
    assert (y.double() - nrm(zz2, t[3])).norm() < 0.04 * y.double().norm()
    for got, want in ((dx, t[0].grad), (dx, t[1].grad), (dw1, t[2].grad), (dw2, t[3].grad)):
        assert (got.double() - want).norm() < 0.08 * want.norm()


@pytest.mark.parametrize("d", [192, 128])
@pytest.mark.parametrize("lq,lk,h,hk", [([1], [5000], 8, 8), ([3], [4097], 2, 2), ([130], [4500], 2, 1), ([1], [9000], 1, 1),
                                        ([1, 2, 1, 1], [3000, 1, 130, 4000], 8, 2), ([257], [2200], 1, 1)])
def test_few_rows_of_long_sequences(smla, lq, lk, h, hk, d):
    """A tile's keys shared out over the CTAs of a cluster, down to CTAs with none."""
    _run(smla, sum(lk), lq, lk, h, hk, d, tail=2)


@pytest.mark.parametrize("what", [NAN, INF])
def test_few_rows_and_values_that_are_not_finite(smla, what):
    q, k, v, _, cq, ck = _inputs(15, [100], [3100], 2, 2, 128)
    want = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
    v[3060, :, 7] = what      # seen by the rows from 60 on
    v[5, 1, 9] = what         # by all
    out, lse = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
    assert torch.equal(lse, want[1])
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[60:, :, 7] = True
    bad[:, 1, 9] = True
    assert not out[bad].isfinite().any() and torch.equal(out[~bad], want[0][~bad])


@pytest.mark.parametrize("d,h,hk,lq,lk", [
    (192, 64, 64, [1100], [1100]), (128, 64, 8, [1300], [1300]), (192, 64, 8, [900, 1300, 600], [1000, 1300, 700]),
    (128, 160, 32, [513], [900]), (192, 96, 96, [700, 1025], [640, 1025]), (128, 128, 1, [700], [700])])
def test_many_tiles(smla, d, h, hk, lq, lk):
    """Two tiles to a CTA; rows that end in either, and before them."""
    _run(smla, h + lq[0], lq, lk, h, hk, d, tail=3)


@pytest.mark.parametrize("what", [NAN, INF])
@pytest.mark.parametrize("at", [300, 511, 512, 1000])
def test_many_tiles_and_hidden_values_that_are_not_finite(smla, at, what):
    n, h = 1050, 64
    q, k, v, *_ = _inputs(16, [n], [n], h, h, 128)
    want = smla.dense_mha_fwd(q, k, v, 0.1)
    v2, k2 = v.clone(), k.clone()
    v2[at, :, 5::60] = what
    k2[at, :, 3] = what
    out, lse = smla.dense_mha_fwd(q, k, v2, 0.1)
    cols = torch.zeros(128, dtype=torch.bool, device=DEV)
    cols[5::60] = True
    assert torch.equal(lse, want[1]) and torch.equal(out[:at], want[0][:at])
    assert torch.equal(out[..., ~cols], want[0][..., ~cols]) and not out[at:][..., cols].isfinite().any()
    out, lse = smla.dense_mha_fwd(q, k2, v2, 0.1)
    assert torch.equal(lse[:at], want[1][:at]) and torch.equal(out[:at], want[0][:at])


@pytest.mark.parametrize("d,h,hk", [(192, 2, 2), (128, 10, 2)])
@pytest.mark.parametrize("lq,lk", [([5, 700, 1], [9000, 700, 4500]), ([4400, 3, 70], [4400, 3, 4300]),
                                   ([30, 1, 2500] + [9] * 40, [30, 6000, 2500] + [11] * 40)])
def test_sequences_of_very_different_lengths(smla, lq, lk, d, h, hk):
    """Tiles of more blocks than a warp has lanes, and more sequences than that."""
    _run(smla, sum(lk), lq, lk, h, hk, d, tail=2)


def test_more_heads_than_run_side_by_side(smla):
    _run(smla, 24, [5200], [5200], 24, 24, 192, dense=True)


def test_two_calls_at_once(smla):
    sets = [_inputs(20 + i, lq, lk, 8, 2, 192) for i, (lq, lk) in
            enumerate((([700, 1, 333], [900, 1, 333]), ([64, 1000], [640, 1000])))]

    def both(q, k, v, do, cq, ck):
        a = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
        return a + smla.dense_mha_bwd(q, k, v, 0.1, *a, do, cq, ck)

    want = [both(*s) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(4):
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(both(*s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i % 2]))

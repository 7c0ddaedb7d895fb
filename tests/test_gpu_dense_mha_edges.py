"""dense_mha_fwd and dense_mha_bwd where their formulas have an edge: orders of a
CTA's stages, values that are not finite, rows that see one key, tiles that take
long, and sizes past what a product of two counters holds.  Helpers and the derivation of the
tolerances are test_gpu_dense_mha's."""
import pytest
import torch

from oracle import dense_mha_oracle as dmo
from tests.test_gpu_dense_mha import _check_bwd, _check_fwd, _inputs, smla  # noqa: F401  (the module's fixture)

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


NAN, INF = float("nan"), float("inf")


def _odd_sums(x):
    """The sums of what is not finite in rows 0 .. i of x (0: there is none), for each i."""
    some = lambda mask: mask.cumsum(0) > 0  # noqa: E731
    up, down, bad = some(x == INF), some(x == -INF), some(x.isnan())
    s = torch.zeros(x.shape, device=x.device)
    s[up], s[down] = INF, -INF
    s[bad | (up & down)] = NAN
    return s


@pytest.mark.parametrize("scores", ["far apart", "rising"])
@pytest.mark.parametrize("lq,lk,h,hk,d", [(300, 300, 2, 2, 192), (1, 5000, 8, 8, 192), (130, 4500, 2, 1, 128),
                                          (1050, 1100, 64, 64, 128), (900, 900, 128, 1, 192), (70, 40, 3, 1, 128)])
def test_a_seen_value_that_is_not_finite_counts_however_small_its_weight(smla, lq, lk, h, hk, d, scores):  # noqa: F811
    """Weights that underflow, in whole blocks, in blocks that some rows do not see all of, in parts of a cluster,
    and behind a maximum that has grown: a column is the sum of what is not finite in it."""
    q, k, v, *_ = _inputs(32, [lq], [lk], h, hk, d)
    q[..., 0], k[..., 0] = 8.0, 0.0
    a, b = 3, lk - 2
    if scores == "rising":
        k[..., 0] = (torch.arange(lk, device=k.device) * 0.5).bfloat16()[:, None]
    else:
        k[a, :, 0] = k[b, :, 0] = -400.0
    want = smla.dense_mha_fwd(q, k, v, 0.5)
    v2 = v.clone()
    v2[a, :, 7], v2[a, :, 9], v2[a, :, 11], v2[b, :, 11], v2[b, :, 13], v2[lk // 2, 0, 40:50] = INF, -INF, INF, -INF, NAN, INF
    out, lse = smla.dense_mha_fwd(q, k, v2, 0.5)
    assert torch.equal(lse, want[1])
    first = max(0, lq - lk)   # rows before it see nothing
    assert torch.equal(out[:first], want[0][:first])
    odd = _odd_sums(v2)[lk - lq + first:].repeat_interleave(h // hk, 1).float()
    ref = torch.where(odd == 0, want[0][first:].float(), odd)
    assert torch.equal(torch.nan_to_num(out[first:].float(), nan=12345.0), torch.nan_to_num(ref, nan=12345.0))


def test_a_row_whose_scores_are_not_finite_is_nan(smla):  # noqa: F811
    """Its weights are NaN: an infinity among its values changes nothing."""
    q, k, v, *_ = _inputs(33, [300], [300], 2, 2, 128)
    k[150, 0, 5] = NAN
    v[140, 0, 3], v[160, 0, 4] = INF, INF
    out, lse = smla.dense_mha_fwd(q, k, v, 0.1)
    assert out[150:, 0].isnan().all() and lse[150:, 0].isnan().all() and lse[:150].isfinite().all()
    assert (out[140:150, 0, 3] == INF).all() and out[:140].isfinite().all() and out[:, 1].isfinite().all()


def test_waits_that_run_out_are_reported_and_the_next_call_is_right(smla):  # noqa: F811
    """A 1 ns bound on a wait: the loading threads, whose waits for the stages before them are the longest, give up at
    once, and the other warps by the CTA's flag; the kernels record a code, wait for their copies and products, free
    TMEM and return."""
    for lq, lk, h, hk, d in (([1100, 2], [1100, 900], 64, 64, 128), ([4100], [4100], 16, 4, 192)):
        q, k, v, do, cq, ck = _inputs(34, lq, lk, h, hk, d)
        want = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
        grads = smla.dense_mha_bwd(q, k, v, 0.1, *want, do, cq, ck)
        torch.cuda.synchronize()
        codes = []
        for call in (lambda: smla.dense_mha_fwd(q, k, v, 0.1, cq, ck),
                     lambda: smla.dense_mha_bwd(q, k, v, 0.1, *want, do, cq, ck)):
            try:
                smla.set_wait_timeout_ns(1)
                call()
                torch.cuda.synchronize()
                codes.append(smla.get_device_error())
            finally:
                smla.set_wait_timeout_ns(0)
                smla.clear_device_error()
        assert 0x701 <= codes[0] <= 0x703 and 0x711 <= codes[1] <= 0x724, codes
        assert smla.get_device_error() == 0
        assert all(torch.equal(a, b) for a, b in zip(smla.dense_mha_fwd(q, k, v, 0.1, cq, ck), want))
        assert all(torch.equal(a, b) for a, b in zip(smla.dense_mha_bwd(q, k, v, 0.1, *want, do, cq, ck), grads))


@pytest.mark.parametrize("d", [192, 128])
def test_the_bound_is_a_waits_not_a_tiles(smla, d):  # noqa: F811
    """Tiles of 1 to 2 ms under a bound of 0.5: each has hundreds of waits of some microseconds."""
    n = 131072
    q, k, v, do, *_ = _inputs(35, [n], [n], 1, 1, d)
    want = smla.dense_mha_fwd(q, k, v, 0.1)
    grads = smla.dense_mha_bwd(q, k, v, 0.1, *want, do)
    torch.cuda.synchronize()
    try:
        smla.set_wait_timeout_ns(500000)
        got = smla.dense_mha_fwd(q, k, v, 0.1)
        got += smla.dense_mha_bwd(q, k, v, 0.1, *want, do)
        torch.cuda.synchronize()
        code = smla.get_device_error()
    finally:
        smla.set_wait_timeout_ns(0)
        smla.clear_device_error()
    assert code == 0 and all(torch.equal(a, b) for a, b in zip(got, want + grads))


@pytest.mark.parametrize("d", [192, 128])
@pytest.mark.parametrize("h,hk", [(2, 2), (64, 1), (128, 1), (48, 1), (5, 1), (6, 2)])
def test_rows_that_see_one_key_have_no_gradient_of_scores(smla, h, hk, d):  # noqa: F811
    """P is 1 and out is v there, so dS = dout v - dout out is 0, and with it dq and the row's part of dk."""
    # sequences of one token, of one key, of one query
    q, k, v, do, cq, ck = _inputs(36, [1, 1, 300, 1, 1, 0], [1, 1, 1, 1, 0, 3], h, hk, d)
    out, lse = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
    dq, dk, dv = smla.dense_mha_bwd(q, k, v, 0.1, out, lse, do, cq, ck)
    assert (dq == 0).all() and (dk == 0).all()
    # dv is the one row's dout, summed over the heads: dout is bf16, P within 2^-16 of 1 and rounded, 2^-8
    rows = [0, 1, 301, 302]
    want = do[rows].double().view(4, hk, h // hk, 128)
    assert ((dv[:4].double() - want.sum(2)).abs() <= 2.0 ** -7 * want.abs().sum(2)).all() and (dv[4:] == 0).all()
    # the first row of longer sequences, of all keys' tiles: other rows get no upstream gradient
    for lq, lk in (([300, 129, 40], [300, 129, 40]), ([300, 200], [150, 3])):
        q, k, v, do, cq, ck = _inputs(37, lq, lk, h, hk, d)
        first = [sum(lq[:i]) + lq[i] - lk[i] for i in range(len(lq))]
        only = torch.zeros_like(do)
        only[first] = do[first]
        out, lse = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
        dq, dk, dv = smla.dense_mha_bwd(q, k, v, 0.1, out, lse, only, cq, ck)
        assert (dq == 0).all() and (dk == 0).all() and (dv[[sum(lk[:i]) for i in range(len(lk))]] != 0).any()
        assert (smla.dense_mha_bwd(q, k, v, 0.1, out, lse, do, cq, ck)[0][first] == 0).all()


BACK = [([300], [300], 2, 2, 192), ([1100, 70], [1300, 70], 4, 4, 128), ([200, 90], [200, 40], 64, 1, 192),
        ([400], [450], 5, 1, 128), ([260], [260], 6, 2, 192)]


@pytest.mark.parametrize("lq,lk,h,hk,d", BACK)
def test_dv_does_not_depend_on_values(smla, lq, lk, h, hk, d):  # noqa: F811
    """An infinite value makes out and D of the rows that see it infinite: their dq and what they give dk is NaN;
    dv = P^T dout stays."""
    q, k, v, do, cq, ck = _inputs(38, lq, lk, h, hk, d)
    want = smla.dense_mha_bwd(q, k, v, 0.1, *smla.dense_mha_fwd(q, k, v, 0.1, cq, ck), do, cq, ck)
    for at in (0, 37, 127, 128, lk[0] - 1):
        if at >= lk[0]:
            continue
        v2 = v.clone()
        v2[at, :, 9] = INF
        dq, dk, dv = smla.dense_mha_bwd(q, k, v2, 0.1, *smla.dense_mha_fwd(q, k, v2, 0.1, cq, ck), do, cq, ck)
        assert torch.equal(dv, want[2])
        sees = max(0, at + lq[0] - lk[0])   # the first row that sees the key
        assert torch.equal(dq[:sees], want[0][:sees]) and torch.equal(dq[lq[0]:], want[0][lq[0]:])
        assert dq[sees:lq[0]].isnan().all() and dk[:lk[0]].isnan().all()
        assert torch.equal(dk[lk[0]:], want[1][lk[0]:])


@pytest.mark.parametrize("scores", ["near", "far apart"])
@pytest.mark.parametrize("lq,lk,h,hk,d", BACK)
def test_upstream_gradients_that_are_not_finite(smla, lq, lk, h, hk, d, scores):  # noqa: F811
    """A column of dv is the sum of what is not finite in the rows that see the key, also where weights underflow;
    the other columns, and the keys that those rows do not see, have what they had."""
    q, k, v, do, cq, ck = _inputs(39, lq, lk, h, hk, d)
    if scores == "far apart":
        q[..., 0], k[..., 0] = 8.0, 0.0
        k[1::3, :, 0] = -2000.0
    out, lse = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
    want = smla.dense_mha_bwd(q, k, v, 0.1, out, lse, do, cq, ck)
    n, g = lq[0], h // hk
    first = max(0, n - lk[0])   # rows before it see nothing
    do2 = do.clone()
    rows = sorted({first, first + 5, n // 2, n - 1})
    for i, r in enumerate(rows):
        do2[r, i % h, 3], do2[r, -1, 70], do2[r, 0, 90] = INF, (INF, -INF)[i % 2], (NAN, 1.0)[i % 2]
    dq, dk, dv = smla.dense_mha_bwd(q, k, v, 0.1, out, lse, do2, cq, ck)
    # suffix sums over the rows of the first sequence, then over the heads of a group
    odd = torch.where(do2[first:n].isfinite(), 0.0, do2[first:n].float()).flip(0)
    odd = _odd_sums(odd).flip(0).view(n - first, hk, g, 128).sum(2)
    at = (torch.arange(lk[0], device=q.device) - (lk[0] - n)).clamp(min=first) - first   # first row that sees a key
    odd = torch.cat([odd[at], torch.zeros_like(dv[lk[0]:], dtype=torch.float32)])
    ref = torch.where(odd == 0, want[2].float(), odd)
    # columns with a changed but finite entry (1.0) are not compared
    cols = torch.ones(128, dtype=torch.bool, device=q.device)
    cols[90] = False
    same = lambda a, b: torch.equal(torch.nan_to_num(a, nan=12345.0), torch.nan_to_num(b, nan=12345.0))  # noqa: E731
    assert same(dv[..., cols].float(), ref[..., cols])
    assert (dv[..., 90].isfinite() == odd[..., 90].isfinite()).all()
    # dq: the heads' rows with such an entry; dk: the keys that one of them sees
    bad = ~do2.isfinite().all(-1)
    assert dq[bad].isnan().all()
    keep = ~bad
    keep[rows] = False   # their finite heads may have the changed entry
    assert torch.equal(dq[keep], want[0][keep])
    bad_key = torch.zeros(dk.shape[:2], dtype=torch.bool, device=q.device)
    for r, j in bad.nonzero().tolist():
        bad_key[:min(lk[0], r + lk[0] - n + 1), j // g] = True
    assert dk[bad_key].isnan().all() and dk[~bad_key].isfinite().all()


def test_dv_of_rows_whose_scores_are_not_finite(smla):  # noqa: F811
    """A NaN key: the rows that see it have NaN weights, whatever their upstream gradient is."""
    q, k, v, do, *_ = _inputs(40, [300], [300], 4, 2, 128)
    k[150, 0, 5] = NAN
    do[[20, 100, 200, 290], :, 7] = INF
    out, lse = smla.dense_mha_fwd(q, k, v, 0.1)
    dq, dk, dv = smla.dense_mha_bwd(q, k, v, 0.1, out, lse, do)
    assert dv[:, 0].isnan().all() and dq[150:, :2].isnan().all() and dk[:, 0].isnan().all()
    assert (dv[:291, 1, 7] == INF).all() and dv[291:, 1].isfinite().all()
    assert dv[:, 1, :7].isfinite().all() and dv[:, 1, 8:].isfinite().all()


@pytest.mark.parametrize("lq,lk,h,hk,d", BACK)
def test_seen_keys_whose_scores_are_minus_infinite(smla, lq, lk, h, hk, d):  # noqa: F811
    """Weight 0 and dS 0: NaN in dq where the key is not finite (0 times an infinity), whether all rows of a block see
    it or not; all else as with a key that is only far away.  (No row sees such a key alone.)  A block whose heads
    side by side leave rows unused gives them no weight."""
    q, k, v, do, cq, ck = _inputs(41, lq, lk, h, hk, d)
    q[..., 5] = 1.0
    for at in (1, 90, 95, 96, 130, 199, 200, 255, lk[0] - 1):
        if at >= lk[0]:
            continue
        k2, far = k.clone(), k.clone()
        k2[at, :, 5], far[at, :, 5] = -INF, -1e30
        a, b = smla.dense_mha_fwd(q, k2, v, 0.1, cq, ck), smla.dense_mha_fwd(q, far, v, 0.1, cq, ck)
        sees = max(0, at + lq[0] - lk[0])
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        got, want = (smla.dense_mha_bwd(q, x, v, 0.1, *y, do, cq, ck) for x, y in ((k2, a), (far, b)))
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        assert got[0][sees:lq[0], :, 5].isnan().all()
        got[0][sees:lq[0], :, 5] = want[0][sees:lq[0], :, 5]
        assert torch.equal(got[0], want[0])


def test_keys_times_heads_past_32_bits(smla):  # noqa: F811
    """One token of 32 heads over 2^26 keys and more: every key has the same weight and the same dv."""
    n, h, d = (1 << 26) + 1000, 32, 128
    q, _, _, do, *_ = _inputs(42, [1], [1], h, 1, d)
    k, v = (torch.zeros(n, 1, d, dtype=torch.bfloat16, device=q.device) for _ in range(2))
    out, lse = smla.dense_mha_fwd(q, k, v, 0.1)
    # ln n is 18.02: fp32's half step there and the sum's roundings (2^-20 of n)
    assert (out == 0).all() and ((lse.double() - torch.tensor(float(n)).log()).abs() <= 2.0 ** -19).all()
    dq, dk, dv = smla.dense_mha_bwd(q, k, v, 0.1, out, lse, do)
    assert (dq == 0).all() and not dk.count_nonzero()
    row = dv[-1].double()
    # P is rounded to bf16 and off by lse's error, dv rounded once more
    assert ((row - do.double().sum(1) / n).abs() <= 2.0 ** -7 * do.double().abs().sum(1) / n).all() and (row != 0).any()
    assert all(torch.equal(x, dv[-1:].expand_as(x)) for x in dv.split(1 << 22))


def test_gradients_under_offsets_outside_of_the_tensors(smla):  # noqa: F811
    """Offsets are cut to the tensors in the backward as in the forward."""
    q, k, v, do, *_ = _inputs(7, [90], [90], 2, 1, 128)
    offsets = lambda *x: torch.tensor(x, dtype=torch.int32, device=q.device)  # noqa: E731
    cut = offsets(0, 60, 500, 10), offsets(-4, 60, 1000, 2000)
    good = (offsets(0, 60, 90),) * 2
    a, b = smla.dense_mha_fwd(q, k, v, 0.1, *cut), smla.dense_mha_fwd(q, k, v, 0.1, *good)
    a += smla.dense_mha_bwd(q, k, v, 0.1, *a, do, *cut)
    b += smla.dense_mha_bwd(q, k, v, 0.1, *b, do, *good)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("lq,lk,h,hk,d", [([900, 130], [900, 300], 4, 2, 192), ([1500], [1500], 8, 1, 128)])
def test_gradients_2_norm(smla, lq, lk, h, hk, d):  # noqa: F811
    """P and dS are rounded to bf16 once, a value once more on its way out: each is spread over half a step, 2^-8 /
    sqrt(3) in the mean square at most.  The inputs' keys, queries and upstream rows have independent signs, so a sum's
    terms add up in the mean square as their errors do: sqrt(2 / 3) 2^-8 in all.  fp32's 2^-16 of the terms of
    T - D, some 10 times its size, is 2^-12.  Together less than 2^-8."""
    q, k, v, do, cq, ck = _inputs(43, lq, lk, h, hk, d)
    out, lse = smla.dense_mha_fwd(q, k, v, d ** -0.5, cq, ck)
    grads = smla.dense_mha_bwd(q, k, v, d ** -0.5, out, lse, do, cq, ck)
    ref, _ = dmo.bwd(q, k, v, d ** -0.5, out, lse, do, cq, ck)
    for g, r, name in zip(grads, ref, ("dq", "dk", "dv")):
        assert (g.double() - r).norm() <= 2.0 ** -8 * r.norm(), name


@pytest.mark.parametrize("n", [300, 2000])
def test_many_short_sequences(smla, n):  # noqa: F811
    """Far more sequences than a warp has lanes, some without rows, against the same in a few calls."""
    g = torch.Generator().manual_seed(44)
    lq = torch.randint(0, 7, (n,), generator=g).tolist()
    lk = [x + int(y) for x, y in zip(lq, torch.randint(0, 40, (n,), generator=g))]
    q, k, v, do, cq, ck = _inputs(45, lq, lk, 4, 2, 128, tail=3)
    out, lse = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
    dq, dk, dv = smla.dense_mha_bwd(q, k, v, 0.1, out, lse, do, cq, ck)
    assert (out[-3:] == 0).all() and all((t[-3:] == 0).all() for t in (dq, dk, dv))
    a, b = cq.tolist(), ck.tolist()
    for i in range(0, n, 25):
        j = min(n, i + 25)
        rows, keys = slice(a[i], a[j]), slice(b[i], b[j])
        c, e = (t[i:j + 1] - t[i] for t in (cq, ck))
        if a[i] == a[j] or b[i] == b[j]:
            continue
        want = smla.dense_mha_fwd(q[rows], k[keys], v[keys], 0.1, c, e)
        assert torch.equal(want[0], out[rows]) and torch.equal(want[1], lse[rows])
        back = smla.dense_mha_bwd(q[rows], k[keys], v[keys], 0.1, *want, do[rows], c, e)
        assert all(torch.equal(x, y) for x, y in zip(back, (dq[rows], dk[keys], dv[keys])))


def test_a_long_request_beside_short_ones(smla):  # noqa: F811
    """16 tokens behind 30000 keys beside 31 short texts: the layout goes by mean lengths, the rows do not."""
    lq, lk = [16] + [20 + i for i in range(31)], [30000] + [20 + 2 * i for i in range(31)]
    q, k, v, do, cq, ck = _inputs(46, lq, lk, 8, 8, 192)
    out, lse = smla.dense_mha_fwd(q, k, v, 0.1, cq, ck)
    _check_fwd(out, lse, q, k, v, 0.1, cq, ck)
    _check_bwd(smla.dense_mha_bwd(q, k, v, 0.1, out, lse, do, cq, ck), q, k, v, 0.1, out, lse, do, cq, ck)


@pytest.mark.parametrize("lq,lk,h,hk,d", [(1, 5000, 8, 8, 192), (130, 4500, 2, 1, 128), (300, 1200, 2, 2, 192),
                                          (1050, 1100, 64, 64, 128), (900, 1700, 128, 1, 192)])
def test_seen_values_of_keys_of_weight_zero(smla, lq, lk, h, hk, d):  # noqa: F811
    """Keys whose scores are -infinite, whole parts of a cluster among them, have no weight; their values that are not
    finite count as all others do."""
    q, k, v, *_ = _inputs(47, [lq], [lk], h, hk, d)
    q[..., 0] = 1.0
    n = min(700, lk - lq)   # all rows see more than these
    k[:n, :, 0] = -INF
    want = smla.dense_mha_fwd(q, k, v, 0.1)
    assert want[0].isfinite().all() and want[1].isfinite().all()
    v2 = v.clone()
    v2[5, :, 7], v2[n // 2, :, 9], v2[n - 1, :, 9], v2[n - 1, :, 100] = INF, INF, -INF, NAN
    out, lse = smla.dense_mha_fwd(q, k, v2, 0.1)
    assert torch.equal(lse, want[1])
    ref = want[0].clone()
    ref[..., 7], ref[..., 9], ref[..., 100] = INF, NAN, NAN
    assert torch.equal(torch.nan_to_num(out, nan=12345.0), torch.nan_to_num(ref, nan=12345.0))

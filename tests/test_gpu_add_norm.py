"""mla_add_norm and mla_add_norm_bwd against the float64 oracle.

Tolerances.  The sum is one rounding; normed rows are rounded once from 46
bits: equal to the oracle's, and so are codes and scales.  A gradient dx is
within half a bf16 step of its value, 2^-8 of it, plus fp32 arithmetic on its
terms: sums of up to 16384 terms, 32 in a thread and the rest in a tree, are
within 45 roundings, under 2^-18 of the terms' magnitudes.  dweight is a sum of
at most 200 terms in a row and a tree of their sums."""
import numpy as np
import pytest
import torch

from oracle import add_norm_oracle as ano
from oracle.norm_rope_oracle import round_bf16

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 1e-6


@pytest.fixture(scope="module")
def smla(cuda_lib):
    import serving_sparse_mla_gb300 as pkg
    pkg.clear_device_error()
    yield pkg
    assert pkg.get_device_error() == 0


def _f64(t):
    return t.double().cpu().numpy()


def _rows(seed, n, d, wide=0):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(0.7 * torch.randn(d, generator=g))
    make = lambda: (torch.randn(n, d, generator=g) * size * torch.exp(torch.randn(n, 1, generator=g))).bfloat16()  # noqa: E731
    x, r = make().to(DEV), make().to(DEV)
    if wide:
        x = torch.cat([torch.full((n, 8), float("nan"), dtype=x.dtype, device=DEV), x,
                       torch.full((n, wide), float("nan"), dtype=x.dtype, device=DEV)], 1)[:, 8:8 + d]
    return x, r, (1 + 0.2 * torch.randn(d, generator=g)).bfloat16().to(DEV)


def _check(x, r, w, group, got):
    out, scales, z = got
    rz = ano.add(_f64(x), None if r is None else _f64(r))
    assert np.array_equal(_f64(z), rz)
    y = round_bf16(ano.norm(rz, _f64(w), EPS))
    if group is None:
        assert scales is None and np.array_equal(_f64(out), y)
        return
    v, s = ano.codes(y, group or y.shape[1])
    assert out.dtype == torch.float8_e4m3fn and scales.shape == s.shape
    assert np.array_equal(_f64(scales), s) and np.array_equal(_f64(out), v)


@pytest.mark.parametrize("group", [None, 128, 0])
@pytest.mark.parametrize("n,d", [(1, 8), (1, 7168), (3, 128), (2, 136), (5, 1000), (7, 2048), (3, 2056), (2, 4096), (3, 4104),
                                 (4, 5120), (2, 8192), (1, 16384), (700, 1544), (1300, 64)])
def test_add_norm(smla, n, d, group):
    x, r, w = _rows(n * 7 + d, n, d, wide=16)
    _check(x, r, w, group, smla.mla_add_norm(x, w, r, eps=EPS, group=group))
    _check(x, None, w, group, smla.mla_add_norm(x, w, eps=EPS, group=group))


@pytest.mark.parametrize("group", [None, 128, 0])
def test_in_place_and_given_outputs(smla, group):
    x, r, w = _rows(5, 900, 1032)
    kind = torch.bfloat16 if group is None else torch.float8_e4m3fn
    want = smla.mla_add_norm(x, w, r, eps=EPS, group=group)
    for where in ("residual", "x"):
        a, b = x.clone(), r.clone()
        out = torch.empty(900, 1032, dtype=kind, device=DEV)
        scales = None if group is None else torch.empty_like(want[1])
        got = smla.mla_add_norm(a, w, b, eps=EPS, group=group, out=out, scales=scales,
                                residual_out=b if where == "residual" else a)
        assert got[0] is out and got[2] is (b if where == "residual" else a)
        for u, v in zip(got, want):
            assert u is v is None or torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def test_scales_at_their_borders(smla):
    """Rows whose largest value is at, just under and just over 448 times a power of two; zeros; subnormals."""
    n, d = 24, 256
    z = torch.zeros(n, d)
    for i in range(n - 2):
        z[i, 3], z[i, 200] = (1.75 + (i % 3 - 1) / 128) * 2.0 ** (i - 10), 0.01
    z[n - 1] = 1e-30
    z, w = z.bfloat16().to(DEV), torch.ones(d, dtype=torch.bfloat16, device=DEV)
    for group in (128, 0):
        _check(z, None, w, group, smla.mla_add_norm(z, w, eps=EPS, group=group))


def test_values_that_are_not_finite(smla):
    x, r, w = _rows(6, 8, 384)
    x[1, 5], x[2, 200], x[3, 383] = float("nan"), float("inf"), float("-inf")
    w2 = w.clone()
    w2[130] = float("nan")
    for group in (None, 128, 0):
        out, scales, _ = smla.mla_add_norm(x, w, r, eps=EPS, group=group)
        clean = smla.mla_add_norm(x[4:], w, r[4:], eps=EPS, group=group)
        assert torch.equal(out[4:].view(torch.uint8), clean[0].view(torch.uint8))
        if group is None:
            assert out[1].isnan().all()
            # an infinity's row: the factor is 0
            assert out[2, 200].isnan() and (out[2, :200] == 0).all() and (out[2, 201:] == 0).all()
        else:
            bad = scales.isnan().cpu()
            assert bad[1].all() and bad[2:4].any(1).all() and not bad[0].any() and not bad[4:].any()
            assert (group == 0) or (bad[2].tolist() == [False, True, False] and bad[3].tolist() == [False, False, True])
        out, scales, _ = smla.mla_add_norm(x[4:], w2, r[4:], eps=EPS, group=group)
        if group == 128:
            assert scales.isnan().cpu().tolist() == [[False, True, False]] * 4


def _check_grads(z, w, do, dr, got):
    dx, dw, sx, sw = ano.grads(_f64(z), _f64(w), EPS, _f64(do), None if dr is None else _f64(dr))
    assert (np.abs(_f64(got[0]) - dx) <= 2.0 ** -8 * np.abs(dx) + 2.0 ** -18 * sx + 1e-38).all()
    assert got[1].dtype == torch.float32
    assert (np.abs(_f64(got[1]) - dw) <= (2.0 ** -19 + 2.0 ** -24 * min(len(dx), 200)) * sw + 1e-38).all()


@pytest.mark.parametrize("n,d", [(1, 8), (1, 7168), (3, 136), (257, 2048), (150, 2056), (77, 4104), (5, 16384),
                                 (2000, 320), (1500, 1000)])
def test_gradients(smla, n, d):
    z, do, w = _rows(n + d, n, d, wide=8)
    do = do * 0.01
    dr = _rows(n + d + 1, n, d, wide=24)[0]
    _check_grads(z, w, do, dr, smla.mla_add_norm_bwd(z, w, do, dr, eps=EPS))
    _check_grads(z, w, dr, None, smla.mla_add_norm_bwd(z, w, dr, eps=EPS))
    first = smla.mla_add_norm_bwd(z, w, do, dr, eps=EPS)
    a, b = do.clone(), dr.clone()
    assert smla.mla_add_norm_bwd(z, w, a, dr, eps=EPS, dx=a)[0] is a and torch.equal(a, first[0])
    assert smla.mla_add_norm_bwd(z, w, do, b, eps=EPS, dx=b)[0] is b and torch.equal(b, first[0])
    assert all(torch.equal(u, v) for u, v in zip(first, smla.mla_add_norm_bwd(z, w, do, dr, eps=EPS)))


def test_gradients_are_differences(smla):
    """d(sum(y dout) + sum(z dres)) along random directions, from the oracle's unrounded forward."""
    z, do, w = _rows(9, 6, 264)
    dr = _rows(10, 6, 264)[0]
    dx, dw = smla.mla_add_norm_bwd(z, w, do, dr, eps=EPS)
    rng = np.random.default_rng(3)
    f = lambda a, b: (ano.norm(a, b, EPS) * _f64(do)).sum() + (a * _f64(dr)).sum()  # noqa: E731
    for _ in range(4):
        u, v = rng.standard_normal((6, 264)), rng.standard_normal(264)
        diff = (f(_f64(z) + 1e-6 * u, _f64(w) + 1e-6 * v) - f(_f64(z) - 1e-6 * u, _f64(w) - 1e-6 * v)) / 2e-6
        got = (_f64(dx) * u).sum() + (_f64(dw) * v).sum()
        # dx is rounded by up to 2^-8 of itself, each value by itself
        assert abs(got - diff) <= 2.0 ** -8 * np.abs(_f64(dx) * u).sum() + 1e-5 * abs(diff)


def test_no_rows(smla):
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    out, scales, z = smla.mla_add_norm(x, w, x, group=128)
    assert out.shape == (0, 64) and scales.shape == (0, 1) and z.shape == (0, 64)
    dx, dw = smla.mla_add_norm_bwd(x, w, x, x, dweight=torch.full((64,), 3.0, device=DEV))
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_rows_past_32_bit_offsets(smla):
    """Rows 2^31 elements and more from the tensor's start."""
    d, n = 16384, (1 << 17) + 3
    x = torch.zeros(n, d, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    last, r, _ = _rows(11, 2, d)
    x[-2:] = last
    out, scales, z = smla.mla_add_norm(x, w, x, eps=EPS, group=128)
    want = smla.mla_add_norm(last, w, last, eps=EPS, group=128)
    assert torch.equal(out[-2:].view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(scales[-2:], want[1]) and torch.equal(z[-2:], want[2])
    dx, _ = smla.mla_add_norm_bwd(x, w, x, eps=EPS)
    assert torch.equal(dx[-2:], smla.mla_add_norm_bwd(last, w, last, eps=EPS)[0])


def test_streams_and_graphs(smla):
    x, r, w = _rows(12, 300, 7168)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = smla.mla_add_norm(x, w, r, eps=EPS, group=128, stream=side)
    g = smla.mla_add_norm_bwd(a[2], w, x, r, eps=EPS, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b = smla.mla_add_norm(x, w, r, eps=EPS, group=128)
    h = smla.mla_add_norm_bwd(b[2], w, x, r, eps=EPS)
    assert all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(a + g, b + h))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = smla.mla_add_norm(x, w, r, eps=EPS, group=128)
        k = smla.mla_add_norm_bwd(c[2], w, x, r, eps=EPS)
    x2, r2, _ = _rows(13, 300, 7168)
    x.copy_(x2)
    r.copy_(r2)
    graph.replay()
    d = smla.mla_add_norm(x2, w, r2, eps=EPS, group=128)
    m = smla.mla_add_norm_bwd(d[2], w, x2, r2, eps=EPS)
    torch.cuda.synchronize()
    assert all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(c + k, d + m))

"""Refusals of mla_add_norm, mla_add_norm_bwd, dense_mha_fwd and dense_mha_bwd
(no GPU): status codes of the C entry points before any device is touched, and
the binding's checks with the library replaced by a recorder."""
import glob
import os
import re

import math

import pytest
import torch

from tests.test_binding_checks import STREAM, _ok, _refused, b  # noqa: F401  (the recorder fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from serving_sparse_mla_gb300 import binding, build
    build.build()
    return binding.load()


def test_header_functions_are_exported_and_bound(lib):
    from serving_sparse_mla_gb300 import binding
    text = ""
    for h in glob.glob(os.path.join(ROOT, "include", "*.h")):
        text += re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
    names = set(re.findall(r"\b(mla_add_\w+|dense_mha_\w+)\s*\(", text))
    assert names == {"mla_add_norm", "mla_add_norm_bwd", "mla_add_norm_bwd_workspace_size", "dense_mha_fwd",
                     "dense_mha_bwd", "dense_mha_bwd_workspace_size"}
    for n in names:
        assert hasattr(lib, n) and n in binding.SIGNATURES


def _norm(lib, **kw):
    a = dict(x=16, xs=64, res=16, rs=64, w=16, eps=1e-6, out=16, sc=16, form=1, z=16, n=3, d=64, stream=None)
    a.update(kw)
    return lib.mla_add_norm(*a.values())


def _grad(lib, **kw):
    a = dict(x=16, xs=64, w=16, eps=1e-6, do=16, ds=64, res=16, rs=64, dx=16, dw=16, n=3, d=64, ws=16, wb=1 << 24,
             stream=None)
    a.update(kw)
    return lib.mla_add_norm_bwd(*a.values())


@pytest.mark.parametrize("call", [_norm, _grad])
def test_norm_argument_codes(lib, call):
    for bad in (dict(d=60), dict(d=16392), dict(d=1)):
        assert call(lib, **bad) == 2, bad
    for bad in (dict(n=-1), dict(d=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None),
                dict(w=None), dict(x=24), dict(w=8), dict(xs=65), dict(rs=4), dict(res=24)):
        assert call(lib, **bad) == 1, bad


def test_norm_output_codes(lib):
    for bad in (dict(out=None), dict(out=24), dict(sc=None), dict(sc=18), dict(z=None), dict(z=24), dict(form=3),
                dict(form=-1)):
        assert _norm(lib, **bad) == 1, bad
    for bad in (dict(do=None), dict(do=24), dict(ds=9), dict(dx=None), dict(dx=24), dict(dw=None), dict(dw=18)):
        assert _grad(lib, **bad) == 1, bad
    for n, d in ((0, 64), (-1, 64), (4, 60), (4, 0), (4, 1 << 20)):
        assert lib.mla_add_norm_bwd_workspace_size(n, d) == 0


def _fwd(lib, **kw):
    a = dict(q=16, qt=1536, qh=192, k=16, kt=768, kh=192, v=16, vt=512, vh=128, cq=16, ck=16, b=2, scale=0.1, out=16,
             lse=16, fill=0, nq=5, nk=9, h=8, hk=4, d=192, dv=128, stream=None)
    a.update(kw)
    return lib.dense_mha_fwd(*a.values())


def _bwd(lib, **kw):
    a = dict(q=16, qt=1536, qh=192, k=16, kt=768, kh=192, v=16, vt=512, vh=128, cq=16, ck=16, b=2, scale=0.1, out=16,
             lse=16, do=16, dt=1024, dh=128, dq=16, dk=16, dvo=16, nq=5, nk=9, h=8, hk=4, d=192, dv=128, ws=16,
             wb=1 << 24, stream=None)
    a.update(kw)
    return lib.dense_mha_bwd(*a.values())


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_attention_argument_codes(lib, call):
    for bad in (dict(d=64), dict(d=576), dict(d=0), dict(dv=192), dict(dv=64)):
        assert call(lib, **bad) == 2, bad
    big = 2 ** 31 - 1
    for bad in (dict(nq=-1), dict(nk=-1), dict(h=0), dict(hk=0), dict(hk=3), dict(h=4, hk=8), dict(scale=-0.1),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(cq=None), dict(ck=None), dict(b=0), dict(b=-1),
                dict(cq=18), dict(ck=18), dict(q=None), dict(k=None), dict(v=None), dict(q=24), dict(k=8), dict(v=24),
                dict(qt=1540), dict(qh=100), dict(kt=4), dict(vh=12), dict(qt=0), dict(kh=0), dict(vt=-8),
                dict(out=None), dict(out=24), dict(lse=None), dict(lse=18), dict(nq=big), dict(nk=big), dict(b=big),
                dict(h=1 << 20, hk=1)):
        assert call(lib, **bad) == 1, bad


def test_attention_output_codes(lib):
    for bad in (dict(fill=4), dict(fill=-1)):
        assert _fwd(lib, **bad) == 1, bad
    for bad in (dict(do=None), dict(do=24), dict(dt=4), dict(dh=0), dict(dq=None), dict(dk=None), dict(dvo=None),
                dict(dq=24), dict(dk=24), dict(dvo=24)):
        assert _bwd(lib, **bad) == 1, bad


# ------------------------------------------------------------------ binding

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _norm_args(n=5, d=64):
    return dict(x=torch.zeros(n, d, dtype=BF), weight=torch.zeros(d, dtype=BF), residual=torch.zeros(n, d, dtype=BF))


def test_add_norm_hands_over(b):  # noqa: F811
    for kw in (dict(), dict(group=128), dict(group=0), dict(residual=None), dict(x=torch.zeros(5, 128, dtype=BF)[:, 64:])):
        _ok(b, "mla_add_norm", b.mla_add_norm, **dict(_norm_args(), **kw))
    a = _norm_args()
    out, scales, z = b.mla_add_norm(**a, group=128, stream=STREAM)
    assert out.dtype == torch.float8_e4m3fn and scales.shape == (5, 1) and z.shape == (5, 64) and z.dtype == BF
    assert b.mla_add_norm(a["x"], a["weight"], stream=STREAM)[2] is a["x"]
    assert b.mla_add_norm(**a, residual_out=a["residual"], stream=STREAM)[2] is a["residual"]


@pytest.mark.parametrize("kw", [
    dict(x=torch.zeros(5, 64)), dict(x=torch.zeros(5, 1, 64, dtype=BF)), dict(x=torch.zeros(64, 5, dtype=BF).T),
    dict(x=torch.zeros(5, 65, dtype=BF)[:, :64]), dict(x=torch.zeros(321, dtype=BF)[1:].view(5, 64)),
    dict(weight=torch.zeros(65, dtype=BF)), dict(weight=torch.zeros(63, dtype=BF)), dict(weight=torch.zeros(64)),
    dict(residual=torch.zeros(4, 64, dtype=BF)), dict(residual=torch.zeros(5, 72, dtype=BF)), dict(group=64),
    dict(out=torch.zeros(5, 64)), dict(out=torch.zeros(4, 64, dtype=BF)), dict(scales=torch.zeros(5, 1)),
    dict(group=128, out=torch.zeros(5, 64, dtype=BF)), dict(group=128, scales=torch.zeros(4, 1)),
    dict(residual=None, residual_out=torch.zeros(5, 64, dtype=BF)), dict(residual_out=torch.zeros(5, 64)),
    dict(residual_out=torch.zeros(4, 64, dtype=BF)),
])
def test_add_norm_refuses(b, kw):  # noqa: F811
    _refused(b, b.mla_add_norm, **dict(_norm_args(), **kw))


def test_add_norm_refuses_memory_that_it_reads_later(b):  # noqa: F811
    pool = torch.zeros(12, 64, dtype=BF)
    w = torch.zeros(64, dtype=BF)
    _refused(b, b.mla_add_norm, pool[:5], w, pool[6:11], residual_out=pool[1:6])
    _refused(b, b.mla_add_norm, pool[:5], w, out=pool[:5])
    wide = torch.zeros(5, 128, dtype=BF)
    _refused(b, b.mla_add_norm, wide[:, :64], w, pool[:5], residual_out=wide.view(10, 64)[:5])
    _refused(b, b.mla_add_norm_bwd, pool[:5], w, pool[6:11], dx=pool[:5])
    _refused(b, b.mla_add_norm_bwd, pool[:5], w, pool[6:11], dx=pool[7:12])
    _ok(b, "mla_add_norm_bwd", b.mla_add_norm_bwd, pool[:5], w, pool[6:11], dx=pool[6:11])


def _grad_args(n=5, d=64):
    return dict(z=torch.zeros(n, d, dtype=BF), weight=torch.zeros(d, dtype=BF), dout=torch.zeros(n, d, dtype=BF),
                dresidual=torch.zeros(n, d, dtype=BF))


def test_add_norm_bwd_checks(b):  # noqa: F811
    for kw in (dict(), dict(dresidual=None), dict(dout=torch.zeros(5, 128, dtype=BF)[:, :64])):
        _ok(b, "mla_add_norm_bwd", b.mla_add_norm_bwd, **dict(_grad_args(), **kw))
    for kw in (dict(z=torch.zeros(5, 64)), dict(z=torch.zeros(64, dtype=BF)), dict(weight=torch.zeros(8, dtype=BF)),
               dict(dout=torch.zeros(5, 64)), dict(dout=torch.zeros(4, 64, dtype=BF)),
               dict(dresidual=torch.zeros(5, 63, dtype=BF)), dict(dx=torch.zeros(5, 64)),
               dict(dx=torch.zeros(2, 64, dtype=BF)), dict(dweight=torch.zeros(64, dtype=BF)),
               dict(dweight=torch.zeros(63))):
        _refused(b, b.mla_add_norm_bwd, **dict(_grad_args(), **kw))


def _mha_args(n=5, m=9, h=8, hk=4, d=192):
    return dict(q=torch.zeros(n, h, d, dtype=BF), k=torch.zeros(m, hk, d, dtype=BF), v=torch.zeros(m, hk, 128, dtype=BF),
                sm_scale=0.1, cu_seqlens_q=torch.tensor([0, 2, 5], dtype=I32),
                cu_seqlens_kv=torch.tensor([0, 2, 9], dtype=I32))


BAD_MHA = [
    dict(q=torch.zeros(5, 8, 192)), dict(q=torch.zeros(5, 8 * 192, dtype=BF)), dict(k=torch.zeros(9, 4, 128, dtype=BF)),
    dict(k=torch.zeros(9, 3, 192, dtype=BF)), dict(k=torch.zeros(9, 0, 192, dtype=BF)),
    dict(v=torch.zeros(8, 4, 128, dtype=BF)), dict(v=torch.zeros(9, 2, 128, dtype=BF)), dict(v=torch.zeros(9, 4, 128)),
    dict(q=torch.zeros(5, 192, 8, dtype=BF).transpose(1, 2)), dict(k=torch.zeros(9, 4, 196, dtype=BF)[..., :192]),
    dict(k=torch.zeros(9, 1, 192, dtype=BF).expand(9, 4, 192)), dict(v=torch.zeros(1, 4, 128, dtype=BF).expand(9, 4, 128)),
    dict(q=torch.zeros(5 * 8 * 192 + 1, dtype=BF)[1:].view(5, 8, 192)), dict(cu_seqlens_kv=None),
    dict(cu_seqlens_q=None), dict(cu_seqlens_q=torch.tensor([0, 5])), dict(cu_seqlens_kv=torch.tensor([0, 9], dtype=I32)),
    dict(cu_seqlens_kv=torch.tensor([0, 1, 2, 9], dtype=I32)),
]


@pytest.mark.parametrize("kw", BAD_MHA + [dict(out=torch.zeros(5, 8, 128)), dict(out=torch.zeros(4, 8, 128, dtype=BF)),
                                          dict(lse=torch.zeros(39)), dict(lse=torch.zeros(40, dtype=BF))])
def test_dense_mha_fwd_refuses(b, kw):  # noqa: F811
    _refused(b, b.dense_mha_fwd, **dict(_mha_args(), **kw))


def test_dense_mha_fwd_hands_over(b):  # noqa: F811
    heads_first = torch.zeros(8, 5, 192, dtype=BF).transpose(0, 1)
    latent = torch.zeros(9, 4, 256, dtype=BF)   # keys and values of one projection
    for kw in (dict(), dict(q=heads_first), dict(v=latent[..., 128:]), dict(cu_seqlens_q=None, cu_seqlens_kv=None),
               dict(_mha_args(d=128)), dict(q=torch.zeros(0, 8, 192, dtype=BF), cu_seqlens_q=None, cu_seqlens_kv=None)):
        _ok(b, "dense_mha_fwd", b.dense_mha_fwd, **dict(_mha_args(), **kw))
    out, lse = b.dense_mha_fwd(**_mha_args(), stream=STREAM)
    assert out.shape == (5, 8, 128) and out.dtype == BF and lse.shape == (5, 8) and lse.dtype == F32


def _bwd_args(**kw):
    a = dict(_mha_args(), out=torch.zeros(5, 8, 128, dtype=BF), lse=torch.zeros(5, 8), dout=torch.zeros(5, 8, 128, dtype=BF))
    return dict(a, **kw)


@pytest.mark.parametrize("kw", BAD_MHA + [
    dict(out=torch.zeros(5, 8, 128)), dict(out=torch.zeros(4, 8, 128, dtype=BF)), dict(lse=torch.zeros(39)),
    dict(dout=torch.zeros(5, 8, 128)), dict(dout=torch.zeros(5, 4, 128, dtype=BF)),
    dict(dout=torch.zeros(1, 8, 128, dtype=BF).expand(5, 8, 128)), dict(dq=torch.zeros(5, 8, 192)),
    dict(dq=torch.zeros(4, 8, 192, dtype=BF)), dict(dk=torch.zeros(9, 4, 128, dtype=BF)),
    dict(dv=torch.zeros(8, 4, 128, dtype=BF))])
def test_dense_mha_bwd_refuses(b, kw):  # noqa: F811
    _refused(b, b.dense_mha_bwd, **_bwd_args(**kw))


def test_dense_mha_bwd_hands_over(b):  # noqa: F811
    for kw in (dict(), dict(dout=torch.zeros(8, 5, 128, dtype=BF).transpose(0, 1)),
               dict(dq=torch.zeros(5, 8, 192, dtype=BF))):
        _ok(b, "dense_mha_bwd", b.dense_mha_bwd, **_bwd_args(**kw))
    dq, dk, dv = b.dense_mha_bwd(**_bwd_args(), stream=STREAM)
    assert dq.shape == (5, 8, 192) and dk.shape == (9, 4, 192) and dv.shape == (9, 4, 128)


def test_dense_mha_refuses_memory_that_it_reads(b):  # noqa: F811
    def part(pool, start, *shape):
        n = math.prod(shape)
        return pool[start:start + n].view(*shape)

    pool = torch.zeros(1 << 16, dtype=BF)
    q, out = part(pool, 0, 5, 8, 192), part(pool, 7680, 5, 8, 128)
    _ok(b, "dense_mha_fwd", b.dense_mha_fwd, **dict(_mha_args(), q=q, out=out))
    for kw in (dict(out=part(pool, 7672, 5, 8, 128)), dict(out=part(pool, 0, 5, 8, 128)),
               dict(lse=part(pool, 7600, 80).view(F32)), dict(out=out, lse=part(pool, 12720, 80).view(F32))):
        _refused(b, b.dense_mha_fwd, **dict(_mha_args(), q=q, **kw))
    latent = part(pool, 0, 9, 4, 384)   # an output between the rows' parts that are read
    _refused(b, b.dense_mha_fwd, **dict(_mha_args(), k=latent[..., :192], out=part(pool, 192, 5, 8, 128)))
    a = _bwd_args(q=q, out=out)
    dk, dv = part(pool, 16384, 9, 4, 192), part(pool, 24576, 9, 4, 128)
    _ok(b, "dense_mha_bwd", b.dense_mha_bwd, **dict(a, dk=dk, dv=dv, dq=part(pool, 32768, 5, 8, 192)))
    for kw in (dict(dq=q), dict(dk=part(pool, 12792, 9, 4, 192)), dict(dk=dk, dv=part(pool, 16384, 9, 4, 128)),
               dict(dv=part(pool, 0, 9, 4, 128)),
               dict(dv=dv, workspace=dv.view(torch.uint8).view(-1))):
        _refused(b, b.dense_mha_bwd, **dict(a, **kw))

"""Refusals of mla_norm_rope, mla_norm_rope_bwd and sparse_mla_decode_fp4 (no
GPU): status codes of the C entry points before any device is touched, and
the binding's checks with the library replaced by a recorder."""
import glob
import os
import re
import types

import pytest
import torch

import mla_inputs as mi
from tests.test_binding_checks import _ok, _refused, b  # noqa: F401  (the recorder fixture)

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
    names = set(re.findall(r"\b(mla_norm_\w+|sparse_mla_decode_fp4\w*)\s*\(", text))
    assert names == {"mla_norm_rope", "mla_norm_rope_bwd", "mla_norm_rope_bwd_workspace_size",
                     "sparse_mla_decode_fp4", "sparse_mla_decode_fp4_workspace_size"}
    for n in names:
        assert hasattr(lib, n) and n in binding.SIGNATURES


def _norm(lib, **kw):
    a = dict(q=16, qt=4608, qh=576, kv=16, kt=576, pos=16, cs=16, n_pos=10, qw=None, kw=16, eps=1e-6, il=1, qo=16, ko=16,
             cache=16, form=2, ks=1.0, slots=16, n_slots=64, n=3, h=8, d=576, stream=None)
    a.update(kw)
    return lib.mla_norm_rope(*a.values())


def _grad(lib, **kw):
    a = dict(q=16, qt=4608, qh=576, kv=16, kt=576, pos=16, cs=16, n_pos=10, qw=None, kw=16, eps=1e-6, il=1, dq=16, dkv=16,
             dqi=16, dki=16, dqw=None, dkw=16, n=3, h=8, d=576, ws=16, wb=1 << 24, stream=None)
    a.update(kw)
    return lib.mla_norm_rope_bwd(*a.values())


def _fp4(lib, **kw):
    a = dict(q=16, kv=16, table=16, lens=16, idx=16, scale=0.1, ks=1.0, out=16, lse=16, b=2, s=3, h=8, d=576, dv=512,
             topk=64, page=64, mb=4, nb=4, ws=None, wb=0, stream=None)
    a.update(kw)
    return lib.sparse_mla_decode_fp4(*a.values())


@pytest.mark.parametrize("call", [_norm, _grad])
def test_norm_argument_codes(lib, call):
    assert call(lib, d=512) == 2
    for bad in (dict(h=0), dict(n=-1), dict(n_pos=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(q=None),
                dict(kv=None), dict(pos=None), dict(cs=None), dict(q=24), dict(kv=8), dict(pos=18), dict(cs=20),
                dict(qt=4), dict(qh=577), dict(kt=580), dict(kw=24)):
        assert call(lib, **bad) == 1, bad


def test_norm_output_and_cache_codes(lib):
    for bad in (dict(qo=None), dict(qo=24), dict(ko=24), dict(cache=24), dict(slots=None), dict(slots=18),
                dict(n_slots=-1), dict(form=3), dict(form=-1), dict(ks=0.0), dict(ks=-1.0), dict(ks=float("inf")),
                dict(form=0, ks=0.5), dict(form=1, ks=0.5)):
        assert _norm(lib, **bad) == 1, bad


def test_grad_output_codes(lib):
    for bad in (dict(dq=None), dict(dkv=None), dict(dqi=None), dict(dki=None), dict(dq=24), dict(dkv=24),
                dict(dqi=24), dict(dki=24), dict(dkw=None), dict(dqw=16), dict(dkw=18)):
        assert _grad(lib, **bad) == 1, bad


def test_fp4_argument_codes(lib):
    assert _fp4(lib, d=512) == 2 and _fp4(lib, dv=256) == 2
    for bad in (dict(q=None), dict(q=24), dict(out=None), dict(lse=None), dict(idx=18), dict(table=None),
                dict(lens=None), dict(page=0), dict(b=-1), dict(h=0), dict(topk=0), dict(nb=1 << 30)):
        assert _fp4(lib, **bad) == 1, bad
    assert lib.sparse_mla_decode_fp4_workspace_size(0, 1, 8, 512, 64) == 0
    assert lib.sparse_mla_decode_fp4_workspace_size(1, 1, 8, 256, 64) == 0
    assert lib.mla_norm_rope_bwd_workspace_size(0, 8) == 0


def test_a_cache_factor_near_the_ends_of_fp32_is_refused(lib):
    """A group's step is 2^-9 .. 448 factors; it and its reciprocal have to be normal."""
    for ks in (2.0 ** -65, 1e-38, 1e-45, 2.0 ** 65, 3e38):
        assert _norm(lib, ks=ks) == 1 and _fp4(lib, ks=ks) == 1, ks


def test_sizes_past_the_counters_are_refused(lib):
    """Lists, rows and blocks whose counts would leave their integers."""
    big = 2 ** 31 - 1
    for bad in (dict(topk=big), dict(topk=big - 1000), dict(h=big), dict(b=big), dict(b=big, s=big),
                dict(b=1 << 27, s=1, h=16), dict(b=1 << 27, s=1, h=8, topk=1 << 30)):
        assert _fp4(lib, **bad) == 1, bad
        a = dict(dict(b=2, s=3, h=8, topk=64), **bad)
        assert lib.sparse_mla_decode_fp4_workspace_size(a["b"], a["s"], a["h"], 512, a["topk"]) == 0, bad
    for call in (_norm, _grad):
        assert call(lib, h=big) == 1 and call(lib, n=big) == 1


# ------------------------------------------------------------------ binding

def _args(n=5, h=3, n_pos=20):
    q, kv, qw, kw = mi.norm_rows(1, n, h)
    return [q, kv, torch.arange(n, dtype=torch.int32), mi.rope_table(n_pos)], dict(q_weight=qw, kv_weight=kw)


def test_norm_binding_accepts(b):  # noqa: F811
    a, w = _args()
    sl = torch.arange(5, dtype=torch.int32)
    f = b.mla_norm_rope
    _ok(b, "mla_norm_rope", f, *a)
    _ok(b, "mla_norm_rope", f, *a, **w)
    _ok(b, "mla_norm_rope", f, a[0], a[1].view(5, 1, 576), *a[2:])
    for cache in (torch.zeros(2, 16, 576, dtype=torch.bfloat16), torch.zeros(2, 16, 656, dtype=torch.uint8),
                  torch.zeros(2, 16, 416, dtype=torch.uint8)):
        _ok(b, "mla_norm_rope", f, *a, kv_cache=cache, slots=sl)
    wide = torch.zeros(5, 3, 640, dtype=torch.bfloat16)[..., :576]
    _ok(b, "mla_norm_rope", f, wide, torch.zeros(5, 1024, dtype=torch.bfloat16)[:, 64:640], *a[2:])
    _ok(b, "mla_norm_rope", f, a[0][:0], a[1][:0], a[2][:0], a[3])
    g = b.mla_norm_rope_bwd
    _ok(b, "mla_norm_rope_bwd", g, *a, a[0].float(), a[1].float())


def test_norm_binding_refuses(b):  # noqa: F811
    a, w = _args()
    q, kv, pos, cs = a
    f, g = b.mla_norm_rope, lambda *x, **k: b.mla_norm_rope_bwd(*x, q.float(), kv.float(), **k)
    for call in (f, g):
        _refused(b, call, q.float(), kv, pos, cs, match="q must be")
        _refused(b, call, q[..., :512], kv, pos, cs, match="q must be")
        _refused(b, call, q, kv[:4], pos, cs, match="kv has 4 rows")
        _refused(b, call, q, kv.to("meta"), pos, cs, match="kv is on meta")
        _refused(b, call, q, kv, pos[:4], cs, match="positions")
        _refused(b, call, q, kv, pos.long(), cs, match="positions")
        _refused(b, call, q, kv, pos, cs[:, :32].contiguous(), match="cos_sin")
        _refused(b, call, q, kv, pos, cs.double(), match="cos_sin")
        _refused(b, call, q, kv, pos, cs, q_weight=w["q_weight"][:511], match="q_weight")
        _refused(b, call, q, kv, pos, cs, kv_weight=w["kv_weight"].float(), match="kv_weight")
        odd = torch.zeros(5, 3, 580, dtype=torch.bfloat16)[..., :576]
        _refused(b, call, odd, kv, pos, cs, match="16 bytes")
        off = torch.zeros(5 * 3 * 576 + 4, dtype=torch.bfloat16)[4:].view(5, 3, 576)
        _refused(b, call, off, kv, pos, cs, match="16 bytes")
        _refused(b, call, torch.zeros(5, 576, 3, dtype=torch.bfloat16).transpose(1, 2), kv, pos, cs, match="contiguous")
    sl = torch.arange(5, dtype=torch.int32)
    c4 = torch.zeros(2, 16, 416, dtype=torch.uint8)
    _refused(b, f, *a, kv_cache=c4, match="slots")
    _refused(b, f, *a, slots=sl, match="kv_cache")
    _refused(b, f, *a, kv_cache=c4[..., :400].contiguous(), slots=sl, match="kv_cache must be")
    _refused(b, f, *a, kv_cache=c4.view(torch.int8), slots=sl, match="kv_cache must be")
    _refused(b, f, *a, kv_cache=c4[:, :8], slots=sl, match="contiguous")
    _refused(b, f, *a, kv_cache=c4, slots=sl[:3], match="slots")
    _refused(b, f, *a, q_out=torch.empty(5, 3, 512, dtype=torch.bfloat16), match="q_out")
    _refused(b, f, *a, kv_out=torch.empty(5, 576), match="kv_out")


def test_grad_binding_refuses(b):  # noqa: F811
    a, w = _args()
    dq, dkv = a[0].float(), a[1].float()
    g = b.mla_norm_rope_bwd
    _refused(b, g, *a, dq[:4], dkv, match="dq")
    _refused(b, g, *a, dq, dkv.bfloat16(), match="dkv")
    _refused(b, g, *a, dq, dkv, dq_in=torch.empty(5, 3, 576), match="dq_in")
    _refused(b, g, *a, dq, dkv, dq_weight=torch.empty(512), match="without its weight")
    _refused(b, g, *a, dq, dkv, dkv_weight=torch.empty(511), **w, match="dkv_weight")


def test_fp4_binding(b):  # noqa: F811
    c, u = mi.decode_case_fp4(2, batch=2, s_next=2, h_q=4, lo=20, hi=40, topk=32, page=16, spare_pages=2)
    a = [c.q, u, c.block_table, c.cache_seqlens, c.indices, c.sm_scale]
    f = b.sparse_mla_decode_fp4
    _ok(b, "sparse_mla_decode_fp4", f, *a)
    _ok(b, "sparse_mla_decode_fp4", f, *a, kv_scale=0.5, out=torch.empty(2, 2, 4, 512, dtype=torch.bfloat16))
    _refused(b, f, a[0], u[..., :400].contiguous(), *a[2:], match="416")
    _refused(b, f, *a[:4], c.indices[:1], a[5], match="indices")
    _refused(b, f, *a, lse=torch.empty(2, 2, 3), match="lse")
    _refused(b, f, *a, out=torch.empty(2, 2, 4, 512), match="out")
    _refused(b, f, a[0].float(), *a[1:], match="q must be")
    _refused(b, f, *a, page_size=17, match="kv_cache")


def test_a_stream_of_another_device_is_refused(b):  # noqa: F811
    a, _ = _args()
    with pytest.raises(ValueError, match="stream is on"):
        b.mla_norm_rope(*a, stream=types.SimpleNamespace(cuda_stream=0, device=torch.device("meta")))

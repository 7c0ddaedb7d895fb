"""Decode over a 4-bit cache against the float64 oracle: the allclose bar of
the other decodes on every element, and a tight bound from the kernel's
arithmetic.  The rows are exact in f16 and bf16; P is rounded to f16 (half a
step 2^-11 relative, an eighth of the bf16 P that pv_rounding_sigma takes) and
the output to bf16.  LSE: scores are fp32 sums of 576 exact products; 2e-5
covers 2^-22 of the sum of their sizes at these inputs."""
import numpy as np
import pytest
import torch

import mla_inputs as mi
from oracle import fp4_kv_oracle as f4
from oracle import sparse_mla_oracle as orc
from tests.parity import compare, pv_rounding_sigma, record, tight_ratio

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def smla(cuda_lib):
    import serving_sparse_mla_gb300 as pkg
    pkg.clear_device_error()
    yield pkg
    assert pkg.get_device_error() == 0


def _run(smla, c, u, ks=1.0, **kw):
    d = lambda t: t.to(DEV)  # noqa: E731
    r = smla.sparse_mla_decode_fp4(d(c.q), d(u), d(c.block_table), d(c.cache_seqlens), d(c.indices), c.sm_scale,
                                   c.page_size, kv_scale=ks, **kw)
    torch.cuda.synchronize()
    return r


def _check(smla, c, u, what, ks=1.0):
    out, lse = _run(smla, c, u, ks)
    n = c.batch * c.s_next
    o = out.float().cpu().numpy().reshape(n, c.h_q, 512)
    l = lse.cpu().numpy().reshape(n, c.h_q)
    ro, rl = f4.sparse_mla_decode_fp4(c.q, u, c.block_table, c.cache_seqlens, c.indices, c.sm_scale, c.page_size, ks)
    do, dl = compare(o, l, ro, rl, what)
    X = f4.dequantize_slots(u, ks).reshape(-1, 576)
    idx, tab, lens = c.indices.numpy().astype(np.int64), c.block_table.numpy().astype(np.int64), c.cache_seqlens.numpy()
    worst = 0.0
    for t in range(n):
        b, j = divmod(t, c.s_next)
        r = orc.rows_paged(idx[b, j], tab[b], int(lens[b]), c.page_size, u.shape[0])
        if r.size:
            sig = pv_rounding_sigma(c.q[b, j].double().numpy().reshape(c.h_q, 576), X[r], c.sm_scale) / 8
            worst = max(worst, tight_ratio(o[t], ro[t], sig))
    record(what, max_dout=do, max_dlse=dl, tight_ratio=worst)
    assert worst <= 1.0, f"{what}: tight ratio {worst:.3f}"
    assert dl <= 2e-5, f"{what}: lse {dl:.3e}"


@pytest.mark.parametrize("h_q", [1, 2, 7, 8, 9, 16, 17, 24, 33, 64, 128])
def test_heads(smla, h_q):
    c, u = mi.decode_case_fp4(900 + h_q, batch=3, s_next=2, h_q=h_q, lo=100, hi=900, topk=256, page=64, spare_pages=3)
    _check(smla, c, u, f"fp4 decode h={h_q}")


@pytest.mark.parametrize("h_q,topk,page,ks", [(8, 1, 16, 1.0), (8, 63, 16, 1.0), (3, 65, 32, 0.3), (16, 200, 16, 1.0),
                                             (40, 129, 64, 4.0), (64, 1000, 16, 0.01)])
def test_ragged_lists_small_pages(smla, h_q, topk, page, ks):
    c, u = mi.decode_case_fp4(930 + topk, batch=4, s_next=3, h_q=h_q, lo=1, hi=1500, topk=topk, page=page,
                              spare_pages=5, kv_scale=ks)
    _check(smla, c, u, f"fp4 decode h={h_q} topk={topk} page={page}", ks)


@pytest.mark.parametrize("h_q", [8, 64])
def test_long_lists_cut_over_ctas(smla, h_q):
    c, u = mi.decode_case_fp4(951, batch=1, s_next=1, h_q=h_q, lo=9000, hi=9001, topk=2048, spare_pages=2)
    _check(smla, c, u, f"fp4 decode one token h={h_q}")
    c, u = mi.decode_case_fp4(952, batch=3, s_next=2, h_q=h_q, lo=1, hi=200, topk=2048, page=64, spare_pages=2)
    _check(smla, c, u, f"fp4 decode short lists h={h_q}")


@pytest.mark.parametrize("h_q", [8, 16, 40])
@pytest.mark.parametrize("tokens,topk", [(1, 70), (2, 2048), (9, 640), (20, 1100), (60, 2048), (120, 500)])
def test_every_split_of_the_lists(smla, h_q, tokens, topk):
    """From one token to more units than clusters fit: clusters of 16 to 2 CTAs,
    ranges with a merge, and whole units."""
    c, u = mi.decode_case_fp4(1000 + tokens, batch=1, s_next=tokens, h_q=h_q, lo=2500, hi=2500, topk=topk, page=64,
                              spare_pages=2)
    _check(smla, c, u, f"fp4 decode {tokens} tokens, {topk} entries h={h_q}")


@pytest.mark.parametrize("h_q", [8, 16, 40])
@pytest.mark.parametrize("tokens,topk", [(1, 9000), (3, 5000), (150, 256), (300, 100)])
def test_lists_longer_and_shorter_than_usual(smla, h_q, tokens, topk):
    """Few long lists (ranges of at most 64 pieces a list) and many short ones
    (a list a CTA)."""
    c, u = mi.decode_case_fp4(1200 + tokens, batch=1, s_next=tokens, h_q=h_q, lo=9500, hi=9500, topk=topk, page=64,
                              spare_pages=2)
    _check(smla, c, u, f"fp4 decode {tokens} tokens, {topk} entries h={h_q}")


@pytest.mark.parametrize("h_q", [8, 16, 40])
@pytest.mark.parametrize("tokens,topk", [(4, 700), (40, 700), (300, 300), (300, 700)])
def test_masked_tiles_blocks_and_tokens(smla, h_q, tokens, topk):
    """-1 in single entries, in 16-entry tiles, in whole blocks and in whole
    lists, wherever the lists are cut; unnamed slots hold NaN scales."""
    c, u = mi.decode_case_fp4(1300 + tokens, batch=1, s_next=tokens, h_q=h_q, lo=1500, hi=1500, topk=topk, page=64,
                              spare_pages=2)
    g = torch.Generator().manual_seed(tokens + topk)
    i = c.indices[0]
    i[torch.rand(tokens, topk, generator=g) < 0.2] = -1
    tile = torch.rand(tokens, (topk + 15) // 16, generator=g) < 0.3
    i[tile.repeat_interleave(16, 1)[:, :topk]] = -1
    block = torch.rand(tokens, (topk + 127) // 128, generator=g) < 0.4
    i[block.repeat_interleave(128, 1)[:, :topk]] = -1
    i[torch.rand(tokens, generator=g) < 0.2] = -1
    i[0] = -1
    named = i[i >= 0].long()
    slot = c.block_table[0, named // 64].long() * 64 + named % 64
    keep = torch.zeros(u.shape[0] * 64, dtype=torch.bool)
    keep[slot] = True
    u.view(-1, 416)[~keep, 256:288] = 0x7F
    _check(smla, c, u, f"fp4 decode masked {tokens} tokens, {topk} entries h={h_q}")
    out, lse = _run(smla, c, u)
    empty = (i < 0).all(1)
    assert bool((out[0, empty] == 0).all()) and bool(torch.isneginf(lse[0, empty]).all())


@pytest.mark.parametrize("h_q", [8, 24])
@pytest.mark.parametrize("page", [1, 7, 48])
def test_repeated_entries_and_odd_pages(smla, h_q, page):
    """An entry counts once for every time it is listed (a list of one entry
    only among them); pages of 1, 7 and 48 slots, requests that share pages."""
    c, u = mi.decode_case_fp4(1400 + page, batch=3, s_next=2, h_q=h_q, lo=100, hi=400, topk=90, page=page, spare_pages=3)
    c.indices[0, 0, 45:] = c.indices[0, 0, :45]
    c.indices[0, 1, :] = c.indices[0, 1, 0]
    c.indices[1, 0, 3:30] = c.indices[1, 0, 2]
    c.indices[2] = c.indices[1]
    c.cache_seqlens[2] = c.cache_seqlens[1]
    c.block_table[2] = c.block_table[1]
    _check(smla, c, u, f"fp4 decode repeated entries h={h_q} page={page}")


@pytest.mark.parametrize("h_q", [8, 16, 64])
def test_many_tokens_of_one_request(smla, h_q):
    """More units than CTAs, so that a CTA works through several."""
    c, u = mi.decode_case_fp4(961, batch=1, s_next=400, h_q=h_q, lo=700, hi=700, topk=130, page=64, spare_pages=2)
    _check(smla, c, u, f"fp4 decode 400 tokens h={h_q}")


@pytest.mark.parametrize("h_q", [8, 24])
@pytest.mark.parametrize("f", [2.0 ** -20, 2.0 ** 12])
def test_small_and_large_factors(smla, h_q, f):
    """A cache factor of 2^-20 or 2^12 with the same codes: out scales with it
    exactly as the oracle's does (checked relative to f)."""
    c, u = mi.decode_case_fp4(970, batch=2, s_next=2, h_q=h_q, lo=300, hi=600, topk=256, page=64, spare_pages=2)
    out, lse = _run(smla, c, u, f)
    ro, rl = f4.sparse_mla_decode_fp4(c.q, u, c.block_table, c.cache_seqlens, c.indices, c.sm_scale, 64, f)
    o = out.float().cpu().numpy().reshape(ro.shape) / f
    # at 2^12 one row takes all: its weight's rounding and its neighbours' are what is left
    assert np.all(np.abs(o - ro / f) <= 2.0 ** -8 * np.abs(ro / f) + 5e-3)
    tol = 1e-4 if f < 1 else 2.0 ** -20 * 4096 * 300
    assert np.all(np.abs(lse.cpu().numpy().reshape(rl.shape) - rl) <= tol)


@pytest.mark.parametrize("h_q", [8, 16, 64])
def test_masked_rows(smla, h_q):
    """Tokens whose list leaves nothing, entries past the context, page entries
    outside the pool or the table, lengths 0 and 1: masked rows are never read
    (every slot that no valid entry names holds a NaN scale)."""
    c, u = mi.decode_case_fp4(980, batch=5, s_next=2, h_q=h_q, lo=70, hi=200, topk=150, page=16, spare_pages=3)
    c.indices[0] = -1
    c.cache_seqlens[1] = 0
    c.cache_seqlens[2] = 1
    c.indices[2, :, :] = -1
    c.indices[2, 0, 149] = 0                       # one valid entry, the list's last
    u.view(-1, 416)[int(c.block_table[2, 0]) * 16] = mi.quantize_fp4_slots(torch.full((576,), 0.5).bfloat16())
    c.indices[3, 0, :40] = torch.arange(40, dtype=torch.int32) * 10 ** 7     # past everything
    c.indices[3, 0, 40:80] = -(2 ** 31)
    c.block_table[4, 1] = u.shape[0]               # outside the pool
    c.block_table[4, 2] = -5
    _check(smla, c, u, f"fp4 decode masked h={h_q}")
    out, lse = _run(smla, c, u)
    assert bool(torch.isneginf(lse[0]).all()) and bool((out[0] == 0).all())
    assert bool(torch.isneginf(lse[1]).all()) and bool(torch.isneginf(lse[2, 1]).all())
    # 0.5 / 6 rounds to the scale 11 * 2^-7: the row stands for 6 * 11 * 2^-7
    assert bool((out[2, 0] == 0.515625).all())


def test_empty_pool_and_table(smla):
    q = torch.randn(2, 1, 8, 576, device=DEV).bfloat16()
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    u = torch.zeros(0, 64, 416, dtype=torch.uint8, device=DEV)
    o, l = smla.sparse_mla_decode_fp4(q, u, z(2, 3), z(2) + 5, z(2, 1, 8), 0.1)
    assert bool((o == 0).all()) and bool(torch.isneginf(l).all())
    o, l = smla.sparse_mla_decode_fp4(q[:0], u, z(0, 3), z(0), z(0, 1, 8), 0.1)
    assert o.shape == (0, 1, 8, 512)


@pytest.mark.parametrize("h_q", [8, 64])
def test_a_nan_scale_reads_as_nan(smla, h_q):
    c, u = mi.decode_case_fp4(985, batch=1, s_next=1, h_q=h_q, lo=100, hi=100, topk=64, page=64, spare_pages=1)
    pos = int(c.indices[0, 0, 0])
    u.view(-1, 416)[int(c.block_table[0, pos // 64]) * 64 + pos % 64, 256 + 5] = 0x7F
    out, lse = _run(smla, c, u)
    assert bool(torch.isnan(lse).all()) and bool(torch.isnan(out).all())


@pytest.mark.parametrize("h_q", [8, 64])
def test_queries_of_any_size(smla, h_q):
    """Queries scaled by a power of two with sm_scale scaled back: the same
    scores, so the same results (f16 operands must not over- or underflow)."""
    c, u = mi.decode_case_fp4(990, batch=2, s_next=1, h_q=h_q, lo=200, hi=300, topk=128, page=64, spare_pages=1)
    o, l = _run(smla, c, u)
    for f in (2.0 ** -40, 2.0 ** 30):
        q = c.q
        c.q, c.sm_scale = (q.float() * f).bfloat16(), c.sm_scale / f
        o2, l2 = _run(smla, c, u)
        c.q, c.sm_scale = q, c.sm_scale * f
        assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("h_q,s_next", [(8, 2), (64, 2), (8, 90), (64, 90)])
def test_workspace_streams_and_graphs(smla, h_q, s_next):
    """A dirty workspace of exactly the size asked for (few tokens ask for none:
    their pieces meet in a cluster); two decodes on two streams with their own
    workspaces; two captured graphs replayed."""
    cases = [mi.decode_case_fp4(995 + k, batch=2, s_next=s_next, h_q=h_q, lo=2100, hi=3000, topk=2048, spare_pages=2)
             for k in range(2)]
    want = [_run(smla, c, u) for c, u in cases]
    need = smla.decode_fp4_workspace_size(2, s_next, h_q, 2048)
    assert need > 0 if s_next == 90 else (need == 0 or h_q > 8)
    ws = [torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device=DEV) for _ in cases]
    args = [([t.to(DEV) for t in (c.q, u, c.block_table, c.cache_seqlens, c.indices)], c.sm_scale) for c, u in cases]
    if need:
        with pytest.raises(smla.SparseMLAError):
            smla.sparse_mla_decode_fp4(*args[0][0], args[0][1], workspace=ws[0][:need - 16])
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for (a, sc), w, s in zip(args, ws, streams):
        for _ in range(3):
            with torch.cuda.stream(s):
                r = smla.sparse_mla_decode_fp4(*a, sc, workspace=w)
        got.append(r)
    torch.cuda.synchronize()
    for r, x in zip(got, want):
        assert torch.equal(r[0], x[0]) and torch.equal(r[1], x[1])
    graphs = []
    for (a, sc), w in zip(args, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = smla.sparse_mla_decode_fp4(*a, sc, workspace=w)
        graphs.append((g, r))
    for _ in range(2):
        for g, r in graphs:
            r[0].zero_()
            g.replay()
        torch.cuda.synchronize()
        for (g, r), x in zip(graphs, want):
            assert torch.equal(r[0], x[0]) and torch.equal(r[1], x[1])


def test_a_given_stream_owns_what_the_call_allocates(smla):
    """stream=s with the call's own outputs and workspace.  s held up: memory
    that the current stream takes next is not the call's workspace.  The current
    stream held up: the outputs are not memory that it has yet to write."""
    c, u = mi.decode_case_fp4(51, batch=2, s_next=90, h_q=8, lo=2100, hi=3000, topk=2048, spare_pages=2)
    want = _run(smla, c, u)
    need = smla.decode_fp4_workspace_size(2, 90, 8, 2048)
    assert need > 0
    a = [t.to(DEV) for t in (c.q, u, c.block_table, c.cache_seqlens, c.indices)]
    s = torch.cuda.Stream()

    def nan():
        return [torch.full((need // 4,), float("nan"), device=DEV), torch.full_like(want[0], float("nan")),
                torch.full_like(want[1], float("nan"))]

    for late in (s, torch.cuda.current_stream()):
        smla.sparse_mla_decode_fp4(*a, c.sm_scale, stream=s)   # every block of memory is there before the streams wait
        nan()
        torch.cuda.synchronize()
        with torch.cuda.stream(late):
            torch.cuda._sleep(100_000_000)   # some 50 ms
        if late is not s:
            nan()                            # written late, free at once
        got = smla.sparse_mla_decode_fp4(*a, c.sm_scale, stream=s)
        took = nan() if late is s else []
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert all(bool(torch.isnan(t).all()) for t in took)
        del got, took

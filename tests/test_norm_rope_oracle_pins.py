"""Pins of the 4-bit cache's and of mla_norm_rope's float64 oracles (CPU)."""
import numpy as np
import pytest
import torch

import mla_inputs as mi
from oracle import fp4_kv_oracle as f4
from oracle import norm_rope_oracle as nro
from oracle import sparse_mla_oracle as orc


def test_e2m1_values():
    assert list(f4.E2M1_TABLE[:8]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert np.array_equal(f4.E2M1_TABLE[8:], -f4.E2M1_TABLE[:8])


def test_slot_by_hand():
    slot = np.zeros(416, dtype=np.uint8)
    slot[0] = 0x72            # codes 0 and 1: 1.0 and 6.0
    slot[255] = 0x9F          # codes 510 and 511: -6.0 and -0.5
    slot[256] = 0x40          # scale 0: 2.0
    slot[287] = 0x30          # scale 31: 0.5
    slot[288:290] = [0x80, 0x3F]   # bf16 1.0
    slot[414:416] = [0x00, 0xC0]   # bf16 -2.0
    x = f4.dequantize_slots(slot, 0.5)
    want = np.zeros(576)
    want[[0, 1, 510, 511, 512, 575]] = [1.0, 6.0, -1.5, -0.125, 1.0, -2.0]
    assert np.array_equal(x, want)


def test_generator_slots_read_back():
    """The generator's slots stand for values within half a step of the rows."""
    x = mi.randn_bf16(torch.Generator().manual_seed(5), (50, 576))
    for ks in (1.0, 0.3):
        y = f4.dequantize_slots(mi.quantize_fp4_slots(x, ks), ks)
        v = x.double().numpy()
        assert np.array_equal(y[:, 512:], v[:, 512:])
        top = np.abs(v[:, :512]).reshape(50, 32, 16).max(-1, keepdims=True).repeat(16, -1).reshape(50, 512)
        # scale rounding moves the largest by at most 1/16, half of the widest step is 1/6 of it
        assert np.all(np.abs(y[:, :512] - v[:, :512]) <= top * (1 / 6 * 17 / 16 + 1e-6))


def test_decode_equals_decode_of_the_rows():
    c, u = mi.decode_case_fp4(31, batch=2, s_next=2, h_q=4, lo=20, hi=90, topk=40, page=16, spare_pages=2, kv_scale=0.5)
    o, l = f4.sparse_mla_decode_fp4(c.q, u, c.block_table, c.cache_seqlens, c.indices, c.sm_scale, 16, 0.5)
    x = f4.dequantize_slots(u, 0.5)
    po, pl = orc.sparse_mla_decode(c.q, x, c.block_table, c.cache_seqlens, c.indices, c.sm_scale, 16)
    assert np.array_equal(o, po) and np.array_equal(l, pl) and np.all(np.isfinite(l))


def test_bf16_rounding_is_torchs():
    y = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * torch.logspace(-5, 5, 20000)
    assert np.array_equal(nro.round_bf16(y.double().numpy()), y.bfloat16().double().numpy())
    tie = 1 + np.array([1, 3]) / 256.0          # halfway: to even
    assert np.array_equal(nro.round_bf16(tie), [1.0, 1 + 4 / 256.0])


@pytest.mark.parametrize("grid", [nro.E2M1_POS, nro.E4M3_POS])
def test_nearest_code_on_borders(grid):
    mid = (grid[1:] + grid[:-1]) / 2
    even = np.where(np.arange(len(mid)) % 2 == 0, np.arange(len(mid)), np.arange(len(mid)) + 1)
    assert np.array_equal(nro.nearest_code(mid, grid), even)
    assert np.array_equal(nro.nearest_code(np.nextafter(mid, 0), grid), np.arange(len(mid)))
    assert np.array_equal(nro.nearest_code(np.nextafter(mid, 1e9), grid), np.arange(len(mid)) + 1)
    assert nro.nearest_code(grid[-1] * 1.2, grid) == len(grid) - 1


def test_fp8_scale_rule():
    y = np.zeros((1, 512))
    y[0, 0], y[0, 128], y[0, 256] = 448.0, 450.0, 2.0 ** -80
    _, scale, val = nro.quantize_fp8(y)
    assert np.array_equal(scale[0], [1.0, 2.0, 2.0 ** -64, 1.0])
    assert val[0, 0] == 448 and val[0, 128] == 448 and val[0, 256] == 0


def test_codes_match_the_generators_writer():
    """quantize_fp4 against the generator's own writer: the same scales, the
    same codes but for halfway values (which the generator sends down)."""
    x = mi.randn_bf16(torch.Generator().manual_seed(9), (64, 576))
    u = mi.quantize_fp4_slots(x).numpy()
    c, s, v = nro.quantize_fp4(x.double().numpy()[:, :512])
    assert np.array_equal(s, u[:, 256:288])
    y = f4.dequantize_slots(u)[:, :512]
    d = np.abs(np.abs(y - x.double().numpy()[:, :512]) - np.abs(v - x.double().numpy()[:, :512]))
    assert d.max() == 0.0


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("normed", [True, False])
def test_gradients_against_differences(interleaved, normed):
    rng = np.random.default_rng(3)
    x, dy = rng.normal(size=(3, 576)), rng.normal(size=(3, 576))
    w = 1 + 0.2 * rng.normal(size=512) if normed else None
    cs = mi.rope_table(10).double().numpy()[[0, 3, 9]]
    f = lambda x, w: (nro.norm_rope(x, cs, w, 1e-6, interleaved) * dy).sum()  # noqa: E731
    dx, dw = nro.norm_rope_bwd(x, dy, cs, w, 1e-6, interleaved)
    for _ in range(6):
        u = rng.normal(size=x.shape)
        h = 1e-6
        assert abs((f(x + h * u, w) - f(x - h * u, w)) / (2 * h) - (dx * u).sum()) < 1e-6 * np.abs(dx * u).sum()
        if normed:
            v = rng.normal(size=512)
            assert abs((f(x, w + h * v) - f(x, w - h * v)) / (2 * h) - (dw * v).sum()) < 1e-6 * np.abs(dw * v).sum()


def test_rotation_keeps_lengths_and_planes():
    rng = np.random.default_rng(4)
    r = rng.normal(size=(7, 64))
    cs = mi.rope_table(500).double().numpy()[[0, 1, 2, 50, 100, 200, 499]]
    for il in (True, False):
        t = nro.rotate(r, cs, il)
        assert np.allclose((t * t).sum(-1), (r * r).sum(-1), rtol=1e-6)
        assert np.allclose(nro.rotate(t, cs, il, back=True), r, atol=1e-6)
        assert np.array_equal(t[0], r[0])      # position 0
    assert nro.planes(True)[1][0] == 1 and nro.planes(False)[1][0] == 32

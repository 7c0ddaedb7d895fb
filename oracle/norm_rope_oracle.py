"""CPU float64 oracle of mla_norm_rope and its gradients.

TEST INFRASTRUCTURE ONLY: plain NumPy from the definitions, sharing no code
with the CUDA path.  A row x has 512 latent values a and 64 rotated values r:

    a' = a / sqrt(mean(a^2) + eps) * w          (no w: a' = a)
    plane i of r, (x, y) -> (x cos - y sin, y cos + x sin)

The latent row's a' is rounded to bf16 (8 significant bits, ties to even) and
then to the cache's codes, the nearest of the format's values (ties to the
even code), found here by comparing with every value.  The 4-bit cache's factor
is an fp32 number, and what is formed with it before a code is chosen (6 factors,
a group's step, the quotients) is rounded to fp32 as its definition says.

Pins (tests/test_norm_rope_oracle_pins.py): the rounding against torch's; the
codes against brute force on the borders; the gradients against differences.
"""
from __future__ import annotations

import numpy as np

from oracle.fp4_kv_oracle import E2M1_TABLE
from oracle.fp8_kv_oracle import E4M3_TABLE

E2M1_POS = E2M1_TABLE[:8]
E4M3_POS = E4M3_TABLE[:127]


def round_bf16(y):
    """Nearest bf16 value (normal range), ties to even, in float64."""
    y = np.asarray(y, dtype=np.float64)
    m, e = np.frexp(y)
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(y), np.ldexp(np.rint(np.where(np.isfinite(y), m, 0.0) * 256.0), e - 8), y)


def nearest_code(mag, grid):
    """Code of the nearest grid value (grid ascending, code = index), ties to
    the even code, above the last value the last code."""
    mag = np.asarray(mag, dtype=np.float64)
    hi = np.clip(np.searchsorted(grid, mag), 1, len(grid) - 1)
    below, above = mag - grid[hi - 1], grid[hi] - mag
    return np.where((below < above) | ((below == above) & (hi % 2 == 1)), hi - 1, hi)


def planes(interleaved):
    i = np.arange(32)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + 32)


def rotate(r, cos_sin, interleaved, back=False):
    """r [..., 64], cos_sin [..., 64]."""
    a, b = planes(interleaved)
    c, s = cos_sin[..., :32], cos_sin[..., 32:] * (-1.0 if back else 1.0)
    out = np.empty_like(r)
    out[..., a] = r[..., a] * c - r[..., b] * s
    out[..., b] = r[..., b] * c + r[..., a] * s
    return out


def rms_norm(a, w, eps):
    return a if w is None else a / np.sqrt((a * a).mean(axis=-1, keepdims=True) + eps) * w


def quantize_fp8(y):
    """y [n, 512] bf16 values -> (codes uint8 [n, 512], scales [n, 4], values)."""
    t = y.reshape(-1, 4, 128)
    bad = ~np.isfinite(t).all(axis=-1)
    t = np.where(bad[..., None], 0.0, t)
    top = np.abs(t).max(axis=-1)
    scale = np.ones_like(top)
    for k in range(31, -65, -1):   # the smallest 2^k with top / 2^k <= 448
        scale = np.where((top > 0) & (top <= 448.0 * 2.0 ** k), 2.0 ** k, scale)
    scale = np.where(top > 448.0 * 2.0 ** 31, 2.0 ** 31, scale)
    code = nearest_code(np.abs(t) / scale[..., None], E4M3_POS).astype(np.uint8)
    val = np.copysign(E4M3_POS[code], t) * scale[..., None]
    code = code | (np.signbit(t).astype(np.uint8) << 7)
    code[bad] = 0
    scale = np.where(bad, np.nan, scale)
    val[bad] = np.nan
    return code.reshape(-1, 512), scale, val.reshape(-1, 512)


def quantize_fp4(y, kv_scale=1.0):
    """y [n, 512] bf16 values -> (code bytes [n, 256], scale bytes [n, 32], values)."""
    f = np.float32(kv_scale)
    f6 = np.float32(6.0 * np.float64(f))
    t = y.reshape(-1, 32, 16)
    bad = ~np.isfinite(t).all(axis=-1)
    t = np.where(bad[..., None], 0.0, t)
    top = np.abs(t).max(axis=-1)
    with np.errstate(over="ignore", under="ignore"):
        sc = nearest_code(np.clip(top.astype(np.float32) / f6, 2.0 ** -9, 448.0), E4M3_POS).astype(np.uint8)
        step = E4M3_POS[sc].astype(np.float32) * f
        code = nearest_code(np.abs(t).astype(np.float32) / step[..., None], E2M1_POS).astype(np.uint8)
    step = step.astype(np.float64)
    val = np.copysign(E2M1_POS[code], t) * step[..., None]
    code = (code | (np.signbit(t).astype(np.uint8) << 3))
    code[bad] = 0
    val[bad] = np.nan
    sc[bad] = 0x7F
    c = code.reshape(-1, 256, 2)
    return c[..., 0] | (c[..., 1] << 4), sc, val.reshape(-1, 512)


def norm_rope(x, cos_sin, w, eps, interleaved):
    """Rows x [..., 576] float64 with their angles cos_sin [..., 64], unrounded."""
    return np.concatenate([rms_norm(x[..., :512], w, eps), rotate(x[..., 512:], cos_sin, interleaved)], axis=-1)


def norm_rope_bwd(x, dy, cos_sin, w, eps, interleaved):
    """(dx, dw) of rows x, dy [..., 576] float64 (dw None where w is)."""
    a, g = x[..., :512], dy[..., :512]
    dr = rotate(dy[..., 512:], cos_sin, interleaved, back=True)
    if w is None:
        return np.concatenate([g, dr], axis=-1), None
    r = 1.0 / np.sqrt((a * a).mean(axis=-1, keepdims=True) + eps)
    xhat = a * r
    dw = (g * xhat).reshape(-1, 512).sum(axis=0)
    g = g * w
    return np.concatenate([r * (g - xhat * (g * xhat).mean(axis=-1, keepdims=True)), dr], axis=-1), dw

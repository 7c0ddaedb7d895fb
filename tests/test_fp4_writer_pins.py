"""Pins of the 4-bit cache writer's oracle where the factor has many bits (CPU)."""
import numpy as np
import torch

import mla_inputs as mi
from oracle import norm_rope_oracle as nro


def test_codes_of_a_factor_with_many_bits_by_hand():
    """The factor 0.3 as fp32: every product and quotient rounded to fp32 before
    the code is chosen, checked value by value in plain Python arithmetic."""
    f = float(np.float32(0.3))
    r32 = lambda v: float(np.float32(v))  # noqa: E731
    x = mi.randn_bf16(torch.Generator().manual_seed(10), (40, 512)).double().numpy()
    c, s, v = nro.quantize_fp4(x, 0.3)
    exact = fp32 = 0
    for row in range(40):
        for g in range(32):
            t = np.abs(x[row, 16 * g:16 * g + 16])
            sc = min(range(1, 127), key=lambda k: (abs(nro.E4M3_POS[k] - r32(t.max() / r32(6 * f))), k % 2))
            assert s[row, g] == sc
            step = r32(nro.E4M3_POS[sc] * f)
            for i, a in enumerate(t):
                near = lambda q: min(range(8), key=lambda k: (abs(nro.E2M1_POS[k] - q), k % 2))  # noqa: E731
                code = (c[row, 8 * g + i // 2] >> (4 * (i % 2))) & 7
                assert code == near(r32(a / step))
                exact += code != near(a / (nro.E4M3_POS[sc] * f))
                fp32 += 1
    assert 0 < exact < fp32 / 100     # the rounding decides some codes, few

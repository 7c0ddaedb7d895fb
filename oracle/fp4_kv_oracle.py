"""CPU float64 oracle of the sparse-MLA decode over a 4-bit KV cache.

TEST INFRASTRUCTURE ONLY, as fp8_kv_oracle.  One cache slot is 416 bytes:

    bytes [0, 256)    512 e2m1 codes, code 2i in the low and 2i + 1 in the high
                      four bits of byte i;
    bytes [256, 288)  32 e4m3 scales (codes 0x7F / 0xFF are NaN); scale k
                      applies to codes 16 k .. 16 k + 15;
    bytes [288, 416)  64 bf16 values (little-endian).

    x[d] = e2m1(code[d]) * e4m3(scale[d // 16]) * kv_scale      d < 512

and the decode is the paged decode of sparse_mla_oracle over those rows.

e2m1: bit 3 sign s, bits 2..1 exponent e, bit 0 mantissa m, bias 1:
    e = 0:       (-1)^s * m / 2
    e = 1 .. 3:  (-1)^s * 2^(e - 1) * (1 + m / 2)
"""
from __future__ import annotations

import numpy as np

from oracle import sparse_mla_oracle as orc
from oracle.fp8_kv_oracle import E4M3_TABLE

SLOT_BYTES = 416
SCALE_OFF = 256
ROPE_OFF = 288
GROUP = 16


def e2m1_value(code: int) -> float:
    """The value of one e2m1 code, from the format definition."""
    s = -1.0 if (code >> 3) & 1 else 1.0
    e, m = (code >> 1) & 3, code & 1
    return s * (m / 2.0 if e == 0 else 2.0 ** (e - 1) * (1.0 + m / 2.0))


E2M1_TABLE = np.array([e2m1_value(c) for c in range(16)], dtype=np.float64)


def dequantize_slots(cache_u8, kv_scale: float = 1.0) -> np.ndarray:
    """uint8 [..., 416] -> float64 [..., 576] latent rows."""
    import torch
    b = cache_u8.cpu().numpy() if isinstance(cache_u8, torch.Tensor) else np.asarray(cache_u8)
    b = np.ascontiguousarray(b, dtype=np.uint8)
    lead = b.shape[:-1]
    flat = b.reshape(-1, SLOT_BYTES)
    out = np.empty((flat.shape[0], 576), dtype=np.float64)
    out[:, 0:512:2] = E2M1_TABLE[flat[:, :SCALE_OFF] & 15]
    out[:, 1:512:2] = E2M1_TABLE[flat[:, :SCALE_OFF] >> 4]
    scales = E4M3_TABLE[flat[:, SCALE_OFF:ROPE_OFF]]
    out[:, :512] *= np.repeat(scales, GROUP, axis=1) * float(np.float32(kv_scale))
    bits = flat[:, ROPE_OFF:].copy().view("<u2").astype(np.uint32) << 16
    out[:, 512:] = bits.astype(np.uint32).view(np.float32).astype(np.float64)
    return out.reshape(*lead, 576)


def sparse_mla_decode_fp4(q, cache_u8, block_table, cache_seqlens, indices, sm_scale: float, page_size: int = 64,
                          kv_scale: float = 1.0, d_v: int = 512, tokens=None):
    """Paged decode over a 4-bit cache uint8 [num_blocks, page_size, 416]."""
    return orc.sparse_mla_decode(q, dequantize_slots(cache_u8, kv_scale), block_table, cache_seqlens, indices,
                                 sm_scale, page_size, d_v, tokens=tokens)

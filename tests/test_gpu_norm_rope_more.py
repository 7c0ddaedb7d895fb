"""mla_norm_rope and mla_norm_rope_bwd: cache factors that are not powers of
two, byte by byte; rows at the ends of the norm's range; padding rows of
outputs that the call allocates; more rows than the backward's warps."""
import numpy as np
import pytest
import torch

import mla_inputs as mi
from oracle import fp4_kv_oracle as f4
from oracle import norm_rope_oracle as nro
from tests import test_gpu_norm_rope as base

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def smla(cuda_lib):
    import serving_sparse_mla_gb300 as pkg
    pkg.clear_device_error()
    yield pkg
    assert pkg.get_device_error() == 0


@pytest.mark.parametrize("normed", [True, False])
@pytest.mark.parametrize("ks", [0.3, 0.1, 0.7, 1.7, 0.01, 1 / 3, 12345.678, 3e-19, 1.7e19])
def test_cache_bytes_with_any_factor(smla, ks, normed):
    """Scales and codes where the factor rounds: unnormed rows have few bits, so
    that many quotients lie at a border."""
    base._run_and_check(smla, 91, 700, 1, "fp4", True, q_norm=False, kv_norm=normed, kv_scale=ks, page=64)

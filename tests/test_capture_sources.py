"""The sources of the attention's and the indexer's kernels are apart from those
around the latent cache: a capture is shown with a benchmark's line while its
family's sources hash as they did when it was taken (CPU)."""
import os

import bench
from serving_sparse_mla_gb300 import build


def test_the_families_sources_hold_nothing_of_the_latent_caches_kernels():
    for name in {n for names in bench.KERNEL_SOURCES.values() for n in names}:
        text = open(os.path.join(build.CSRC, name)).read()
        for word in ("fp4", "f4_", "norm_rope", "latent_api"):
            assert word not in text, (name, word)


def test_the_build_depends_on_every_source():
    assert sorted(build.DEPS) == sorted(f for f in os.listdir(build.CSRC) if f.endswith((".cu", ".cuh")))

"""Set-up and size checks of the C entry points on a stand-in device (no GPU):
the library's one source is compiled with the runtime's queries replaced, so
that a device can be described that refuses some of them.  Calls that would
launch are not made."""
import ctypes
import subprocess
import sys

import pytest

from serving_sparse_mla_gb300 import build

SOURCE = r"""
#include <cuda_runtime.h>
#include <type_traits>
#include "fp4_decode_kernel.cuh"
namespace fake {
int refuse_clusters, refuse_fp4, asked;
cudaError_t pending;   // what cudaGetLastError would report to the next launch
inline cudaError_t fail(cudaError_t e) { return pending = e; }
inline cudaError_t device(int* d) { *d = 0; return cudaSuccess; }
inline cudaError_t attribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
  return cudaSuccess;
}
template <class T>
cudaError_t function(T*, cudaFuncAttribute, int) {
  if (!std::is_same<T, void(const smla::Fp4Params)>::value && !std::is_same<T, void(smla::Fp4Params)>::value) return cudaSuccess;
  ++asked;
  return refuse_fp4 ? fail(cudaErrorInvalidValue) : cudaSuccess;
}
template <class T>
cudaError_t clusters(int* n, T*, const cudaLaunchConfig_t* c) {
  ++asked;
  const int size = static_cast<int>(c->attrs[0].val.clusterDim.x);
  if (size >= refuse_clusters && refuse_clusters > 0) return fail(cudaErrorInvalidClusterSize);
  *n = 152 / size - 1;
  return cudaSuccess;
}
inline cudaError_t last() { const cudaError_t e = pending; pending = cudaSuccess; return e; }
}  // namespace fake
#define cudaGetDevice fake::device
#define cudaDeviceGetAttribute fake::attribute
#define cudaFuncSetAttribute fake::function
#define cudaOccupancyMaxActiveClusters fake::clusters
#define cudaGetLastError fake::last
#include "library.cu"
extern "C" {
void fake_refuse(int clusters, int fp4) { fake::refuse_clusters = clusters; fake::refuse_fp4 = fp4; }
int fake_pending() { return fake::pending; }
int fake_asked() { return fake::asked; }
}
"""


@pytest.fixture(scope="module")
def lib_path(tmp_path_factory):
    d = tmp_path_factory.mktemp("setup")
    (d / "fake.cu").write_text(SOURCE)
    # host code only matters: device code stays PTX, without optimisation
    cmd = [build.nvcc_path(), "-gencode", "arch=compute_103a,code=compute_103a", "-O1", "-Xcicc", "-O0", "-std=c++17",
           "-Xcompiler", "-fPIC", "-shared", "-I", build.INCLUDE, "-I", build.CSRC, "-o", str(d / "fake.so"),
           str(d / "fake.cu")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(d / "fake.so")


def _run(lib_path, refuse, body):
    """`body` in a process of its own (the set-up is made once per process)."""
    code = f"""
import ctypes, sys
from serving_sparse_mla_gb300.binding import SIGNATURES
lib = ctypes.CDLL({lib_path!r})
for n, (res, args) in SIGNATURES.items():
    f = getattr(lib, n); f.restype, f.argtypes = res, args
lib.fake_refuse({refuse})
def fwd(): return lib.sparse_mla_fwd(16, 16, 16, 0.1, 16, 16, 0, 8, 8, 576, 512, 64, None)
def norm(): return lib.mla_norm_rope(16, 4608, 576, 16, 576, 16, 16, 9, None, 16, 1e-6, 1, 16, 16, 16, 2, 1.0, 16, 9, 0, 8, 576, None)
def fp4(n=0, h=8, topk=64, nb=4, ws=None, wb=0):
    return lib.sparse_mla_decode_fp4(16, 16, 16, 16, 16, 0.1, 1.0, 16, 16, n, 1, h, 576, 512, topk, 64, 4, nb, ws, wb, None)
def need(n, h, topk): return lib.sparse_mla_decode_fp4_workspace_size(n, 1, h, 512, topk)
{body}
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=build.ROOT)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("refuse", ["16, 0", "2, 0", "0, 1", "2, 1"])
def test_other_calls_work_where_the_4bit_kernels_are_refused(lib_path, refuse):
    """Neither a cluster size that the device does not take nor any other
    refusal of the 4-bit kernels' set-up stops the library's other calls."""
    _run(lib_path, refuse, """
assert fwd() == 0 and norm() == 0, (fwd(), norm())
assert lib.fake_asked() == 0 and lib.fake_pending() == 0
""")


@pytest.mark.parametrize("refuse", ["16, 0", "4, 0", "2, 0"])
def test_a_refused_cluster_size_is_not_used(lib_path, refuse):
    """The 4-bit decode takes smaller clusters, or ranges and a workspace, where
    the device refuses a size; no error is left behind for the next launch."""
    _run(lib_path, refuse, f"""
refused = ({refuse})[0]
assert fp4() == 0 and fwd() == 0
# 16 tokens of 2048 entries go to clusters of 8, 50 of 500 to clusters of 2: no workspace
assert (need(16, 8, 2048) > 0) == (refused <= 8) and (need(50, 8, 500) > 0) == (refused <= 2)
assert need(200, 8, 2048) > 0
assert lib.fake_pending() == 0
""")


def test_the_4bit_decode_itself_says_that_it_was_refused(lib_path):
    _run(lib_path, "0, 1", """
assert fp4(1) == 4 and need(1, 8, 2048) == 0 and fwd() == 0
assert lib.fake_pending() == 0
""")


def test_ctas_with_more_blocks_than_an_int_counts_are_refused(lib_path):
    """60 million heads over a list of 2^31 entries is 10^11 blocks for a CTA."""
    _run(lib_path, "0, 0", """
big = 2 ** 31 - 1025
for n, h, topk in ((1, 60_000_000, big), (10, 6_000_000, big), (16_000_000, 8, big)):
    assert need(n, h, topk) == 0, (n, h, topk)
    assert fp4(n, h, topk) == 1, (n, h, topk)
for n, h, topk in ((2000, 64, 100_000), (1, 128, big), (500_000, 128, 2048)):
    assert need(n, h, topk) > 0, (n, h, topk)
""")


def test_the_stand_in_has_every_entry_point(lib_path):
    from serving_sparse_mla_gb300.binding import SIGNATURES
    lib = ctypes.CDLL(lib_path)
    assert all(hasattr(lib, n) for n in SIGNATURES)

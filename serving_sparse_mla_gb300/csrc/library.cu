// The library's one translation unit.  The entry points of the attention and the
// indexer and those around the latent cache are two files, so that a capture of a
// kernel, recorded with the hash of its family's sources (bench.py), stays current while
// the other family changes.
#include "sparse_mla_api.cu"

#include "latent_api.cuh"

// The library's one translation unit.  The entry points of the attention and the
// indexer, those around the latent cache and those around a layer's dense attention are
// three files, so that a capture of a kernel, recorded with the hash of its family's
// sources (bench.py), stays current while the other families change.
#include "sparse_mla_api.cu"

#include "latent_api.cuh"

#include "layer_api.cuh"

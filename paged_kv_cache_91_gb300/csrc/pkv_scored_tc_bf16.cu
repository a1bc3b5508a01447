// Scored paged attention on the tensor-memory tile: bf16 pools.
#include "pkv_internal.h"
#include "pkv_scored_tc.cuh"

namespace pkv {

cudaError_t scored_tc_bf16(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, int head_dim, int block_size, int num_seqs, cudaStream_t stream) {
  using T = __nv_bfloat16;
  if (head_dim == 128) {
    if (block_size == 16) return launch_scored_tc<T, 128, 16, false>(p, sc, kmap, vmap, num_seqs, stream);
    if (block_size == 8) return launch_scored_tc<T, 128, 8, false>(p, sc, kmap, vmap, num_seqs, stream);
    if (block_size == 32) return launch_scored_tc<T, 128, 32, false>(p, sc, kmap, vmap, num_seqs, stream);
  } else if (head_dim == 64) {
    if (block_size == 16) return launch_scored_tc<T, 64, 16, false>(p, sc, kmap, vmap, num_seqs, stream);
    if (block_size == 8) return launch_scored_tc<T, 64, 8, false>(p, sc, kmap, vmap, num_seqs, stream);
    if (block_size == 32) return launch_scored_tc<T, 64, 32, false>(p, sc, kmap, vmap, num_seqs, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pkv

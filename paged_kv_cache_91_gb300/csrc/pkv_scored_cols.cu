// Scored paged attention on the 8-column tile: f16 and bf16 pools.
#include "pkv_internal.h"
#include "pkv_scored_cols.cuh"

namespace pkv {

template <typename T>
static cudaError_t dispatch(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, int head_dim, int block_size, int num_seqs, cudaStream_t stream) {
  if (head_dim == 128) {
    if (block_size == 16) return launch_scored_cols<ScoredTile<T, 128, 16>, T>(p, sc, kmap, vmap, num_seqs, stream);
    if (block_size == 8) return launch_scored_cols<ScoredTile<T, 128, 8>, T>(p, sc, kmap, vmap, num_seqs, stream);
    if (block_size == 32) return launch_scored_cols<ScoredTile<T, 128, 32>, T>(p, sc, kmap, vmap, num_seqs, stream);
  } else if (head_dim == 64) {
    if (block_size == 16) return launch_scored_cols<ScoredTile<T, 64, 16>, T>(p, sc, kmap, vmap, num_seqs, stream);
    if (block_size == 8) return launch_scored_cols<ScoredTile<T, 64, 8>, T>(p, sc, kmap, vmap, num_seqs, stream);
    if (block_size == 32) return launch_scored_cols<ScoredTile<T, 64, 32>, T>(p, sc, kmap, vmap, num_seqs, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t scored_cols_16(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, bool f16, int head_dim, int block_size, int num_seqs,
                           cudaStream_t stream) {
  return f16 ? dispatch<__half>(p, sc, kmap, vmap, head_dim, block_size, num_seqs, stream)
             : dispatch<__nv_bfloat16>(p, sc, kmap, vmap, head_dim, block_size, num_seqs, stream);
}

}  // namespace pkv

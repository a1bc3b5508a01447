// Scored paged attention on the 8-column tile: FP8 (E4M3) pools, head_dim 128.
#include "pkv_internal.h"
#include "pkv_scored_cols.cuh"

namespace pkv {

template <typename T>
static cudaError_t dispatch(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, int block_size, int num_seqs, cudaStream_t stream) {
  constexpr int R = PKV_MMA_FP8_RING_BYTES, D = 128;
  using C = __nv_fp8_e4m3;
  if (block_size == 16) return launch_scored_cols<ScoredTileE4M3<T, D, 16>, C, R>(p, sc, kmap, vmap, num_seqs, stream);
  if (block_size == 8) return launch_scored_cols<ScoredTileE4M3<T, D, 8>, C, R>(p, sc, kmap, vmap, num_seqs, stream);
  if (block_size == 32) return launch_scored_cols<ScoredTileE4M3<T, D, 32>, C, R>(p, sc, kmap, vmap, num_seqs, stream);
  return cudaErrorInvalidValue;
}

cudaError_t scored_cols_fp8(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, bool f16, int block_size, int num_seqs, cudaStream_t stream) {
  return f16 ? dispatch<__half>(p, sc, kmap, vmap, block_size, num_seqs, stream)
             : dispatch<__nv_bfloat16>(p, sc, kmap, vmap, block_size, num_seqs, stream);
}

}  // namespace pkv

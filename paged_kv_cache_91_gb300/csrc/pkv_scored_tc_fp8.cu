// Scored paged attention on the tensor-memory tile: FP8 (E4M3) pools, head_dim 128.
#include "pkv_internal.h"
#include "pkv_scored_tc.cuh"

namespace pkv {

template <typename T>
static cudaError_t dispatch(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, int block_size, int num_seqs, cudaStream_t stream) {
  if (block_size == 16) return launch_scored_tc<T, 128, 16, true>(p, sc, kmap, vmap, num_seqs, stream);
  if (block_size == 8) return launch_scored_tc<T, 128, 8, true>(p, sc, kmap, vmap, num_seqs, stream);
  if (block_size == 32) return launch_scored_tc<T, 128, 32, true>(p, sc, kmap, vmap, num_seqs, stream);
  return cudaErrorInvalidValue;
}

cudaError_t scored_tc_fp8(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                          const CUtensorMap& vmap, bool f16, int block_size, int num_seqs, cudaStream_t stream) {
  return f16 ? dispatch<__half>(p, sc, kmap, vmap, block_size, num_seqs, stream)
             : dispatch<__nv_bfloat16>(p, sc, kmap, vmap, block_size, num_seqs, stream);
}

}  // namespace pkv

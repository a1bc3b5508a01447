// Tree attention on the tensor-memory tile: dispatch over the pool's type, head_dim and block size.
#pragma once

#include "pkv_scored_tc.cuh"

namespace pkv {

template <typename T, int D, bool F8>
cudaError_t dispatch_tree_block(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, int block_size, int num_seqs, cudaStream_t stream) {
  if (block_size == 16) return launch_tree_tc<T, D, 16, F8>(p, sc, kmap, vmap, num_seqs, stream);
  if (block_size == 8) return launch_tree_tc<T, D, 8, F8>(p, sc, kmap, vmap, num_seqs, stream);
  if (block_size == 32) return launch_tree_tc<T, D, 32, F8>(p, sc, kmap, vmap, num_seqs, stream);
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t dispatch_tree_tc(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, bool fp8, int head_dim, int block_size, int num_seqs,
                             cudaStream_t stream) {
  if (fp8) return dispatch_tree_block<T, 128, true>(p, sc, kmap, vmap, block_size, num_seqs, stream);
  if (head_dim == 128) return dispatch_tree_block<T, 128, false>(p, sc, kmap, vmap, block_size, num_seqs, stream);
  if (head_dim == 64) return dispatch_tree_block<T, 64, false>(p, sc, kmap, vmap, block_size, num_seqs, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkv

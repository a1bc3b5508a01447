// Tree attention on the tensor-memory tile: f16 queries.
#include "pkv_internal.h"
#include "pkv_tree_tc.cuh"

namespace pkv {

cudaError_t tree_tc_f16(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap, const CUtensorMap& vmap,
                     bool fp8, int head_dim, int block_size, int num_seqs, cudaStream_t stream) {
  return dispatch_tree_tc<__half>(p, sc, kmap, vmap, fp8, head_dim, block_size, num_seqs, stream);
}

}  // namespace pkv

// Tree attention on the 8-column tile.
#include "pkv_internal.h"
#include "pkv_scored_cols.cuh"

namespace pkv {

template <template <typename, int, int> class Tile, typename T, typename C, int D, int RING>
static cudaError_t of_block(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, int block_size, int num_seqs, cudaStream_t stream) {
  if (block_size == 16) return launch_scored_cols<Tile<T, D, 16>, C, RING, true>(p, sc, kmap, vmap, num_seqs, stream);
  if (block_size == 8) return launch_scored_cols<Tile<T, D, 8>, C, RING, true>(p, sc, kmap, vmap, num_seqs, stream);
  if (block_size == 32) return launch_scored_cols<Tile<T, D, 32>, C, RING, true>(p, sc, kmap, vmap, num_seqs, stream);
  return cudaErrorInvalidValue;
}

template <typename T>
static cudaError_t dispatch(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, bool fp8, int head_dim, int block_size, int num_seqs,
                            cudaStream_t stream) {
  constexpr int R16 = PKV_MMA_RING_BYTES, R8 = PKV_MMA_FP8_RING_BYTES;
  if (fp8)
    return of_block<ScoredTileE4M3, T, __nv_fp8_e4m3, 128, R8>(p, sc, kmap, vmap, block_size, num_seqs, stream);
  if (head_dim == 128) return of_block<ScoredTile, T, T, 128, R16>(p, sc, kmap, vmap, block_size, num_seqs, stream);
  if (head_dim == 64) return of_block<ScoredTile, T, T, 64, R16>(p, sc, kmap, vmap, block_size, num_seqs, stream);
  return cudaErrorInvalidValue;
}

cudaError_t tree_cols(const DecodeParams& p, const ScoreParams& sc, const CUtensorMap& kmap, const CUtensorMap& vmap,
                      bool f16, bool fp8, int head_dim, int block_size, int num_seqs, cudaStream_t stream) {
  return f16 ? dispatch<__half>(p, sc, kmap, vmap, fp8, head_dim, block_size, num_seqs, stream)
             : dispatch<__nv_bfloat16>(p, sc, kmap, vmap, fp8, head_dim, block_size, num_seqs, stream);
}

}  // namespace pkv

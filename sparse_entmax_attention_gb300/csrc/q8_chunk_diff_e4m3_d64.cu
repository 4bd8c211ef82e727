// q8_chunk_diff_e4m3_d64.cu -- differential chunk attention over e4m3 codes, head dimension 64.
#include "q8_chunk.cuh"

namespace ekv {

template <>
cudaError_t chunk_run<false, 64, true>(const ChunkArgs& g, cudaStream_t st) {
  return chunk_pages<false, 64, true>(g, st);
}

}  // namespace ekv

// q8_chunk_diff_e4m3_d128.cu -- differential chunk attention over e4m3 codes, head dimension 128.
#include "q8_chunk.cuh"

namespace ekv {

template <>
cudaError_t chunk_run<false, 128, true>(const ChunkArgs& g, cudaStream_t st) {
  return chunk_pages<false, 128, true>(g, st);
}

}  // namespace ekv

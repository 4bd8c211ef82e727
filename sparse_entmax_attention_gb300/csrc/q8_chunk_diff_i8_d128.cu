// q8_chunk_diff_i8_d128.cu -- differential chunk attention over whole-number codes, head dimension 128.
#include "q8_chunk.cuh"

namespace ekv {

template <>
cudaError_t chunk_run<true, 128, true>(const ChunkArgs& g, cudaStream_t st) {
  return chunk_pages<true, 128, true>(g, st);
}

}  // namespace ekv

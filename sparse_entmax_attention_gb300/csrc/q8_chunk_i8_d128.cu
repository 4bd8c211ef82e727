// q8_chunk_i8_d128.cu -- chunk attention over whole-number codes, head dimension 128.
#include "q8_chunk.cuh"

namespace ekv {

template <>
cudaError_t chunk_run<true, 128, false>(const ChunkArgs& g, cudaStream_t st) {
  return chunk_pages<true, 128, false>(g, st);
}

}  // namespace ekv

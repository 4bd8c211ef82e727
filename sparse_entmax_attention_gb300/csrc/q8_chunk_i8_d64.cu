// q8_chunk_i8_d64.cu -- chunk attention over whole-number codes, head dimension 64.
#include "q8_chunk.cuh"

namespace ekv {

template <>
cudaError_t chunk_run<true, 64, false>(const ChunkArgs& g, cudaStream_t st) {
  return chunk_pages<true, 64, false>(g, st);
}

}  // namespace ekv

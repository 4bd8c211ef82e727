// q8_chunk_e4m3_d64.cu -- chunk attention over e4m3 codes, head dimension 64.
#include "q8_chunk.cuh"

namespace ekv {

template <>
cudaError_t chunk_run<false, 64>(const ChunkArgs& g, cudaStream_t st) {
  return chunk_pages<false, 64>(g, st);
}

}  // namespace ekv

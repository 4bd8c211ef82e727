// q8_weigh_chunk_i8_d64.cu -- weights of many rows over whole-number codes, head dimension 64.
#include "q8_weigh_chunk.cuh"

namespace ekv {

template <>
cudaError_t weigh_chunk_run<true, 64>(const WcArgs& g, cudaStream_t st) {
  return weigh_chunk_pages<true, 64>(g, st);
}

}  // namespace ekv

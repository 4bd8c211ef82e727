// q8_weigh_chunk_i8_d128.cu -- weights of many rows over whole-number codes, head dimension 128.
#include "q8_weigh_chunk.cuh"

namespace ekv {

template <>
cudaError_t weigh_chunk_run<true, 128>(const WcArgs& g, cudaStream_t st) {
  return weigh_chunk_pages<true, 128>(g, st);
}

}  // namespace ekv

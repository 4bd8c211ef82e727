// q8_weigh_chunk_e4m3_d64.cu -- weights of many rows over e4m3 codes, head dimension 64.
#include "q8_weigh_chunk.cuh"

namespace ekv {

template <>
cudaError_t weigh_chunk_run<false, 64>(const WcArgs& g, cudaStream_t st) {
  return weigh_chunk_pages<false, 64>(g, st);
}

}  // namespace ekv

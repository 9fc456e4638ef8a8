// decode_list.cu -- the decode kernel's variants that read listed blocks (sparse attention).
#include "decode_kernel.cuh"

namespace kvinc {

cudaError_t launch_decode_list(const DecodeParams &p, int D, int n_tiles_heads, cudaStream_t s,
                             bool pdl) {
  return launch_decode_mode<kDecodeList>(p, D, n_tiles_heads, s, pdl);
}

cudaError_t configure_decode_list() { return configure_decode_mode<kDecodeList>(); }

}  // namespace kvinc

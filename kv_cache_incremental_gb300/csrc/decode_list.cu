// decode_list.cu -- the decode kernel's variants that read listed blocks (sparse attention).
// All keep the shallow pipeline: the deep one fills an SM's shared memory, so that neither
// the selection before it nor the launch after it overlaps with it (16 queries x 8 heads x
// 37 blocks: 47.8 us against 44.3).
#include "decode_kernel.cuh"

namespace kvinc {

cudaError_t launch_decode_list(const DecodeParams &p, int D, int n_tiles_heads, cudaStream_t s,
                             bool pdl) {
  if (p.n_items <= 0) return cudaSuccess;
  constexpr int M = kDecodeList;
  if (D == 128)
    return n_tiles_heads == 1 ? launch_decode_t<128, 1, false, M>(p, s, pdl)
                              : launch_decode_t<128, 2, false, M>(p, s, pdl);
  if (D == 64)
    return n_tiles_heads == 1 ? launch_decode_t<64, 1, false, M>(p, s, pdl)
                              : launch_decode_t<64, 2, false, M>(p, s, pdl);
  return cudaErrorInvalidValue;
}

cudaError_t configure_decode_list() {
  constexpr int M = kDecodeList;
  cudaError_t e = configure_decode_t<128, 1, false, M>();
  if (e == cudaSuccess) e = configure_decode_t<128, 2, false, M>();
  if (e == cudaSuccess) e = configure_decode_t<64, 1, false, M>();
  if (e == cudaSuccess) e = configure_decode_t<64, 2, false, M>();
  return e;
}

}  // namespace kvinc

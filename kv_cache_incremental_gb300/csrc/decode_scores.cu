// decode_scores.cu -- the decode kernel's variants that also store each head's softmax maximum and
// sum and, if wanted, every key's scores (accumulated weights).
#include "decode_kernel.cuh"

namespace kvinc {

cudaError_t launch_decode_scores(const DecodeParams &p, int D, int n_tiles_heads, cudaStream_t s,
                             bool pdl) {
  return launch_decode_mode<kDecodeScores>(p, D, n_tiles_heads, s, pdl);
}

cudaError_t configure_decode_scores() { return configure_decode_mode<kDecodeScores>(); }

}  // namespace kvinc

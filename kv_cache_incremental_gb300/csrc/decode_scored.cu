// decode_scored.cu -- the decode kernel's variants with changed scores, documents and prefixes
// (kv_append_scored).  Bound by HBM like the ordinary ones: 64 rows of 1k to 8k keys, Hq 32, Hk 8,
// D 128, capped, 176 us, 99% of the copy rate; a mode of its own keeps the changes out of their registers.
#include "decode_kernel.cuh"

namespace kvinc {

cudaError_t launch_decode_scored(const ScoredDecodeParams &p, int D, int n_tiles_heads,
                                 cudaStream_t s, bool pdl) {
  return launch_decode_mode<kDecodeScored>(p, D, n_tiles_heads, s, pdl);
}

cudaError_t configure_decode_scored() { return configure_decode_mode<kDecodeScored>(); }

}  // namespace kvinc

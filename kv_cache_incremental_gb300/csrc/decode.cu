// decode.cu -- the decode kernel's ordinary variants (decode_kernel.cuh), as launches and as
// graph nodes; the variants that read listed blocks or store the scores are compiled in
// files of their own (decode_list.cu, decode_scores.cu).
#include "decode_kernel.cuh"

namespace kvinc {

cudaError_t launch_decode_list(const DecodeParams &p, int D, int n_tiles_heads, cudaStream_t s,
                               bool pdl);
cudaError_t launch_decode_scores(const DecodeParams &p, int D, int n_tiles_heads, cudaStream_t s,
                                 bool pdl);
cudaError_t configure_decode_list();
cudaError_t configure_decode_scores();

namespace {

// Function and shared memory of the variant for (D, tiles of heads, deep pipeline).
template <int D, int NT>
bool pick_t(bool deep, void **fn, int *smem) {
  if (deep) {
    *fn = reinterpret_cast<void *>(decode_kernel<D, NT, true, kDecodePlain>);
    *smem = decode_smem_bytes<D, NT, true>();
  } else {
    *fn = reinterpret_cast<void *>(decode_kernel<D, NT, false, kDecodePlain>);
    *smem = decode_smem_bytes<D, NT, false>();
  }
  return true;
}

bool pick(int D, int n_tiles_heads, bool deep, void **fn, int *smem) {
  if (D == 128) return n_tiles_heads == 1 ? pick_t<128, 1>(deep, fn, smem)
                                          : pick_t<128, 2>(deep, fn, smem);
  if (D == 64) return n_tiles_heads == 1 ? pick_t<64, 1>(deep, fn, smem)
                                         : pick_t<64, 2>(deep, fn, smem);
  return false;
}

}  // namespace

cudaError_t launch_decode(const DecodeParams &p, int D, int n_tiles_heads, cudaStream_t s,
                          bool pdl) {
  if (p.list) return launch_decode_list(p, D, n_tiles_heads, s, pdl);
  if (p.row_ml) return launch_decode_scores(p, D, n_tiles_heads, s, pdl);
  return launch_decode_mode<kDecodePlain>(p, D, n_tiles_heads, s, pdl);
}

// The same launch as a graph kernel node: function, grid, block, shared memory and the one
// argument (the node copies *p when it is added or its parameters are set).
cudaError_t decode_node(const DecodeParams *p, int D, int n_tiles_heads, void **args,
                        cudaKernelNodeParams *kp) {
  if (p->n_items <= 0) return cudaErrorInvalidValue;
  args[0] = const_cast<DecodeParams *>(p);
  kp->gridDim = dim3(p->n_items, p->Hk);
  kp->blockDim = dim3(kThreads);
  kp->kernelParams = args;
  kp->extra = nullptr;
  int smem = 0;
  if (!pick(D, n_tiles_heads, p->deep_pipeline != 0, &kp->func, &smem))
    return cudaErrorInvalidValue;
  kp->sharedMemBytes = smem;
  return cudaSuccess;
}

cudaError_t configure_decode() {
  cudaError_t e = configure_decode_mode<kDecodePlain>();
  if (e == cudaSuccess) e = configure_decode_list();
  if (e == cudaSuccess) e = configure_decode_scores();
  return e;
}

}  // namespace kvinc

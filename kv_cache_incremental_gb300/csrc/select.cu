// select.cu -- the two kernels in front of sparse attention: 8-bit bounds of the key
// blocks, and each query's choice of blocks by them.
//
// Bounds.  For a block of 64 cached (post-RoPE) keys of one kv head let, per head
// dimension d, lo_d and hi_d be the smallest and largest K_jd, and m the largest
// magnitude among them.  Stored are, with inv = 127 / m (one float32 division), the
// levels hi8_d = ceil(hi_d inv) and lo8_d = floor(lo_d inv), clamped to +-127, and the
// step m * fl(1 / 127).  Rounding outwards keeps them bounds: q_d K_jd <= max(q_d lo_d,
// q_d hi_d) for every key of the block.  A block whose m is below 1e-30 counts as zero.
//
// Score.  A query head rotated and rounded to bf16 is taken to 127 levels the same way,
// rounded to nearest: q8_d, step qs.  The head's score of a block is the bound on q . K_j,
//   (float)(sum_d max(q8_d lo8_d, q8_d hi8_d)) * (qs * step),
// and a block's score for the kv head the largest over the group's query heads, since
// the group reads its blocks together.  With q+ = max(q8, 0) and q- = min(q8, 0) the sum
// is sum_d (q+_d hi8_d + q-_d lo8_d): two dp4a per four dimensions.  It is a whole number
// below 2^24 (D = 128: 128 x 127 x 127), so every order of summing gives the same score
// and the chosen blocks are the same on every run and every machine; that, and one byte
// per bound, are what 8 bits are taken for.  Ties go to the lower block; a NaN score
// counts below every number.
#include "kvinc_internal.h"
#include "ptx.cuh"

namespace kvinc {
namespace {

constexpr float kTiny = 1e-30f;
constexpr float kStep = (float)(1.0 / 127.0);

// ---------------------------------------------------------------- bounds
constexpr int kBoundsWarps = 4;

__device__ __forceinline__ int find_bounds_row(const BoundsParams &p, int item) {
  int lo = 0, hi = p.n_rows - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.rows[mid].item0 <= item) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int level(float x) {  // to -127 .. 127; NaN gives -127
  return __float2int_rn(fminf(fmaxf(x, -127.f), 127.f));
}

// One warp per (block, kv head).  A lane owns a 16-byte chunk of the head dimension and
// every (32 / chunks)-th key; loads of eight keys are in flight at a time.
template <int D>
__global__ void __launch_bounds__(kBoundsWarps * 32)
    bounds_kernel(const __grid_constant__ BoundsParams p) {
  ptx::grid_dep_wait();  // the keys come from the launches before
  ptx::grid_dep_launch();
  constexpr int kChunks = D / 8, kKeysPer = 32 / kChunks;
  const int item = blockIdx.x * kBoundsWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (item >= p.n_items) return;
  const int g = blockIdx.y;
  const BoundsRow &row = p.rows[find_bounds_row(p, item)];
  const int blk = row.blk0 + item - row.item0;
  const int chunk = lane % kChunks, key0 = lane / kChunks;
  float lo[8], hi[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo[j] = INFINITY;
    hi[j] = -INFINITY;
  }
  constexpr int kLoads = 8;
  for (int k0 = 0; k0 < kSparseBlock; k0 += kLoads * kKeysPer) {
    uint4 x[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int slot = blk * kSparseBlock + k0 + i * kKeysPer + key0;
      x[i] = *reinterpret_cast<const uint4 *>(
          p.K + kv_row(p.pt, row.cache_row, p.Hk, g, p.seg_rows, slot) * D + 8 * chunk);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(&x[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = __bfloat162float(v[j]);
        lo[j] = fminf(lo[j], f);
        hi[j] = fmaxf(hi[j], f);
      }
    }
  }
#pragma unroll
  for (int off = kChunks; off < 32; off <<= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo[j] = fminf(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], off));
      hi[j] = fmaxf(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], off));
    }
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(lo[j]), fabsf(hi[j])));
#pragma unroll
  for (int off = 1; off < kChunks; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  const bool some = m >= kTiny;
  const float inv = some ? __fdiv_rn(127.f, m) : 0.f;
  const int64_t at = ((int64_t)row.cache_row * p.Hk + g) * p.nb_cap + blk;
  if (lane < kChunks) {
    uint32_t h[2] = {0, 0}, l[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[j / 4] |= (uint32_t)(level(ceilf(__fmul_rn(hi[j], inv))) & 255) << (8 * (j % 4));
      l[j / 4] |= (uint32_t)(level(floorf(__fmul_rn(lo[j], inv))) & 255) << (8 * (j % 4));
    }
    uint2 *dst = reinterpret_cast<uint2 *>(p.bound + at * 2 * D);
    dst[chunk] = make_uint2(h[0], h[1]);
    dst[D / 8 + chunk] = make_uint2(l[0], l[1]);
    if (lane == 0) p.scale[at] = some ? __fmul_rn(m, kStep) : 0.f;
  }
}

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 128, kSelWarps = kSelThreads / 32;

// Order-preserving whole number of a score: NaN lowest, -0 and +0 alike.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int D>  // q+ and q- levels and steps of up to kMaxRep heads
constexpr int kSelHead = kMaxRep * 2 * D + kMaxRep * 4;

// One CTA per (query, kv head).
template <int D>
__global__ void __launch_bounds__(kSelThreads)
    select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kHalf = D / 2;
  extern __shared__ __align__(16) uint8_t sm[];
  int8_t *q8 = reinterpret_cast<int8_t *>(sm);                     // [rep][2][D]: q+, q-
  float *qs = reinterpret_cast<float *>(sm + kMaxRep * 2 * D);     // [rep]
  uint32_t *keys = reinterpret_cast<uint32_t *>(sm + kSelHead<D>);  // [max_cand]
  __shared__ int hist[256];
  __shared__ int warp_n[kSelWarps][2];
  __shared__ int pick[2];  // the digit that holds the threshold, keys above it

  const SelectQuery &qu = p.queries[blockIdx.x];
  const int g = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nb = qu.slot / kSparseBlock + 1;
  const int per = p.sink + p.top_k + p.recent;
  const int n_sel = min(nb, per);
  const int n_cand = nb > per ? nb - p.sink - p.recent : 0;
  int32_t *list = p.list + ((int64_t)blockIdx.x * p.Hk + g) * p.list_stride;
  int32_t *user = p.selected ? p.selected + ((int64_t)qu.tok * p.Hk + g) * per : nullptr;

  ptx::grid_dep_wait();  // bounds, and the lists that the launch before read
  ptx::grid_dep_launch();
  const auto put = [&](int i, int blk) {
    list[i] = blk;
    if (user) user[i] = blk;
  };
  if (user)
    for (int i = n_sel + tid; i < per; i += kSelThreads) user[i] = -1;
  if (n_cand == 0) {  // everything there is
    for (int i = tid; i < n_sel; i += kSelThreads) put(i, i);
    return;
  }
  for (int i = tid; i < p.sink; i += kSelThreads) put(i, i);
  for (int i = tid; i < p.recent; i += kSelThreads)
    put(p.sink + p.top_k + i, nb - p.recent + i);

  // The group's query heads, one warp each: rotate (float products without contraction,
  // one rounding to bf16, as the attention does), find the largest magnitude, quantise.
  const float2 *cs = p.rope + (int64_t)qu.pos * kHalf;
  for (int h = warp; h < p.rep; h += kSelWarps) {
    const __nv_bfloat16 *q = p.q + ((int64_t)qu.tok * p.Hq + g * p.rep + h) * D;
    float a[kHalf / 32], b[kHalf / 32], m = 0.f;
#pragma unroll
    for (int i = 0; i < kHalf / 32; ++i) {
      const int d = lane + 32 * i;
      const float x1 = __bfloat162float(q[d]), x2 = __bfloat162float(q[d + kHalf]);
      const float2 r = cs[d];
      a[i] = __bfloat162float(
          __float2bfloat16_rn(__fsub_rn(__fmul_rn(x1, r.x), __fmul_rn(x2, r.y))));
      b[i] = __bfloat162float(
          __float2bfloat16_rn(__fadd_rn(__fmul_rn(x1, r.y), __fmul_rn(x2, r.x))));
      m = fmaxf(m, fmaxf(fabsf(a[i]), fabsf(b[i])));
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const bool some = m >= kTiny;
    const float inv = some ? __fdiv_rn(127.f, m) : 0.f;
#pragma unroll
    for (int i = 0; i < kHalf / 32; ++i) {
      const int d = lane + 32 * i;
      const int la = level(rintf(__fmul_rn(a[i], inv))), lb = level(rintf(__fmul_rn(b[i], inv)));
      q8[h * 2 * D + d] = (int8_t)max(la, 0);
      q8[h * 2 * D + D + d] = (int8_t)min(la, 0);
      q8[h * 2 * D + d + kHalf] = (int8_t)max(lb, 0);
      q8[h * 2 * D + D + d + kHalf] = (int8_t)min(lb, 0);
    }
    if (lane == 0) qs[h] = some ? __fmul_rn(m, kStep) : 0.f;
  }
  __syncthreads();

  // Scores: eight lanes per block, each D / 8 of the head dimension.
  {
    constexpr int kWords = D / 32;  // 4-byte words per lane
    const int sub = tid & 7;
    const int8_t *bound = p.bound + ((int64_t)qu.cache_row * p.Hk + g) * p.nb_cap * 2 * D;
    const float *scale = p.scale + ((int64_t)qu.cache_row * p.Hk + g) * p.nb_cap;
    // every lane of a warp takes the same number of passes (the shuffles below)
    for (int c0 = 0; c0 < n_cand; c0 += kSelThreads / 8) {
      const int c = c0 + tid / 8;
      const int blk = p.sink + min(c, n_cand - 1);
      const int *hi = reinterpret_cast<const int *>(bound + (int64_t)blk * 2 * D) + sub * kWords;
      const int *lo = hi + D / 4;
      int h4[kWords], l4[kWords];
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        h4[w] = hi[w];
        l4[w] = lo[w];
      }
      const float st = scale[blk];
      uint32_t best = 0;
      for (int h = 0; h < p.rep; ++h) {
        const int *qp = reinterpret_cast<const int *>(q8 + h * 2 * D) + sub * kWords;
        int dot = 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          dot = __dp4a(h4[w], qp[w], dot);
          dot = __dp4a(l4[w], qp[D / 4 + w], dot);
        }
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        best = max(best, order_key(__fmul_rn((float)dot, __fmul_rn(qs[h], st))));
      }
      if (sub == 0 && c < n_cand) keys[c] = best;
    }
  }
  if (p.top_k == 0) return;
  __syncthreads();

  // The top_k-th largest key, one 8-bit digit at a time: `above` keys are larger than the
  // prefix found so far, and the next digit is the one whose bin holds rank top_k.
  uint32_t prefix = 0;
  int above = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int c = tid; c < n_cand; c += kSelThreads)
      if ((keys[c] & mask) == prefix) atomicAdd(&hist[(keys[c] >> shift) & 255], 1);
    __syncthreads();
    if (warp == 0) {  // bins from the largest down, eight per lane
      int sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += hist[255 - 8 * lane - i];
      int incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
      }
      int run = above + incl - sum;
      if (run < p.top_k && above + incl >= p.top_k) {
        for (int i = 0; i < 8; ++i) {
          const int n = hist[255 - 8 * lane - i];
          if (run + n >= p.top_k) {
            pick[0] = 255 - 8 * lane - i;
            pick[1] = run;
            break;
          }
          run += n;
        }
      }
    }
    __syncthreads();
    prefix |= (uint32_t)pick[0] << shift;
    above = pick[1];
  }
  // Blocks above the threshold, and the first top_k - above at it, in ascending order.
  const int ties = p.top_k - above;
  int base_gt = 0, base_eq = 0;
  for (int c0 = 0; c0 < n_cand; c0 += kSelThreads) {
    const int c = c0 + tid;
    const uint32_t key = c < n_cand ? keys[c] : 0;
    const bool gt = c < n_cand && key > prefix, eq = c < n_cand && key == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      warp_n[warp][0] = __popc(bg);
      warp_n[warp][1] = __popc(be);
    }
    __syncthreads();
    int ng = base_gt, ne = base_eq;
    for (int w = 0; w < kSelWarps; ++w) {
      if (w < warp) {
        ng += warp_n[w][0];
        ne += warp_n[w][1];
      }
      base_gt += warp_n[w][0];
      base_eq += warp_n[w][1];
    }
    const uint32_t below = (1u << lane) - 1;
    ng += __popc(bg & below);
    ne += __popc(be & below);
    if (gt || (eq && ne < ties)) put(p.sink + ng + min(ne, ties), p.sink + c);
    __syncthreads();
  }
}

template <int D>
cudaError_t launch_select_t(const SelectParams &p, cudaStream_t s, bool pdl) {
  const int smem = kSelHead<D> + 4 * p.max_cand;
  return launch_k(select_kernel<D>, dim3(p.n_queries, p.Hk), dim3(kSelThreads), smem, s, p, pdl);
}

}  // namespace

cudaError_t launch_bounds(const BoundsParams &p, cudaStream_t s, bool pdl) {
  if (p.n_items <= 0) return cudaSuccess;
  const dim3 grid((p.n_items + kBoundsWarps - 1) / kBoundsWarps, p.Hk);
  return p.D == 128 ? launch_k(bounds_kernel<128>, grid, dim3(kBoundsWarps * 32), 0, s, p, pdl)
                    : launch_k(bounds_kernel<64>, grid, dim3(kBoundsWarps * 32), 0, s, p, pdl);
}

cudaError_t launch_select(const SelectParams &p, cudaStream_t s, bool pdl) {
  if (p.n_queries <= 0) return cudaSuccess;
  return p.D == 128 ? launch_select_t<128>(p, s, pdl) : launch_select_t<64>(p, s, pdl);
}

// Keys of the longest row (max_len = 2^20: 16384 blocks) take 64 KB of shared memory.
cudaError_t configure_select() {
  constexpr int cand = (1 << 20) / kSparseBlock;
  const cudaError_t e =
      cudaFuncSetAttribute(select_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSelHead<128> + 4 * cand);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(select_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kSelHead<64> + 4 * cand);
}

}  // namespace kvinc

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

// Bounds of block `blk` of (row, kv head), by one warp.  A lane owns a 16-byte chunk of the
// head dimension and every (32 / chunks)-th key; loads of eight keys are in flight at a time.
template <int D>
__device__ __forceinline__ void bounds_of_block(const __nv_bfloat16 *K, const PageTable &pt,
                                                int seg_rows, int cache_row, int Hk, int g, int blk,
                                                int nb_cap, int8_t *bound, float *scale,
                                                int lane) {
  constexpr int kChunks = D / 8, kKeysPer = 32 / kChunks;
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
      x[i] = *reinterpret_cast<const uint4 *>(K + kv_row(pt, cache_row, Hk, g, seg_rows, slot) * D +
                                              8 * chunk);
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
  const int64_t at = ((int64_t)cache_row * Hk + g) * nb_cap + blk;
  if (lane < kChunks) {
    uint32_t h[2] = {0, 0}, l[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[j / 4] |= (uint32_t)(level(ceilf(__fmul_rn(hi[j], inv))) & 255) << (8 * (j % 4));
      l[j / 4] |= (uint32_t)(level(floorf(__fmul_rn(lo[j], inv))) & 255) << (8 * (j % 4));
    }
    uint2 *dst = reinterpret_cast<uint2 *>(bound + at * 2 * D);
    dst[chunk] = make_uint2(h[0], h[1]);
    dst[D / 8 + chunk] = make_uint2(l[0], l[1]);
    if (lane == 0) scale[at] = some ? __fmul_rn(m, kStep) : 0.f;
  }
}

// One warp per (block, kv head).
template <int D>
__global__ void __launch_bounds__(kBoundsWarps * 32)
    bounds_kernel(const __grid_constant__ BoundsParams p) {
  ptx::grid_dep_wait();  // the keys come from the launches before
  ptx::grid_dep_launch();
  const int item = blockIdx.x * kBoundsWarps + (threadIdx.x >> 5);
  if (item >= p.n_items) return;
  const BoundsRow &row = p.rows[find_bounds_row(p, item)];
  bounds_of_block<D>(p.K, p.pt, p.seg_rows, row.cache_row, p.Hk, blockIdx.y,
                     row.blk0 + item - row.item0, p.nb_cap, p.bound, p.scale, threadIdx.x & 31);
}

// ---------------------------------------------------------------- selection
// Up to this many candidates a block's rank is counted directly (every candidate against
// every other), above it found by radix selection (16 to 125 candidates, 64 rows, the whole
// call: counted 58.0 us, by radix 59.1; 29 candidates, one row: 9.9 and 11.1).
constexpr int kCountMax = 256;

// Order-preserving whole number of a score: NaN lowest, -0 and +0 alike.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int D>  // q+ and q- levels and steps of up to kMaxRep heads
constexpr int kSelHead = kMaxRep * 2 * D + kMaxRep * 4;

template <int W>  // W consecutive 4-byte words
struct Words {
  int w[W];
};
template <int W>
__device__ __forceinline__ Words<W> load_words(const void *p) {
  Words<W> r;
  if constexpr (W == 4) {
    const int4 x = *reinterpret_cast<const int4 *>(p);
    r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
  } else {
    static_assert(W == 2, "D is 64 or 128");
    const int2 x = *reinterpret_cast<const int2 *>(p);
    r.w[0] = x.x, r.w[1] = x.y;
  }
  return r;
}

// One CTA per (query, kv head).  APPEND (calls of single-token rows): the CTA first rotates
// and stores its row's new key and value, and computes the bounds of the row's pending
// blocks, so that a step needs no launches of their own for them.
// T threads; the bound keeps a batch of 512 (query, kv head) pairs at D = 128 in one wave.
template <int D, bool APPEND, int T>
__global__ void __launch_bounds__(T, T == 1024 ? 1 : D == 64 ? 5 : 4)
    select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kSelThreads = T, kSelWarps = T / 32;
  static_assert(T >= kCountMax && T >= 256, "a thread per counted candidate and per bin");
  constexpr int kHalf = D / 2;
  extern __shared__ __align__(16) uint8_t sm[];
  int8_t *q8 = reinterpret_cast<int8_t *>(sm);                     // [rep][2][D]: q+, q-
  float *qs = reinterpret_cast<float *>(sm + kMaxRep * 2 * D);     // [rep]
  uint32_t *keys = reinterpret_cast<uint32_t *>(sm + kSelHead<D>);  // [max_cand], to a 4
  __shared__ int hist[256];
  __shared__ int warp_n[kSelWarps][2];
  __shared__ int pick[3];  // the digit that holds the threshold, keys above it and in it

  int r = blockIdx.x;  // the query's row: single tokens, a row each
  if (!APPEND) {
    int hi = p.n_rows - 1;
    r = 0;
    while (r < hi) {
      const int mid = (r + hi + 1) >> 1;
      if (p.rows[mid].q0 <= (int)blockIdx.x) r = mid;
      else hi = mid - 1;
    }
  }
  const SelectRow &row = p.rows[r];
  const int nth = APPEND ? 0 : (int)blockIdx.x - row.q0;
  const int slot = row.slot + nth, pos = row.pos + nth, tok = row.tok + nth;
  const int g = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nb = slot / kSparseBlock + 1;
  const int per = p.sink + p.top_k + p.recent;
  const int n_sel = min(nb, per);
  const int n_cand = nb > per ? nb - p.sink - p.recent : 0;
  int32_t *list = p.list + ((int64_t)blockIdx.x * p.Hk + g) * p.list_stride;
  int32_t *user = p.selected ? p.selected + ((int64_t)tok * p.Hk + g) * per : nullptr;

  // APPEND: q, k and v may come from the kernel before; else an append of this call lies
  // between, and whatever ran before that append has completed.
  if (APPEND) {
    // The bounds start into L2 meanwhile (a hint, whoever writes them still: 9.8 -> 9.4 us for
    // one row of 2k keys, 58.3 -> 57.9 for 64 of 1k-8k).  The same for the first one, two or
    // four blocks chosen below lost (60.6, 61.5, 62.9): the known blocks fill that time.
    if (tid == 0 && n_cand > 0)
      ptx::prefetch_l2(p.bound + (((int64_t)row.cache_row * p.Hk + g) * p.nb_cap + p.sink) * 2 * D,
                       (uint32_t)n_cand * 2 * D);
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
  }
  const float2 *cs = p.rope + (int64_t)pos * kHalf;
  if (APPEND && warp == kSelWarps - 1) {  // the new key and value, 8 pairs per lane
    const int64_t dst = kv_row(p.pt, row.cache_row, p.Hk, g, p.seg_rows, slot) * D;
    const int64_t src = ((int64_t)tok * p.Hk + g) * D;
    if (lane < kHalf / 8) {
      const uint4 k1 = *reinterpret_cast<const uint4 *>(p.k + src + 8 * lane);
      const uint4 k2 = *reinterpret_cast<const uint4 *>(p.k + src + kHalf + 8 * lane);
      const __nv_bfloat16 *x1 = reinterpret_cast<const __nv_bfloat16 *>(&k1);
      const __nv_bfloat16 *x2 = reinterpret_cast<const __nv_bfloat16 *>(&k2);
      uint4 o1, o2;
      __nv_bfloat16 *y1 = reinterpret_cast<__nv_bfloat16 *>(&o1);
      __nv_bfloat16 *y2 = reinterpret_cast<__nv_bfloat16 *>(&o2);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = __bfloat162float(x1[j]), b = __bfloat162float(x2[j]);
        const float2 e = cs[8 * lane + j];
        y1[j] = __float2bfloat16_rn(__fsub_rn(__fmul_rn(a, e.x), __fmul_rn(b, e.y)));
        y2[j] = __float2bfloat16_rn(__fadd_rn(__fmul_rn(a, e.y), __fmul_rn(b, e.x)));
      }
      *reinterpret_cast<uint4 *>(p.cache_k + dst + 8 * lane) = o1;
      *reinterpret_cast<uint4 *>(p.cache_k + dst + kHalf + 8 * lane) = o2;
    } else if (lane < kHalf / 8 + D / 8) {
      const int c = lane - kHalf / 8;
      *reinterpret_cast<uint4 *>(p.cache_v + dst + 8 * c) =
          *reinterpret_cast<const uint4 *>(p.v + src + 8 * c);
    }
  }
  if (n_cand > 0) {
    // The group's query heads, one warp each: rotate (float products without contraction,
    // one rounding to bf16, as the attention does), find the largest magnitude, quantise.
    for (int h = warp; h < p.rep; h += kSelWarps) {
      const __nv_bfloat16 *q = p.q + ((int64_t)tok * p.Hq + g * p.rep + h) * D;
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
  }
  if (!APPEND) {
    ptx::grid_dep_wait();  // bounds, and the lists that the launch before read
    ptx::grid_dep_launch();
  }
  const auto put = [&](int i, int blk) {  // the i-th chosen block, ascending
    list[i] = blk;
    if (user) user[p.sink + i] = blk;
  };
  if (user) {  // the blocks read in any case: everything there is, or the first and last ones
    for (int i = tid; i < per; i += kSelThreads)
      if (n_cand == 0)
        user[i] = i < n_sel ? i : -1;
      else if (i < p.sink)
        user[i] = i;
      else if (i >= p.sink + p.top_k)
        user[i] = nb - per + i;
  }
  __syncthreads();  // q8 and, APPEND, the stored key
  if (APPEND && row.n_pend > 0) {
    for (int i = warp; i < row.n_pend; i += kSelWarps)
      bounds_of_block<D>(p.cache_k, p.pt, p.seg_rows, row.cache_row, p.Hk, g, row.pend0 + i,
                         p.nb_cap, p.bound, p.scale, lane);
    __syncthreads();
  }
  if (n_cand == 0 || p.top_k == 0) return;

  // Scores: eight lanes per four blocks, each D / 8 of the head dimension; the four sums
  // are spread over the lanes while they are added up, so that lanes 2 i and 2 i + 1 of the
  // eight end with block i's.
  {
    constexpr int kWords = D / 32;  // 4-byte words per lane
    const int sub = tid & 7;
    const int8_t *bound = p.bound + ((int64_t)row.cache_row * p.Hk + g) * p.nb_cap * 2 * D +
                          4 * kWords * sub;
    const float *scale = p.scale + ((int64_t)row.cache_row * p.Hk + g) * p.nb_cap;
    // a warp takes 16 blocks per pass, all of its lanes as many passes (the shuffles below)
    for (int c0 = 16 * warp; c0 < n_cand; c0 += kSelThreads / 2) {
      const int cg = c0 + 4 * (lane / 8);
      Words<kWords> hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int8_t *b = bound + (int64_t)(p.sink + min(cg + i, n_cand - 1)) * 2 * D;
        hi[i] = load_words<kWords>(b);
        lo[i] = load_words<kWords>(b + D);
      }
      const int c = cg + (sub >> 1);
      const float st = scale[p.sink + min(c, n_cand - 1)];
      uint32_t best = 0;
      for (int h = 0; h < p.rep; ++h) {
        const int8_t *qp = q8 + h * 2 * D + 4 * kWords * sub;
        const Words<kWords> qa = load_words<kWords>(qp), qb = load_words<kWords>(qp + D);
        int dot[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dot[i] = 0;
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            dot[i] = __dp4a(hi[i].w[w], qa.w[w], dot[i]);
            dot[i] = __dp4a(lo[i].w[w], qb.w[w], dot[i]);
          }
        }
        const bool up = sub & 4, odd = sub & 2;
        const int k0 = up ? dot[2] : dot[0], k1 = up ? dot[3] : dot[1];
        const int s0 = up ? dot[0] : dot[2], s1 = up ? dot[1] : dot[3];
        const int r0 = k0 + __shfl_xor_sync(0xffffffffu, s0, 4);
        const int r1 = k1 + __shfl_xor_sync(0xffffffffu, s1, 4);
        int d = (odd ? r1 : r0) + __shfl_xor_sync(0xffffffffu, odd ? r0 : r1, 2);
        d += __shfl_xor_sync(0xffffffffu, d, 1);
        best = max(best, order_key(__fmul_rn((float)d, __fmul_rn(qs[h], st))));
      }
      if ((sub & 1) == 0 && c < (n_cand + 3) / 4 * 4) keys[c] = c < n_cand ? best : 0;
    }
  }
  __syncthreads();

  uint32_t prefix = 0;  // keys above it are taken, and the first `ties` at it
  int ties = 0;
  if (n_cand <= kCountMax) {
    // Each thread ranks one candidate: equal keys count if they come before it, which only
    // within a warp differs from thread to thread.  (Keys past the last are 0: they count
    // for nobody.)  The taken ones are written in order.
    const uint32_t mine = tid < n_cand ? keys[tid] : 0;
    int rank = 0;
    if (32 * warp < n_cand) {
      const uint4 *keys4 = reinterpret_cast<const uint4 *>(keys);
      const int n4 = (n_cand + 3) / 4, own = 8 * warp, end = min(own + 8, n4);
#pragma unroll 4
      for (int j = 0; j < own; ++j) {
        const uint4 x = keys4[j];
        rank += (x.x >= mine) + (x.y >= mine) + (x.z >= mine) + (x.w >= mine);
      }
#pragma unroll 4
      for (int j = own; j < end; ++j) {
        const uint4 x = keys4[j];
        const int before = tid - 4 * j;  // keys 4 j .. 4 j + before - 1 come before this one
        rank += (x.x > mine || (x.x == mine && before > 0)) +
                (x.y > mine || (x.y == mine && before > 1)) +
                (x.z > mine || (x.z == mine && before > 2)) +
                (x.w > mine || (x.w == mine && before > 3));
      }
#pragma unroll 4
      for (int j = end; j < n4; ++j) {
        const uint4 x = keys4[j];
        rank += (x.x > mine) + (x.y > mine) + (x.z > mine) + (x.w > mine);
      }
    }
    const bool take = tid < n_cand && rank < p.top_k;
    const uint32_t bt = __ballot_sync(0xffffffffu, take);
    if (lane == 0) warp_n[warp][0] = __popc(bt);
    __syncthreads();
    int at = __popc(bt & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) at += warp_n[w][0];
    if (take) put(at, p.sink + tid);
    return;
  }
  // The top_k-th largest key, one 8-bit digit at a time: `above` keys are larger than the
  // prefix found so far, and the next digit is the one whose bin holds rank top_k.  When the
  // whole bin is taken the rest of the digits do not matter.
  int above = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
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
            pick[2] = n;
            break;
          }
          run += n;
        }
      }
    }
    __syncthreads();
    prefix |= (uint32_t)pick[0] << shift;
    above = pick[1];
    ties = p.top_k - above;
    if (pick[2] == ties && prefix > 0) {  // every key from the prefix on
      prefix -= 1;
      ties = 0;
      break;
    }
  }
  int base_gt = 0, base_eq = 0;
  for (int c0 = 0; c0 < n_cand; c0 += kSelThreads) {
    const int c = c0 + tid;
    const uint32_t key = c < n_cand ? keys[c] : 0;
    const bool gt = c < n_cand && key > prefix;
    const bool eq = ties > 0 && c < n_cand && key == prefix;
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
    if (gt || (eq && ne < ties)) put(ng + min(ne, ties), p.sink + c);
    __syncthreads();
  }
}

template <int D, bool APPEND, int T>
cudaError_t launch_select_t(const SelectParams &p, cudaStream_t s, bool pdl) {
  return launch_k(select_kernel<D, APPEND, T>, dim3(p.n_queries, p.Hk), dim3(T),
                  kSelHead<D> + 16 * (((size_t)p.max_cand + 3) / 4), s, p, pdl);
}

// Keys of the longest row (max_len = 2^20: 16384 blocks) take 64 KB of shared memory.
template <int D, bool APPEND, int T>
cudaError_t configure_select_t() {
  constexpr int smem = kSelHead<D> + 4 * ((1 << 20) / kSparseBlock);
  return cudaFuncSetAttribute(select_kernel<D, APPEND, T>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

// Threads per CTA: few while the longest query's candidates fit two passes of scoring, else
// many, since one CTA's chain of passes then bounds the call (16 queries x 8 heads x 240 to
// 500 candidates, Hq = 64, the whole call: 256 threads 44.1 us, 512 42.1, 1024 41.1).
constexpr int kSelSmall = 256, kSelLarge = 1024;

template <int D, bool APPEND>
cudaError_t launch_select_d(const SelectParams &p, cudaStream_t s, bool pdl) {
  return p.max_cand <= 256 ? launch_select_t<D, APPEND, kSelSmall>(p, s, pdl)
                           : launch_select_t<D, APPEND, kSelLarge>(p, s, pdl);
}

template <int D>
cudaError_t configure_select_d() {
  cudaError_t e = configure_select_t<D, true, kSelSmall>();
  if (e == cudaSuccess) e = configure_select_t<D, true, kSelLarge>();
  if (e == cudaSuccess) e = configure_select_t<D, false, kSelSmall>();
  if (e == cudaSuccess) e = configure_select_t<D, false, kSelLarge>();
  return e;
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
  if (p.D == 128)
    return p.k ? launch_select_d<128, true>(p, s, pdl) : launch_select_d<128, false>(p, s, pdl);
  return p.k ? launch_select_d<64, true>(p, s, pdl) : launch_select_d<64, false>(p, s, pdl);
}

cudaError_t configure_select() {
  const cudaError_t e = configure_select_d<128>();
  return e == cudaSuccess ? configure_select_d<64>() : e;
}

}  // namespace kvinc

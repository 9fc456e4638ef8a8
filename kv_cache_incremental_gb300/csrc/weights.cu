// weights.cu -- per-key softmax weights of a call's queries, added to an accumulator.
//
// For a kv head g and a cached key j of a row, with the counted query tokens t (at slots
// s_t = slots + t) and the group's heads h,
//   acc_out[j] = acc_in[j] + sum_t sum_h [j <= s_t] 2^(x_thj - m_th) / l_th,
//   x_thj = log2(e) / sqrt(D) q_th . K_j,  m_th = max_j x_thj,  l_th = sum_j 2^(x_thj - m_th).
// A weight needs its query's m and l over all keys first.  The attention kernels, which run
// before, have both and leave (m, 1 / l) per query vector (decode_kernel.cuh, the scores mode;
// prefill_tc.cu, prefill.cu and its merge); m may be any reference that l was summed from.
//
// Rows with a single new token: the decode kernel stores the scores as well, on its one pass
// over K and V, and the join kernel turns them into weights: 8 bytes of scores per key and
// head, written and read, beside the 4 D bytes of a key and value (64 rows of 1k-8k keys, Hq
// 32, Hk 8, D 128: 190 us, against 489 with two more passes over K).  Chunks, and rows whose
// scores outgrow the room reserved for them, take one more pass over K: S^T = K Q^T with
// mma.sync (keys on M, query vectors on N), so that a key's weights lie in the lanes of one
// quad and their sum over all queries stays in a register.  Nothing is added atomically: the
// result does not depend on the order in which CTAs run.
//
// K goes from global memory straight into MMA fragments: an MMA's contraction index may be
// permuted alike on both sides, so lane (r, c) of a quad row takes 16 consecutive bytes of
// key r and uses them as the fragments of two steps; the query vectors are read from
// shared memory in the same order.
#include "kvinc_internal.h"
#include "ptx.cuh"

namespace kvinc {
namespace {

constexpr int kWarps = 8, kWThreads = kWarps * 32;
// Query vectors are taken in chunks of 8 QT.  A chunk's unused eights are skipped: variants of
// one and two eights for single tokens ran no faster (8 counted vectors, 24 rows of 6k keys:
// 54.7 us with eight, 54.9 with one).
constexpr int QT = 8;
constexpr int kEights = 2;  // eights of vectors that a step takes together
static_assert(kWeightTile == kWarps * 16, "one 16-key fragment per warp");

__device__ __forceinline__ int find_weights_row(const WeightsParams &p, int item) {
  int lo = 0, hi = p.n_rows - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.rows[mid].item0 <= item) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Rows of 2 D bytes padded by 64: the eight lanes that read 16 bytes each of two
// neighbouring rows then cover all 32 banks.
template <int D>
constexpr int kQStride = 2 * D + 64;

// Query vectors [v0, v0 + 8 QT) of the row, rotated and rounded to bf16 as the attention
// rotates them, into shared memory, with their -m and 1 / l and the last slot that each sees.
// sum_step takes them by kEights eights; the vectors that fill up the last of these are copies of
// the row's last one with a 1 / l of 0.  They add 0 wherever that one's weight is a number (zeros
// in their place made NaN of 0 * inf at keys with infinite components that nothing weighs).
template <int D>
__device__ __forceinline__ void load_queries(const WeightsParams &p, const WeightsRow &row, int g,
                                             int v0, int n_vec, uint8_t *qs, float2 *ml,
                                             int *limit) {
  constexpr int kHalf = D / 2, kVec = kHalf / 8, kFill = 8 * kEights;
  const int taken = min(8 * QT, (n_vec - v0 + kFill - 1) / kFill * kFill);
  if (threadIdx.x < taken) {
    const int vec = min(v0 + (int)threadIdx.x, n_vec - 1);
    const bool fill = v0 + (int)threadIdx.x >= n_vec;
    const int t = row.t0 + vec / p.rep;
    const float2 e =
        p.ml[((int64_t)row.call_row * kChunk + t - row.tok0) * p.Hq + g * p.rep + vec % p.rep];
    ml[threadIdx.x] = make_float2(-e.x, fill ? 0.f : e.y);
    limit[threadIdx.x] = fill ? -1 : row.slots + t;
  }
  for (int u = threadIdx.x; u < taken * kVec; u += kWThreads) {
    const int i = u / kVec, c = u % kVec, vec = min(v0 + i, n_vec - 1);
    const int t = row.t0 + vec / p.rep, h = vec % p.rep;
    const __nv_bfloat16 *q = p.q + (int64_t)row.call_row * p.q_row_stride +
                             ((int64_t)t * p.Hq + g * p.rep + h) * D;
    const uint4 x1v = *reinterpret_cast<const uint4 *>(q + 8 * c);
    const uint4 x2v = *reinterpret_cast<const uint4 *>(q + kHalf + 8 * c);
    const __nv_bfloat16 *x1 = reinterpret_cast<const __nv_bfloat16 *>(&x1v);
    const __nv_bfloat16 *x2 = reinterpret_cast<const __nv_bfloat16 *>(&x2v);
    uint4 lo, hi;
    __nv_bfloat16 *o1 = reinterpret_cast<__nv_bfloat16 *>(&lo);
    __nv_bfloat16 *o2 = reinterpret_cast<__nv_bfloat16 *>(&hi);
    const float2 *cs = p.rope + (int64_t)(row.slots + row.shift + t) * kHalf + 8 * c;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = __bfloat162float(x1[j]), b = __bfloat162float(x2[j]);
      const float2 e = cs[j];
      o1[j] = __float2bfloat16_rn(__fsub_rn(__fmul_rn(a, e.x), __fmul_rn(b, e.y)));
      o2[j] = __float2bfloat16_rn(__fadd_rn(__fmul_rn(a, e.y), __fmul_rn(b, e.x)));
    }
    *reinterpret_cast<uint4 *>(qs + i * kQStride<D> + 16 * c) = lo;
    *reinterpret_cast<uint4 *>(qs + i * kQStride<D> + D + 16 * c) = hi;
  }
}

// This lane's part of the 16 keys at `slot0`: 16 bytes of keys gq and gq + 8 per 32
// dimensions.  Slots past the row's last key read that key again (they are masked).
template <int D>
__device__ __forceinline__ void load_keys(const WeightsParams &p, const WeightsRow &row, int g,
                                          int slot0, int last, int lane, uint4 (&a)[D / 32],
                                          uint4 (&b)[D / 32]) {
  const int gq = lane >> 2, qq = lane & 3;
  const __nv_bfloat16 *ka =
      p.K + kv_row(p.pt, row.cache_row, p.Hk, g, p.seg_rows, min(slot0 + gq, last)) * D + 8 * qq;
  const __nv_bfloat16 *kb =
      p.K + kv_row(p.pt, row.cache_row, p.Hk, g, p.seg_rows, min(slot0 + gq + 8, last)) * D +
      8 * qq;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    a[j] = *reinterpret_cast<const uint4 *>(ka + 32 * j);
    b[j] = *reinterpret_cast<const uint4 *>(kb + 32 * j);
  }
}

// The loaded keys as MMA fragments, each in four consecutive registers as the instruction
// takes them (formed once per 16 keys: left to the use of the loaded vectors themselves,
// every MMA was preceded by the moves that gather its operand).
template <int D>
__device__ __forceinline__ void fragments(const uint4 (&a)[D / 32], const uint4 (&b)[D / 32],
                                          uint4 (&f)[D / 16]) {
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    f[2 * j] = make_uint4(a[j].x, b[j].x, a[j].y, b[j].y);
    f[2 * j + 1] = make_uint4(a[j].z, b[j].z, a[j].w, b[j].w);
  }
}

// Scores of the warp's 16 keys with N eights of query vectors of the chunk in qs, from the
// nt-th on; the eights' MMA chains are independent and interleaved.
template <int D, int N>
__device__ __forceinline__ void scores(const uint4 (&f)[D / 16], const uint8_t *qs, int nt,
                                       int lane, float (&s)[N][4]) {
  const int gq = lane >> 2, qq = lane & 3;
  const uint8_t *qr = qs + (8 * nt + gq) * kQStride<D> + 16 * qq;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    uint4 w[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      w[i] = *reinterpret_cast<const uint4 *>(qr + 8 * i * kQStride<D> + 64 * j);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint4 &x = f[2 * j];
      if (j == 0)
        ptx::mma_bf16_zero(s[i], x.x, x.y, x.z, x.w, w[i].x, w[i].y);
      else
        ptx::mma_bf16(s[i], x.x, x.y, x.z, x.w, w[i].x, w[i].y);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint4 &x = f[2 * j + 1];
      ptx::mma_bf16(s[i], x.x, x.y, x.z, x.w, w[i].z, w[i].w);
    }
  }
}

// One step: 16 keys as fragments f against the first n_nt eights of query vectors, whose -m
// and 1 / l are in ml.  FULL: every key is visible to every vector; else key `key` up to
// `limit`.
template <int D, bool FULL>
__device__ __forceinline__ void sum_step(const uint4 (&f)[D / 16], const uint8_t *qs,
                                         const int *limit, const float2 *ml,
                                         int n_nt, int key, float scale, int lane, float &sum0,
                                         float &sum1) {
  constexpr int N = kEights;
  static_assert(QT % N == 0, "whole steps");
#pragma unroll
  for (int nt0 = 0; nt0 < QT; nt0 += N) {
    if (nt0 >= n_nt) break;
    float sc[N][4];
    scores<D, N>(f, qs, nt0, lane, sc);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float(&s)[4] = sc[i];
      const int nt = nt0 + i;
      const float4 e = *reinterpret_cast<const float4 *>(&ml[8 * nt + 2 * (lane & 3)]);
      float w0 = ptx::ex2(fmaf(s[0], scale, e.x)), w1 = ptx::ex2(fmaf(s[1], scale, e.z));
      float w2 = ptx::ex2(fmaf(s[2], scale, e.x)), w3 = ptx::ex2(fmaf(s[3], scale, e.z));
      if (!FULL) {
        const int l0 = limit[8 * nt + 2 * (lane & 3)], l1 = limit[8 * nt + 2 * (lane & 3) + 1];
        if (key > l0) w0 = 0.f;
        if (key > l1) w1 = 0.f;
        if (key + 8 > l0) w2 = 0.f;
        if (key + 8 > l1) w3 = 0.f;
      }
      sum0 = fmaf(w0, e.y, fmaf(w1, e.w, sum0));
      sum1 = fmaf(w2, e.y, fmaf(w3, e.w, sum1));
    }
  }
}

// One CTA per (row, kWeightTiles tiles of 128 keys, kv head).  Bound by instruction issue (per
// 16 keys and 8 vectors D / 16 MMAs, 4 ex2 and about 20 others), so by the warps to issue from.
// D = 64: two tiles leave room for three CTAs per SM: 126.1 us for a call (24 rows, chunks of up
// to 64 tokens, the last 32 counted, Hq 16, Hk 4); four tiles and two CTAs 128.9, two and two
// 130.7, four and three (spilling) 139.1.  D = 128: two CTAs by its registers, where more tiles
// read the queries less often: four 65.0 us, two 69.1 (24 rows of 6k keys, 8 counted, Hq 32).
template <int D>
__global__ void __launch_bounds__(kWThreads, D == 64 ? 3 : 2)
    weights_kernel(const __grid_constant__ WeightsParams p) {
  constexpr int kTiles = kWeightTiles<D>;
  __shared__ __align__(16) uint8_t qs[8 * QT * kQStride<D>];
  __shared__ __align__(16) float2 ml[8 * QT];
  __shared__ int limit[8 * QT];
  const WeightsRow &row = p.rows[find_weights_row(p, blockIdx.x)];
  const int g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, qq = lane & 3;
  const int n_vec = (row.t1 - row.t0) * p.rep;
  const int keys = row.slots + row.t1;  // slots whose accumulator the launch defines
  const int kb0 = ((int)blockIdx.x - row.item0) * kTiles * kWeightTile + 16 * warp;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  float sum[kTiles][2];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) sum[i][0] = sum[i][1] = 0.f;
  for (int v0 = 0; v0 < n_vec; v0 += 8 * QT) {
    const int n_nt = min(QT, (n_vec - v0 + 7) / 8);
    uint4 a[D / 32], b[D / 32];
    load_keys<D>(p, row, g, kb0, keys - 1, lane, a, b);
    __syncthreads();
    load_queries<D>(p, row, g, v0, n_vec, qs, ml, limit);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int kb = kb0 + i * kWeightTile;
      if (kb >= keys) break;
      uint4 f[D / 16];
      fragments<D>(a, b, f);
      if (i + 1 < kTiles && kb + kWeightTile < keys)  // the next keys, meanwhile
        load_keys<D>(p, row, g, kb + kWeightTile, keys - 1, lane, a, b);
      if (kb + 15 <= row.slots + row.t0)
        sum_step<D, true>(f, qs, limit, ml, n_nt, kb + gq, p.scale_log2, lane, sum[i][0],
                          sum[i][1]);
      else
        sum_step<D, false>(f, qs, limit, ml, n_nt, kb + gq, p.scale_log2, lane, sum[i][0],
                           sum[i][1]);
    }
  }
  const float *before = row.first ? p.acc_in : p.acc_out;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      sum[i][0] += __shfl_xor_sync(0xffffffffu, sum[i][0], off);
      sum[i][1] += __shfl_xor_sync(0xffffffffu, sum[i][1], off);
    }
    if (qq < 2) {  // lanes 0 and 1 of a quad write its two keys
      const int slot = kb0 + i * kWeightTile + gq + 8 * qq;
      const int64_t at = ((int64_t)row.cache_row * p.Hk + g) * p.acc_stride + slot;
      if (slot < keys)
        p.acc_out[at] = (slot < row.known ? before[at] : 0.f) + (qq == 0 ? sum[i][0] : sum[i][1]);
    }
  }
}

// Single-token rows: the scores are there already.  One CTA per (row, 1024 slots, kv head),
// coalesced over slots; a thread's loads of its four slots are independent.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ float2 ml[kMaxRep];
  int lo = 0, hi = p.n_rows - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.rows[mid].item0 <= (int)blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const JoinRow &row = p.rows[lo];
  const int g = blockIdx.y;
  const int s0 = ((int)blockIdx.x - row.item0) * kJoinSlots + threadIdx.x;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  if (threadIdx.x < p.rep)
    ml[threadIdx.x] =
        p.row_ml[(int64_t)row.call_row * kChunk * p.Hq + g * p.rep + threadIdx.x];
  __syncthreads();
  const float *sc = p.scores + ((int64_t)lo * p.Hq + g * p.rep) * p.score_stride + s0;
  const int64_t at = ((int64_t)row.cache_row * p.Hk + g) * p.acc_stride + s0;
  constexpr int kPer = kJoinSlots / 256;
  float sum[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    sum[i] = s0 + 256 * i < row.keys - 1 ? p.acc_in[at + 256 * i] : 0.f;
  for (int h = 0; h < p.rep; ++h) {
    const float2 e = ml[h];
    float x[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      x[i] = s0 + 256 * i < row.keys ? sc[h * p.score_stride + 256 * i] : -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum[i] += exp2f(x[i] - e.x) * e.y;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (s0 + 256 * i < row.keys) p.acc_out[at + 256 * i] = sum[i];
}

}  // namespace

cudaError_t launch_join(const JoinParams &p, cudaStream_t s, bool pdl) {
  if (p.n_items <= 0) return cudaSuccess;
  return launch_k(join_kernel, dim3(p.n_items, p.Hk), dim3(256), 0, s, p, pdl);
}

cudaError_t launch_weights(const WeightsParams &p, cudaStream_t s, bool pdl) {
  if (p.n_items <= 0) return cudaSuccess;
  const dim3 grid(p.n_items, p.Hk), block(kWThreads);
  return p.D == 128 ? launch_k(weights_kernel<128>, grid, block, 0, s, p, pdl)
                    : launch_k(weights_kernel<64>, grid, block, 0, s, p, pdl);
}

}  // namespace kvinc

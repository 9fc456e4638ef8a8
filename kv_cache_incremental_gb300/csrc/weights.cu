// weights.cu -- per-key softmax weights of a call's queries, added to an accumulator.
//
// For a kv head g and a cached key j of a row, with the counted query tokens t (at slots
// s_t = slots + t) and the group's heads h,
//   acc_out[j] = acc_in[j] + sum_t sum_h [j <= s_t] 2^(x_thj - m_th) / l_th,
//   x_thj = log2(e) / sqrt(D) q_th . K_j,  m_th = max_j x_thj,  l_th = sum_j 2^(x_thj - m_th).
// A weight needs its query's m and l over all keys first.  For rows with a single new token
// the decode kernel stores the scores on its one pass over K and V (decode_kernel.cuh, the
// scores mode) and the join kernel turns them into weights: 8 bytes of scores per key and
// head, written and read, beside the 4 D bytes of a key and value (64 rows of 1k-8k keys, Hq
// 32, Hk 8, D 128: 190 us, 489 with two passes).  For chunks, and for rows whose scores
// outgrow the room reserved for them, there are two passes over K: the first leaves (m, l) per query vector and key split, the second joins the splits and
// sums the weights per key.  Both form S^T = K Q^T with mma.sync (keys on M, query vectors
// on N): a key's weights then lie in the lanes of one quad and its sum over the queries
// stays in a register; a query's running (m, l) over its lane's keys stays in registers
// too, with one exchange between lanes at the end.  Nothing is added atomically, so the
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
constexpr int kSumTiles = kWeightSumTiles;
// Query vectors are taken in chunks of 8 QT.  A chunk's unused eights are skipped: variants of
// one and two eights for single tokens ran no faster (8 counted vectors, 24 rows of 6k keys:
// 54.7 us with eight, 54.9 with one).
constexpr int QT = 8;
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
// rotates them, into shared memory, and the last slot that each sees; vectors past the last
// are zero and see nothing.
template <int D>
__device__ __forceinline__ void load_queries(const WeightsParams &p, const WeightsRow &row, int g,
                                             int v0, int n_vec, uint8_t *qs, int *limit) {
  constexpr int kHalf = D / 2, kVec = kHalf / 8;
  if (threadIdx.x < 8 * QT)
    limit[threadIdx.x] = v0 + (int)threadIdx.x < n_vec
                             ? row.slots + row.t0 + (v0 + (int)threadIdx.x) / p.rep
                             : -1;
  for (int u = threadIdx.x; u < 8 * QT * kVec; u += kWThreads) {
    const int i = u / kVec, c = u % kVec, vec = v0 + i;
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (vec < n_vec) {
      const int t = row.t0 + vec / p.rep, h = vec % p.rep;
      const __nv_bfloat16 *q = p.q + (int64_t)row.call_row * p.q_row_stride +
                               ((int64_t)t * p.Hq + g * p.rep + h) * D;
      const uint4 x1v = *reinterpret_cast<const uint4 *>(q + 8 * c);
      const uint4 x2v = *reinterpret_cast<const uint4 *>(q + kHalf + 8 * c);
      const __nv_bfloat16 *x1 = reinterpret_cast<const __nv_bfloat16 *>(&x1v);
      const __nv_bfloat16 *x2 = reinterpret_cast<const __nv_bfloat16 *>(&x2v);
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

// The exponent's reference of a query vector that has seen no key yet, and how far a score
// may lie above the reference before the sum is rescaled: sums then stay below 2^(64 + 31).
constexpr float kNoRef = -1e30f, kSlack = 64.f;

// Pass 1: one CTA per (row, key split, kv head); a reference m and the sum l = sum_j 2^(x_j -
// m) of every query vector over the split's keys.  m need not be the maximum: it moves only
// when a score exceeds it by kSlack, so that a score costs one multiply-add, one ex2 and
// one addition.
//
// One step: 16 keys as fragments f against the first n_nt eights of query vectors.  FULL: every key
// is visible to every vector; else key gq is visible up to `limit` and below k1.
template <int D, bool FULL>
__device__ __forceinline__ void stats_step(const uint4 (&f)[D / 16], const uint8_t *qs,
                                           const int *limit, int n_nt, int key, int k1,
                                           float scale, int lane, float (&nm)[QT][2],
                                           float (&l)[QT][2]) {
  constexpr int N = 2;
#pragma unroll
  for (int nt0 = 0; nt0 < QT; nt0 += N) {
    if (nt0 >= n_nt) break;
    float sc[N][4];
    scores<D, N>(f, qs, nt0, lane, sc);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float(&s)[4] = sc[i];
      const int nt = nt0 + i;
      if (!FULL) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int lim = min(k1 - 1, limit[8 * nt + 2 * (lane & 3) + j]);
          if (key > lim) s[j] = -INFINITY;
          if (key + 8 > lim) s[2 + j] = -INFINITY;
        }
      }
      float d0 = fmaf(s[0], scale, nm[nt][0]), d2 = fmaf(s[2], scale, nm[nt][0]);
      float d1 = fmaf(s[1], scale, nm[nt][1]), d3 = fmaf(s[3], scale, nm[nt][1]);
      if (__any_sync(0xffffffffu, fmaxf(fmaxf(d0, d2), fmaxf(d1, d3)) > kSlack)) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float m = -nm[nt][j], mn = fmaxf(m, fmaxf(s[j] * scale, s[2 + j] * scale));
          l[nt][j] *= ptx::ex2(m - mn);
          nm[nt][j] = -mn;
        }
        d0 = fmaf(s[0], scale, nm[nt][0]);
        d2 = fmaf(s[2], scale, nm[nt][0]);
        d1 = fmaf(s[1], scale, nm[nt][1]);
        d3 = fmaf(s[3], scale, nm[nt][1]);
      }
      l[nt][0] += ptx::ex2(d0) + ptx::ex2(d2);
      l[nt][1] += ptx::ex2(d1) + ptx::ex2(d3);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kWThreads, 2)
    weights_stats_kernel(const __grid_constant__ WeightsParams p) {
  __shared__ __align__(16) uint8_t qs[8 * QT * kQStride<D>];
  __shared__ float2 red[kWarps][8 * QT];
  __shared__ int limit[8 * QT];
  const WeightsRow &row = p.rows[find_weights_row(p, blockIdx.x)];
  const int g = blockIdx.y, split = blockIdx.x - row.item0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, qq = lane & 3;
  const int n_vec = (row.t1 - row.t0) * p.rep;
  const int keys = row.slots + row.t1;  // visible to the last counted token
  const int k0 = split * row.split_tiles * kWeightTile;
  const int k1 = min(keys, k0 + row.split_tiles * kWeightTile);
  ptx::grid_dep_wait();  // keys come from the launches before; partials are read by them
  ptx::grid_dep_launch();
  for (int v0 = 0; v0 < n_vec; v0 += 8 * QT) {
    const int n_nt = min(QT, (n_vec - v0 + 7) / 8);
    uint4 a[D / 32], b[D / 32];
    if (k0 + 16 * warp < k1) load_keys<D>(p, row, g, k0 + 16 * warp, keys - 1, lane, a, b);
    __syncthreads();
    load_queries<D>(p, row, g, v0, n_vec, qs, limit);
    __syncthreads();
    if (split == 0) {  // pass 2 takes the rotated vectors as they are
      uint4 *dst = reinterpret_cast<uint4 *>(p.rotated + (row.part + (int64_t)g * n_vec + v0) * D);
      for (int u = threadIdx.x; u < min(8 * QT, n_vec - v0) * (D / 8); u += kWThreads)
        dst[u] = *reinterpret_cast<const uint4 *>(qs + u / (D / 8) * kQStride<D> +
                                                  16 * (u % (D / 8)));
    }
    float nm[QT][2], l[QT][2];  // -m, l
#pragma unroll
    for (int nt = 0; nt < QT; ++nt) {
      nm[nt][0] = nm[nt][1] = -kNoRef;
      l[nt][0] = l[nt][1] = 0.f;
    }
    for (int kb = k0 + 16 * warp; kb < k1; kb += kWeightTile) {
      uint4 f[D / 16];
      fragments<D>(a, b, f);
      if (kb + kWeightTile < k1)  // the next keys, while these are used
        load_keys<D>(p, row, g, kb + kWeightTile, keys - 1, lane, a, b);
      if (kb + 16 <= k1 && kb + 15 <= row.slots + row.t0)
        stats_step<D, true>(f, qs, limit, n_nt, kb + gq, k1, p.scale_log2, lane, nm, l);
      else
        stats_step<D, false>(f, qs, limit, n_nt, kb + gq, k1, p.scale_log2, lane, nm, l);
    }
#pragma unroll
    for (int nt = 0; nt < QT; ++nt) {
      if (nt >= n_nt) break;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float m = -nm[nt][j];
        float mm = m;
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, off));
        float ll = l[nt][j] * ptx::ex2(m - mm);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) ll += __shfl_xor_sync(0xffffffffu, ll, off);
        if (gq == 0) red[warp][8 * nt + 2 * qq + j] = make_float2(mm, ll);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 8 * QT; i += kWThreads) {
      if (v0 + i >= n_vec) continue;
      float mm = kNoRef, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, red[w][i].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ll += red[w][i].y * ptx::ex2(red[w][i].x - mm);
      p.part_ml[row.part + (int64_t)(split * p.Hk + g) * n_vec + v0 + i] = make_float2(mm, ll);
    }
  }
}

// Pass 2: one CTA per (row, kSumTiles tiles of 128 keys, kv head).  One step as in pass 1; ml holds -m and the reciprocal of the sum.
template <int D, bool FULL>
__device__ __forceinline__ void sum_step(const uint4 (&f)[D / 16], const uint8_t *qs,
                                         const int *limit, const float2 *ml,
                                         int n_nt, int key, float scale, int lane, float &sum0,
                                         float &sum1) {
  constexpr int N = 2;
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

template <int D>
__global__ void __launch_bounds__(kWThreads, 2)
    weights_sum_kernel(const __grid_constant__ WeightsParams p) {
  __shared__ __align__(16) uint8_t qs[8 * QT * kQStride<D>];
  __shared__ __align__(16) float2 ml[8 * QT];
  __shared__ int limit[8 * QT];
  const WeightsRow &row = p.rows[find_weights_row(p, blockIdx.x)];
  const int g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, qq = lane & 3;
  const int n_vec = (row.t1 - row.t0) * p.rep;
  const int keys = row.slots + row.n;  // slots whose accumulator the call defines
  const int kb0 = ((int)blockIdx.x - row.item0) * kSumTiles * kWeightTile + 16 * warp;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  float sum[kSumTiles][2];
#pragma unroll
  for (int i = 0; i < kSumTiles; ++i) sum[i][0] = sum[i][1] = 0.f;
  for (int v0 = 0; v0 < n_vec; v0 += 8 * QT) {
    const int n_nt = min(QT, (n_vec - v0 + 7) / 8);
    uint4 a[D / 32], b[D / 32];
    load_keys<D>(p, row, g, kb0, keys - 1, lane, a, b);
    __syncthreads();
    const uint4 *src = reinterpret_cast<const uint4 *>(
        p.rotated + (row.part + (int64_t)g * n_vec + v0) * D);
    for (int u = threadIdx.x; u < 8 * QT * (D / 8); u += kWThreads) {
      const int i = u / (D / 8);
      *reinterpret_cast<uint4 *>(qs + i * kQStride<D> + 16 * (u % (D / 8))) =
          v0 + i < n_vec ? src[u] : make_uint4(0, 0, 0, 0);
    }
    for (int i = threadIdx.x; i < 8 * QT; i += kWThreads) {
      float mm = kNoRef, ll = 0.f;
      if (v0 + i < n_vec) {
        const float2 *part = p.part_ml + row.part + (int64_t)g * n_vec + v0 + i;
        const int64_t stride = (int64_t)p.Hk * n_vec;
        for (int s = 0; s < row.n_splits; ++s) mm = fmaxf(mm, part[s * stride].x);
        for (int s = 0; s < row.n_splits; ++s) {
          const float2 x = part[s * stride];
          ll += x.y * ptx::ex2(x.x - mm);
        }
      }
      // a vector past the last: weights 2^(0 - inf) * 0
      ml[i] = v0 + i < n_vec ? make_float2(-mm, 1.f / ll) : make_float2(-INFINITY, 0.f);
      limit[i] = v0 + i < n_vec ? row.slots + row.t0 + (v0 + i) / p.rep : -1;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSumTiles; ++i) {
      const int kb = kb0 + i * kWeightTile;
      if (kb >= keys) break;
      uint4 f[D / 16];
      fragments<D>(a, b, f);
      if (i + 1 < kSumTiles && kb + kWeightTile < keys)
        load_keys<D>(p, row, g, kb + kWeightTile, keys - 1, lane, a, b);
      if (kb + 15 <= row.slots + row.t0)
        sum_step<D, true>(f, qs, limit, ml, n_nt, kb + gq, p.scale_log2, lane, sum[i][0],
                              sum[i][1]);
      else
        sum_step<D, false>(f, qs, limit, ml, n_nt, kb + gq, p.scale_log2, lane, sum[i][0],
                               sum[i][1]);
    }
  }
#pragma unroll
  for (int i = 0; i < kSumTiles; ++i) {
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      sum[i][0] += __shfl_xor_sync(0xffffffffu, sum[i][0], off);
      sum[i][1] += __shfl_xor_sync(0xffffffffu, sum[i][1], off);
    }
    if (qq < 2) {  // lanes 0 and 1 of a quad write its two keys
      const int slot = kb0 + i * kWeightTile + gq + 8 * qq;
      const int64_t at = ((int64_t)row.cache_row * p.Hk + g) * p.acc_stride + slot;
      if (slot < keys) {
        const float before = slot < row.slots || !row.first ? p.acc_in[at] : 0.f;
        p.acc_out[at] = before + (qq == 0 ? sum[i][0] : sum[i][1]);
      }
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
  if (threadIdx.x < p.rep) ml[threadIdx.x] = p.row_ml[(int64_t)lo * p.Hq + g * p.rep + threadIdx.x];
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

cudaError_t launch_weights(const WeightsParams &p, int pass, cudaStream_t s, bool pdl) {
  if (p.n_items <= 0) return cudaSuccess;
  const dim3 grid(p.n_items, p.Hk), block(kWThreads);
  if (p.D == 128)
    return pass == 1 ? launch_k(weights_stats_kernel<128>, grid, block, 0, s, p, pdl)
                     : launch_k(weights_sum_kernel<128>, grid, block, 0, s, p, pdl);
  return pass == 1 ? launch_k(weights_stats_kernel<64>, grid, block, 0, s, p, pdl)
                   : launch_k(weights_sum_kernel<64>, grid, block, 0, s, p, pdl);
}

}  // namespace kvinc

// weights.cu -- per-key softmax weights of a call's queries, added to an accumulator.
//
// For a kv head g and a cached key j of a row, with the counted query tokens t (at slots
// s_t = slots + t) and the group's heads h,
//   acc_out[j] = acc_in[j] + sum_t sum_h [j <= s_t] 2^(x_thj - m_th) / l_th,
//   x_thj = log2(e) / sqrt(D) q_th . K_j,  m_th = max_j x_thj,  l_th = sum_j 2^(x_thj - m_th).
// A weight needs its query's m and l over all keys first.  For rows with a single new token
// the decode kernel stores the scores on its one pass over K and V (decode_kernel.cuh, the
// scores mode) and the join kernel turns them into weights: 8 bytes of scores per key and
// head, written and read, beside the 4 D bytes of a key and value.  For chunks, and for rows
// whose scores outgrow the room reserved for them, there are two passes over K: the first leaves (m, l) per query vector and key split, the second joins the splits and
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
// rotates them, into shared memory; vectors past the last are zero.
template <int D, int QT>
__device__ __forceinline__ void load_queries(const WeightsParams &p, const WeightsRow &row, int g,
                                             int v0, int n_vec, uint8_t *qs) {
  constexpr int kHalf = D / 2, kVec = kHalf / 8;
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

// Scores of the warp's 16 keys with query vectors 8 nt .. 8 nt + 7 of the chunk in qs.
template <int D>
__device__ __forceinline__ void scores8(const uint4 (&a)[D / 32], const uint4 (&b)[D / 32],
                                        const uint8_t *qs, int nt, int lane, float (&s)[4]) {
  const int gq = lane >> 2, qq = lane & 3;
  s[0] = s[1] = s[2] = s[3] = 0.f;
  const uint8_t *qr = qs + (8 * nt + gq) * kQStride<D> + 16 * qq;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    const uint4 w = *reinterpret_cast<const uint4 *>(qr + 64 * j);
    ptx::mma_bf16(s, a[j].x, b[j].x, a[j].y, b[j].y, w.x, w.y);
    ptx::mma_bf16(s, a[j].z, b[j].z, a[j].w, b[j].w, w.z, w.w);
  }
}

// Pass 1: one CTA per (row, key split, kv head); (m, l) of every query vector over the
// split's keys.
template <int D, int QT>
__global__ void __launch_bounds__(kWThreads)
    weights_stats_kernel(const __grid_constant__ WeightsParams p) {
  __shared__ __align__(16) uint8_t qs[8 * QT * kQStride<D>];
  __shared__ float2 red[kWarps][8 * QT];
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
    __syncthreads();
    load_queries<D, QT>(p, row, g, v0, n_vec, qs);
    __syncthreads();
    float m[QT][2], l[QT][2];
#pragma unroll
    for (int nt = 0; nt < QT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
    for (int kb = k0 + 16 * warp; kb < k1; kb += kWeightTile) {
      uint4 a[D / 32], b[D / 32];
      load_keys<D>(p, row, g, kb, keys - 1, lane, a, b);
#pragma unroll
      for (int nt = 0; nt < QT; ++nt) {
        float s[4];
        scores8<D>(a, b, qs, nt, lane, s);
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // query vector of this column
          const int limit = row.slots + row.t0 + (v0 + 8 * nt + 2 * qq + j) / p.rep;
          const float x0 = kb + gq < k1 && kb + gq <= limit ? s[j] * p.scale_log2 : -INFINITY;
          const float x1 =
              kb + gq + 8 < k1 && kb + gq + 8 <= limit ? s[2 + j] * p.scale_log2 : -INFINITY;
          const float mn = fmaxf(m[nt][j], fmaxf(x0, x1));
          const float base = mn == -INFINITY ? 0.f : mn;
          l[nt][j] = l[nt][j] * exp2f(m[nt][j] - base) + (exp2f(x0 - base) + exp2f(x1 - base));
          m[nt][j] = mn;
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < QT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mm = m[nt][j], ll = l[nt][j];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          const float mo = __shfl_xor_sync(0xffffffffu, mm, off);
          const float lo = __shfl_xor_sync(0xffffffffu, ll, off);
          const float mn = fmaxf(mm, mo), base = mn == -INFINITY ? 0.f : mn;
          ll = ll * exp2f(mm - base) + lo * exp2f(mo - base);
          mm = mn;
        }
        if (gq == 0) red[warp][8 * nt + 2 * qq + j] = make_float2(mm, ll);
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 8 * QT; i += kWThreads) {
      if (v0 + i >= n_vec) continue;
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, red[w][i].x);
      const float base = mm == -INFINITY ? 0.f : mm;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ll += red[w][i].y * exp2f(red[w][i].x - base);
      p.part_ml[row.part + (int64_t)(split * p.Hk + g) * n_vec + v0 + i] = make_float2(mm, ll);
    }
  }
}

// Pass 2: one CTA per (row, 128-key tile, kv head).
template <int D, int QT>
__global__ void __launch_bounds__(kWThreads)
    weights_sum_kernel(const __grid_constant__ WeightsParams p) {
  __shared__ __align__(16) uint8_t qs[8 * QT * kQStride<D>];
  __shared__ float2 ml[8 * QT];  // max, 1 / sum of the chunk's query vectors
  const WeightsRow &row = p.rows[find_weights_row(p, blockIdx.x)];
  const int g = blockIdx.y, tile = blockIdx.x - row.item0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, qq = lane & 3;
  const int n_vec = (row.t1 - row.t0) * p.rep;
  const int keys = row.slots + row.n;  // slots whose accumulator the call defines
  const int kb = tile * kWeightTile + 16 * warp;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  uint4 a[D / 32], b[D / 32];
  load_keys<D>(p, row, g, kb, keys - 1, lane, a, b);
  float sum0 = 0.f, sum1 = 0.f;
  for (int v0 = 0; v0 < n_vec; v0 += 8 * QT) {
    __syncthreads();
    load_queries<D, QT>(p, row, g, v0, n_vec, qs);
    for (int i = threadIdx.x; i < 8 * QT; i += kWThreads) {
      float mm = -INFINITY, ll = 0.f;
      if (v0 + i < n_vec) {
        const float2 *part = p.part_ml + row.part + (int64_t)g * n_vec + v0 + i;
        const int64_t stride = (int64_t)p.Hk * n_vec;
        for (int s = 0; s < row.n_splits; ++s) mm = fmaxf(mm, part[s * stride].x);
        for (int s = 0; s < row.n_splits; ++s) {
          const float2 x = part[s * stride];
          ll += x.y * exp2f(x.x - mm);
        }
      }
      ml[i] = make_float2(mm, 1.f / ll);
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < QT; ++nt) {
      if (v0 + 8 * nt >= n_vec) break;
      float s[4];
      scores8<D>(a, b, qs, nt, lane, s);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int vec = v0 + 8 * nt + 2 * qq + j;
        const int limit = vec < n_vec ? row.slots + row.t0 + vec / p.rep : -1;
        const float2 e = ml[8 * nt + 2 * qq + j];
        if (kb + gq <= limit) sum0 += exp2f(s[j] * p.scale_log2 - e.x) * e.y;
        if (kb + gq + 8 <= limit) sum1 += exp2f(s[2 + j] * p.scale_log2 - e.x) * e.y;
      }
    }
  }
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    sum0 += __shfl_xor_sync(0xffffffffu, sum0, off);
    sum1 += __shfl_xor_sync(0xffffffffu, sum1, off);
  }
  if (qq < 2) {  // lanes 0 and 1 of a quad write its two keys
    const int slot = kb + gq + 8 * qq;
    const int64_t at = ((int64_t)row.cache_row * p.Hk + g) * p.acc_stride + slot;
    if (slot < keys) {
      const float before = slot < row.slots || !row.first ? p.acc_in[at] : 0.f;
      p.acc_out[at] = before + (qq == 0 ? sum0 : sum1);
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

template <int D, int QT>
cudaError_t launch_weights_t(const WeightsParams &p, int pass, cudaStream_t s, bool pdl) {
  const dim3 grid(p.n_items, p.Hk), block(kWThreads);
  return pass == 1 ? launch_k(weights_stats_kernel<D, QT>, grid, block, 0, s, p, pdl)
                   : launch_k(weights_sum_kernel<D, QT>, grid, block, 0, s, p, pdl);
}

}  // namespace

cudaError_t launch_join(const JoinParams &p, cudaStream_t s, bool pdl) {
  if (p.n_items <= 0) return cudaSuccess;
  return launch_k(join_kernel, dim3(p.n_items, p.Hk), dim3(256), 0, s, p, pdl);
}

// Rows of a launch are of one kind: at most 8 query vectors (single tokens of groups of up
// to 8 heads) in one fragment, at most 16 in two, else chunks of 64.
cudaError_t launch_weights(const WeightsParams &p, int pass, cudaStream_t s, bool pdl) {
  if (p.n_items <= 0) return cudaSuccess;
  int most = 0;
  for (int i = 0; i < p.n_rows; ++i)
    most = p.rows[i].t1 - p.rows[i].t0 > most ? p.rows[i].t1 - p.rows[i].t0 : most;
  most *= p.rep;
  if (p.D == 128) {
    if (most <= 8) return launch_weights_t<128, 1>(p, pass, s, pdl);
    if (most <= 16) return launch_weights_t<128, 2>(p, pass, s, pdl);
    return launch_weights_t<128, 8>(p, pass, s, pdl);
  }
  if (most <= 8) return launch_weights_t<64, 1>(p, pass, s, pdl);
  if (most <= 16) return launch_weights_t<64, 2>(p, pass, s, pdl);
  return launch_weights_t<64, 8>(p, pass, s, pdl);
}

}  // namespace kvinc

// evict.cu -- eviction: which keys of a row stay, and moving them together.
//
// Per (row, global layer, kv head) the last `recent` of the row's keys stay, and of the
// others the keep - recent with the largest accumulated weight (ties: the lower slot; NaN
// below every number).  The kept keys keep their order: destination slot i takes the i-th
// smallest kept slot, so that "recent" still means the last slots afterwards.
//
// The choice is a radix selection: the (keep - recent)-th largest weight is found 11, 11
// and 10 bits at a time from histograms of the order-preserving whole numbers of the
// weights, then the slots above it (and the first of its ties) are written in order from
// per-warp counts.  One CTA per (row, layer, kv head); the weights stay in shared memory
// while they fit.
#include "kvinc_internal.h"
#include "ptx.cuh"

namespace kvinc {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 2048;
// Weights held in shared memory at most (192 KB); a longer row's are read again per pass (8
// rows of 16k-32k keys, the whole call: 78.2 us held, 93.3 read again).
constexpr int kHeld = 48 * 1024;

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 as +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The number order_key makes, back to its weight (a NaN to the plain one, -0 to +0).
__device__ __forceinline__ float key_weight(uint32_t k) {
  if (k == 0) return __int_as_float(0x7FC00000);
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// HELD: the row's weights stay in shared memory (every launch whose rows fit).
template <bool HELD>
__global__ void __launch_bounds__(kThreads)
    evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t held[];  // order keys
  __shared__ int hist[kBins];
  __shared__ int warp_n[kWarps][2];
  __shared__ int pick[3];  // the digit that holds the threshold, keys above it and in it
  const EvictItem &it = p.items[blockIdx.x];
  const int g = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float *acc = it.acc_in + (int64_t)g * p.acc_in_stride;
  float *out = it.acc_out ? it.acc_out + (int64_t)g * p.acc_out_stride : nullptr;
  int32_t *kept = it.kept + (int64_t)g * p.keep;
  const bool cut = it.slots > p.keep;
  const int n = cut ? it.slots - p.recent : it.slots;  // slots that compete
  const int want = cut ? p.keep - p.recent : n;
  for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
  __syncthreads();
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  if (HELD) {  // one read of the weights, with the first digit's histogram
    constexpr int kPer = 8;
    for (int i0 = 0; i0 < it.slots; i0 += kPer * kThreads) {
      float x[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = i0 + j * kThreads + tid;
        x[j] = i < it.slots ? acc[i] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = i0 + j * kThreads + tid;
        const uint32_t k = order_key(x[j]);
        if (i < it.slots) held[i] = k;
        if (cut && i < n) atomicAdd(&hist[k >> 21], 1);
      }
    }
    // Whatever follows reads keys that other threads stored -- also when nothing competes
    // (recent == keep, or a row that keeps everything) -- and may write acc_out over acc_in.
    __syncthreads();
  }
  const auto key_at = [&](int i) { return HELD ? held[i] : order_key(acc[i]); };
  uint32_t prefix = 0;  // keys above it are kept, and the first `ties` at it
  int ties = n;         // a row that keeps everything: every key is at or above 0
  if (cut && want > 0) {
    uint32_t mask = 0;
    int above = 0;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digit = pass == 2 ? 1023 : 2047;
      if (pass > 0) {
        for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
      }
      if (!HELD || pass > 0) {  // HELD: the first digit's was made with the load
#pragma unroll 4
        for (int i = tid; i < n; i += kThreads) {
          const uint32_t k = key_at(i);
          if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & digit], 1);
        }
        __syncthreads();
      }
      // Bins from the largest down, two per thread; each warp scans its 64, then adds the
      // totals of the warps before it.
      const int top = kBins - 1 - 2 * tid;
      const int c0 = hist[top], c1 = hist[top - 1];
      int incl = c0 + c1;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
      }
      if (lane == 31) warp_n[warp][0] = incl;
      __syncthreads();
      int before = lane < warp ? warp_n[lane][0] : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
      const int run = above + before + incl - c0 - c1;  // keys above this thread's bins
      if (run < want && run + c0 >= want) {
        pick[0] = top;
        pick[1] = run;
        pick[2] = c0;
      } else if (run + c0 < want && run + c0 + c1 >= want) {
        pick[0] = top - 1;
        pick[1] = run + c0;
        pick[2] = c1;
      }
      __syncthreads();
      prefix |= (uint32_t)pick[0] << shift;
      mask |= digit << shift;
      above = pick[1];
      ties = want - above;
      if (pick[2] == ties && prefix > 0) {  // every key from the prefix on: no more digits
        prefix -= 1;
        ties = 0;
        break;
      }
    }
  }
  if (want > 0) {
    // Each warp writes the kept slots of one contiguous range, after those of the warps
    // before it.
    const int per = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int a = min(warp * per, n), b = min(a + per, n);
    const auto keep_slot = [&](int at, int i, uint32_t k) {
      kept[at] = i;
      if (HELD && out) out[at] = key_weight(k);
    };
    const uint32_t below = (1u << lane) - 1;
    int gt = 0, eq = 0;
#pragma unroll 4
    for (int i = a + lane; i < b; i += 32) {
      const uint32_t k = key_at(i);
      gt += k > prefix;
      if (ties > 0) eq += k == prefix;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    __syncthreads();  // warp_n of the last digit has been read
    if (lane == 0) {
      warp_n[warp][0] = gt;
      warp_n[warp][1] = eq;
    }
    __syncthreads();
    gt = __reduce_add_sync(0xffffffffu, lane < warp ? warp_n[lane][0] : 0);
    eq = __reduce_add_sync(0xffffffffu, lane < warp ? warp_n[lane][1] : 0);
    if (ties == 0) {
#pragma unroll 4
      for (int i0 = a; i0 < b; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < b ? key_at(i) : 0;
        const bool is_gt = i < b && k > prefix;
        const uint32_t bg = __ballot_sync(0xffffffffu, is_gt);
        if (is_gt) keep_slot(gt + __popc(bg & below), i, k);
        gt += __popc(bg);
      }
    } else {
      for (int i0 = a; i0 < b; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < b ? key_at(i) : 0;
        const bool is_gt = i < b && k > prefix, is_eq = i < b && k == prefix;
        const uint32_t bg = __ballot_sync(0xffffffffu, is_gt);
        const uint32_t be = __ballot_sync(0xffffffffu, is_eq);
        const int ng = gt + __popc(bg & below), ne = eq + __popc(be & below);
        if (is_gt || (is_eq && ne < ties)) keep_slot(ng + min(ne, ties), i, k);
        gt += __popc(bg);
        eq += __popc(be);
      }
    }
  }
  if (cut) {
    for (int i = tid; i < p.recent; i += kThreads) {
      kept[want + i] = n + i;
      if (HELD && out) out[want + i] = key_weight(held[n + i]);
    }
  } else {
    for (int i = it.slots + tid; i < p.keep; i += kThreads) kept[i] = -1;
  }
  if (HELD || !out) return;
  // The kept accumulators, moved together.  acc_out may be acc_in: a kept slot never lies
  // below its destination, so what a pass writes has been read by it or an earlier one.
  const int m = min(it.slots, p.keep);
  __syncthreads();
  for (int i0 = 0; i0 < m; i0 += kThreads) {
    const int i = i0 + tid;
    const float x = i < m ? acc[kept[i]] : 0.f;
    __syncthreads();
    if (i < m) out[i] = x;
    __syncthreads();
  }
}

constexpr int kMoveThreads = 256;
// Destination slots per CTA and pass.
constexpr int kMoveSlots = 64, kMoveSlotsInPlace = 256;

// Kept keys and values of one (row, layer, kv head) to their destination slots.  Out of
// place, blockIdx.x numbers (item, 64 destination slots).  IN_PLACE: one CTA walks all of
// an item's slots from the first that moves, 256 at a time with a barrier between a pass's
// loads and its stores -- a source slot never lies below its destination, so what a pass
// overwrites has been read; blockIdx.z takes one of four quarters of the head dimension.
template <int D, bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads)
    evict_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kChunks = IN_PLACE ? D / 32 : D / 8;  // 16-byte chunks of a slot per CTA
  constexpr int kSlots = IN_PLACE ? kMoveSlotsInPlace : kMoveSlots;
  constexpr int kUnits = kSlots * kChunks / kMoveThreads;
  static_assert(kUnits >= 1, "every thread has a chunk");
  const int passes = (p.keep + kSlots - 1) / kSlots;
  const EvictItem &it = p.items[IN_PLACE ? blockIdx.x : blockIdx.x / passes];
  const int g = blockIdx.y;
  const int m = min(it.slots, p.keep);
  const int32_t *kept = it.kept + (int64_t)g * p.keep;
  const int chunk0 = IN_PLACE ? blockIdx.z * kChunks : 0;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  int i0 = IN_PLACE ? 0 : (blockIdx.x % passes) * kSlots;
  if (i0 >= m) return;
  if (IN_PLACE) {  // kept[i] - i never falls: the first slot that moves
    int lo = 0, hi = m;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (kept[mid] > mid) hi = mid;
      else lo = mid + 1;
    }
    i0 = lo;
  }
  for (; i0 < m; i0 += kSlots) {
    uint4 k[kUnits], v[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int x = threadIdx.x + u * kMoveThreads, i = i0 + x / kChunks;
      if (i >= m) continue;
      const int64_t s = kv_row(p.src_pt, it.src_row, p.Hk, g, p.src_seg, kept[i]) * D +
                        8 * (chunk0 + x % kChunks);
      k[u] = *reinterpret_cast<const uint4 *>(it.src_k + s);
      v[u] = *reinterpret_cast<const uint4 *>(it.src_v + s);
    }
    if (IN_PLACE) __syncthreads();
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int x = threadIdx.x + u * kMoveThreads, i = i0 + x / kChunks;
      if (i >= m) continue;
      const int64_t d = kv_row(p.dst_pt, it.dst_row, p.Hk, g, p.dst_seg, i) * D +
                        8 * (chunk0 + x % kChunks);
      *reinterpret_cast<uint4 *>(it.dst_k + d) = k[u];
      *reinterpret_cast<uint4 *>(it.dst_v + d) = v[u];
    }
    if (!IN_PLACE) return;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictParams &p, cudaStream_t s, bool pdl) {
  if (p.n_items <= 0) return cudaSuccess;
  const dim3 grid(p.n_items, p.Hk);
  if (p.max_slots <= kHeld)
    return launch_k(evict_select_kernel<true>, grid, dim3(kThreads), 4 * (size_t)p.max_slots, s, p,
                    pdl);
  return launch_k(evict_select_kernel<false>, grid, dim3(kThreads), 0, s, p, pdl);
}

cudaError_t launch_evict_move(const EvictParams &p, bool in_place, cudaStream_t s, bool pdl) {
  if (p.n_items <= 0) return cudaSuccess;
  const dim3 block(kMoveThreads);
  if (in_place) {
    const dim3 grid(p.n_items, p.Hk, 4);
    return p.D == 128 ? launch_k(evict_move_kernel<128, true>, grid, block, 0, s, p, pdl)
                      : launch_k(evict_move_kernel<64, true>, grid, block, 0, s, p, pdl);
  }
  const dim3 grid(p.n_items * ((p.keep + kMoveSlots - 1) / kMoveSlots), p.Hk);
  return p.D == 128 ? launch_k(evict_move_kernel<128, false>, grid, block, 0, s, p, pdl)
                    : launch_k(evict_move_kernel<64, false>, grid, block, 0, s, p, pdl);
}

cudaError_t configure_evict() {
  return cudaFuncSetAttribute(evict_select_kernel<true>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kHeld);
}

}  // namespace kvinc

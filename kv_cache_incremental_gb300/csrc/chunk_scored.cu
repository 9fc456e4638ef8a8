// chunk_scored.cu -- attention of chunk rows and drafted trees with changed scores
// (kv_append_scored, kv_append_tree) on the 5th-generation tensor cores.
//
// What is computed: query row rho of a (row, kv head) is token t = rho / rep, head rho % rep of the
// GQA group.  With x its score (scaled, capped by cap tanh(x / cap), less slope |distance|; log2
// units), out = sum_j 2^(x_j - m) V_j / sum_j 2^(x_j - m) over the keys it sees.
//
// One CTA owns up to 128 query rows (the MMA's M) of one (row, kv head) and a range of its keys, in
// blocks of 128 (two 64-key TMA tiles): S = Q K^T into one of three buffers in TMEM, softmax,
// O += P_hi V + P_lo V with P over S's columns (bf16 high and low parts: 16 bits of a weight; one
// part would cost 2^-9 of it, and a token would not get the same from a draft as from a decode
// step).  S of the next block is computed during the softmax of this one, and O of this one
// during that of the next.
//
// What bounds such a chain is latency, not a pipe: with four softmax warps per 128 rows
// (as in prefill_tc.cu) 32 rows of 4096 keys, 16 tokens, Hq 32, Hk 8, D 128, kept the issue slots
// at 26% and the tensor pipe at 24% busy (225 us).  So the softmax has as many warps as registers
// allow, sixteen: four threads per query row, 32 of the block's keys each, which a thread holds
// in registers from TMEM to TMEM.  The four keep the same maximum; it moves, and O is rescaled,
// only when a score exceeds it by kRise, on a vote of their warps.  Weights up to 2^kRise cost
// no accuracy (floats and bf16 halves are relative), but with values above 2^95 a sum may overflow.
//
// Measured: 64 rows of 1k to 8k keys, 4 to 16 drafts, Hq 32, Hk 8, D 128, 196 us: 92% of the
// copy rate.  16 rows of 16k to 32k keys, 8 to 32 drafts, Hq 64, Hk 8, capped, 463 us.  A block takes
// 2 700 to 2 800 cycles, 2 000 to 2 200 without a cap, its products 1 540; a CTA 15 000 beside its
// blocks.
//
// A hidden key's weight is 0, but 0 times infinity is NaN.  So when an output is not finite, the
// CTA runs over its blocks a second time with such values set to 0 and the maximum exact at every
// block (weights up to 1), and the rows that see none of them take that.  (Values are looked at only
// then: a scan of every tile would be on the chain.)
//
// A piece of a split row's keys may hold no block for a query tile.  Such a CTA has no MMAs to wait
// for, so it commits none either: a commit's arrival that nothing waits for could come after the
// CTA's end, in shared memory that is the next CTA's.
//
// Warps: 0-15 softmax (quarter of the block, 32 rows); 16 and 19 load K and V; 17 (which owns
// TMEM) issues the MMAs of S, 18 those of O.  Each is one thread's work: a TMA box takes its
// issuer about 200 cycles, an MMA 60 to 100, and a read of shared memory after MMAs stalls for
// 500 (24 rows of 4096 keys, 32 tokens, Hq 64, Hk 8: one thread for both loads 165 us, or for S
// and O 182, four threads 153).  Every mbarrier is waited for phase by phase by the same
// thread, or the argument is given at the wait.  Every wait is bounded; on a timeout the CTA
// records the error, keeps passing its named barriers, lets its own loads and MMAs finish
// (bounded), frees its TMEM and returns.
#include <type_traits>

#include "kvinc_internal.h"
#include "ptx.cuh"
#include "score_mod.cuh"

namespace kvinc {
namespace {

constexpr int kRows = 128;        // query rows of a tile (MMA M)
constexpr int kKeys = kTileKeys;  // keys per TMA tile
constexpr int kBlockKeys = 2 * kKeys;
constexpr int kPart = 32;         // keys of a softmax thread
constexpr int kSoftWarps = 16, kSoftThreads = 32 * kSoftWarps;
constexpr int kWarpK = kSoftWarps, kWarpS = kWarpK + 1, kWarpO = kWarpS + 1, kWarpV = kWarpO + 1;
constexpr int kThreads = 32 * (kWarpV + 1);  // 20 warps: five per sub-partition, 96 registers
constexpr float kRise = 32.f;  // of the first run
constexpr int kBufs = 3;  // S buffers: one in the softmax, one ahead, one whose P is read
constexpr int kFar = 1 << 30;  // past any position
// Named barriers: 1-4 the four warps of 32 query rows, 5-8 of a quarter of the keys, 15 all
// softmax.
constexpr int kBarRows = 1, kBarQuarter = 5, kBarAll = 15;

// What a CTA works on, in shared memory: the softmax warps have no registers for it.
struct Geo {
  int entry, head, rho0, n_rho;
  int lens, prefix;
  // Key segments: 0 the layer storage (sl0 keys), 2 the chunk scratch of a sliding layer or a
  // tree's draft room (sl2 keys), whose 64-key tiles start at tile st2; j_end: past the last
  // tile.
  int sl0, sl2, st2, j_end;
  // Of the blocks that count, those from i0 on are this entry's.  Those between the prefix and the
  // first key that any of the CTA's tokens sees do not: the first b_near blocks follow one another,
  // the others start b_gap blocks further on.
  int i0, n_blocks, b_near, b_gap;
  // Block of turn `it`, the newest first: a bias that falls with the distance then leaves the
  // maximum where the first block put it.
  __device__ __forceinline__ int block(int it) const volatile {
    const int i = i0 + n_blocks - 1 - it;
    return i + (i >= b_near ? b_gap : 0);
  }
};
struct Flags {
  uint32_t tmem;
  int fail;
  int again;  // an output is not finite
  int issued_k, issued_v;  // blocks
  int last;                // this CTA merges
  uint32_t row_bad[4];     // rows that see a value that is not finite, a bit for each
  uint32_t key_bad[4];     // and the keys of the block's quarters that have one
};

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kStages = D == 128 ? 3 : 6;       // of the K ring and of the V ring
  static constexpr int kQBytes = kPanels * kRows * 128;  // one Q tile, K-major, 128B swizzle
  static constexpr int kPanelBytes = kBlockKeys * 128;   // 64 dims of one K or V block
  static constexpr int kTileBytes = kKeys * 128;         // one 64-key TMA box of a panel
  static constexpr int kBlockBytes = kPanels * kPanelBytes;
  static constexpr int kOff_Q = 0;
  static constexpr int kOff_K = kQBytes;
  static constexpr int kOff_V = kOff_K + kStages * kBlockBytes;
  static constexpr int kOff_Row = kOff_V + kStages * kBlockBytes;  // [4][128] per quarter and row
  static constexpr int kOff_Parents = kOff_Row + 4 * kRows * 4;    // [64]
  static constexpr int kOff_Geo = kOff_Parents + kChunk * 4;
  static constexpr int kOff_Bar = kOff_Geo + (sizeof(Geo) + 7) / 8 * 8;
  static constexpr int kBars = 4 * kStages + 3 * kBufs + 2;  // of one run over the blocks
  static constexpr int kOff_Flags = kOff_Bar + 2 * kBars * 8;
  static constexpr int kSmem = kOff_Flags + sizeof(Flags);
  static_assert(kSmem <= 232448, "shared memory per CTA");
};
// TMEM columns: S of block b at 128 (b % 3) (per 16 keys then 8 columns of P's high part and 8
// of its low one, two keys each), O behind.
constexpr int kColO = kBufs * kBlockKeys, kTmemCols = 512;

// A run's barriers, in this order; a second run has its own.
template <int D>
struct Bars {
  uint64_t *b;
  __device__ __forceinline__ Bars(uint8_t *smem, int run)
      : b(reinterpret_cast<uint64_t *>(smem + Cfg<D>::kOff_Bar) + run * Cfg<D>::kBars) {}
  static constexpr int kSt = Cfg<D>::kStages, kP = 4 * kSt + 2 * kBufs + 1;
  __device__ __forceinline__ uint64_t *k_full(int s) const { return b + s; }  // [stage] TMA -> MMA
  __device__ __forceinline__ uint64_t *v_full(int s) const { return b + kSt + s; }
  __device__ __forceinline__ uint64_t *k_empty(int s) const { return b + 2 * kSt + s; }  // S -> TMA
  __device__ __forceinline__ uint64_t *v_empty(int s) const { return b + 3 * kSt + s; }  // O -> TMA
  // [buffer] S done -> softmax; O of the block done -> MMA, softmax
  __device__ __forceinline__ uint64_t *s_full(int i) const { return b + 4 * kSt + i; }
  __device__ __forceinline__ uint64_t *o_done(int i) const { return b + 4 * kSt + kBufs + i; }
  __device__ __forceinline__ uint64_t *drain() const { return b + kP - 1; }  // every MMA done
  // Sixteen warps each: [buffer] softmax wrote P -> MMA; rotated queries stored -> MMA
  __device__ __forceinline__ uint64_t *p_full(int i) const { return b + kP + i; }
  __device__ __forceinline__ uint64_t *q_ready() const { return b + kP + kBufs; }
};
template <int D>
__device__ __forceinline__ volatile Flags *flags_of(uint8_t *smem) {
  return reinterpret_cast<volatile Flags *>(smem + Cfg<D>::kOff_Flags);
}
template <int D>
__device__ __forceinline__ volatile Geo *geo_of(uint8_t *smem) {
  return reinterpret_cast<volatile Geo *>(smem + Cfg<D>::kOff_Geo);
}
template <int D>
__device__ __forceinline__ void give_up(const ScoredPrefillParams &p, uint8_t *smem) {
  atomicExch(p.err, 1);
  flags_of<D>(smem)->fail = 1;
}

// A work item: the entry, its kv head and its query tile; items go by entry, then by kv head,
// then by tile, so that the tiles that share keys run together.  A division when all entries
// have the same number of tiles (each probe of the search is a dependent parameter load, slow at
// kernel start).
struct Item {
  int entry, head, tile;
};
__device__ __forceinline__ Item find_item(const ScoredPrefillParams &p, int w) {
  Item it;
  int first = 0, tiles = p.uniform_tiles;
  if (tiles > 0) {
    it.entry = w / (tiles * p.Hk);
    first = it.entry * tiles;
  } else {
    int lo = 0, hi = p.n_rows - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.rows[mid].cta0 * p.Hk <= w) lo = mid;
      else hi = mid - 1;
    }
    it.entry = lo;
    first = p.rows[lo].cta0;
    tiles = (lo + 1 < p.n_rows ? (int)p.rows[lo + 1].cta0 : p.n_ctas) - first;
  }
  const int rest = w - first * p.Hk;
  it.head = rest / tiles;
  it.tile = rest % tiles;
  return it;
}

// Token of a query row (its head is the rest): an exact product with 2^32 / rep, rounded up, since
// rows times rep stay below 2^32.
__device__ __forceinline__ int token_of(const ScoredPrefillParams &p, int rho) {
  return p.rep_inv ? (int)__umulhi(rho, p.rep_inv) : rho;
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Barrier of `threads` threads, and whether any of them says so.
__device__ __forceinline__ bool bar_any(int id, int threads, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"((uint32_t)mine), "r"(threads)
      : "memory");
  return any != 0;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Largest and smallest of 32 values, 16 three-input instructions each.
template <class F>
__device__ __forceinline__ float reduce32(const float (&v)[32], F f3) {
  float a[11];
#pragma unroll
  for (int k = 0; k < 10; ++k) a[k] = f3(v[3 * k], v[3 * k + 1], v[3 * k + 2]);
  a[10] = f3(v[30], v[31], v[31]);
#pragma unroll
  for (int k = 0; k < 3; ++k) a[k] = f3(a[3 * k], a[3 * k + 1], a[3 * k + 2]);
  return f3(f3(a[0], a[1], a[2]), a[9], a[10]);
}
__device__ __forceinline__ float max32(const float (&v)[32]) { return reduce32(v, fmax3); }
__device__ __forceinline__ float min32(const float (&v)[32]) { return reduce32(v, fmin3); }

// 32 consecutive columns of the lane's TMEM row (as tc::ld16), and the wait for them.
__device__ __forceinline__ void ld32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
        "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
        "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
        "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]),
        "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
// O's columns of a thread times alpha.
template <int D>
__device__ __noinline__ void rescale(uint32_t tO, float alpha) {
#pragma unroll 1
  for (int c = 0; c < D / 64; ++c) {
    float o16[16];
    tc::ld16(tO + 16 * c, o16);
    tc::wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) o16[k] *= alpha;
    tc::st16(tO + 16 * c, o16);
  }
  tc::wait_st();
}

// A bounded wait; over when another warp has given up.  (A flag read after tcgen05 instructions
// stalls for hundreds of cycles, so it is read only when there is time.)
template <int D>
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, uint8_t *smem) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (flags_of<D>(smem)->fail) return false;
  }
  return false;
}

// Values of a quarter of a V block (the second run): infinities and NaN become 0, and their
// keys' bits are set in *keys.  `u0` of 128 threads.
template <int D>
__device__ __noinline__ void clean_values(uint8_t *vt, int key0, int u0, uint32_t *keys) {
  for (int u = u0; u < kPart * (D / 8); u += 128) {
    const int key = u / (D / 8), ch = u % (D / 8);
    uint4 *at = reinterpret_cast<uint4 *>(vt + (ch / 8) * (kBlockKeys * 128) +
                                          ptx::swz128(key0 + key, ch % 8));
    uint4 x = *at;
    uint32_t *w = reinterpret_cast<uint32_t *>(&x);
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if ((w[k] & 0x7f80u) == 0x7f80u) w[k] &= 0xffff0000u, bad = true;
      if ((w[k] & 0x7f800000u) == 0x7f800000u) w[k] &= 0xffffu, bad = true;
    }
    if (bad) {
      *at = x;
      atomicOr(keys, 1u << key);
    }
  }
}

// The loads of K or of V of a run: one thread.
template <int D>
__device__ __forceinline__ void load_run(const ScoredPrefillParams &p, uint8_t *smem, Bars<D> bar,
                                         bool value) {
  using C = Cfg<D>;
  const volatile Geo &geo = *geo_of<D>(smem);
  const int cache_row = p.rows[geo.entry].cache_row, g = geo.head, n_blocks = geo.n_blocks;
  const int st2 = geo.st2, j_end = geo.j_end;
  const int64_t rh = (int64_t)cache_row * p.Hk + g;
  ptx::prefetch_tmap(value ? &p.tmap_v : &p.tmap_k);
  for (int it = 0; it < n_blocks; ++it) {
    const int s = it % C::kStages;
    if (it >= C::kStages && !wait<D>(value ? bar.v_empty(s) : bar.k_empty(s),
                                     ((it / C::kStages) - 1) & 1, smem))
      return give_up<D>(p, smem);
    uint8_t *dst = smem + (value ? C::kOff_V : C::kOff_K) + s * C::kBlockBytes;
    uint64_t *full = value ? bar.v_full(s) : bar.k_full(s);
    const int b = geo.block(it);
    const int halves = min(2, j_end - 2 * b);  // a last block may hold one tile
    ptx::mbar_arrive_expect_tx(full, halves * C::kPanels * C::kTileBytes);
    for (int h = 0; h < halves; ++h) {
      const int j = 2 * b + h;
      const bool stored = j < st2;
      const int y = static_cast<int>(stored ? rh * p.seg_rows + (int64_t)j * kKeys
                                            : rh * kChunk + (int64_t)(j - st2) * kKeys);
      int4 y4 = make_int4(y, y + kBlockTokens, y + 2 * kBlockTokens, y + 3 * kBlockTokens);
      if (stored && p.pt.max_blocks) y4 = kv_rows4(p.pt, cache_row, g, j * kKeys);
      uint8_t *at = dst + h * C::kTileBytes;
      if (rows4_contiguous(y4)) {  // dense, or a paged tile of consecutive blocks
        const CUtensorMap *m =
            value ? (stored ? &p.tmap_v : &p.tmap_sv) : (stored ? &p.tmap_k : &p.tmap_sk);
#pragma unroll
        for (int pn = 0; pn < C::kPanels; ++pn)
          ptx::tma_load_2d(at + pn * C::kPanelBytes, m, pn * 64, y4.x, full);
      } else {  // paged: four 16-key blocks, 16-row boxes
        const CUtensorMap *m = value ? &p.tmap_v16 : &p.tmap_k16;
        const int ys[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int pn = 0; pn < C::kPanels; ++pn)
            ptx::tma_load_2d(at + pn * C::kPanelBytes + i * kBlockTokens * 128, m, pn * 64, ys[i],
                             full);
      }
    }
    (value ? flags_of<D>(smem)->issued_v : flags_of<D>(smem)->issued_k) = it + 1;
  }
}

// The MMAs of S of a run: one thread.
template <int D>
__device__ __forceinline__ void s_run(const ScoredPrefillParams &p, uint8_t *smem, Bars<D> bar,
                                      uint32_t tmem) {
  using C = Cfg<D>;
  constexpr uint32_t kIdS = tc::idesc_bf16_f32(kRows, kBlockKeys);
  const int n_blocks = geo_of<D>(smem)->n_blocks;
  // (descriptors of later addresses: the address / 16 is added)
  const uint64_t q_desc = tc::desc_sw128(ptx::smem_u32(smem + C::kOff_Q));
  const uint64_t k_desc = tc::desc_sw128(ptx::smem_u32(smem + C::kOff_K));
  // S of block b into buffer b % 3, over the columns of P of block b - 3, once O has read it.  A
  // block with one tile still multiplies all 128 rows of its K stage; the softmax masks the
  // absent half.
  bool ok = n_blocks == 0 || wait<D>(bar.q_ready(), 0, smem);
  int s = 0, buf = 0;
  uint32_t k_phase = 0, o_phase = 1;
  for (int b = 0; ok && b < n_blocks; ++b) {
    ok = wait<D>(bar.k_full(s), k_phase, smem) &&
         (b < kBufs || wait<D>(bar.o_done(buf), o_phase, smem));
    if (!ok) break;
    tc::fence_after();
    const uint64_t kd = k_desc + s * (C::kBlockBytes >> 4);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      tc::mma(tmem + kBlockKeys * buf, q_desc + (((kk / 4) * (kRows * 128) + 32 * (kk % 4)) >> 4),
              kd + (((kk / 4) * C::kPanelBytes + 32 * (kk % 4)) >> 4), kIdS, kk > 0);
    tc::commit(bar.s_full(buf));
    tc::commit(bar.k_empty(s));
    if (++s == C::kStages) s = 0, k_phase ^= 1;
    if (++buf == kBufs) buf = 0, o_phase ^= 1;
  }
  if (!ok) give_up<D>(p, smem);
  if (n_blocks > 0) tc::commit(bar.drain());  // (without a block no one waits for it)
}

// The MMAs of O of a run: one thread.
template <int D>
__device__ __forceinline__ void o_run(const ScoredPrefillParams &p, uint8_t *smem, Bars<D> bar,
                                      uint32_t tmem) {
  using C = Cfg<D>;
  constexpr uint32_t kIdO = tc::idesc_bf16_f32(kRows, D, /*b_mn_major=*/true);
  const int n_blocks = geo_of<D>(smem)->n_blocks;
  const uint64_t v_desc = tc::desc_sw128_mn(ptx::smem_u32(smem + C::kOff_V), C::kPanelBytes, 1024);
  bool ok = true;
  int s = 0, buf = 0;
  uint32_t v_phase = 0, p_phase = 0;
  for (int b = 0; ok && b < n_blocks; ++b) {
    ok = wait<D>(bar.v_full(s), v_phase, smem) && wait<D>(bar.p_full(buf), p_phase, smem);
    if (!ok) break;
    tc::fence_after();
    const uint64_t vd = v_desc + s * (C::kBlockBytes >> 4);
#pragma unroll
    for (int ks = 0; ks < kBlockKeys / 16; ++ks) {
      const uint32_t tP = tmem + kBlockKeys * buf + 16 * ks;
      tc::mma_ts(tmem + kColO, tP, vd + (ks * 16 * 128 >> 4), kIdO, b > 0 || ks > 0);
      tc::mma_ts(tmem + kColO, tP + 8, vd + (ks * 16 * 128 >> 4), kIdO, true);
    }
    tc::commit(bar.o_done(buf));
    tc::commit(bar.v_empty(s));
    if (++s == C::kStages) s = 0, v_phase ^= 1;
    if (++buf == kBufs) buf = 0, p_phase ^= 1;
  }
  if (!ok) give_up<D>(p, smem);
  if (n_blocks > 0) tc::commit(bar.drain());  // (without a block no one waits for it)
}

// What a softmax thread's query row sees: positions from `first` to `pos` (a tree: all cached ones
// from `first` on), the prefix, or of the drafts those of its lineage (within the window); its
// head's slope in log2 units.  Of the turns [open0, open1) of blocks all of the warp's rows see all
// of the thread's keys: those of full-length storage between the latest first position and the
// earliest own one.
struct Sees {
  uint64_t line;
  int pos, first;
  float slope;
  int open0, open1;
};

// Query row o of a (row, kv head) in the output.
__device__ __forceinline__ __nv_bfloat16 *out_row(const ScoredPrefillParams &p, int entry, int g,
                                                  int o, int D) {
  const int t = token_of(p, o);
  return p.out + (int64_t)p.rows[entry].call_row * p.out_row_stride +
         ((int64_t)t * p.Hq + g * p.rep + o - t * p.rep) * D;
}

// A softmax warp's run over the blocks, and the rows' outputs.  kClean: the second run, without
// values that are not finite and with weights up to 1.
template <int D, bool kClean>
__device__ __forceinline__ void softmax_run(const ScoredPrefillParams &p, uint8_t *smem,
                                            Bars<D> bar, uint32_t tmem, const Sees &see) {
  using C = Cfg<D>;
  constexpr int kStages = C::kStages;
  volatile Flags *fl = flags_of<D>(smem);
  volatile Geo *geo = geo_of<D>(smem);
  float *row_num = reinterpret_cast<float *>(smem + C::kOff_Row);  // [quarter][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp / 4;       // of the block's keys
  const int r = threadIdx.x % kRows;  // query row of this thread = TMEM lane
  const uint32_t lane_off = (uint32_t)(32 * (warp % 4)) << 16;
  const uint32_t tO = tmem + kColO + D / 4 * quarter + lane_off;  // this thread's quarter of O
  const int rows_bar = kBarRows + warp % 4;
  float *num_mine = row_num + quarter * kRows + r;
  const bool tree = p.parents != nullptr;
  const bool capped = p.cap_in > 0.f, sloped = p.slopes != nullptr;
  const float sc = capped || sloped ? 1.f : p.scale_log2;
  const int n_blocks = geo->n_blocks;
  const bool qvalid = geo->rho0 + r < geo->n_rho;
  // A warp whose rows are all past the last one computes nothing: O reads its lanes' P (stale),
  // which only reach O rows that are never stored.
  const bool idle = geo->rho0 + 32 * (warp % 4) >= geo->n_rho;
  // Bits lo..hi of the thread's 32 keys (none when lo > hi).
  const auto range_bits = [](int lo, int hi) -> uint32_t {
    lo = max(lo, 0);
    hi = min(hi, kPart - 1);
    if (lo > hi) return 0u;
    return (hi == 31 ? ~0u : (2u << hi) - 1u) & ~((1u << lo) - 1u);
  };
  float m_used = -INFINITY;
  uint64_t l2[2] = {ptx::f2_pack(0.f, 0.f), ptx::f2_pack(0.f, 0.f)};  // sums of the weights
  bool ok = true;
  int buf = 0;         // S buffer of the block
  uint32_t phase = 0;  // of its barriers
#pragma unroll 1
  for (int it = 0; it < n_blocks; ++it) {
    const uint32_t tS = tmem + kBlockKeys * buf + kPart * quarter + lane_off;
    const bool whole = it >= see.open0 && it < see.open1;
    bool open = whole;
    int left = kPart;     // of the thread's 32 keys, those that exist
    uint32_t bits = ~0u;  // and those that the row sees
    // Key k of them is at position at + k, in a ring past its newest slot (k > wrap) R lower; ln:
    // drafts, the row's lineage from the first of them on.
    int at = 0, wrap = kPart;
    uint64_t ln = 0;
    if (whole) {
      if (sloped) at = geo->block(it) * kBlockKeys + kPart * quarter;
    } else {
      const int j = 2 * geo->block(it) + quarter / 2;
      const bool more = j >= geo->st2;  // in the scratch or the draft room
      const int ki = (more ? j - geo->st2 : j) * kKeys + quarter % 2 * kPart;
      left = j < geo->j_end ? min(kPart, (more ? geo->sl2 : geo->sl0) - ki) : 0;
      const int lens = geo->lens;
      at = ki + (more ? lens : 0);
      if (!more && p.sliding && lens > p.ring_R) {
        at += (lens - 1) / p.ring_R * p.ring_R;
        wrap = (lens - 1) % p.ring_R - ki;
      }
      if (more && tree) {
        ln = see.line >> ki;
        bits = (uint32_t)ln;
        wrap = INT32_MIN;  // told by ln
      } else {
        const int hi = tree ? INT32_MAX - at : see.pos - at, lo = see.first - at;
        bits = wrap >= kPart - 1
                   ? range_bits(lo, hi)
                   : (range_bits(lo, min(hi, wrap)) |
                      range_bits(max(lo + p.ring_R, wrap + 1), kPart - 1));
        const int prefix = geo->prefix;
        if (!more && prefix > ki) bits |= range_bits(0, prefix - 1 - ki);
      }
      if (left < kPart) bits &= left > 0 ? range_bits(0, left - 1) : 0u;
      if (!qvalid) bits = 0;
      open = __all_sync(0xffffffffu, bits == ~0u);
    }
    // warp-uniform decisions: tcgen05.ld / st are warp-collective
    ok = ok && __all_sync(0xffffffffu, wait<D>(bar.s_full(buf), phase, smem));
    tc::fence_after();
    if (left < kPart || kClean) {
      // (The phases of v_full before this one are done, as O of their blocks is, and the next ones
      // cannot be before O of this block.)
      const int s = it % kStages;
      ok = ok && __all_sync(0xffffffffu, wait<D>(bar.v_full(s), (it / kStages) & 1, smem));
      uint8_t *vt = smem + C::kOff_V + s * C::kBlockBytes;
      // Values past a segment's end may be anything: zeros, so that 0 * V stays 0.
      const int from = max(left, 0);
      for (int u = r; ok && u < (kPart - from) * (D / 8); u += kRows) {
        const int vr = kPart * quarter + from + u / (D / 8), ch = u % (D / 8);
        *reinterpret_cast<uint4 *>(vt + (ch / 8) * C::kPanelBytes + ptx::swz128(vr, ch % 8)) =
            make_uint4(0, 0, 0, 0);
      }
      if (kClean) {
        uint32_t *keys = const_cast<uint32_t *>(&fl->key_bad[quarter]);
        bar_sync(kBarQuarter + quarter, kRows);  // the zeros are written, *keys is 0
        if (ok) clean_values<D>(vt, kPart * quarter, r, keys);
        bar_sync(kBarQuarter + quarter, kRows);
        if (bits & *(volatile uint32_t *)keys)
          atomicOr(const_cast<uint32_t *>(&fl->row_bad[r / 32]), 1u << (r % 32));
        bar_sync(kBarQuarter + quarter, kRows);
        if (r == 0) *keys = 0;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (!idle) {
      // With `top` the largest of the scores: the maximum of the row, then the weights 2^(x -
      // m), x = scaled(v), over the columns of the scores.
      const auto finish = [&](const float (&v)[kPart], float top, auto scaled) {
        const bool rise =
            m_used == -INFINITY ? top > -INFINITY : top > m_used + (kClean ? 0.f : kRise);
        if (bar_any(rows_bar, 128, rise)) {
          *num_mine = top;
          bar_sync(rows_bar, 128);
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, row_num[k * kRows + r]);
          // (the barrier of the next vote keeps the next exchange apart)
          float alpha = 1.f;
          if (m_used == -INFINITY) m_used = top;  // O and l of this row are still zero
          else if (top > m_used + (kClean ? 0.f : 8.f)) alpha = exp2f(m_used - top), m_used = top;
          if (it > 0) {
            // O of the block before may still run.  (Its barrier's phase before is that of four
            // blocks before this one, done before S of the block before was issued over its P.)
            const int b1 = buf == 0 ? kBufs - 1 : buf - 1;
            ok = ok &&
                 __all_sync(0xffffffffu, wait<D>(bar.o_done(b1), phase ^ (buf == 0), smem));
            tc::fence_after();
            if (ok) rescale<D>(tO, alpha);
            l2[0] = ptx::f2_mul(l2[0], ptx::f2_pack(alpha, alpha));
            l2[1] = ptx::f2_mul(l2[1], ptx::f2_pack(alpha, alpha));
          }
        }
        const float low = m_used == -INFINITY ? 0.f : -m_used;
        const uint64_t nb = ptx::f2_pack(low, low);
#pragma unroll
        for (int c = 0; c < kPart / 16; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float x0, x1;
            ptx::f2_unpack(scaled(ptx::f2_pack(v[16 * c + 2 * k], v[16 * c + 2 * k + 1]), nb), x0,
                           x1);
            const uint64_t e = ptx::f2_pack(ptx::ex2(x0), ptx::ex2(x1));
            l2[k & 1] = ptx::f2_add(l2[k & 1], e);
            ptx::split_bf16x2(e, w[k], w[8 + k]);
          }
          tc::st16(tS + 16 * c, w);
        }
      };
      const auto plain = [&](uint64_t x, uint64_t nb) {
        return ptx::f2_fma(x, ptx::f2_pack(sc, sc), nb);
      };
      // The paths are apart from the load to the store, so that scores stay in the registers they
      // were loaded to.
      if (whole && !sloped) {
        // All of the scores count.  Capping is monotone: the maximum comes first, and the cap,
        // while none is near it, with the exponentials.
        float v[kPart];
        ld32(tS, v);  // (anything, once `ok` is false)
        float top = max32(v);
        if (!capped) {
          finish(v, top * sc, plain);
        } else {
          const float big = fmaxf(top, -min32(v)) * p.cap_in;
          top = p.cap_out * tanh_any(top * p.cap_in);
          const auto capped_by = [&](auto cs) {
            finish(v, top, [&](uint64_t x, uint64_t nb) {
              return ptx::f2_fma(x, cap_factor(cs, x), nb);
            });
          };
          if (!__any_sync(0xffffffffu, big > kTanhTiny)) {
            capped_by(cap_small<4>(p.cap_in, p.cap_out));
          } else if (!__any_sync(0xffffffffu, big > kTanhSmall)) {
            capped_by(cap_small(p.cap_in, p.cap_out));
          } else {
            cap_any(v, p.cap_in, p.cap_out);
            finish(v, top, plain);
          }
        }
      } else if (whole && !capped) {
        // A bias is linear in the key's index, since no key lies behind the queries.
        float v[kPart];
        ld32(tS, v);
        const uint64_t s2 = ptx::f2_pack(p.scale_log2, p.scale_log2);
        const uint64_t up2 = ptx::f2_pack(see.slope, see.slope);
        const float b0 = see.slope * (float)(at - see.pos);
        const uint64_t base2 = ptx::f2_pack(b0, b0);
#pragma unroll
        for (int e = 0; e < kPart; e += 2) {
          const uint64_t bias = ptx::f2_fma(ptx::f2_pack((float)e, (float)(e + 1)), up2, base2);
          ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(v[e], v[e + 1]), s2, bias), v[e], v[e + 1]);
        }
        finish(v, max32(v), [&](uint64_t x, uint64_t nb) { return ptx::f2_add(x, nb); });
      } else {
        float v[kPart];
        ld32(tS, v);
        if (capped) {
          // (which form of the cap is taken is the seen keys' to decide)
          if (!open) {
#pragma unroll
            for (int e = 0; e < kPart; ++e) v[e] = bits >> e & 1u ? v[e] : 0.f;
          }
          if (__any_sync(0xffffffffu, fmaxf(max32(v), -min32(v)) * p.cap_in > kTanhSmall)) {
            cap_any(v, p.cap_in, p.cap_out);
          } else {
            const auto cs = cap_small(p.cap_in, p.cap_out);
#pragma unroll
            for (int e = 0; e < kPart; e += 2) {
              const uint64_t x = ptx::f2_pack(v[e], v[e + 1]);
              ptx::f2_unpack(ptx::f2_mul(x, cap_factor(cs, x)), v[e], v[e + 1]);
            }
          }
        }
        if (sloped) {
          const float s0 = capped ? 1.f : p.scale_log2;
          if (wrap == INT32_MIN) {
#pragma unroll
            for (int e = 0; e < kPart; ++e)
              v[e] = fmaf(v[e], s0, -see.slope * (float)__popcll(ln >> e >> 1));
          } else {
            const float d0 = (float)(see.pos - at), jump = wrap < kPart ? (float)p.ring_R : 0.f;
#pragma unroll
            for (int e = 0; e < kPart; ++e) {
              const float d = d0 - (float)e + (e > wrap ? jump : 0.f);
              v[e] = fmaf(-see.slope, fabsf(d), v[e] * s0);
            }
          }
        }
        if (!open) {
#pragma unroll
          for (int e = 0; e < kPart; ++e) v[e] = bits >> e & 1u ? v[e] : -INFINITY;
        }
        finish(v, max32(v) * sc, plain);
      }
      tc::wait_st();
    }
    tc::fence_before();
    __syncwarp();
    // (a warp ahead of others arrives at another buffer's barrier; three blocks ahead, it waits for
    // S over the columns of a P that all have published)
    if (ok && lane == 0) ptx::mbar_arrive(bar.p_full(buf));
    if (++buf == kBufs) buf = 0, phase ^= 1;
  }
  // ------------------------------------------------------------ the rows' end
  if (n_blocks > 0) {
    ok = ok && __all_sync(0xffffffffu, wait<D>(bar.drain(), 0, smem));
    tc::fence_after();
  }
  if (!ok && lane == 0) give_up<D>(p, smem);
  float l0, l1;
  ptx::f2_unpack(ptx::f2_add(l2[0], l2[1]), l0, l1);
  bar_sync(rows_bar, 128);  // the last exchange has been read
  *num_mine = l0 + l1;
  bar_sync(rows_bar, 128);
  const float l =
      (row_num[r] + row_num[kRows + r]) + (row_num[2 * kRows + r] + row_num[3 * kRows + r]);
  const int entry = geo->entry, g = geo->head, rho0 = geo->rho0, n_rho = geo->n_rho;
  const int part0 = p.rows[entry].part;
  const bool part = part0 >= 0, any = n_blocks > 0 && m_used != -INFINITY;
  const float f = part ? 1.f : 1.f / l;
  const int64_t vec0 = part ? (int64_t)part0 + (int64_t)g * n_rho + rho0 : 0;
  if (part && qvalid && quarter == 0 && !(kClean && fl->row_bad[r / 32] >> (r % 32) & 1u))
    p.part_ml[vec0 + r] = make_float2(m_used, l);
  // Through shared memory (every block has been consumed), so that whole rows are stored: bf16
  // outputs, or a key split's floats.
  const int pitch = part ? 4 * D + 16 : 2 * D + 16;  // bytes; 16-byte columns on distinct banks
  uint8_t *staged = smem + C::kOff_K;
  uint8_t *mine = staged + r * pitch + (part ? D : D / 2) * quarter;
  bool finite = true;
#pragma unroll 1
  for (int c = 0; c < D / 64; ++c) {
    float o16[16];
    tc::ld16(tO + 16 * c, o16);
    tc::wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      o16[k] = any ? o16[k] * f : 0.f;  // (no key seen: zeros)
      finite = finite && fabsf(o16[k]) < INFINITY;
    }
    if (part) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<float4 *>(mine + 64 * c + 16 * k) =
            make_float4(o16[4 * k], o16[4 * k + 1], o16[4 * k + 2], o16[4 * k + 3]);
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint4 w;
        w.x = ptx::pack_bf16(o16[8 * k], o16[8 * k + 1]);
        w.y = ptx::pack_bf16(o16[8 * k + 2], o16[8 * k + 3]);
        w.z = ptx::pack_bf16(o16[8 * k + 4], o16[8 * k + 5]);
        w.w = ptx::pack_bf16(o16[8 * k + 6], o16[8 * k + 7]);
        *reinterpret_cast<uint4 *>(mine + 32 * c + 16 * k) = w;
      }
    }
  }
  if (!finite && qvalid) fl->again = 1;
  bar_sync(rows_bar, 128);
  const int per_row = part ? D / 4 : D / 8;  // 16-byte pieces of a row
  for (int u = 32 * quarter + lane; u < 32 * per_row; u += 128) {
    const int rr = 32 * (warp % 4) + u / per_row, c = u % per_row, o = rho0 + rr;
    if (o >= n_rho) break;
    // (rows that see a value that is not finite keep what they got the first time)
    if (kClean && fl->row_bad[warp % 4] >> (rr % 32) & 1u) continue;
    const uint4 w = *reinterpret_cast<const uint4 *>(staged + rr * pitch + 16 * c);
    if (part)
      *reinterpret_cast<uint4 *>(p.part_o + (vec0 + rr) * D + 4 * c) = w;
    else
      *reinterpret_cast<uint4 *>(out_row(p, entry, g, o, D) + 8 * c) = w;
  }
  if (!kClean) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // a second run's loads
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_scored_kernel(const __grid_constant__ ScoredPrefillParams p) {
  using C = Cfg<D>;
  constexpr int kHalf = D / 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (ptx::smem_u32(smem) & 1023) {  // the swizzled tiles' alignment, which the layout counts on
    if (threadIdx.x == 0) atomicExch(p.err, 1);
    return;
  }
  volatile Flags *fl = flags_of<D>(smem);
  int *parents = reinterpret_cast<int *>(smem + C::kOff_Parents);

  const Item item = find_item(p, blockIdx.x);
  const PrefillRow &row = p.rows[item.entry];
  const int g = item.head, n_rho = row.n * p.rep, lens = row.lens;
  // The later queries of a long chunk see the most keys: their CTAs start first.
  const int rho0 = (n_rho - 1) / kRows * kRows - item.tile * kRows;
  const int t_max = token_of(p, min(rho0 + kRows, n_rho) - 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const bool tree = p.parents != nullptr;
  const bool soft = warp < kSoftWarps;
  ptx::grid_dep_wait();  // the previous grid on the stream has completed
  ptx::grid_dep_launch();

  // The call's queries, 8 rotary pairs at a time, neighbouring lanes on neighbouring pairs, and
  // what its tokens see are on their way while the barriers and TMEM are set up.
  constexpr int kPairs = kHalf / 8, kUnits = kRows * kPairs / kSoftThreads;
  uint4 x1[kUnits], x2[kUnits];
  Sees see = {0ull, INT32_MAX - 1, 0, 0.f, 0, 0};
  const int quarter = warp / 4, r = threadIdx.x % kRows, rho = rho0 + r;
  const bool qvalid = soft && rho < n_rho;
  if (soft) {
    if (tree && threadIdx.x < row.n) parents[threadIdx.x] = p.parents[row.call_row + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = threadIdx.x + kSoftThreads * i, c = u % kPairs, o = rho0 + u / kPairs;
      x1[i] = x2[i] = make_uint4(0, 0, 0, 0);  // rows past the last one are zero
      if (o >= n_rho) continue;
      const int t = token_of(p, o);
      const __nv_bfloat16 *q = p.q + (int64_t)row.call_row * p.q_row_stride +
                               ((int64_t)t * p.Hq + g * p.rep + o - t * p.rep) * D + 8 * c;
      x1[i] = *reinterpret_cast<const uint4 *>(q);
      x2[i] = *reinterpret_cast<const uint4 *>(q + kHalf);
    }
    if (qvalid) {
      const int t = token_of(p, rho);
      see.pos = lens + t;
      // (positions lie well below kFar, and sums with it below 2^31)
      if (p.first) see.first = min(max(0, p.first[(int64_t)row.call_row + t]), kFar);
      if (p.slopes) see.slope = p.slopes[g * p.rep + rho - t * p.rep] * kLog2e;
    }
  } else if (warp == kWarpO) {
    for (int i = lane; i < 2 * C::kBars; i += 32) {
      const int k = i % C::kBars - Bars<D>::kP;
      ptx::mbar_init(reinterpret_cast<uint64_t *>(smem + C::kOff_Bar) + i,
                     k >= 0 ? kSoftWarps : k == -1 ? 2 : 1);
    }
    if (lane < 4) fl->row_bad[lane] = fl->key_bad[lane] = 0;
    if (lane == 0) fl->fail = fl->again = fl->issued_k = fl->issued_v = 0;
    ptx::fence_barrier_init();
  } else if (warp == kWarpS) {
    tc::alloc(const_cast<uint32_t *>(&fl->tmem), kTmemCols);
  } else if (warp == kWarpK) {
    Geo geo;
    geo.entry = item.entry;
    geo.head = g;
    geo.rho0 = rho0;
    geo.n_rho = n_rho;
    geo.lens = lens;
    geo.prefix = p.prefix[item.entry];
    geo.sl0 = p.sliding ? min(lens, p.ring_R)
              : tree    ? lens
                        : max(lens + t_max + 1, geo.prefix);
    geo.sl2 = p.sliding || tree ? t_max + 1 : 0;
    geo.st2 = (geo.sl0 + kKeys - 1) / kKeys;
    geo.j_end = geo.st2 + (geo.sl2 + kKeys - 1) / kKeys;
    if (p.first && !p.sliding) {
      int lo = INT32_MAX;
      for (int t = token_of(p, rho0) + lane; t <= t_max; t += 32)
        lo = min(lo, p.first[(int64_t)row.call_row + t]);
      lo = max(__reduce_min_sync(0xffffffffu, lo), 0);
      const int all = (geo.j_end + 1) / 2;
      geo.b_near = min(all, (geo.prefix + kBlockKeys - 1) / kBlockKeys);
      geo.b_gap = max(0, min(lo / kBlockKeys, all) - geo.b_near);
      // piece tile0 of tile1: an equal share of what counts
      const int n = all - geo.b_gap;
      geo.i0 = n * row.tile0 / row.tile1;
      geo.n_blocks = n * (row.tile0 + 1) / row.tile1 - geo.i0;
    } else {
      geo.j_end = min(geo.j_end, row.tile1);
      geo.i0 = row.tile0 / 2;
      geo.n_blocks = max(0, (geo.j_end + 1) / 2 - geo.i0);
      geo.b_near = INT32_MAX;
      geo.b_gap = 0;
    }
    if (lane == 0) *const_cast<Geo *>(geo_of<D>(smem)) = geo;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = fl->tmem;

  if (soft) {
    // The rotated queries into the 128-byte-swizzled Q tile, times a power of two.
    const float qs = p.q_scale;
    uint8_t *q_tile = smem + C::kOff_Q;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = threadIdx.x + kSoftThreads * i, c = u % kPairs, qr = u / kPairs;
      const int t = token_of(p, min(rho0 + qr, n_rho - 1));
      const int pos = lens + row.shift + (tree ? lineage(parents, t, 0).depth : t);
      const float4 *cs = reinterpret_cast<const float4 *>(p.rope + (int64_t)pos * kHalf + 8 * c);
      uint32_t *w1 = reinterpret_cast<uint32_t *>(&x1[i]);
      uint32_t *w2 = reinterpret_cast<uint32_t *>(&x2[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 e = cs[j];
        const float a0 = __uint_as_float(w1[j] << 16), a1 = __uint_as_float(w1[j] & 0xffff0000u);
        const float b0 = __uint_as_float(w2[j] << 16), b1 = __uint_as_float(w2[j] & 0xffff0000u);
        w1[j] = ptx::pack_bf16(qs * __fsub_rn(__fmul_rn(a0, e.x), __fmul_rn(b0, e.y)),
                               qs * __fsub_rn(__fmul_rn(a1, e.z), __fmul_rn(b1, e.w)));
        w2[j] = ptx::pack_bf16(qs * __fadd_rn(__fmul_rn(a0, e.y), __fmul_rn(b0, e.x)),
                               qs * __fadd_rn(__fmul_rn(a1, e.w), __fmul_rn(b1, e.z)));
      }
      const int c_hi = kPairs + c;  // 16-byte chunks along D
      *reinterpret_cast<uint4 *>(q_tile + (c / 8) * kRows * 128 + ptx::swz128(qr, c % 8)) = x1[i];
      *reinterpret_cast<uint4 *>(q_tile + (c_hi / 8) * kRows * 128 +
                                 ptx::swz128(qr, c_hi % 8)) = x2[i];
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // Q -> tensor core
    __syncwarp();
    if (lane < 2) ptx::mbar_arrive(Bars<D>(smem, lane).q_ready());
    if (qvalid) {
      if (tree) {
        const Lineage ln = lineage(parents, token_of(p, rho), p.sliding ? p.window : INT32_MAX);
        see.line = ln.bits;
        see.pos = lens + ln.depth;
      }
      if (p.sliding) see.first = max(see.first, see.pos - p.window + 1);
    }
    const volatile Geo &geo = *geo_of<D>(smem);
    const int from = __reduce_max_sync(0xffffffffu, see.first) - kPart * quarter;
    const int to =
        min(geo.sl0, __reduce_min_sync(0xffffffffu, tree ? INT32_MAX - 1 : see.pos) + 1) -
        kPart * (quarter + 1);
    const int gap = geo.b_gap, end = geo.i0 + geo.n_blocks;
    const int i0 = max((max(from, 0) + kBlockKeys - 1) / kBlockKeys - gap, gap ? geo.b_near : 0);
    const int i1 = p.sliding || to < 0 ? 0 : to / kBlockKeys + 1 - gap;
    see.open0 = end - i1;  // the newest first
    see.open1 = end - i0;
  }

  // The runs over the blocks: one, or a second one when an output is not finite.
  const auto run_blocks = [&](auto clean) {
    constexpr bool kClean = decltype(clean)::value;
    const Bars<D> bar(smem, kClean);
    if (warp == kWarpK || warp == kWarpV) {
      if (lane == 0) load_run<D>(p, smem, bar, warp == kWarpV);
    } else if (warp == kWarpS) {
      if (lane == 0) s_run<D>(p, smem, bar, tmem);
    } else if (warp == kWarpO) {
      if (lane == 0) o_run<D>(p, smem, bar, tmem);
    } else {
      softmax_run<D, kClean>(p, smem, bar, tmem, see);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
  };
  run_blocks(std::integral_constant<bool, false>{});
  const bool rerun = fl->again && !fl->fail;
  if (rerun) {
    __syncthreads();
    if (threadIdx.x == 0) fl->issued_k = fl->issued_v = 0;
    __syncthreads();
    run_blocks(std::integral_constant<bool, true>{});
  }

  // A key split: the last CTA of the tile merges all of them, out = sum_s 2^(m_s - M) O_s / sum_s
  // 2^(m_s - M) l_s, a row at a time.
  volatile Geo *geo = geo_of<D>(smem);
  const int ns = p.splits[geo->entry];
  if (ns > 0 && soft) {
    __threadfence();
    bar_sync(kBarAll, kSoftThreads);
    int32_t *ticket = p.counters + (int64_t)p.rows[geo->entry].cache_row * p.Hk + geo->head;
    const int n_rho = geo->n_rho, rho0 = geo->rho0;
    const int shift = 5 * (((n_rho - 1) / kRows * kRows - rho0) / kRows);
    if (threadIdx.x == 0) {
      fl->last = (atomicAdd(ticket, 1 << shift) >> shift & 31) == ns - 1;
      if (fl->last) atomicSub(ticket, ns << shift);  // as it was
    }
    bar_sync(kBarAll, kSoftThreads);
    if (fl->last) {
      __threadfence();
      constexpr int kPer = D / 32;  // dims per lane
      const int64_t stride = (int64_t)p.Hk * n_rho;
      const int64_t v0 = (int64_t)p.part0[geo->entry] + (int64_t)geo->head * n_rho + rho0;
#pragma unroll 2
      for (int rr = warp; rr < min(kRows, n_rho - rho0); rr += kSoftWarps) {
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < ns) ml = __ldcg(&p.part_ml[v0 + rr + lane * stride]);
        float top = ml.x;
#pragma unroll
        for (int off = 8; off > 0; off >>= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        top = __shfl_sync(0xffffffffu, top, 0);
        float wt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top), sum = wt * ml.y;
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        sum = __shfl_sync(0xffffffffu, sum, 0);
        wt = sum > 0.f || sum != sum ? wt / sum : 0.f;
        float acc[kPer] = {};
#pragma unroll 4
        for (int s = 0; s < ns; ++s) {
          const float ws = __shfl_sync(0xffffffffu, wt, s);
          const float *po = p.part_o + (v0 + rr + s * stride) * D + kPer * lane;
          float x[kPer];
          if (kPer == 4) {
            const float4 y = __ldcg(reinterpret_cast<const float4 *>(po));
            x[0] = y.x, x[1] = y.y, x[2 % kPer] = y.z, x[3 % kPer] = y.w;
          } else {
            const float2 y = __ldcg(reinterpret_cast<const float2 *>(po));
            x[0] = y.x, x[1] = y.y;
          }
#pragma unroll
          for (int k = 0; k < kPer; ++k) acc[k] += ws * x[k];
        }
        __nv_bfloat16 *dst = out_row(p, geo->entry, geo->head, geo->rho0 + rr, D) + kPer * lane;
        if (kPer == 4)
          *reinterpret_cast<uint2 *>(dst) = make_uint2(ptx::pack_bf16(acc[0], acc[1]),
                                                       ptx::pack_bf16(acc[2 % kPer], acc[3 % kPer]));
        else
          *reinterpret_cast<uint32_t *>(dst) = ptx::pack_bf16(acc[0], acc[1]);
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  if (fl->fail && threadIdx.x == 0) {
    // Every MMA issued completes before TMEM is released, every TMA load before the shared memory.
    const Bars<D> bar(smem, rerun);
    ptx::mbar_wait(bar.drain(), 0, kWaitLimit);
    for (int s = 0; s < C::kStages && s < fl->issued_k; ++s)
      ptx::mbar_wait(bar.k_full(s), (fl->issued_k - 1 - s) / C::kStages & 1, kWaitLimit);
    for (int s = 0; s < C::kStages && s < fl->issued_v; ++s)
      ptx::mbar_wait(bar.v_full(s), (fl->issued_v - 1 - s) / C::kStages & 1, kWaitLimit);
  }
  __syncthreads();
  if (warp == kWarpS) {
    tc::fence_after();
    tc::dealloc(tmem, kTmemCols);
  }
}

}  // namespace

template <int D>
static cudaError_t launch_t(const ScoredPrefillParams &p, cudaStream_t s, bool pdl) {
  return launch_k(chunk_scored_kernel<D>, dim3(p.n_ctas * p.Hk), dim3(kThreads), Cfg<D>::kSmem,
                  s, p, pdl);
}

cudaError_t launch_chunk_scored(const ScoredPrefillParams &p, int D, cudaStream_t s, bool pdl) {
  if (p.n_ctas <= 0) return cudaSuccess;
  if (D == 128) return launch_t<128>(p, s, pdl);
  if (D == 64) return launch_t<64>(p, s, pdl);
  return cudaErrorInvalidValue;
}

cudaError_t configure_chunk_scored() {
  cudaError_t e = cudaFuncSetAttribute(chunk_scored_kernel<128>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<128>::kSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(chunk_scored_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<64>::kSmem);
  return e;
}

}  // namespace kvinc

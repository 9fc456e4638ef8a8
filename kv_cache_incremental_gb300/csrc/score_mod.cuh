// score_mod.cuh -- changed attention scores (kv_append_scored, kv_append_tree): the tanh cap, and
// the ancestors of a drafted token.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace kvinc {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// tanh(x) = x P(x^2) for |x| <= 0.6: P is the polynomial of degree 4 in x^2 with the smallest
// largest relative error on [0, 0.36], fitted to tanh itself a coefficient at a time, each rounded to
// float before the next ones are fitted (7.5e-8; 7.3e-8 unrounded, 9.1e-8 if rounded at the end).
// A score is that close to its cap only rarely, and while none of a warp's is, the polynomial leaves
// the special-function unit, which the weights' exponentials keep busy, alone.
constexpr float kTanhSmall = 0.6f;
__host__ __device__ constexpr float tanh_coef(int i) {
  constexpr float c[5] = {0.99999994f, -0.3333236f, 0.13310668f, -0.05211966f, 0.015497749f};
  return c[i];
}
// And of degree 3 for |x| <= 0.38 (6.7e-8): a cap of 30 has most scores below 11, and a packed product
// less per two scores is 5% of a capped block (chunk_scored.cu: 16 rows of 16k to 32k keys, 8 to 32
// drafts, Hq 64, Hk 8: 500 us with degree 4 alone, 477 with both; degree 2 for |x| <= 0.18 as well, 484).
constexpr float kTanhTiny = 0.38f;
__host__ __device__ constexpr float tanh_coef3(int i) {
  constexpr float c[4] = {0.99999994f, -0.333319f, 0.13282442f, -0.048148867f};
  return c[i];
}
__device__ __forceinline__ float tanh_small(float x) {
  const float t = x * x;
  float r = tanh_coef(4);
#pragma unroll
  for (int i = 3; i >= 0; --i) r = fmaf(r, t, tanh_coef(i));
  return x * r;
}
// tanh(x) = 1 - 2 / (e^2x + 1) for any x, absolute error about 2e-7.
__device__ __forceinline__ float tanh_any(float x) {
  return fmaf(-2.f, __fdividef(1.f, ptx::ex2(x * (2.f * kLog2e)) + 1.f), 1.f);
}

// The polynomial r, of N coefficients, of a capped score cap_out tanh(v cap_in) = v r(v^2) while |v|
// cap_in <= kTanhSmall (N = 5) or kTanhTiny (4), for two scores at a time: N packed instructions.
// Its coefficients hold powers of cap_in up to the ninth; the host scales the products v so that all
// of them are normal floats (kMinCapIn).
template <int N>
struct CapSmall {
  uint64_t c[N];
};
template <int N = 5>
__device__ __forceinline__ CapSmall<N> cap_small(float cap_in, float cap_out) {
  CapSmall<N> s;
  const float in2 = cap_in * cap_in;
  float k = cap_in * cap_out;
#pragma unroll
  for (int i = 0; i < N; ++i, k *= in2) {
    const float c = k * (N == 5 ? tanh_coef(i) : tanh_coef3(i < 4 ? i : 0));
    s.c[i] = ptx::f2_pack(c, c);
  }
  return s;
}
template <int N>
__device__ __forceinline__ uint64_t cap_factor(const CapSmall<N> &s, uint64_t v2) {
  const uint64_t t = ptx::f2_mul(v2, v2);
  uint64_t r = s.c[N - 1];
#pragma unroll
  for (int k = N - 2; k >= 0; --k) r = ptx::f2_fma(r, t, s.c[k]);
  return r;
}
template <int N>
__device__ __forceinline__ void cap_any(float (&v)[N], float cap_in, float cap_out) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = cap_out * tanh_any(v[i] * cap_in);
}

// A drafted token's ancestors and itself, the `window` nearest of them, a bit for each; and its
// depth (0: a child of the row's last token).  A parent is an earlier token: any other number
// stands for none.
struct Lineage {
  uint64_t bits;
  int depth;
};
__device__ __forceinline__ Lineage lineage(const int32_t *parents, int t, int window) {
  Lineage ln = {0, -1};
  for (int i = t; i >= 0;) {
    if (++ln.depth < window) ln.bits |= 1ull << i;
    const int up = parents[i];
    i = up < i ? up : -1;
  }
  return ln;
}

}  // namespace
}  // namespace kvinc

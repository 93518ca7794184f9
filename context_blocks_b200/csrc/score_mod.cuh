// Attention with modified scores: the arithmetic shared by the prefill kernel
// (attn_mod.cuh) and the shared-prefix decoding kernel (attn_shared.cuh).
//
//     s_ij = scale * q_i . k_j
//     capped:  s_ij <- c * tanh(s_ij / c)
//     biased:  s_ij <- s_ij - slope_h * |p_i - j|      (p_i: the row's position)
//     hidden keys:  s_ij <- -inf, chosen by comparison, never added, so that a
//                   NaN or Inf score of a hidden key does not reach the softmax
//
// Everything is kept in log2 units (x = s * log2 e), fp32.  tanh(u), u = s / c, is
// u * g(u^2) with a degree-5 polynomial g (relative error 5.9e-7,
// gen_tanh_poly.py) for |u| <= 1, and 1 - 2 / (2^(2 u log2 e) + 1) beyond: ex2 and
// rcp of the special-function unit, whose errors (2^-22 relative) become at most
// c * 2^-21 in the capped score.  Against the fixed reference (c <= 52, cap_top) that
// is 4e-5 even for small scores, and a warp with a score beyond takes all of a
// tile's in this way; elsewhere c may be anything, and each score goes by its own u.
// The polynomial takes half the special-function work of a score away, which bounded
// the kernels (8192 capped causal keys, 24 heads: 800 us before, 639 us with it).
// The unit's own tanh has a relative error of 2^-11, which at c = 50 would be 0.02 in
// the exponent.  Scores of 4096 causal keys, 24 heads, normal with deviation 3, cap
// 20, 12 and 4: 130, 160 and 224 us; each by its own u against the fixed reference
// too: 132, 181 and 249.
// Roundings to fewer bits than fp32, and why.
//   Weights to bf16 for P.V: a matrix instruction takes A and B of one type, and V is
//   bf16; a second product with the weights' lower halves would cost half the matrix
//   rate again.  Half a step is 2^-8 of a weight; their sum is taken before it, which
//   leaves the errors of a row's weights independent.  O errs by 0.8e-3 to 1.7e-3
//   (relative L2, normal values), its own rounding to bf16 by 1.65e-3.
//   One in four exponentials by a degree-3 polynomial (1.4e-4, a thirtieth of the
//   above) where nothing is hidden or capped: 1 in 8 gave the plain forward 0.4 to 1 %
//   and 1 in 4 another 1 to 2 % on short keys.
//   ex2, lg2 and rcp of the special-function unit: 2^-22, below fp32 sums of a row.
#pragma once

#include <cuda_bf16.h>
#include <cfloat>
#include <cstdint>

#include "fwd_common.cuh"

namespace pa {
namespace mod {

constexpr int kPParts = 2;                     // P is handed to the MMA warp in two halves
constexpr uint32_t kSuspendHintNs = 1000000;   // see attn_fwd.cuh; the waits stay bounded
// Share of the exponentials on the FMA pipe in tiles without hidden keys: 1 in
// 4 pairs, as in attn_fwd.cuh.  Tiles with hidden keys take all of them on the
// special-function unit, which gives exactly 0 for -inf (the polynomial gives
// 2^-126, and a hidden value row may be as large as 2^127).
constexpr uint32_t kPolyPairs = 0x8888u;

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(u) = u * sum_i kTanhC[i] u^(2 i) for |u| <= 1 (gen_tanh_poly.py).
constexpr float kTanhC[6] = {9.999994040e-01f,  -3.332904279e-01f, 1.328143328e-01f,
                             -5.160567537e-02f, 1.674311422e-02f,  -3.067060374e-03f};

__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Load 16 consecutive 32-bit TMEM columns of this thread's lane; waits for completion.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// max(|a|, |b|, |c|), NaN where one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Scalars of the score modification, set by the host.
struct ScoreMod {
  float scale_log2;     // scale * log2(e)
  float cap_log2;       // c * log2(e)
  float cap_u;          // scale / c
  float cap_g[6];       // cap_log2 * (coefficients of g)
  float cap_ref;        // cap_log2 - cap_top(): the fixed reference maximum of capped scores
  bool cap_fixed;       // whether the weights fit that reference (see cap_top)
  const float* slopes;  // [Hq], natural units; read where the kernel is built for a bias
};

// Capped scores without a bias lie in [-c, c], so the softmax needs no running
// maximum: with x = s log2 e and the fixed reference m = c log2 e - top, the weights
// 2^(x - m) lie in [2^(top - 2 c log2 e), 2^top].  top is 8, as far as a running
// maximum may lag (kRescaleLog2), and where that would bring the smallest weights
// below 2^-64 just as much more as keeps them there; c log2 e <= kCapMax (c <= 52)
// keeps it at 86 or less, so a sum of 2^30 weights is finite.  Values down to 2^-62
// keep their bits even where every score of a row is -c.  Values above some
// 2^(127 - top) may overflow the accumulator; such rows are done again with weights
// that sum to one (repair_rows in attn_mod.cuh, redo_row in attn_shared.cuh).
constexpr float kCapMax = 75.f;
inline float cap_top(float cap_log2) { return fmaxf(kRescaleLog2, 2.f * cap_log2 - 64.f); }

// The capped score for |u| > 1, plus top - c log2 e.
__device__ __forceinline__ float cap_far(float u, float cap_log2, float top) {
  return fmaf(rcp_approx(ex2_approx(u * (2.f * 1.4426950408889634f)) + 1.f), -2.f * cap_log2, top);
}

// A row's constants in one tile: dist0 = p_i - (first key of the tile).
__device__ __forceinline__ float mod_one(float s, const ScoreMod& m, bool cap, bool bias, float slope2, float dist) {
  float x = s * m.scale_log2;
  if (cap) {
    const float u = s * m.cap_u, w = u * u;
    float y = m.cap_g[5];
#pragma unroll
    for (int i = 4; i >= 0; --i) y = fmaf(y, w, m.cap_g[i]);
    x = fabsf(u) <= 1.f ? y * u : cap_far(u, m.cap_log2, m.cap_log2);
  }
  if (bias) x = fmaf(-slope2, fabsf(dist), x);
  return x;
}

// Whether all of the warp's scores lie where the polynomial holds; those of a thread
// whose row does not count are whatever its Q rows in shared memory were left with.
template <int kPairs>
__device__ __forceinline__ bool cap_by_polynomial(const uint64_t (&x)[kPairs], const ScoreMod& sm, bool counts) {
  float a4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < kPairs; ++e) {
    float x0, x1;
    f2_split(x[e], x0, x1);
    a4[e & 3] = max3_abs(a4[e & 3], x0, x1);
  }
  const float amax = max3_abs(max3_abs(a4[0], a4[1], a4[2]), a4[3], 0.f) * sm.cap_u;
  return __all_sync(0xffffffffu, amax <= 1.f || !counts);
}

// kPairs pairs of raw scores to capped scores (log2 units) plus `add`, by the
// polynomial.  The steps go over the pairs in turn, so that each has the others'
// latency to wait in.
template <int kPairs>
__device__ __forceinline__ void cap_near(uint64_t (&x)[kPairs], const ScoreMod& sm, float add) {
  constexpr int kGroup = kPairs < 8 ? kPairs : 8;
  const uint64_t k2 = f2(sm.cap_u, sm.cap_u), add2 = f2(add, add);
  uint64_t g[6];
#pragma unroll
  for (int u = 0; u < 6; ++u) g[u] = f2(sm.cap_g[u], sm.cap_g[u]);
#pragma unroll
  for (int e0 = 0; e0 < kPairs; e0 += kGroup) {
    uint64_t w[kGroup], y[kGroup];
#pragma unroll
    for (int e = 0; e < kGroup; ++e) x[e0 + e] = f2_mul(x[e0 + e], k2);
#pragma unroll
    for (int e = 0; e < kGroup; ++e) w[e] = f2_mul(x[e0 + e], x[e0 + e]);
#pragma unroll
    for (int e = 0; e < kGroup; ++e) y[e] = f2_fma(g[5], w[e], g[4]);
#pragma unroll
    for (int u = 3; u >= 0; --u)
#pragma unroll
      for (int e = 0; e < kGroup; ++e) y[e] = f2_fma(y[e], w[e], g[u]);
#pragma unroll
    for (int e = 0; e < kGroup; ++e) x[e0 + e] = f2_fma(y[e], x[e0 + e], add2);
  }
}

// The same for any scores and any cap: those of |u| > 1 once more from their raw
// values, still in tensor memory at tS.
template <int kPairs>
__device__ __forceinline__ void cap_scores(uint64_t (&x)[kPairs], uint32_t tS, const ScoreMod& sm, bool counts) {
  const bool near = cap_by_polynomial<kPairs>(x, sm, counts);
  cap_near<kPairs>(x, sm, 0.f);
  if (near) return;
#pragma unroll
  for (int e0 = 0; e0 < kPairs; e0 += 8) {
    uint32_t r[16];
    tmem_ld_x16(tS + 2 * e0, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u0 = __uint_as_float(r[2 * e]) * sm.cap_u, u1 = __uint_as_float(r[2 * e + 1]) * sm.cap_u;
      float y0, y1;
      f2_split(x[e0 + e], y0, y1);
      x[e0 + e] = f2(fabsf(u0) <= 1.f ? y0 : cap_far(u0, sm.cap_log2, sm.cap_log2),
                     fabsf(u1) <= 1.f ? y1 : cap_far(u1, sm.cap_log2, sm.cap_log2));
    }
  }
}

// Raw scores to packed weights against the fixed reference, polynomial only; l
// grows by their sum.  The exponentials of eight pairs are issued among the
// polynomial steps of the next eight, so that the special-function and the FMA
// pipe work at the same time.
template <int kPairs>
__device__ __forceinline__ void capped_weights(uint64_t (&x)[kPairs], const ScoreMod& sm, uint32_t (&pk)[kPairs],
                                               float& l) {
  constexpr int kGroup = 8;
  const uint64_t k2 = f2(sm.cap_u, sm.cap_u), add2 = f2(-sm.cap_ref, -sm.cap_ref);
  uint64_t g[6], l2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
  for (int u = 0; u < 6; ++u) g[u] = f2(sm.cap_g[u], sm.cap_g[u]);
#pragma unroll
  for (int e0 = 0; e0 <= kPairs; e0 += kGroup) {
    uint64_t w[kGroup], y[kGroup];
#pragma unroll
    for (int step = 0; step < 8; ++step) {
      if (e0 < kPairs) {
#pragma unroll
        for (int e = 0; e < kGroup; ++e) {
          uint64_t& v = x[e0 < kPairs ? e0 + e : 0];
          if (step == 0) v = f2_mul(v, k2);
          if (step == 1) w[e] = f2_mul(v, v);
          if (step == 2) y[e] = f2_fma(g[5], w[e], g[4]);
          if (step >= 3 && step < 7) y[e] = f2_fma(y[e], w[e], g[6 - step]);
          if (step == 7) v = f2_fma(y[e], v, add2);
        }
      }
      if (e0 > 0) {  // pair `step` of the eight before
        const int e = e0 - kGroup + step;
        float x0, x1;
        f2_split(x[e], x0, x1);
        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
        l2[e & 1] = f2_add(l2[e & 1], f2(p0, p1));
        pk[e] = pack_bf16x2(p0, p1);
      }
    }
  }
  float s0, s1;
  f2_split(f2_add(l2[0], l2[1]), s0, s1);
  l += s0 + s1;
}

// `with` where key 2 e or 2 e + 1 of the pairs is not in [a, b).
template <int kPairs>
__device__ __forceinline__ void hide(uint64_t (&x)[kPairs], int a, int b, float with = -INFINITY) {
#pragma unroll
  for (int e = 0; e < kPairs; ++e) {
    float x0, x1;
    f2_split(x[e], x0, x1);
    x[e] = f2((2 * e < a || 2 * e >= b) ? with : x0, (2 * e + 1 < a || 2 * e + 1 >= b) ? with : x1);
  }
}

// x <- x * mul - slope2 * |dist0 - key| for kPairs pairs of keys 0, 1, .., of
// which those in [a, b) count.  The distance is linear in the key on either side
// of the row's own position: unless a row sees keys on both sides, the bias is
// a base for every eight keys plus one of four pairs of multiples of the slope,
// two packed operations a pair.  In between a score is rounded beside up to seven
// slopes (2^-15 at kLinearSlope), so beyond that every key's distance is taken by
// itself.  Adding the base and the multiple first would do for all slopes, but made 4096
// causal biased keys, 24 heads, take 130 us instead of 118.
constexpr float kLinearSlope = 64.f;  // log2 units
template <int kPairs, bool kMul>
__device__ __forceinline__ void bias_scores(uint64_t (&x)[kPairs], float mul, float slope2, float dist0, int a, int b) {
  const bool behind = dist0 >= static_cast<float>(min(b, 2 * kPairs) - 1);  // all keys that count
  if (__all_sync(0xffffffffu,
                 (behind || dist0 <= static_cast<float>(max(a, 0))) && fabsf(slope2) <= kLinearSlope)) {
    const float sl = behind ? slope2 : -slope2;
    uint64_t step[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) step[u] = f2(sl * static_cast<float>(2 * u), sl * static_cast<float>(2 * u + 1));
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      const float at = sl * (static_cast<float>(2 * (e & ~3)) - dist0);
      x[e] = f2_add(kMul ? f2_fma(x[e], f2(mul, mul), f2(at, at)) : f2_add(x[e], f2(at, at)), step[e & 3]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      float x0, x1;
      f2_split(kMul ? f2_mul(x[e], f2(mul, mul)) : x[e], x0, x1);
      x[e] = f2(fmaf(-slope2, fabsf(dist0 - static_cast<float>(2 * e)), x0),
                fmaf(-slope2, fabsf(dist0 - static_cast<float>(2 * e + 1)), x1));
    }
  }
}

// Weights (bf16 pairs) to tensor memory, handed over on `bar`.
__device__ __forceinline__ void hand_over(uint32_t tP, const uint32_t (&pk)[32], uint32_t bar, int lane) {
  tmem_st_x32(tP, pk);
  tmem_st_wait();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// capped_keys where some key is hidden from some row of the warp or some score is
// past the polynomial's end; returns the sum of the weights.
__device__ __forceinline__ float capped_keys_cut(uint32_t tS, uint32_t tP, int a, int b, bool counts,
                                                 const ScoreMod& sm, uint32_t bar_p, int lane) {
  constexpr int kPairs = 32;
  uint32_t pk[kPairs];
  float l = 0.f;
  if (!__any_sync(0xffffffffu, max(a, 0) < min(b, 2 * kPairs))) {  // no row of this warp sees any of it
#pragma unroll
    for (int e = 0; e < kPairs; ++e) pk[e] = 0u;
  } else {
    uint64_t x[kPairs];
    {
      uint32_t sr[2 * kPairs];
      tmem_ld_x64(tS, sr);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) x[e] = f2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
    }
    const bool edge = __any_sync(0xffffffffu, a > 0 || b < 2 * kPairs);
    if (edge) hide<kPairs>(x, a, b, 0.f);  // so that hidden scores have no part in how the others are taken
    if (cap_by_polynomial<kPairs>(x, sm, counts)) {
      cap_near<kPairs>(x, sm, -sm.cap_ref);
    } else {
      const uint64_t k2 = f2(sm.cap_u, sm.cap_u);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        float u0, u1;
        f2_split(f2_mul(x[e], k2), u0, u1);
        x[e] = f2(cap_far(u0, sm.cap_log2, sm.cap_log2 - sm.cap_ref),
                  cap_far(u1, sm.cap_log2, sm.cap_log2 - sm.cap_ref));
      }
    }
    if (edge) hide<kPairs>(x, a, b);
    uint64_t l2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      float x0, x1;
      f2_split(x[e], x0, x1);
      const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
      l2[e & 1] = f2_add(l2[e & 1], f2(p0, p1));
      pk[e] = pack_bf16x2(p0, p1);
    }
    float s0, s1;
    f2_split(f2_add(l2[0], l2[1]), s0, s1);
    l = s0 + s1;
  }
  hand_over(tP, pk, bar_p, lane);
  return l;
}

// A softmax step of one row a thread over 64 keys with the fixed reference: scores
// at tS in tensor memory, weights (bf16 pairs, 32 columns) to tP, which may lie
// over scores this thread has taken.  The row, where it counts, sees the keys
// [a, b) of the 64.
// No maximum, no rescaling of O, nothing to agree on with another thread; l
// grows by the weights' sum.
__device__ __forceinline__ void capped_keys(uint32_t tS, uint32_t tP, int a, int b, bool counts, const ScoreMod& sm,
                                            float& l, uint32_t bar_p, int lane) {
  constexpr int kPairs = 32;
  if (!__any_sync(0xffffffffu, a > 0 || b < 2 * kPairs)) {
    uint64_t x[kPairs];
    {
      uint32_t sr[2 * kPairs];
      tmem_ld_x64(tS, sr);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) x[e] = f2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
    }
    if (cap_by_polynomial<kPairs>(x, sm, counts)) {
      uint32_t pk[kPairs];
      capped_weights<kPairs>(x, sm, pk, l);
      hand_over(tP, pk, bar_p, lane);
      return;
    }
  }
  l += capped_keys_cut(tS, tP, a, b, counts, sm, bar_p, lane);
}

// One 128-key tile of one row a thread: S from tensor memory at tS, P (bf16
// pairs) written back over it and handed over in two halves.  The row sees
// keys [a, b) of the tile.  m_ref, l: the row's running reference maximum and
// sum; tO: its O accumulator, rescaled when the maximum moves (`have_o`: it
// holds something).  A row that has seen nothing keeps m_ref = -inf and l = 0; one
// that does not count (`counts`) makes no difference to others.  kFixed: capped scores
// may be against the fixed reference (sm.cap_fixed).
template <int D, bool kCap, bool kBias, bool kFixed>
__device__ __forceinline__ void softmax_tile(uint32_t tS, uint32_t tO, int a, int b, float dist0, float slope2,
                                             const ScoreMod& sm, bool counts, bool have_o, float& m_ref, float& l,
                                             uint32_t bar_part, uint32_t bar_full, int lane) {
  if constexpr (kFixed) {
    if (sm.cap_fixed) {
      if (max(a, 0) < min(b, kBN)) m_ref = sm.cap_ref;  // stays -inf until the row sees a key
      capped_keys(tS, tS, a, b, counts, sm, l, bar_part, lane);
      capped_keys(tS + 64, tS + 32, a - 64, b - 64, counts, sm, l, bar_full, lane);
      return;
    }
  }
  constexpr bool kMod = kCap || kBias;
  if (!__any_sync(0xffffffffu, max(a, 0) < min(b, kBN))) {  // no row of this warp sees any of it
    const uint32_t none[16] = {};
#pragma unroll
    for (int ch = 0; ch < kBN / 32; ++ch) tmem_st_x16(tS + ch * 16, none);
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(bar_part);
      mbar_arrive(bar_full);
    }
    return;
  }
  float s[kBN];
  {
    uint32_t sr[kBN];
    tmem_ld_x128(tS, sr);
#pragma unroll
    for (int e = 0; e < kBN; ++e) s[e] = __uint_as_float(sr[e]);
  }
  const float c = sm.scale_log2;
  const bool edge = __any_sync(0xffffffffu, a > 0 || b < kBN);
  float mx;
  if constexpr (kMod) {
    uint64_t x[kBN / 2];
#pragma unroll
    for (int e = 0; e < kBN / 2; ++e) x[e] = f2(s[2 * e], s[2 * e + 1]);
    if constexpr (kCap) cap_scores<kBN / 2>(x, tS, sm, counts);
    if constexpr (kBias) bias_scores<kBN / 2, !kCap>(x, c, slope2, dist0, a, b);
    if (edge) hide<kBN / 2>(x, a, b);
    float m8[8];
#pragma unroll
    for (int e = 0; e < kBN / 2; ++e) {
      f2_split(x[e], s[2 * e], s[2 * e + 1]);
      m8[e & 7] = e < 8 ? fmaxf(s[2 * e], s[2 * e + 1]) : max3f(m8[e & 7], s[2 * e], s[2 * e + 1]);
    }
    mx = fmaxf(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], max3f(m8[5], m8[6], m8[7])));
  } else {
    if (edge) {
#pragma unroll
      for (int e = 0; e < kBN; ++e)
        if (e < a || e >= b) s[e] = -INFINITY;
    }
    float m8[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) m8[k] = fmaxf(s[k], s[k + 8]);
#pragma unroll
    for (int e = 16; e < kBN; e += 16)
#pragma unroll
      for (int k = 0; k < 8; ++k) m8[k] = max3f(m8[k], s[e + k], s[e + 8 + k]);
    mx = fmaxf(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], max3f(m8[5], m8[6], m8[7])));
    mx *= c;
  }
  float alpha = 1.f;
  bool rescale = false;
  if (mx > m_ref + kRescaleLog2) {
    alpha = ex2_approx(m_ref - mx);  // 0 when the row was empty (m_ref = -inf)
    l *= alpha;
    m_ref = mx;
    rescale = have_o;
  }
  if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
    for (int ch = 0; ch < D / 32; ++ch) {
      uint32_t orr[32];
      tmem_ld_x32(tO + ch * 32, orr);
#pragma unroll
      for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
      tmem_st_x32(tO + ch * 32, orr);
    }
  }
  // x - m_ref stays -inf (not NaN) where the row has seen nothing so far.
  const float neg_m = (m_ref == -INFINITY) ? 0.f : -m_ref;
  const float mul = kMod ? 1.f : c;
  const uint64_t mul2 = f2(mul, mul), nm2 = f2(neg_m, neg_m);
  uint64_t l4[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
  auto pass = [&](auto with_poly) {
#pragma unroll
    for (int ch = 0; ch < kBN / 32; ++ch) {
      uint32_t pk[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint64_t s2 = f2(s[ch * 32 + 2 * e], s[ch * 32 + 2 * e + 1]);
        const uint64_t x2 = kMod ? f2_add(s2, nm2) : f2_fma(s2, mul2, nm2);
        float p0, p1;
        if (with_poly() && ((kPolyPairs >> e) & 1)) {
          f2_split(exp2_poly3_x2(x2), p0, p1);
        } else {
          float x0, x1;
          f2_split(x2, x0, x1);
          p0 = ex2_approx(x0);
          p1 = ex2_approx(x1);
        }
        l4[e & 3] = f2_add(l4[e & 3], f2(p0, p1));
        pk[e] = pack_bf16x2(p0, p1);
      }
      tmem_st_x16(tS + ch * 16, pk);
      constexpr int kChPerPart = (kBN / 32) / kPParts;
      if ((ch + 1) % kChPerPart == 0 && ch + 1 < kBN / 32) {
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_part);
      }
    }
  };
  if (edge || kCap)  // capped scores have the FMA pipe busy already
    pass([] { return false; });
  else
    pass([] { return true; });
  const uint64_t sum = f2_add(f2_add(l4[0], l4[1]), f2_add(l4[2], l4[3]));
  float s0, s1;
  f2_split(sum, s0, s1);
  l += s0 + s1;
  tmem_st_wait();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar_full);
}

// Scale this thread's kCols O columns (at tO) by `inv` and store them as bf16
// through the warp's 1 KB staging area, 16 columns (32 bytes of each of the
// warp's 32 rows) at a time: row r of the warp at dst + r * row_stride elements,
// rows r >= rows_left not written.  inv = 0 stores zeros whatever the
// accumulator holds.  Returns whether the row has a value that is not finite.
template <int kCols>
__device__ __noinline__ bool store_cols_bf16(uint32_t tO, uint32_t stg, __nv_bfloat16* dst, long long row_stride,
                                             int rows_left, float inv) {
  const int lane = threadIdx.x % 32;
  float top = 0.f;  // the largest magnitude, or NaN
#pragma unroll 1
  for (int c0 = 0; c0 < kCols; c0 += 16) {
    uint32_t orr[16], pk[8];
    tmem_ld_x16(tO + c0, orr);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x0 = __uint_as_float(orr[2 * e]), x1 = __uint_as_float(orr[2 * e + 1]);
      top = max3_nan(top, x0, x1);
      pk[e] = inv == 0.f ? 0u : pack_bf16x2(x0 * inv, x1 * inv);
    }
    __syncwarp();  // the previous piece has left the staging area
    // Chunk u of row r at position u ^ (r / 4 % 2): eight rows fill the banks.
    const int sw = (lane >> 2) & 1;
    st_shared_v4(stg + lane * 32 + (sw << 4), pk[0], pk[1], pk[2], pk[3]);
    st_shared_v4(stg + lane * 32 + ((sw ^ 1) << 4), pk[4], pk[5], pk[6], pk[7]);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = 16 * k + (lane >> 1), u = lane & 1;
      const uint4 v = ld_shared_v4(stg + r * 32 + ((u ^ ((r >> 2) & 1)) << 4));
      if (r < rows_left) *reinterpret_cast<uint4*>(dst + r * row_stride + c0 + u * 8) = v;
    }
  }
  return !(top <= FLT_MAX);
}

// Scale a thread's O row (TMEM columns [tO, tO + D)) by `inv` and store it as
// bf16, through the warp's staging area (see attn_fwd.cuh).  Row r of the
// warp is at dst + r * row_stride elements; rows r >= rows_left are not written.
// inv = 0 stores zeros whatever the accumulator holds.  Returns whether this
// thread's row has a value that is not finite.
template <int D>
__device__ __noinline__ bool store_rows(uint32_t tO, uint32_t stg, __nv_bfloat16* dst, long long row_stride,
                                        int rows_left, float inv) {
  const int lane = threadIdx.x % 32;
  // 32 columns (64 bytes of each row) at a time, in a loop that stays short: it runs
  // once an item, mostly from beyond the instruction cache.
  float top[2] = {0.f, 0.f};  // the largest magnitude, or NaN
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 32) {
    uint32_t orr[32], pk[16];
    tmem_ld_x32(tO + c0, orr);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float x0 = __uint_as_float(orr[2 * e]), x1 = __uint_as_float(orr[2 * e + 1]);
      top[e & 1] = max3_nan(top[e & 1], x0, x1);
      pk[e] = inv == 0.f ? 0u : pack_bf16x2(x0 * inv, x1 * inv);
    }
    __syncwarp();  // the previous piece has left the staging area
    // Chunk u of row r at position u ^ (r / 2 % 4): eight rows fill the banks twice.
#pragma unroll
    for (int u = 0; u < 4; ++u)
      st_shared_v4(stg + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4), pk[4 * u], pk[4 * u + 1], pk[4 * u + 2],
                   pk[4 * u + 3]);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 8 * k + (lane >> 2), u = lane & 3;
      const uint4 v = ld_shared_v4(stg + r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
      if (r < rows_left) *reinterpret_cast<uint4*>(dst + r * row_stride + c0 + u * 8) = v;
    }
  }
  return !(max3_nan(top[0], top[1], 0.f) <= FLT_MAX);
}

// What a warp does again, where an accumulator is not finite: lane l holds columns
// l * kV .. of the rows it is given.  Rare, and written for shortness.

// n bf16 from an address that is a multiple of their size.
template <int n>
__device__ __forceinline__ void load_row_part(const __nv_bfloat16* p, float (&x)[n]) {
  static_assert(n == 1 || n == 2 || n == 4, "as many columns as a lane may hold");
  if constexpr (n == 1) {
    x[0] = __bfloat162float(*p);
  } else {
    uint32_t w[n / 2];
    if constexpr (n == 2) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
#pragma unroll
    for (int u = 0; u < n / 2; ++u)
      x[2 * u] = __uint_as_float(w[u] << 16), x[2 * u + 1] = __uint_as_float(w[u] & 0xffff0000u);
  }
}

// Columns with +Inf or NaN (`up`) and with -Inf or NaN (`down`) among the value rows
// [j0, j1): bit u of a lane's masks for its column u.  Ends early where all are both.
template <int kV>
__device__ __forceinline__ void scan_values(const __nv_bfloat16* v, long long v_stride, int j0, int j1, unsigned& up,
                                            unsigned& down) {
  constexpr int kStep = 8;
  const int lane = threadIdx.x % 32;
#pragma unroll 1
  for (int j = j0; j < j1; j += kStep) {
    if (__all_sync(0xffffffffu, (up & down) == (1u << kV) - 1)) return;
    float x[kStep][kV];
#pragma unroll
    for (int e = 0; e < kStep; ++e) load_row_part<kV>(v + min(j + e, j1 - 1) * v_stride + lane * kV, x[e]);
#pragma unroll
    for (int e = 0; e < kStep; ++e)
#pragma unroll
      for (int u = 0; u < kV; ++u) {
        if (!(x[e][u] < INFINITY)) up |= 1u << u;
        if (!(x[e][u] > -INFINITY)) down |= 1u << u;
      }
  }
}

// The value of a column whose visible value rows are not all finite (every weight
// is greater than 0).
__device__ __forceinline__ float not_finite(bool up, bool down) {
  return up && down ? __int_as_float(0x7fffffff) : up ? INFINITY : -INFINITY;
}

// Attention of one row over the keys [j0, j1), by the whole warp: acc += 2^(x_j - ref)
// v_j.  Lane l holds D / 32 of the query's columns in qv.  kStep keys at a time, so
// that their loads and sums wait together; all fp32.  8 and 4 in repair_rows: 67 and
// 83 ns a key and row (4096 keys, d 64); the merge's registers allow 4.
template <int D, int kV, int kStep = 8>
__device__ __forceinline__ void add_keys(const float (&qv)[D / 32], const __nv_bfloat16* k, const __nv_bfloat16* v,
                                         long long k_stride, long long v_stride, int j0, int j1, int pos, float ref,
                                         float slope2, const ScoreMod& sm, bool cap, bool bias,
                                         float (&acc)[kV]) {
  constexpr int kQk = D / 32;
  const int lane = threadIdx.x % 32;
#pragma unroll 1
  for (int j = j0; j < j1; j += kStep) {
    float dot[kStep], kk[kStep][kQk], vv[kStep][kV];
#pragma unroll
    for (int e = 0; e < kStep; ++e) {
      const long long at = min(j + e, j1 - 1);  // past the end: the last key once more, without weight
      load_row_part<kQk>(k + at * k_stride + lane * kQk, kk[e]);
      load_row_part<kV>(v + at * v_stride + lane * kV, vv[e]);
    }
#pragma unroll
    for (int e = 0; e < kStep; ++e) {
      dot[e] = 0.f;
#pragma unroll
      for (int u = 0; u < kQk; ++u) dot[e] = fmaf(qv[u], kk[e][u], dot[e]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
      for (int e = 0; e < kStep; ++e) dot[e] += __shfl_xor_sync(0xffffffffu, dot[e], off);
#pragma unroll
    for (int e = 0; e < kStep; ++e) {
      if (j + e >= j1) continue;
      const float p = ex2_approx(mod_one(dot[e], sm, cap, bias, slope2, static_cast<float>(pos - (j + e))) - ref);
#pragma unroll
      for (int u = 0; u < kV; ++u) acc[u] = fmaf(p, vv[e][u], acc[u]);
    }
  }
}

// 4-D tiled load (coordinates innermost first); c0 * element size must be a
// multiple of 16 bytes.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

}  // namespace mod
}  // namespace pa

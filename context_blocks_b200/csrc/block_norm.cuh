// A block's gated residual update with the norms around it
// (pa_gate_residual_norm), one pass over the data:
//     t  = post_norm(y) * post_weight
//     x' = a * x + gate[b] * t
//     h  = norm(x') * norm_weight * (1 + scale[b]) + shift[b]
// rms:   v * rsqrt(mean(v^2) + eps)
// layer: (v - mean) * rsqrt(mean((v - mean)^2) + eps), the deviations squared
//        after the mean is known (the difference of two large sums would lose
//        the variance of a row far from zero)
// All in fp32, rounded once on output; h is taken from x' before its rounding.
//
// HBM-bound: 8 bytes an element with a bf16 residual stream, 12 with fp32.  A row
// stays in the registers of a group of warps (kVecs 16-byte vectors a thread) from
// its loads to its stores, so every input is read once whatever the norms need.
// All loads of a thread are issued before the first reduction.  60000 rows of 1536
// with an fp32 stream, both norms, gate and modulation: 207 us, 5.3 TB/s under
// counters that show 1.06 GB of HBM traffic for 1.11 GB of tensors.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "fwd_common.cuh"
#include "lse_merge.cuh"  // unpack_bf16x8

namespace pa {
namespace norm {

constexpr int kThreads = 256;
constexpr int kNone = 0, kRms = 1, kLayer = 2;

struct Params {
  const __nv_bfloat16* y;
  const void* x;
  void* x_out;
  __nv_bfloat16* h;  // null without a norm
  const __nv_bfloat16* post_weight;
  const __nv_bfloat16* norm_weight;
  const __nv_bfloat16* gate;
  const __nv_bfloat16* scale;
  const __nv_bfloat16* shift;
  long long gate_stride, scale_stride, shift_stride;  // elements between batch entries
  long long rows;
  int rows_per_batch;
  int D;
  int post, norm;
  float residual_scale, eps;
};

// Sum over the `warps` warps of a row's group, the same bits in all of them.
__device__ __forceinline__ float group_sum(float v, float* red, int group, int warps) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (warps > 1) {
    const int first = group * warps;
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(warps * 32) : "memory");
    v = 0.f;
    for (int u = 0; u < warps; ++u) v += red[first + u];
  }
  return v;
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(p)), f);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// v <- norm(v), in the registers of the row's group.  Every sum of a row has its
// own line of `red`, and rows have two tables in turn, so that none is
// overwritten while a slower warp reads it.
template <int kVecs>
__device__ __forceinline__ void normalise(float (&v)[kVecs][8], int kind, const Params& p, float (&red)[4][8],
                                          int first, int group, int t, int warps) {
  const float inv_d = 1.f / static_cast<float>(p.D);
  if (kind == kLayer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[i][e];
    const float mean = group_sum(s, red[first], group, warps) * inv_d;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if ((t + i * warps * 32) * 8 < p.D)  // vectors past the row stay zero
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] -= mean;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(v[i][e], v[i][e], s);
  const float r = rsqrtf(group_sum(s, red[first + 1], group, warps) * inv_d + p.eps);
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] *= r;
}

// One row: from the raw vectors to the outputs; `next` asks for the next row's
// vectors as soon as this one's are taken.
template <bool kX32, int kVecs, int kXWords, typename Next>
__device__ __forceinline__ void one_row(const Params& p, long long row, const uint4 (&ry)[kVecs],
                                        const uint4 (&rx)[kVecs][kXWords], float (&red)[4][8], int group, int t,
                                        int warps, Next next) {
  const long long b = p.rows_per_batch == p.rows ? 0 : row / p.rows_per_batch;
  const long long at = row * p.D;
  float v[kVecs][8], x[kVecs][8];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if ((t + i * warps * 32) * 8 < p.D) {
      unpack_bf16x8(ry[i], v[i]);
      if constexpr (kX32) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          x[i][4 * u] = __uint_as_float(rx[i][u].x), x[i][4 * u + 1] = __uint_as_float(rx[i][u].y);
          x[i][4 * u + 2] = __uint_as_float(rx[i][u].z), x[i][4 * u + 3] = __uint_as_float(rx[i][u].w);
        }
      } else {
        unpack_bf16x8(rx[i][0], x[i]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = x[i][e] = 0.f;
    }
  }
  next();
  if (p.post != kNone) normalise<kVecs>(v, p.post, p, red, 0, group, t, warps);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (t + i * warps * 32) * 8;
    if (c < p.D) {
      float w[8];
      if (p.post_weight) {
        load8(p.post_weight + c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= w[e];
      }
      if (p.gate) {
        load8(p.gate + b * p.gate_stride + c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = fmaf(p.residual_scale, x[i][e], v[i][e]);
      if constexpr (kX32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.x_out) + at + c);
        __stcs(dst, make_float4(v[i][0], v[i][1], v[i][2], v[i][3]));
        __stcs(dst + 1, make_float4(v[i][4], v[i][5], v[i][6], v[i][7]));
      } else {
        __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.x_out) + at + c), pack8(v[i]));
      }
    }
  }
  if (p.norm == kNone) return;
  normalise<kVecs>(v, p.norm, p, red, 2, group, t, warps);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (t + i * warps * 32) * 8;
    if (c < p.D) {
      float w[8];
      if (p.norm_weight) {
        load8(p.norm_weight + c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= w[e];
      }
      if (p.scale) {
        load8(p.scale + b * p.scale_stride + c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= 1.f + w[e];
      }
      if (p.shift) {
        load8(p.shift + b * p.shift_stride + c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] += w[e];
      }
      __stcs(reinterpret_cast<uint4*>(p.h + at + c), pack8(v[i]));
    }
  }
}

__host__ __device__ constexpr bool stays(bool x32) { return !x32; }
// Blocks of 8 warps an SM, where blocks stay.
__host__ __device__ constexpr int resident_blocks(int vecs) { return vecs <= 2 ? 3 : vecs == 4 ? 2 : 1; }

template <bool kX32, int kVecs>
__global__ void __launch_bounds__(kThreads, stays(kX32) ? resident_blocks(kVecs) : 1)
    gate_residual_norm_kernel(const Params p, int warps) {
  __shared__ float red[2][4][8];
  const int group = threadIdx.x / (warps * 32), t = threadIdx.x % (warps * 32);
  const int groups = blockDim.x / (warps * 32);
  // This thread's vectors of a row, as they lie in memory.
  constexpr int kXWords = kX32 ? 2 : 1;
  uint4 ry[kVecs], rx[kVecs][kXWords];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = (t + i * warps * 32) * 8;
      if (row >= p.rows || c >= p.D) continue;
      const long long at = row * p.D + c;
      ry[i] = __ldcs(reinterpret_cast<const uint4*>(p.y + at));
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(p.x) + at * (kX32 ? 4 : 2));
#pragma unroll
      for (int u = 0; u < kXWords; ++u) rx[i][u] = __ldcs(src + u);
    }
  };
  long long row = static_cast<long long>(blockIdx.x) * groups + group;
  fetch(row);
  // Groups of warps leave alone: their barrier is their own.
  if constexpr (stays(kX32)) {
    const long long step = static_cast<long long>(gridDim.x) * groups;
    for (int it = 0; row < p.rows; row += step, ++it)
      one_row<kX32, kVecs>(p, row, ry, rx, red[it & 1], group, t, warps, [&] { fetch(row + step); });
  } else {
    if (row < p.rows) one_row<kX32, kVecs>(p, row, ry, rx, red[0], group, t, warps, [] {});
  }
}

}  // namespace norm
}  // namespace pa

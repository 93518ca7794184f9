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
// stays in the registers of a group of warps (kVecs 16-byte vectors a thread) from its loads to its stores, so every input is read once whatever the
// norms need.  All loads of a thread are issued before the first reduction.
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

// v <- norm(v), in the registers of the row's group.  Every sum has a row of
// `red` of its own, so that none is overwritten while a slower warp reads it.
template <int kVecs>
__device__ __forceinline__ void normalise(float (&v)[kVecs][8], int kind, const Params& p, float (&red)[4][8], int first,
                                          int group, int t, int warps) {
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

template <bool kX32, int kVecs>
__global__ void __launch_bounds__(kThreads) gate_residual_norm_kernel(const Params p, int warps) {
  __shared__ float red[4][8];
  const int group = threadIdx.x / (warps * 32), t = threadIdx.x % (warps * 32);
  const long long row = static_cast<long long>(blockIdx.x) * (blockDim.x / (warps * 32)) + group;
  if (row >= p.rows) return;  // whole groups leave: their barrier is their own
  const long long b = row / p.rows_per_batch;
  const long long at = row * p.D;
  float v[kVecs][8], x[kVecs][8];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (t + i * warps * 32) * 8;
    if (c < p.D) {
      unpack_bf16x8(__ldcs(reinterpret_cast<const uint4*>(p.y + at + c)), v[i]);
      if constexpr (kX32) {
        const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + at + c);
        const float4 a = __ldcs(src), d = __ldcs(src + 1);
        x[i][0] = a.x, x[i][1] = a.y, x[i][2] = a.z, x[i][3] = a.w;
        x[i][4] = d.x, x[i][5] = d.y, x[i][6] = d.z, x[i][7] = d.w;
      } else {
        unpack_bf16x8(__ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + at + c)), x[i]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = x[i][e] = 0.f;
    }
  }
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

}  // namespace norm
}  // namespace pa

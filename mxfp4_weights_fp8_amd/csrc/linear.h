// What the dense product's kernels share: the argument block, the choice of how a
// product runs, and the epilogue.
#pragma once

#include <math.h>

#include "device_common.h"
#include "host_internal.h"

namespace moe {

// y[m, n] = act(sum_c X[m, c] W[n, c] + bias[n]) + residual[m, n]. An operand lies in
// memory either as [rows, C] with the contraction along memory (C a multiple of 128),
// or as [C, rows], which the tiled kernel reads transposed. Strides are in elements,
// multiples of 8.
struct LinearArgs {
  const uint16_t* x;
  const uint16_t* w;
  int64_t xs, ws;         // elements from one memory row of x (w) to the next
  const float* bias;      // [N], optional
  const void* res;        // [M, N] of the output's type, optional; may be y
  void* y;                // [M, N] bf16 or fp32
  float* z;               // [M, N] pre-activation values, optional
  float* parts;           // [splits, M, N] fp32 partial sums where splits > 1
  int M, N, C;
  int w_rows;             // memory rows of a transposed w (at most C; rows past them count as zeros)
  int act, splits;
  bool out_f32;
};
enum class Layout { kRows, kWTrans, kBothTrans };   // neither, w, or both as [C, rows]

// How a product runs: `small` (weights streamed, the contraction split over the waves
// of a workgroup), or in tiles of 32 ft rows x 32 fw columns, the contraction split
// `splits` times over workgroups.
struct LinearPlan {
  bool small;
  int ft, fw, splits;
};
LinearPlan linear_plan(int M, int N, int C, Layout l);
size_t linear_plan_parts(int M, int N, const LinearPlan& p);   // bytes of `parts`
hipError_t launch_linear_plan(const LinearArgs& a, const LinearPlan& p, Layout l, hipStream_t s);
void launch_tiles(const LinearArgs& a, const LinearPlan& p, Layout l, hipStream_t s);

__device__ __forceinline__ float sigmoid_f(float z) { return 1.f / (1.f + expf(-z)); }

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z < 0.f ? 0.f : z;   // NaN stays NaN
    case MOE_ACT_SILU: return z * sigmoid_f(z);
    case MOE_ACT_GELU: return 0.5f * z * erfcf(z * -0.707106781f);
    case MOE_ACT_SIGMOID: return sigmoid_f(z);
    default: return z;
  }
}

__device__ __forceinline__ float activate_slope(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case MOE_ACT_SILU: {
      const float p = sigmoid_f(z);
      return p * (1.f + z * (1.f - p));
    }
    case MOE_ACT_GELU: return 0.5f * erfcf(z * -0.707106781f) + z * expf(-0.5f * z * z) * 0.398942280f;
    case MOE_ACT_SIGMOID: {
      const float p = sigmoid_f(z);
      return p * (1.f - p);
    }
    default: return 1.f;
  }
}

// The epilogue of columns n .. n + 3 of row m (those below N), from their sums.
__device__ __forceinline__ void finish4(const LinearArgs& a, int64_t m, int n, v4f v) {
  if (m >= a.M || n >= a.N) return;
  const int64_t at = m * a.N + n;
  if (a.N % 4 == 0) {
    if (a.bias) v += *reinterpret_cast<const v4f*>(a.bias + n);
    if (a.z) *reinterpret_cast<v4f*>(a.z + at) = v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = activate(v[i], a.act);
    if (a.out_f32) {
      if (a.res) v += *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(a.res) + at);
      *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.y) + at) = v;
    } else {
      if (a.res) {
        const uint2 r = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(a.res) + at);
        v += v4f{__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                 __uint_as_float(r.y & 0xFFFF0000u)};
      }
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + at) =
          make_uint2(bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= a.N) break;
    float f = v[i] + (a.bias ? a.bias[n + i] : 0.f);
    if (a.z) a.z[at + i] = f;
    f = activate(f, a.act);
    if (a.out_f32) {
      if (a.res) f += reinterpret_cast<const float*>(a.res)[at + i];
      reinterpret_cast<float*>(a.y)[at + i] = f;
    } else {
      if (a.res) f += bf16_to_float(reinterpret_cast<const uint16_t*>(a.res)[at + i]);
      reinterpret_cast<uint16_t*>(a.y)[at + i] = (uint16_t)bf16_pack2(f, 0.f);
    }
  }
}

// The same for columns n .. n + 7.
__device__ __forceinline__ void finish8(const LinearArgs& a, int64_t m, int n, v4f lo, v4f hi) {
  if (a.N % 8 != 0 || a.out_f32) {
    finish4(a, m, n, lo);
    finish4(a, m, n + 4, hi);
    return;
  }
  if (m >= a.M || n >= a.N) return;
  const int64_t at = m * a.N + n;
  if (a.bias) {
    lo += *reinterpret_cast<const v4f*>(a.bias + n);
    hi += *reinterpret_cast<const v4f*>(a.bias + n + 4);
  }
  if (a.z) {
    *reinterpret_cast<v4f*>(a.z + at) = lo;
    *reinterpret_cast<v4f*>(a.z + at + 4) = hi;
  }
  v4i r{0, 0, 0, 0};
  if (a.res) r = *reinterpret_cast<const v4i*>(reinterpret_cast<const uint16_t*>(a.res) + at);
  v4i o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v0 = activate(i < 2 ? lo[2 * i] : hi[2 * i - 4], a.act);
    float v1 = activate(i < 2 ? lo[2 * i + 1] : hi[2 * i - 3], a.act);
    if (a.res) {
      v0 += __uint_as_float((uint32_t)r[i] << 16);
      v1 += __uint_as_float((uint32_t)r[i] & 0xFFFF0000u);
    }
    o[i] = (int)bf16_pack2(v0, v1);
  }
  *reinterpret_cast<v4i*>(reinterpret_cast<uint16_t*>(a.y) + at) = o;
}

}  // namespace moe

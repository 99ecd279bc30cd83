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
// multiples of 8. X may be the sum of two bf16 values per element, its low parts x_low
// elements behind the high ones: both products go into the same accumulators.
struct LinearArgs {
  const uint16_t* x;
  const uint16_t* w;
  int64_t xs, ws;         // elements from one memory row of x (w) to the next
  int x_low;              // 0: x is one bf16 value per element
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

// How a product runs: few rows on the vector units (kDot) or with the weights streamed
// past the matrix cores (kSmall), a contraction of at most 384 with rows of x kept in
// registers (kShort), or in tiles of 32 ft rows x 32 fw columns; the
// contraction split `splits` times over workgroups (kSmall and kTiles).
enum class Path { kDot, kSmall, kShort, kTiles };
struct LinearPlan {
  Path path;
  int ft, fw, splits;
};
// plain: a bf16 result without bias, residual, activation or z. two: x in two parts (the
// gradients' layouts alone).
LinearPlan linear_plan(int M, int N, int C, Layout l, bool plain, bool two = false);
size_t linear_plan_parts(int M, int N, const LinearPlan& p);   // bytes of `parts`
hipError_t launch_linear_plan(const LinearArgs& a, const LinearPlan& p, Layout l, hipStream_t s);
int short_tiles_per_cta(int M, int N, bool two);
void launch_short(const LinearArgs& a, Layout l, hipStream_t s);
void launch_tiles(const LinearArgs& a, const LinearPlan& p, Layout l, hipStream_t s);

__device__ __forceinline__ float sigmoid_f(float z) { return 1.f / (1.f + expf(-z)); }

// act of N values: one branch for all of them.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];   // NaN stays NaN
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] * sigmoid_f(v[i]);
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.5f * v[i] * erfcf(v[i] * -0.707106781f);
      break;
    case MOE_ACT_SIGMOID:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = sigmoid_f(v[i]);
      break;
    default: break;
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
    case MOE_ACT_SIGMOID: {   // p (1 - p) without the difference, which cancels for z > 0
      const float e = expf(-fabsf(z)), r = 1.f / (1.f + e);
      return e * r * r;
    }
    default: return 1.f;
  }
}

// The epilogue of V (1, 4 or 8) neighbouring columns n .. n + V - 1 of row m, those below
// N. The residual is loaded apart, so that a caller can have several on their way.
template <int V>
struct Residual {
  float v[V];
};

template <int V>
__device__ __forceinline__ Residual<V> load_residual(const LinearArgs& a, int64_t m, int n) {
  Residual<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = 0.f;
  if (!a.res || m >= a.M || n >= a.N) return r;
  const int64_t at = m * a.N + n;
  if (V > 1 && a.N % V == 0) {
    if (a.out_f32) {
#pragma unroll
      for (int k = 0; k < V / 4 * 4; k += 4) {
        const v4f t = *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(a.res) + at + k);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.v[k + i] = t[i];
      }
    } else {
      uint32_t t[V / 2 + 1];
      if constexpr (V == 8) {
        const v4i x = *reinterpret_cast<const v4i*>(reinterpret_cast<const uint16_t*>(a.res) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = (uint32_t)x[i];
      } else if constexpr (V == 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(a.res) + at);
        t[0] = x.x;
        t[1] = x.y;
      }
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        r.v[2 * i] = __uint_as_float(t[i] << 16);
        r.v[2 * i + 1] = __uint_as_float(t[i] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (n + i < a.N)
        r.v[i] = a.out_f32 ? reinterpret_cast<const float*>(a.res)[at + i]
                           : bf16_to_float(reinterpret_cast<const uint16_t*>(a.res)[at + i]);
  }
  return r;
}

template <int V>
__device__ __forceinline__ void finish(const LinearArgs& a, int64_t m, int n, float (&v)[V], const Residual<V>& r) {
  if (m >= a.M || n >= a.N) return;
  const int64_t at = m * a.N + n;
  const bool whole = a.N % V == 0;
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (whole || n + i < a.N) v[i] += a.bias[n + i];
  }
  if (a.z) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (whole || n + i < a.N) a.z[at + i] = v[i];
  }
  activate(v, a.act);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = a.res ? v[i] + r.v[i] : v[i];
  if (V > 1 && whole && a.out_f32) {
#pragma unroll
    for (int k = 0; k < V / 4 * 4; k += 4)
      *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.y) + at + k) = v4f{v[k], v[k + 1], v[k + 2], v[k + 3]};
  } else if (V > 1 && whole) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(a.y) + at;
    if constexpr (V == 8)
      *reinterpret_cast<v4i*>(dst) = v4i{(int)bf16_pack2(v[0], v[1]), (int)bf16_pack2(v[2], v[3]),
                                         (int)bf16_pack2(v[4], v[5]), (int)bf16_pack2(v[6], v[7])};
    else if constexpr (V == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (n + i < a.N) {
        if (a.out_f32) reinterpret_cast<float*>(a.y)[at + i] = v[i];
        else reinterpret_cast<uint16_t*>(a.y)[at + i] = (uint16_t)bf16_pack2(v[i], 0.f);
      }
  }
}

// The tiled kernels' epilogue of products without activation and without z, N a multiple
// of 8: bias and residual only, little code, so that it unrolls. RES: there is a
// residual; F32: of y and the residual.
inline __device__ bool is_affine(const LinearArgs& a) { return a.N % 8 == 0 && !a.z && a.act == MOE_ACT_NONE; }

template <bool RES, bool F32>
struct Residual8 {
  v4i r[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const LinearArgs& a, int64_t m, int n) {
    if (!RES || m >= a.M || n >= a.N) return;
    const char* p = reinterpret_cast<const char*>(a.res) + (m * a.N + n) * (F32 ? 4 : 2);
    r[0] = load16(p);
    if constexpr (F32) r[1] = load16(p + 16);
  }
};

template <bool RES, bool F32>
__device__ __forceinline__ void finish_affine(const LinearArgs& a, int64_t m, int n, v4f lo, v4f hi,
                                              const Residual8<RES, F32>& res) {
  if (m >= a.M || n >= a.N) return;
  if (a.bias) {
    lo += *reinterpret_cast<const v4f*>(a.bias + n);
    hi += *reinterpret_cast<const v4f*>(a.bias + n + 4);
  }
  char* p = reinterpret_cast<char*>(a.y) + (m * a.N + n) * (F32 ? 4 : 2);
  if constexpr (F32) {
    if constexpr (RES) {
      lo += __builtin_bit_cast(v4f, res.r[0]);
      hi += __builtin_bit_cast(v4f, res.r[1]);
    }
    *reinterpret_cast<v4f*>(p) = lo;
    *reinterpret_cast<v4f*>(p + 16) = hi;
  } else {
    v4i o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v0 = i < 2 ? lo[2 * i] : hi[2 * i - 4], v1 = i < 2 ? lo[2 * i + 1] : hi[2 * i - 3];
      if constexpr (RES) {
        v0 += __uint_as_float((uint32_t)res.r[0][i] << 16);
        v1 += __uint_as_float((uint32_t)res.r[0][i] & 0xFFFF0000u);
      }
      o[i] = (int)bf16_pack2(v0, v1);
    }
    *reinterpret_cast<v4i*>(p) = o;
  }
}

// Calls f<RES, F32>() for a product's residual and type.
template <typename F>
__device__ __forceinline__ void by_affine(const LinearArgs& a, F f) {
  if (a.res) {
    if (a.out_f32) f(Residual8<true, true>{});
    else f(Residual8<true, false>{});
  } else {
    if (a.out_f32) f(Residual8<false, true>{});
    else f(Residual8<false, false>{});
  }
}

// Partial sums of V (4 or 8) neighbouring columns of a split product.
template <int V>
__device__ __forceinline__ void store_part(const LinearArgs& a, int split, int64_t m, int n, const float (&v)[V]) {
  if (m >= a.M || n >= a.N) return;
  float* dst = a.parts + ((int64_t)split * a.M + m) * a.N + n;
  if (a.N % 4 == 0) {
#pragma unroll
    for (int k = 0; k < V; k += 4)
      if (n + k < a.N) *reinterpret_cast<v4f*>(dst + k) = v4f{v[k], v[k + 1], v[k + 2], v[k + 3]};
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (n + k < a.N) dst[k] = v[k];
  }
}

}  // namespace moe

// What the dense product's forward and gradient launchers share: the argument block
// of the tiled kernel and the epilogue's activation.
#pragma once

#include <math.h>

#include "device_common.h"
#include "host_internal.h"

namespace moe {

// y[m, n] = act(sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n]; x, w bf16
// row-major with K a multiple of 128.
struct LinearArgs {
  const uint16_t* x;      // [M, K]
  const uint16_t* w;      // [N, K]
  const float* bias;      // [N], optional
  const void* res;        // [M, N] of the output's type, optional; may be y
  void* y;                // [M, N] bf16 or fp32
  float* z;               // [M, N] pre-activation values, optional
  float* parts;           // [splits, M, N] fp32 partial sums where splits > 1
  int M, N, K, act, splits;
  bool out_f32;
};

// How a product runs: `small` (weights streamed, K split over the waves of a
// workgroup) or in tiles of 32 fw columns x 128 rows, K split `splits` times over
// workgroups.
struct LinearPlan {
  bool small;
  int fw, splits;
};
LinearPlan linear_plan(int M, int N, int K);
hipError_t launch_linear_plan(const LinearArgs& a, const LinearPlan& p, hipStream_t s);

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

}  // namespace moe

// What the router's kernels share: scores of the logits, row loads, reductions over
// the lanes of a row, and the choice of a layout for the number of experts.
//
// Layout: LPR lanes per row (16: four rows per wave; or 64), each holding NV groups
// of four neighbouring experts: expert 4 (j LPR + lane) + i, so a row is read in 16
// byte (bf16: 8 byte) loads. A logit of -inf or NaN masks its expert (score 0, never
// picked), +inf counts as the largest float.
#pragma once

#include <float.h>
#include <math.h>

#include "device_common.h"
#include "host_internal.h"
#include "lane_reduce.h"

namespace moe {

constexpr int kGateThreads = 256;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kFarBelow = -20.f;   // softplus(l) = e^l here, to fp32
constexpr float kNone = -INFINITY;   // a masked expert's logit, or a key that is taken

// e^x, x <= 88: 2^(x log2 e) with the product's rounding error put back (about 1.5
// ulp; results below 2^-126 are 0).
__device__ __forceinline__ float exp_f(float x) {
  x = fmaxf(x, -150.f);   // e^x is 0 there already, and the error term stays finite
  const float t = x * kLog2e;
  const float err = __builtin_fmaf(x, kLog2e, -t) + x * 1.925963033e-8f;   // log2 e = kLog2e + 1.92596e-8
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, err * 0.693147181f, e);
}

// NaN -> masked (the maximum is the other operand), +inf -> largest float
__device__ __forceinline__ float clean(float l) { return fminf(fmaxf(l, kNone), FLT_MAX); }

// Four logits of experts e0 .. e0 + 3 of a row; experts from E on are masked.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load_logits4(const void* row, int e0, int E, float (&v)[4]) {
  if constexpr (VEC) {   // E % 4 == 0; groups past the end load any of the row: no branch
    const bool in = e0 < E;
    const int at = in ? e0 : 0;
    if constexpr (BF16) {
      const uint2 r = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(row) + at);
      v[0] = __uint_as_float(r.x << 16);
      v[1] = __uint_as_float(r.x & 0xFFFF0000u);
      v[2] = __uint_as_float(r.y << 16);
      v[3] = __uint_as_float(r.y & 0xFFFF0000u);
    } else {
      const v4f r = *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(row) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = r[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = in ? clean(v[i]) : kNone;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + i;
      if constexpr (BF16)
        v[i] = e < E ? clean(bf16_to_float(reinterpret_cast<const uint16_t*>(row)[e])) : kNone;
      else
        v[i] = e < E ? clean(reinterpret_cast<const float*>(row)[e]) : kNone;
    }
  }
}
template <bool BF16>
__device__ __forceinline__ float load_logit(const void* row, int e) {
  return clean(BF16 ? bf16_to_float(reinterpret_cast<const uint16_t*>(row)[e])
                    : reinterpret_cast<const float*>(row)[e]);
}

// Doubles: by shuffles (only rows with close keys, and one sum per workgroup).
template <int LPR>
__device__ __forceinline__ double row_max(double v) {
#pragma unroll
  for (int m = 1; m < LPR; m <<= 1) v = fmax(v, __shfl_xor(v, m));
  return v;
}
template <int LPR>
__device__ __forceinline__ double row_sum(double v) {
#pragma unroll
  for (int m = 1; m < LPR; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// A score that depends on its own logit alone, and its slope d score / d logit, from one
// exponential: with e = e^-|l| and r = 1 / (1 + e), sigmoid(l) is r or e r, its slope
// e r^2, and softplus(l) = max(l, 0) + log(1 + e), the logarithm as log(u) e / (u - 1)
// with u = 1 + e rounded, which takes the rounding of u out again.
template <int SCORE>
__device__ __forceinline__ void score_and_slope(float l, float& s, float& slope) {
  const float e = exp_f(-fabsf(l)), u = 1.f + e, r = __builtin_amdgcn_rcpf(u);
  const float sig = l >= 0.f ? r : e * r;
  if constexpr (SCORE == MOE_SCORE_SIGMOID) {
    s = sig;
    slope = e * r * r;
  } else {
    const float lg = u == 1.f ? e : __builtin_amdgcn_logf(u) * 0.693147181f * e * __builtin_amdgcn_rcpf(u - 1.f);
    const float half = exp_f(0.5f * fminf(l, 0.f));
    const bool far = l < kFarBelow;   // s^2 = e^l there
    s = far ? half : sqrtf(fmaxf(l, 0.f) + lg);
    slope = far ? 0.5f * half : sig * 0.5f * __builtin_amdgcn_rcpf(s);
  }
  if (l == kNone) s = slope = 0.f;
}

// The score of one logit (softmax: with the row's largest logit and the sum of
// e^(l - top)).
template <int SCORE>
__device__ __forceinline__ float score_of(float l, float top, float sum) {
  float s, slope;
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) s = l == kNone ? 0.f : exp_f(l - top) / sum;
  else score_and_slope<SCORE>(l, s, slope);
  return s;
}

// Calls f with (LPR, NV) as integral constants: 16 lanes per row for at most 512
// experts (NV 1..8), else 64 lanes (NV up to 16: 4096 experts). `wide`: 64 lanes
// whatever E.
template <int V>
struct Int {
  static constexpr int value = V;
};
template <typename F>
void by_few_experts(int E, F f) {   // 16 lanes per row, E <= 512
  if (E <= 64) f(Int<1>{});
  else if (E <= 128) f(Int<2>{});
  else if (E <= 256) f(Int<4>{});
  else if (E <= 384) f(Int<6>{});
  else f(Int<8>{});
}
template <typename F>
void by_experts(int E, bool wide, F f) {
  if (E <= 512 && !wide) {
    by_few_experts(E, [&](auto nv) { f(Int<16>{}, nv); });
  } else {
    if (E <= 512) f(Int<64>{}, Int<2>{});
    else if (E <= 1024) f(Int<64>{}, Int<4>{});
    else if (E <= 2048) f(Int<64>{}, Int<8>{});
    else f(Int<64>{}, Int<16>{});
  }
}
template <typename F>
void by_score(int score, F f) {
  if (score == MOE_SCORE_SOFTMAX) f(Int<MOE_SCORE_SOFTMAX>{});
  else if (score == MOE_SCORE_SIGMOID) f(Int<MOE_SCORE_SIGMOID>{});
  else f(Int<MOE_SCORE_SQRTSOFTPLUS>{});
}
template <typename F>
void by_layout(bool bf16, bool vec, F f) {
  if (bf16) {
    if (vec) f(Int<1>{}, Int<1>{});
    else f(Int<1>{}, Int<0>{});
  } else {
    if (vec) f(Int<0>{}, Int<1>{});
    else f(Int<0>{}, Int<0>{});
  }
}

// 64 lanes per row also where a lane would have more than one pick otherwise
inline bool wide_rows(const moe_gate_dims& d) { return d.K > 16; }

}  // namespace moe

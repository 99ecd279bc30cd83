// The router's gate: scores of the logits, top-K selection and routing weights.
//
//   s = softmax(l) | sigmoid(l) | sqrt(softplus(l)),   picks = top-K of s + bias,
//   w_j = scale * s_j / (sum of the picked s + 1e-20)  (or scale * s_j)
//
// Order of the picks. Every score rises with its logit, so without a bias the
// logits themselves are compared, which is exact. With one, the keys s + b are
// formed in fp32 from fast functions together with a bound on their error; where
// two neighbours among the K + 1 best lie within the bound, the row is selected
// again from keys in fp64. Equal keys go to the lowest index.
//
// A selection round is a maximum over the lane's values, a butterfly over the row's
// lanes, and the same for the lowest index that holds the maximum.
#include "router.h"

namespace moe {
namespace {

// log(1 + e), 0 <= e <= 1, relative error about 1e-7 for small e (series) and e
// near 1 (logarithm), at most 7e-6 in between
__device__ __forceinline__ float log1p_fast(float e) {
  const float series = e * (1.f - e * (0.5f - e * 0.333333333f));
  const float full = __builtin_amdgcn_logf(1.f + e) * 0.693147181f;
  return e < 0.01f ? series : full;
}

// A score as a function of its own logit (softmax: e^l relative to the row).
template <int SCORE>
__device__ __forceinline__ float score_fast(float l, float top, float inv_sum) {
  if (l == kNone) return 0.f;
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) return exp_f(l - top) * inv_sum;
  if constexpr (SCORE == MOE_SCORE_SIGMOID) return __builtin_amdgcn_rcpf(1.f + exp_f(fminf(-l, 88.f)));
  return __builtin_amdgcn_sqrtf(fmaxf(l, 0.f) + log1p_fast(exp_f(-fabsf(l))));
}
template <int SCORE>
__device__ __forceinline__ double score_f64(double l, double top, double inv_sum) {
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) return exp(l - top) * inv_sum;
  if constexpr (SCORE == MOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
  return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
}

constexpr int kNoIndex = 0x7FFFFFFF;

// The largest key of the row, its lowest index (kNoIndex if every key is -inf),
// and that key removed.
template <int LPR, int NV, typename F>
__device__ __forceinline__ F take_best(F (&key)[NV][4], int lane, int& index) {
  F best = key[0][0];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) best = key[j][i] > best ? key[j][i] : best;
  best = row_max<LPR>(best);
  int at = kNoIndex;
#pragma unroll
  for (int j = NV - 1; j >= 0; --j)
#pragma unroll
    for (int i = 3; i >= 0; --i) at = key[j][i] == best ? 4 * (j * LPR + lane) + i : at;
  at = row_min<LPR>(at);
  index = best == (F)kNone ? kNoIndex : at;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) key[j][i] = 4 * (j * LPR + lane) + i == at ? (F)kNone : key[j][i];
  return best;
}

struct GateArgs {
  const void* logits;
  const float* bias;        // optional
  const int32_t* n_valid;   // optional: rows from *n_valid on are padding
  int32_t* ids;
  float* w;
  int64_t T;
  int E, K, renorm;
  float scale;
};

template <int LPR, int NV, int SCORE, bool BF16, bool VEC>
__global__ __launch_bounds__(kGateThreads) void k_gate(GateArgs a) {
  const int lane = threadIdx.x & (LPR - 1);
  const int64_t t = (int64_t)blockIdx.x * (kGateThreads / LPR) + threadIdx.x / LPR;
  // every lane of a row's group leaves together; the others keep their butterflies
  // inside their own group
  if (t >= a.T) return;
  int32_t* ids = a.ids + t * a.K;
  float* w = a.w + t * a.K;
  if (a.n_valid && t >= *a.n_valid) {
    if (lane < a.K) {
      ids[lane] = -1;
      w[lane] = 0.f;
    }
    return;
  }
  const char* row = reinterpret_cast<const char*>(a.logits) + t * a.E * (BF16 ? 2 : 4);
  float l[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j) load_logits4<BF16, VEC>(row, 4 * (j * LPR + lane), a.E, l[j]);

  float top = kNone, sum = 1.f;
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, l[j][i]);
    top = row_max<LPR>(top);
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += l[j][i] == kNone ? 0.f : exp_f(l[j][i] - top);
    sum = row_sum<LPR>(sum);
  }

  int mine = kNoIndex;   // lane j keeps pick j (K <= LPR)
  auto keep = [&](int j, int index) { mine = j == lane ? index : mine; };
  if (!a.bias) {
    for (int j = 0; j < a.K; ++j) {
      int index;
      take_best<LPR, NV>(l, lane, index);
      keep(j, index);
    }
  } else {
    const float inv_sum = 1.f / sum;
    float key[NV][4];
    float scale_of_keys = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * (j * LPR + lane) + i;
        const float s = score_fast<SCORE>(l[j][i], top, inv_sum);
        const float b = e < a.E ? a.bias[e] : 0.f;
        key[j][i] = l[j][i] == kNone ? kNone : s + b;
        if (!(key[j][i] == key[j][i])) key[j][i] = kNone;
        scale_of_keys = key[j][i] == kNone ? scale_of_keys : fmaxf(scale_of_keys, s + fabsf(b));
      }
    // each key is off by at most 1e-5 of its score (fast functions) and half an ulp
    // of the sum; two of them are compared
    const float slack = 3e-5f * row_max<LPR>(scale_of_keys) + 1e-18f;
    bool close = false;
    float before = INFINITY;
    for (int j = 0; j <= a.K && j < a.E; ++j) {
      int index;
      const float best = take_best<LPR, NV>(key, lane, index);
      close |= best != kNone && !(before - best > slack);
      before = best;
      if (j < a.K) keep(j, index);
    }
    if (close) {   // the same in all lanes of the row
      double dkey[NV][4], dsum = 1.0;
      if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
        dsum = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) dsum += l[j][i] == kNone ? 0.0 : exp((double)l[j][i] - (double)top);
        dsum = 1.0 / row_sum<LPR>(dsum);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * (j * LPR + lane) + i;
          const double b = e < a.E ? (double)a.bias[e] : 0.0;
          dkey[j][i] = l[j][i] == kNone ? (double)kNone : score_f64<SCORE>(l[j][i], top, dsum) + b;
          if (!(dkey[j][i] == dkey[j][i])) dkey[j][i] = (double)kNone;
        }
      for (int j = 0; j < a.K; ++j) {
        int index;
        take_best<LPR, NV>(dkey, lane, index);
        keep(j, index);
      }
    }
  }

  // weight of the lane's pick, from its logit again
  const float s = mine == kNoIndex ? 0.f : score_f32<SCORE>(load_logit<BF16>(row, mine), top, sum);
  float mul = a.scale;
  if (a.renorm) mul = a.scale / (row_sum<LPR>(s) + 1e-20f);
  if (lane < a.K) {
    ids[lane] = mine == kNoIndex ? -1 : mine;
    w[lane] = s * mul;
  }
}

}  // namespace

hipError_t launch_gate(const moe_gate_dims& d, const void* logits, const float* bias, const int32_t* n_valid,
                       int32_t* ids, float* w, hipStream_t s) {
  const GateArgs a{logits, bias, n_valid, ids, w, d.T, d.E, d.K, d.renorm, d.scale};
  by_experts(d.E, wide_rows(d), [&](auto lpr, auto nv) {
    by_score(d.score, [&](auto score) {
      by_layout(d.logits_type == MOE_TYPE_BF16, d.E % 4 == 0, [&](auto bf16, auto vec) {
        constexpr int L = decltype(lpr)::value;
        hipLaunchKernelGGL((k_gate<L, decltype(nv)::value, decltype(score)::value, decltype(bf16)::value != 0,
                                   decltype(vec)::value != 0>),
                           dim3((unsigned)ceil_div(d.T, kGateThreads / L)), dim3(kGateThreads), 0, s, a);
      });
    });
  });
  return hipGetLastError();
}

}  // namespace moe

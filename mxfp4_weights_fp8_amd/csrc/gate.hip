// The router's gate: scores of the logits, top-K selection and routing weights.
//
//   s = softmax(l) | sigmoid(l) | sqrt(softplus(l)),   picks = top-K of s + bias,
//   w_j = scale * s_j / (sum of the picked s + 1e-20)  (or scale * s_j)
//
// Order of the picks. Every score rises with its logit, so without a bias the
// logits themselves are compared, which is exact. With one, keys s + b are formed in
// fp32 with the hardware's fast functions. A key is off by what its score is, at most half
// of `slack`, and by its own rounding; the size of a bias enters by that rounding alone, so
// that an expert held back by a bias of -1e9 makes nobody else's key uncertain. All
// experts whose key may still reach the K-th best one are taken as candidates, and where
// two neighbours in their order cannot be told apart either, the candidates are ranked again
// by fp64 keys: one fp64 score per lane. Where there are more candidates than lanes (many
// equal keys) the whole row is selected in fp64, in ten to twenty times the time. Equal
// keys go to the lowest index.
//
// Selection. The keys, as integers of the same order, lie in LDS in the lane's groups
// of four, each group's maximum in a register. A round is the maximum over the
// lane's groups, a DPP reduction over the row's lanes, the lowest index that holds
// it (group by group, then in the one group read back), and one group rewritten:
// about 50 instructions instead of the 120 of scanning 24 keys in registers.
//
// 32768 x 384 top-8 with bias (52 MB): 23-27 us, bound by the vector units (scores of 24
// experts per lane, then eight rounds), the same with experts at biases of -1e9 (286-598 us
// when their size went into everybody's bound); 7 x 384 5.2-5.9 us, latency.
#include "router.h"

namespace moe {
namespace {

constexpr int kNoKey = (int)0x807FFFFF;   // to_key(-inf): a masked expert, or a key that is taken
constexpr int kNoIndex = 0x7FFFFFFF;

// Floats as integers of the same order (-0 counts as 0, NaN as -inf).
__device__ __forceinline__ int to_key(float f) {
  const int b = __float_as_int(fmaxf(f, kNone) + 0.f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float from_key(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }

// Scores from the hardware's exp2, log2, rcp and sqrt (1 ulp each): the product
// l log2(e) is off by 2^-24 of itself, at most 127 * 2^-24 where e^l is not out of
// range, so e^l is off by at most 6e-6 of itself, and what follows by no more:
// kSlack score is twice a score's error. One exception: 1 + e^l of sqrt(softplus) is
// rounded to 2^-24, which moves a score s below kLowScore by up to 2^-25 / s, or s itself
// where that is less: by up to 2.5e-4 (kLowSlack is twice that). kRounding |key| is twice
// the rounding of the sum with the bias.
constexpr float kSlack = 1.5e-5f, kLowScore = 0.1f, kLowSlack = 5e-4f, kRounding = 0x1p-23f;
template <int SCORE>
__device__ __forceinline__ float score_fast(float l) {
  if constexpr (SCORE == MOE_SCORE_SIGMOID)
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(l * -kLog2e));
  const float e = __builtin_amdgcn_exp2f(fabsf(l) * -kLog2e);
  return __builtin_amdgcn_sqrtf(fmaxf(l, 0.f) + __builtin_amdgcn_logf(1.f + e) * 0.693147181f);
}
template <int SCORE>
__device__ __forceinline__ double score_f64(double l, double top, double inv_sum) {
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) return exp(l - top) * inv_sum;
  if constexpr (SCORE == MOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
  return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
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

// fp64 key of expert e, minus infinity where it is masked
template <int SCORE, bool BF16>
__device__ __forceinline__ double key_f64(const GateArgs& a, const char* row, int e, double top, double inv_sum) {
  const float l = load_logit<BF16>(row, e);
  if (l == kNone) return -INFINITY;
  const double k = score_f64<SCORE>(l, top, inv_sum) + (double)a.bias[e];
  return k == k ? k : -INFINITY;
}

template <int LPR, int NV, int SCORE, bool BF16, bool VEC>
__global__ __launch_bounds__(kGateThreads) void k_gate(GateArgs a) {
  __shared__ v4i groups[NV][kGateThreads];   // a lane reads and writes its own column only
  const int lane = threadIdx.x & (LPR - 1);
  const int64_t t = (int64_t)blockIdx.x * (kGateThreads / LPR) + threadIdx.x / LPR;
  // every lane of a row leaves together; reductions stay inside a row
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

  // softmax: l becomes e^(l - top), or -1 where masked
  float top = kNone, sum = 1.f;
  auto softmax = [&]() {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, l[j][i]);
    top = row_max<LPR>(top);
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = exp_f(l[j][i] - top);
        sum += l[j][i] == kNone ? 0.f : e;
        if (a.bias) l[j][i] = l[j][i] == kNone ? -1.f : e;
      }
    sum = row_sum<LPR>(sum);
  };
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) softmax();

  int best_of[NV];       // largest key of each group
  float score_size = 0.f;     // the row's largest score
  float bias_top = -INFINITY;   // the largest bias (sqrt(softplus) alone asks)
  if (a.bias) {
    const float inv_sum = 1.f / sum;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e0 = 4 * (j * LPR + lane);
      v4f bias{0.f, 0.f, 0.f, 0.f};
      if constexpr (VEC) {
        bias = *reinterpret_cast<const v4f*>(a.bias + (e0 < a.E ? e0 : 0));   // groups past the end are masked
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e0 + i < a.E) bias[i] = a.bias[e0 + i];
      }
      v4i k;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool masked = SCORE == MOE_SCORE_SOFTMAX ? l[j][i] < 0.f : l[j][i] == kNone;
        float s;
        if constexpr (SCORE == MOE_SCORE_SOFTMAX) s = l[j][i] * inv_sum;
        else s = score_fast<SCORE>(l[j][i]);
        score_size = fmaxf(score_size, s);   // 0 or less where masked
        k[i] = to_key(masked ? kNone : s + bias[i]);
      }
      groups[j][threadIdx.x] = k;
      best_of[j] = max(max(k[0], k[1]), max(k[2], k[3]));
      if constexpr (SCORE == MOE_SCORE_SQRTSOFTPLUS)
        bias_top = fmaxf(fmaxf(bias_top, fmaxf(bias[0], bias[1])), fmaxf(bias[2], bias[3]));
    }
    score_size = row_max<LPR>(score_size);
    if constexpr (SCORE == MOE_SCORE_SQRTSOFTPLUS) bias_top = row_max<LPR>(bias_top);
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      v4i k;
#pragma unroll
      for (int i = 0; i < 4; ++i) k[i] = to_key(l[j][i]);
      groups[j][threadIdx.x] = k;
      best_of[j] = max(max(k[0], k[1]), max(k[2], k[3]));
    }
  }

  // the row's largest key
  auto row_best = [&]() {
    int m = best_of[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) m = max(m, best_of[j]);
    return row_max<LPR>(m);
  };
  // the lowest index that holds `best`, which is removed
  auto take = [&](int best) {
    int mine = NV;
#pragma unroll
    for (int j = NV - 1; j >= 0; --j) mine = best_of[j] == best ? j : mine;
    const int g = min(mine, NV - 1);
    v4i k = groups[g][threadIdx.x];
    int i = 3;
    i = k[2] == best ? 2 : i;
    i = k[1] == best ? 1 : i;
    i = k[0] == best ? 0 : i;
    const int at = mine < NV ? 4 * (mine * LPR + lane) + i : kNoIndex;
    const int first = row_min<LPR>(at);
    if (at == first) {
#pragma unroll
      for (int n = 0; n < 4; ++n) k[n] = n == i ? kNoKey : k[n];
      groups[g][threadIdx.x] = k;
    }
    const int rest = max(max(k[0], k[1]), max(k[2], k[3]));
#pragma unroll
    for (int j = 0; j < NV; ++j) best_of[j] = at == first && j == mine ? rest : best_of[j];
    return first;
  };

  int mine = kNoIndex, pos = lane;   // the lane's pick (K <= LPR) and its place
  if (!a.bias) {
    for (int j = 0; j < a.K; ++j) {
      const int best = row_best();
      const int index = best == kNoKey ? kNoIndex : take(best);
      mine = j == lane ? index : mine;
    }
  } else {
    bool more = true;
    // the key before, the smallest step between keys less their roundings, the bound of
    // two scores' errors, and what a candidate needs once there are K
    float before = INFINITY, step = INFINITY, slack = kSlack * score_size + 1e-18f, least = kNone;
    for (int j = 0; j < LPR && __any(more); ++j) {
      const int best = row_best();
      const float f = from_key(best);
      more = more && best != kNoKey && !(f < least);
      if (!more) continue;   // the same in all lanes of the row
      if (j == a.K - 1) {
        if (SCORE == MOE_SCORE_SQRTSOFTPLUS && !(f > kLowScore + kLowSlack + bias_top + slack)) slack += kLowSlack;
        least = f - slack - 2.f * kRounding * fabsf(f);
      }
      step = fminf(step, before - f - kRounding * (fabsf(before) + fabsf(f)));   // behind infinity NaN, which is passed over
      before = f;
      const int index = take(best);
      mine = j == lane ? index : mine;
    }
    if (SCORE == MOE_SCORE_SQRTSOFTPLUS && least == kNone) slack += kLowSlack;   // fewer than K experts
    const int left = row_best();
    const bool crowd = more && left != kNoKey && !(from_key(left) < least);
    const bool close = !(step > slack);
    if (close || crowd) {
      double dtop = top, inv = 1.0;
      if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
        double ds = 0.0;
#pragma unroll 1
        for (int g = 0; g < NV; ++g)
#pragma unroll 1
          for (int e = 4 * (g * LPR + lane); e < min(4 * (g * LPR + lane) + 4, a.E); ++e)
            ds += exp((double)load_logit<BF16>(row, e) - dtop);   // masked: exp(-inf) is 0
        inv = 1.0 / row_sum<LPR>(ds);
      }
      if (!crowd) {
        const double key = mine == kNoIndex ? -INFINITY : key_f64<SCORE, BF16>(a, row, mine, dtop, inv);
        const int row0 = (threadIdx.x & 63) & ~(LPR - 1);
        int rank = 0;
        for (int r = 0; r < LPR; ++r) {
          const double k = __shfl(key, row0 + r);
          const int i = __shfl(mine, row0 + r);
          if (k > key || (k == key && i < mine)) ++rank;
        }
        if (mine != kNoIndex) pos = rank;   // empty lanes come last already
      } else {
        double last = INFINITY;
        int last_at = -1;
        mine = kNoIndex;
        for (int j = 0; j < a.K; ++j) {   // the best one after `last` in the order
          double best = -INFINITY;
          int at = kNoIndex;
#pragma unroll 1
          for (int g = 0; g < NV; ++g)
#pragma unroll 1
            for (int e = 4 * (g * LPR + lane); e < min(4 * (g * LPR + lane) + 4, a.E); ++e) {
              const double k = key_f64<SCORE, BF16>(a, row, e, dtop, inv);
              if ((k < last || (k == last && e > last_at)) && k > best) {
                best = k;
                at = e;
              }
            }
          last = row_max<LPR>(best);
          last_at = row_min<LPR>(best == last ? at : kNoIndex);
          mine = j == lane ? last_at : mine;
          if (last_at == kNoIndex) break;
        }
      }
    }
  }

  // weight of the lane's pick, from its logit again
  const bool pick = pos < a.K;
  const float s = !pick || mine == kNoIndex ? 0.f : score_of<SCORE>(load_logit<BF16>(row, mine), top, sum);
  const float sum_picked = a.renorm ? row_sum<LPR>(s) + 1e-20f : 1.f;
  if (pick) {
    ids[pos] = mine == kNoIndex ? -1 : mine;
    w[pos] = s / sum_picked * a.scale;   // the quotient first: at most 1, whatever the scale
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

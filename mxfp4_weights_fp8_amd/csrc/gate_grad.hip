// Gradient of the router's gate with respect to the logits, the picks held fixed.
//
// dc_j = scale (dw_j - sum_i dw_i s_i / S) / S with S = sum of the picked scores
// + 1e-20 (renorm), or scale dw_j; ds = the dc of the picks, summed over equal ids;
//   softmax: dl = p (ds - sum p ds);  else dl = ds s'(l).
// 32768 x 384 top-8, softmax, with an added gradient (151 MB): 27-29 us, 5.4 TB/s.
#include "router.h"

namespace moe {
namespace {

struct GateGradArgs {
  const void* logits;
  const int32_t* ids;
  const float* dw;
  const float* add;   // optional; may be dl
  float* dl;
  int64_t T;
  int E, K, renorm;
  float scale;
};

// The picks' gradients are spread over the row through LDS, one pick after another (so
// that equal ids add up in a fixed order): about 60 instructions, where comparing 24
// experts per lane with 8 picks took 480.
template <int LPR, int NV, int SCORE, bool BF16, bool VEC>
__global__ __launch_bounds__(kGateThreads) void k_gate_grad(GateGradArgs a) {
  __shared__ v4f spread[NV][kGateThreads];   // [j][row, lane]: experts 4 (j LPR + lane) ..  of a row
  const int lane = threadIdx.x & (LPR - 1);
  const int64_t t = (int64_t)blockIdx.x * (kGateThreads / LPR) + threadIdx.x / LPR;
  if (t >= a.T) return;
  const char* row = reinterpret_cast<const char*>(a.logits) + t * a.E * (BF16 ? 2 : 4);
  // lane j holds pick j (K <= LPR)
  int id = lane < a.K ? a.ids[t * a.K + lane] : -1;
  if (id < 0 || id >= a.E) id = -1;
  float dc = id >= 0 ? a.dw[t * a.K + lane] : 0.f;
  const float lg = id >= 0 ? load_logit<BF16>(row, id) : kNone;
  float l[SCORE == MOE_SCORE_SOFTMAX ? NV : 1][4];
  if constexpr (SCORE == MOE_SCORE_SOFTMAX)
#pragma unroll
    for (int j = 0; j < NV; ++j) load_logits4<BF16, VEC>(row, 4 * (j * LPR + lane), a.E, l[j]);
#pragma unroll
  for (int j = 0; j < NV; ++j) spread[j][threadIdx.x] = v4f{0.f, 0.f, 0.f, 0.f};

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
      for (int i = 0; i < 4; ++i) {
        l[j][i] = l[j][i] == kNone ? 0.f : exp_f(l[j][i] - top);   // from here on e^(l - top)
        sum += l[j][i];
      }
    sum = row_sum<LPR>(sum);
  }
  const float inv_sum = sum > 0.f ? 1.f / sum : 0.f;

  float s, slope = 0.f;
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) s = score_of<SCORE>(lg, top, sum);
  else score_and_slope<SCORE>(lg, s, slope);
  if (a.renorm) {
    const float S = row_sum<LPR>(s) + 1e-20f;
    dc = (dc - row_sum<LPR>(dc * s) / S) / S;
  }
  dc = id >= 0 ? dc * a.scale : 0.f;
  float pd = 0.f;
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) pd = row_sum<LPR>(dc * s);
  else dc *= slope;

  wave_sync();
  float* flat = reinterpret_cast<float*>(spread);
  const int group = id >= 0 ? id >> 2 : 0;   // expert 4 group + i is spread[group / LPR][row's lane group % LPR][i]
  float* mine = flat + 4 * (group / LPR * kGateThreads + (threadIdx.x & ~(LPR - 1)) + (group & (LPR - 1))) + (id & 3);
  for (int k = 0; k < a.K; ++k) {
    if (lane == k && id >= 0) *mine += dc;
    wave_sync();
  }
  auto gradient = [&](int j) {
    v4f g = spread[j][threadIdx.x];
    if constexpr (SCORE == MOE_SCORE_SOFTMAX)
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = l[j][i] * inv_sum * (g[i] - pd);
    return g;
  };
  float* dl = a.dl + t * a.E;
  if constexpr (VEC) {
    if (a.add) {   // every load ahead of the stores, which may go to the same tensor
      v4f add[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e0 = 4 * (j * LPR + lane);   // past the end: any of the row
        add[j] = *reinterpret_cast<const v4f*>(a.add + t * a.E + (e0 < a.E ? e0 : 0));
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e0 = 4 * (j * LPR + lane);
        if (e0 < a.E) *reinterpret_cast<v4f*>(dl + e0) = gradient(j) + add[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e0 = 4 * (j * LPR + lane);
        if (e0 < a.E) *reinterpret_cast<v4f*>(dl + e0) = gradient(j);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e0 = 4 * (j * LPR + lane);
      const v4f g = gradient(j);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + i < a.E) dl[e0 + i] = g[i] + (a.add ? a.add[t * a.E + e0 + i] : 0.f);
    }
  }
}

}  // namespace

hipError_t launch_gate_grad(const moe_gate_dims& d, const void* logits, const int32_t* ids, const float* dw,
                            const float* add, float* dl, hipStream_t s) {
  const GateGradArgs a{logits, ids, dw, add, dl, d.T, d.E, d.K, d.renorm, d.scale};
  by_experts(d.E, wide_rows(d), [&](auto lpr, auto nv) {
    by_score(d.score, [&](auto score) {
      by_layout(d.logits_type == MOE_TYPE_BF16, d.E % 4 == 0, [&](auto bf16, auto vec) {
        constexpr int L = decltype(lpr)::value;
        hipLaunchKernelGGL((k_gate_grad<L, decltype(nv)::value, decltype(score)::value, decltype(bf16)::value != 0,
                                        decltype(vec)::value != 0>),
                           dim3((unsigned)ceil_div(d.T, kGateThreads / L)), dim3(kGateThreads), 0, s, a);
      });
    });
  });
  return hipGetLastError();
}

}  // namespace moe

// The balance loss of a router with its per-expert counts and its gradient.
//
// Tokens [off_b, off_{b+1}) form sequence b, n_b of them; p = softmax(l) or
// s / sum s; c_be = picks of expert e in sequence b;
//   loss = alpha / B * sum_b sum_e f_be P_be,  f_be = E c_be / (K n_b),
//   P_be = mean of p_te over the sequence.
// With a_be = alpha f_be / (B n_b) the loss is sum_t sum_e a_be p_te, so each token
// adds its own dot product d_t = sum_e a_be p_te, the same sum its gradient needs:
//   softmax: dl = p (a - d);   else dl = (a - d) s'(l) / sum s.
// One pass over the logits, after the counts.
#include "router.h"

namespace moe {
namespace {

struct BalanceArgs {
  const void* logits;
  const int32_t* ids;
  const int32_t* off;   // [B + 1], or null: one sequence of all T tokens
  int32_t* counts;      // [B, E]
  float* dl;
  double* parts;        // one per workgroup
  float* loss;
  int64_t T;
  int E, K, B, rows;    // rows: tokens per workgroup
  float alpha;
};

__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t T) { return v < 0 ? 0 : v > T ? T : v; }

// The sequence that holds token t, or -1 (off is ascending).
__device__ __forceinline__ int find_seq(const BalanceArgs& a, int64_t t) {
  if (!a.off) return 0;
  if (t < a.off[0] || t >= a.off[a.B]) return -1;
  int lo = 0, hi = a.B;   // off[lo] <= t < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.off[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(256) void k_fill_zero(int32_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

// counts, one workgroup per a.rows tokens: an LDS histogram per sequence that the
// tokens touch, added to the global one (integers: any order gives the same).
__global__ __launch_bounds__(256) void k_balance_count(BalanceArgs a) {
  extern __shared__ int32_t hist[];
  const int64_t first = (int64_t)blockIdx.x * a.rows;
  const int64_t end = first + a.rows < a.T ? first + a.rows : a.T;
  for (int64_t t = first; t < end;) {
    const int b = find_seq(a, t);
    if (b < 0) {
      if (a.off && t < a.off[0]) {
        t = clamp_row(a.off[0], a.T);
        continue;
      }
      break;
    }
    int64_t stop = a.off ? clamp_row(a.off[b + 1], a.T) : a.T;
    if (stop > end) stop = end;
    for (int e = threadIdx.x; e < a.E; e += 256) hist[e] = 0;
    __syncthreads();
    for (int64_t i = t * a.K + threadIdx.x; i < stop * a.K; i += 256) {
      const int id = a.ids[i];
      if (id >= 0 && id < a.E) atomicAdd(&hist[id], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 256)
      if (hist[e]) atomicAdd(&a.counts[(int64_t)b * a.E + e], hist[e]);
    __syncthreads();
    t = stop;
  }
}

template <int LPR, int NV, int SCORE, bool BF16, bool VEC>
__global__ __launch_bounds__(kGateThreads) void k_balance(BalanceArgs a) {
  __shared__ double red[kGateThreads / LPR];
  constexpr int kRows = kGateThreads / LPR;   // rows in flight
  const int lane = threadIdx.x & (LPR - 1), sub = threadIdx.x / LPR;
  const int64_t first = (int64_t)blockIdx.x * a.rows;
  const int64_t end = first + a.rows < a.T ? first + a.rows : a.T;
  double mine = 0.0;
  int seq = -2;
  float coef[NV][4];
  for (int64_t t = first + sub; t < end; t += kRows) {
    const int b = find_seq(a, t);
    float l[NV][4];
    const char* row = reinterpret_cast<const char*>(a.logits) + t * a.E * (BF16 ? 2 : 4);
    float* dl = a.dl + t * a.E;
    if (b < 0) {   // behind the last sequence or before the first
      for (int e = lane; e < a.E; e += LPR) dl[e] = 0.f;
      continue;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) load_logits4<BF16, VEC>(row, 4 * (j * LPR + lane), a.E, l[j]);
    if (b != seq) {
      seq = b;
      const float n = a.off ? (float)(a.off[b + 1] - a.off[b]) : (float)a.T;
      const float c = (a.alpha / (float)a.B) * ((float)a.E / (float)a.K) / n / n;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * (j * LPR + lane) + i;
          coef[j][i] = e < a.E ? c * (float)a.counts[(int64_t)b * a.E + e] : 0.f;
        }
    }
    float top = kNone;
    if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, l[j][i]);
      top = row_max<LPR>(top);
    }
    float sum = 0.f, dot = 0.f, s[NV][4];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (SCORE == MOE_SCORE_SOFTMAX) s[j][i] = l[j][i] == kNone ? 0.f : exp_f(l[j][i] - top);
        else s[j][i] = score_f32<SCORE>(l[j][i], top, 1.f);
        sum += s[j][i];
        dot += s[j][i] * coef[j][i];
      }
    sum = row_sum<LPR>(sum);
    dot = row_sum<LPR>(dot);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    dot *= inv;
    if (lane == 0) mine += (double)dot;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e0 = 4 * (j * LPR + lane);
      float o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float g = (coef[j][i] - dot) * inv;
        if constexpr (SCORE == MOE_SCORE_SOFTMAX) o[i] = s[j][i] * g;
        else o[i] = l[j][i] == kNone ? 0.f : g * score_slope<SCORE>(l[j][i], s[j][i]);
      }
      if constexpr (VEC) {
        if (e0 < a.E) *reinterpret_cast<v4f*>(dl + e0) = v4f{o[0], o[1], o[2], o[3]};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e0 + i < a.E) dl[e0 + i] = o[i];
      }
    }
  }
  if (lane == 0) red[sub] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < kRows; ++i) s += red[i];
    a.parts[blockIdx.x] = s;
  }
}

__global__ __launch_bounds__(64) void k_balance_sum(const double* __restrict__ parts, int n, float* loss) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 64) s += parts[i];
  s = row_sum<64>(s);
  if (threadIdx.x == 0) *loss = (float)s;
}

}  // namespace

constexpr int kBalanceRows = 64;   // tokens per workgroup
int balance_parts(const moe_gate_dims& d) { return (int)ceil_div(d.T, kBalanceRows); }

hipError_t launch_balance(const moe_gate_dims& d, int B, float alpha, const void* logits, const int32_t* ids,
                          const int32_t* off, float* loss, int32_t* counts, float* dl, double* parts, hipStream_t s) {
  const int rows = kBalanceRows, n = balance_parts(d);
  const BalanceArgs a{logits, ids, off, counts, dl, parts, loss, d.T, d.E, d.K, B, rows, alpha};
  const int64_t nc = (int64_t)B * d.E;
  hipLaunchKernelGGL(k_fill_zero, dim3((unsigned)(ceil_div(nc, 256) < 1024 ? ceil_div(nc, 256) : 1024)), dim3(256), 0,
                     s, counts, nc);
  if (n > 0) {
    hipLaunchKernelGGL(k_balance_count, dim3((unsigned)n), dim3(256), sizeof(int32_t) * d.E, s, a);
    by_experts(d.E, false, [&](auto lpr, auto nv) {
      by_score(d.score, [&](auto score) {
        by_layout(d.logits_type == MOE_TYPE_BF16, d.E % 4 == 0, [&](auto bf16, auto vec) {
          hipLaunchKernelGGL((k_balance<decltype(lpr)::value, decltype(nv)::value, decltype(score)::value,
                                        decltype(bf16)::value != 0, decltype(vec)::value != 0>),
                             dim3((unsigned)n), dim3(kGateThreads), 0, s, a);
        });
      });
    });
  }
  hipLaunchKernelGGL(k_balance_sum, dim3(1), dim3(64), 0, s, parts, n, loss);
  return hipGetLastError();
}

}  // namespace moe

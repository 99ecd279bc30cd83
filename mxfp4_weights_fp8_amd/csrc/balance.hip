// The balance loss of a router with its per-expert counts and its gradient.
//
// Tokens [off_b, off_{b+1}) form sequence b, n_b of them; p = softmax(l) or
// s / sum s; c_be = picks of expert e in sequence b;
//   loss = alpha / B * sum_b sum_e f_be P_be,  f_be = E c_be / (K n_b),
//   P_be = mean of p_te over the sequence.
// With a_be = alpha f_be / (B n_b) the loss is sum_t sum_e a_be p_te, so each token
// adds its own dot product d_t = sum_e a_be p_te, the same sum its gradient needs:
//   softmax: dl = p (a - d);   else dl = (a - d) s'(l) / sum s.
// One pass over the logits, after the counts. 32768 x 384 top-8 in 17 sequences (102
// MB): 29 us, of which the pass 20-21 (5 TB/s), the counts 5-7, the sum of the parts 4 (1024
// numbers, latency) and clearing the counts 2.
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
  int E, K, B;
  float alpha;
};

__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t T) { return v < 0 ? 0 : v > T ? T : v; }

// The sequence that holds token t, or -1; whatever the offsets hold, an answer b >= 0 has
// off[b] <= t < off[b + 1]. LPR neighbouring lanes search together and call it with the
// same t: up to kSearchAll sequences each is looked at, every load at once, above that by
// halves, one load after another (32768 x 384 in 17 sequences: counts 6.2 us against 8.7 us,
// gradients 20.5 against 21.9).
constexpr int kSearchAll = 256;
template <int LPR>
__device__ __forceinline__ int find_seq(const BalanceArgs& a, int64_t t, int lane) {
  if (!a.off) return 0;
  if (a.B <= kSearchAll) {
    int found = a.B;
#pragma unroll 4
    for (int i = lane; i < a.B; i += LPR)
      if (a.off[i] <= t && t < a.off[i + 1]) found = min(found, i);
    found = row_min<LPR>(found);
    return found < a.B ? found : -1;
  }
  if (t < a.off[0] || t >= a.off[a.B]) return -1;
  int lo = 0, hi = a.B;   // off[lo] <= t < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.off[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// a_be = factor * c_be
__device__ __forceinline__ float seq_factor(const BalanceArgs& a, int b) {
  const float n = a.off ? (float)(a.off[b + 1] - a.off[b]) : (float)a.T;
  return (a.alpha / (float)a.B) * ((float)a.E / (float)a.K) / n / n;
}

template <int LPR, int NV, bool VEC>
__device__ __forceinline__ void load_coef(const int32_t* counts, int E, float factor, int lane, float (&coef)[NV][4]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e0 = 4 * (j * LPR + lane);
    v4i c{0, 0, 0, 0};
    if constexpr (VEC) {
      c = *reinterpret_cast<const v4i*>(counts + (e0 < E ? e0 : 0));   // groups past the end have no scores
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + i < E) c[i] = counts[e0 + i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) coef[j][i] = factor * (float)c[i];
  }
}

template <int LPR, int NV, bool BF16, bool VEC>
__device__ __forceinline__ void load_row(const BalanceArgs& a, int64_t t, int lane, float (&l)[NV][4]) {
  const char* row = reinterpret_cast<const char*>(a.logits) + t * a.E * (BF16 ? 2 : 4);
#pragma unroll
  for (int j = 0; j < NV; ++j) load_logits4<BF16, VEC>(row, 4 * (j * LPR + lane), a.E, l[j]);
}

// The counts of a sequence, and what makes them coefficients.
struct Sequence {
  const int32_t* counts;
  float factor;
};

// A row whose scores come to less than kTinySum has every logit below -40 or so, where
// sigmoid(l) is e^l and sqrt(softplus(l)) e^(l/2) to fp32, so that scores and slopes may be
// taken relative to the largest logit's: their common factor, which fp32 cannot hold below
// 2^-126, leaves p and the gradient alone. Below kLowestLogit a row counts as empty. Such
// rows are rare: they are read again, an expert at a time, so that the others keep their
// registers (32768 x 384 takes as long as without them).
constexpr float kTinySum = 8.67361738e-19f;   // 2^-60
constexpr float kLowestLogit = -690.f;
template <int LPR, int SCORE, bool BF16>
__device__ __forceinline__ float tiny_row(const BalanceArgs& a, int64_t t, int lane, const Sequence& q) {
  constexpr float kPower = SCORE == MOE_SCORE_SIGMOID ? 1.f : 0.5f;   // slope = kPower * score
  const char* row = reinterpret_cast<const char*>(a.logits) + t * a.E * (BF16 ? 2 : 4);
  float top = kNone;
#pragma unroll 1
  for (int e = lane; e < a.E; e += LPR) top = fmaxf(top, load_logit<BF16>(row, e));
  top = row_max<LPR>(top);
  auto score = [&](int e) {
    const float l = load_logit<BF16>(row, e);
    return top < kLowestLogit || l == kNone ? 0.f : exp_f(kPower * (l - top));
  };
  float sum = 0.f, dot = 0.f;
#pragma unroll 1
  for (int e = lane; e < a.E; e += LPR) {
    const float s = score(e);
    sum += s;
    dot += s * (q.factor * (float)q.counts[e]);
  }
  sum = row_sum<LPR>(sum);
  dot = row_sum<LPR>(dot);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  dot *= inv;
#pragma unroll 1
  for (int e = lane; e < a.E; e += LPR)
    a.dl[t * a.E + e] = kPower * score(e) * ((q.factor * (float)q.counts[e] - dot) * inv);
  return dot;
}

// One token of logits s: writes its gradient, returns its part of the loss. coef: factor
// times the counts of its sequence, which `sequence` gives again where it is asked.
template <int LPR, int NV, int SCORE, bool BF16, bool VEC, typename F>
__device__ __forceinline__ float balance_row(const BalanceArgs& a, int64_t t, int lane, const float (&coef)[NV][4],
                                             F sequence, float (&s)[NV][4]) {
  float* dl = a.dl + t * a.E;
  float k[NV][4];   // what multiplies (a - d) / sum in the gradient; s becomes the scores
  float top = kNone;
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s[j][i]);
    top = row_max<LPR>(top);
  }
  float sum = 0.f, dot = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float l = s[j][i];
      if constexpr (SCORE == MOE_SCORE_SOFTMAX) s[j][i] = k[j][i] = l == kNone ? 0.f : exp_f(l - top);
      else score_and_slope<SCORE>(l, s[j][i], k[j][i]);
      sum += s[j][i];
      dot += s[j][i] * coef[j][i];
    }
  sum = row_sum<LPR>(sum);
  dot = row_sum<LPR>(dot);
  if constexpr (SCORE != MOE_SCORE_SOFTMAX)
    if (sum < kTinySum) return tiny_row<LPR, SCORE, BF16>(a, t, lane, sequence());   // all lanes of the row
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  dot *= inv;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e0 = 4 * (j * LPR + lane);
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = k[j][i] * ((coef[j][i] - dot) * inv);
    if constexpr (VEC) {
      if (e0 < a.E) *reinterpret_cast<v4f*>(dl + e0) = v4f{o[0], o[1], o[2], o[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + i < a.E) dl[e0 + i] = o[i];
    }
  }
  return dot;
}

// Picks of tokens [first, end) into an LDS histogram.
__device__ __forceinline__ void count_picks(const BalanceArgs& a, int64_t first, int64_t end, int32_t* hist) {
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  constexpr int kAtOnce = 4;   // loads on their way
  const int64_t n = end * a.K;
  for (int64_t i0 = first * a.K + threadIdx.x; i0 < n; i0 += kAtOnce * blockDim.x) {
    int id[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t i = i0 + u * blockDim.x;
      id[u] = a.ids[i < n ? i : n - 1];
      if (i >= n) id[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (id[u] >= 0 && id[u] < a.E) atomicAdd(&hist[id[u]], 1);
  }
  __syncthreads();
}

// counts, one workgroup per kCountRows tokens: an LDS histogram per sequence that the
// tokens touch, added to the global one (integers: any order gives the same).
constexpr int kCountRows = 256;
__global__ __launch_bounds__(256) void k_balance_count(BalanceArgs a) {
  extern __shared__ int32_t hist[];
  const int64_t first = (int64_t)blockIdx.x * kCountRows;
  const int64_t end = first + kCountRows < a.T ? first + kCountRows : a.T;
  for (int64_t t = first; t < end;) {
    const int b = find_seq<64>(a, t, threadIdx.x & 63);
    if (b < 0) {
      if (t >= a.off[0]) break;   // behind the last sequence
      t = clamp_row(a.off[0], a.T);
      continue;
    }
    int64_t stop = a.off ? clamp_row(a.off[b + 1], a.T) : a.T;
    if (stop > end) stop = end;
    count_picks(a, t, stop, hist);
    for (int e = threadIdx.x; e < a.E; e += 256)
      if (hist[e]) atomicAdd(&a.counts[(int64_t)b * a.E + e], hist[e]);
    __syncthreads();
    t = stop;
  }
}

// The tokens' gradients and parts of the loss, after the counts: kBalanceRows tokens
// per workgroup. A row's lanes keep the coefficients of the sequence they are in.
constexpr int kBalanceRows = 32;
template <int LPR, int NV, int SCORE, bool BF16, bool VEC>
__global__ __launch_bounds__(kGateThreads) void k_balance(BalanceArgs a) {
  constexpr int kRows = kGateThreads / LPR;   // rows in flight
  __shared__ double red[kRows];
  const int lane = threadIdx.x & (LPR - 1), sub = threadIdx.x / LPR;
  const int first = blockIdx.x * kBalanceRows, end = min(first + kBalanceRows, (int)a.T);   // T is at most 2^21
  double mine = 0.0;
  int stop = -1;   // end of the sequence whose coefficients are held
  float coef[NV][4];
  for (int t = first + sub; t < end; t += kRows) {
    float l[NV][4];
    load_row<LPR, NV, BF16, VEC>(a, t, lane, l);
    if (t >= stop) {
      const int b = find_seq<LPR>(a, t, lane);
      if (b < 0) {   // in front of the first sequence or behind the last
        for (int e = lane; e < a.E; e += LPR) a.dl[(int64_t)t * a.E + e] = 0.f;
        continue;
      }
      stop = a.off ? a.off[b + 1] : (int)a.T;
      load_coef<LPR, NV, VEC>(a.counts + (int64_t)b * a.E, a.E, seq_factor(a, b), lane, coef);
    }
    auto sequence = [&]() {
      const int b = find_seq<LPR>(a, t, lane);
      return Sequence{a.counts + (int64_t)b * a.E, seq_factor(a, b)};
    };
    mine += (double)balance_row<LPR, NV, SCORE, BF16, VEC>(a, t, lane, coef, sequence, l);
  }
  if (lane == 0) red[sub] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < kRows; ++i) s += red[i];
    a.parts[blockIdx.x] = s;
  }
}

__global__ __launch_bounds__(256) void k_balance_sum(const double* __restrict__ parts, int n, float* loss) {
  __shared__ double red[4];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) s += parts[i];
  s = row_sum<64>(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) *loss = (float)(red[0] + red[1] + red[2] + red[3]);
}

// Small batches of few sequences in one launch of one workgroup: sequence by sequence,
// the histogram, then its tokens. With many experts half the threads, as 16 waves leave
// each 128 registers and a row's scores and slopes then go to scratch (64 x 512 sigmoid 17.4
// us on 1024 threads, 9.8 on 512; 256 x 384 softmax, which fits, 15.8 and 18.2).
constexpr int one_threads(int nv, int score) {
  return nv <= 4 || (nv <= 6 && score == MOE_SCORE_SOFTMAX) ? 1024 : 512;
}
template <int LPR, int NV, int SCORE, bool BF16, bool VEC>
__global__ __launch_bounds__(one_threads(NV, SCORE)) void k_balance_one(BalanceArgs a) {
  constexpr int kOneThreads = one_threads(NV, SCORE), kRows = kOneThreads / LPR;
  __shared__ __attribute__((aligned(16))) int32_t hist[4 * LPR * NV];   // E at most
  __shared__ double red[kRows];
  const int lane = threadIdx.x & (LPR - 1), sub = threadIdx.x / LPR;
  double mine = 0.0;
  auto clear = [&](int64_t lo, int64_t hi) {   // rows in no sequence
    for (int64_t i = lo * a.E + threadIdx.x; i < hi * a.E; i += kOneThreads) a.dl[i] = 0.f;
  };
  if (a.off) {
    clear(0, clamp_row(a.off[0], a.T));
    clear(clamp_row(a.off[a.B], a.T), a.T);
  }
  for (int b = 0; b < a.B; ++b) {
    const int64_t lo = a.off ? clamp_row(a.off[b], a.T) : 0, hi = a.off ? clamp_row(a.off[b + 1], a.T) : a.T;
    count_picks(a, lo, hi, hist);
    for (int e = threadIdx.x; e < a.E; e += kOneThreads) a.counts[(int64_t)b * a.E + e] = hist[e];
    if (hi > lo) {   // the same for everybody
      float coef[NV][4];
      const float factor = seq_factor(a, b);
      load_coef<LPR, NV, VEC>(hist, a.E, factor, lane, coef);
      auto sequence = [&]() { return Sequence{hist, factor}; };
      for (int64_t t = lo + sub; t < hi; t += kRows) {
        float l[NV][4];
        load_row<LPR, NV, BF16, VEC>(a, t, lane, l);
        mine += (double)balance_row<LPR, NV, SCORE, BF16, VEC>(a, t, lane, coef, sequence, l);
      }
    }
    __syncthreads();   // the histogram is read before the next sequence clears it
  }
  if (lane == 0) red[sub] = mine;
  __syncthreads();
  if (threadIdx.x < 64) {
    double s = 0.0;
    for (int i = threadIdx.x; i < kRows; i += 64) s += red[i];
    s = row_sum<64>(s);
    if (threadIdx.x == 0) *a.loss = (float)s;
  }
}

// One workgroup while its work is small: its rounds over the tokens, one more for each
// further sequence, times the groups of experts that a lane scores, times what a score
// costs. Per call in us (the four launches below take 20-21, bound by the host; in a
// captured graph 9-19), one workgroup at
//   cost up to 48  11, bound by the host
//   64 to 96       512 x 128 softmax 13 and sigmoid 16, 256 x 256 13 and 15, 128 x 512 13
//                  and 16, 256 x 384 softmax 16, sqrtsoftplus 256 x 128 16 and
//                  64 x 512 18
//   from 128 on    512 x 256 softmax 22 and sigmoid 26, 512 x 128 sqrtsoftplus 29
inline bool one_workgroup(const moe_gate_dims& d, int B) {
  if (d.T > 512 || d.E > 512 || B > 4) return false;
  int groups = 0;
  by_few_experts(d.E, [&](auto nv) { groups = decltype(nv)::value; });
  const int rows = one_threads(groups, d.score) / 16;
  const int score = d.score == MOE_SCORE_SOFTMAX ? 2 : d.score == MOE_SCORE_SIGMOID ? 3 : 6;
  return (ceil_div(d.T, rows) + B - 1) * (rows / 32) * groups * score <= 96;
}

}  // namespace

int balance_parts(const moe_gate_dims& d, int B) {
  return one_workgroup(d, B) ? 0 : (int)ceil_div(d.T, kBalanceRows);
}

hipError_t launch_balance(const moe_gate_dims& d, int B, float alpha, const void* logits, const int32_t* ids,
                          const int32_t* off, float* loss, int32_t* counts, float* dl, double* parts, hipStream_t s) {
  const int n = balance_parts(d, B);
  const BalanceArgs a{logits, ids, off, counts, dl, parts, loss, d.T, d.E, d.K, B, alpha};
  const bool bf = d.logits_type == MOE_TYPE_BF16, vec = d.E % 4 == 0;
  if (one_workgroup(d, B)) {
    by_few_experts(d.E, [&](auto nv) {
      by_score(d.score, [&](auto score) {
        by_layout(bf, vec, [&](auto bf16, auto v) {
          hipLaunchKernelGGL((k_balance_one<16, decltype(nv)::value, decltype(score)::value, decltype(bf16)::value != 0,
                                            decltype(v)::value != 0>),
                             dim3(1), dim3(one_threads(decltype(nv)::value, decltype(score)::value)), 0, s, a);
        });
      });
    });
    return hipGetLastError();
  }
  hipError_t err = launch_fill_zero(counts, (int64_t)B * d.E, s);
  if (err != hipSuccess) return err;
  if (n > 0) {
    hipLaunchKernelGGL(k_balance_count, dim3((unsigned)ceil_div(d.T, kCountRows)), dim3(256), sizeof(int32_t) * d.E, s, a);
    by_experts(d.E, false, [&](auto lpr, auto nv) {
      by_score(d.score, [&](auto score) {
        by_layout(bf, vec, [&](auto bf16, auto v) {
          hipLaunchKernelGGL((k_balance<decltype(lpr)::value, decltype(nv)::value, decltype(score)::value,
                                        decltype(bf16)::value != 0, decltype(v)::value != 0>),
                             dim3((unsigned)n), dim3(kGateThreads), 0, s, a);
        });
      });
    });
  }
  hipLaunchKernelGGL(k_balance_sum, dim3(1), dim3(256), 0, s, parts, n, loss);
  return hipGetLastError();
}

}  // namespace moe

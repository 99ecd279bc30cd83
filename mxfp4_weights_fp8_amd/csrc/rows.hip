// Tokens laid out by expert and brought back, with their gradients. Pair p = t K + j is
// pick j of token t, pair_rows[p] its row (the plan's order: by expert, then by pair) or
// -1 where the pick was dropped.
//   sort         rows[r] = x[t]
//   return       y[t] = sum_j w[t, j] rows[r] + add[t]; with w = 1 it is sort's gradient
//   return_grad  d_rows[r] = w[t, j] dy[t],  d_w[t, j] = <rows[r], dy[t]>
// All three walk tokens, so that what a token has once is read once, whatever its K rows
// are; every row has one pair, so each is written (read) once and nothing is added by
// atomics. HBM-bound, all of the traffic whole rows: 32768 tokens x 7168, top-8, by expert
// 777 us (5.4 TB/s; from codes 366 us for half as many), back 716-750 us (5.7 TB/s), the
// gradient of 8191 tokens 388 us (5.1 TB/s). 7 tokens 3.7 us, bound by the launch.
#include "device_common.h"
#include "host_internal.h"
#include "lane_reduce.h"
#include "rows.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kRowThreads = 256;

// 8 values of a token tensor, bf16 or fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if constexpr (F32) {
    const v4f a = *reinterpret_cast<const v4f*>(static_cast<const float*>(p) + at),
              b = *reinterpret_cast<const v4f*>(static_cast<const float*>(p) + at + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    unpack8(load16(static_cast<const uint16_t*>(p) + at), v);
  }
}

// A thread's 8 columns of a token.
struct Place {
  int64_t t;
  int c8;   // group within the row
};
__device__ __forceinline__ Place place_of(int groups) {
  // the workgroup's first group by a scalar division, this thread's by a 32-bit one
  const int64_t g0 = block_id() * kRowThreads, t0 = g0 / groups;
  const uint32_t in = (uint32_t)(g0 - t0 * groups) + threadIdx.x;
  return Place{t0 + in / (uint32_t)groups, (int)(in % (uint32_t)groups)};
}

struct SortArgs {
  const void* x;        // [T, H] bf16, or E4M3 codes
  const uint8_t* x_s;   // [T, H / 128] scales of codes
  const int32_t* pair_rows;
  uint16_t* rows;       // [T K, H], null: the token's values go to `rows` themselves
  int64_t P;
  int T, H, K;
};

// From codes the stores stay cached whatever the size (16K tokens 364 us, nontemporal 378).
template <bool CODES, bool NT>
__global__ __launch_bounds__(kRowThreads) void k_sort_rows(SortArgs a) {
  const int groups = a.H / 8;
  const Place p = place_of(groups);
  if (p.t >= a.T) return;
  const int64_t at = p.t * a.H + 8 * p.c8;
  v4i v;
  if constexpr (CODES) {
    const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + at);
    float f[8];
    decode8(q, (int)a.x_s[at / 128] - 127, f);
    v = pack8(f);   // exact: at most 4 significant bits
  } else {
    v = load16(static_cast<const uint16_t*>(a.x) + at);
  }
  if (!a.pair_rows) {   // unsorted
    *reinterpret_cast<v4i*>(a.rows + at) = v;
    return;
  }
  const int32_t* rows = a.pair_rows + p.t * a.K;
  for (int j = 0; j < a.K; ++j) {
    const uint32_t r = (uint32_t)rows[j];   // -1 is no row
    if (r < a.P) store_row<NT>(a.rows + (int64_t)r * a.H + 8 * p.c8, v);
  }
}

struct ReturnArgs {
  const uint16_t* rows;
  const int32_t* pair_rows;
  const float* w;     // [T, K], optional
  const void* add;    // [T, H] of y's type, optional; may be y
  void* y;
  int64_t P;
  int T, H, K;
};

// Rows on their way at once. A missing row is not read: in a wave that lacks one every load
// has its own condition (in all waves, that costs top-8 1 %). Conditions, and row 0 read in
// place of a missing one, in us: 10595 x 11816 fp32, top-1 153 and 236; 22216 x 576, top-1 16 and
// 28; 32768 x 7168, top-2 248 and 342; 16384 x 7168, top-9 393 and 448; 32768 x 7168, top-8 720
// and 719.
constexpr int kPicks = 8;

template <bool F32, bool NT>
__global__ __launch_bounds__(kRowThreads) void k_return_rows(ReturnArgs a) {
  const int groups = a.H / 8;
  const Place p = place_of(groups);
  if (p.t >= a.T) return;
  const int64_t at = p.t * a.H + 8 * p.c8;
  float acc[8] = {};
  for (int j0 = 0; j0 < a.K; j0 += kPicks) {
    v4i v[kPicks];
    uint32_t r[kPicks];
    float w[kPicks];
    bool ok[kPicks], whole = true;
#pragma unroll
    for (int u = 0; u < kPicks; ++u) {
      const int64_t pair = p.t * a.K + min(j0 + u, a.K - 1);
      r[u] = (uint32_t)a.pair_rows[pair];
      w[u] = a.w ? a.w[pair] : 1.f;
      ok[u] = j0 + u < a.K && r[u] < a.P;
    }
#pragma unroll
    for (int u = 0; u < kPicks; ++u) whole &= ok[u];
    if (__all(whole)) {
#pragma unroll
      for (int u = 0; u < kPicks; ++u) v[u] = load16_nt(a.rows + (int64_t)r[u] * a.H + 8 * p.c8);
    } else {
#pragma unroll
      for (int u = 0; u < kPicks; ++u)
        if (ok[u]) v[u] = load16_nt(a.rows + (int64_t)r[u] * a.H + 8 * p.c8);
    }
#pragma unroll
    for (int u = 0; u < kPicks; ++u)
      if (ok[u]) {
        float f[8];
        unpack8(v[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[u], f[i], acc[i]);
      }
  }
  if (a.add) {
    float f[8];
    load8<F32>(a.add, at, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += f[i];
  }
  if constexpr (F32) {
    float* y = static_cast<float*>(a.y) + at;
    store_row<NT>(reinterpret_cast<uint16_t*>(y), __builtin_bit_cast(v4i, v4f{acc[0], acc[1], acc[2], acc[3]}));
    store_row<NT>(reinterpret_cast<uint16_t*>(y + 4), __builtin_bit_cast(v4i, v4f{acc[4], acc[5], acc[6], acc[7]}));
  } else {
    store_row<NT>(static_cast<uint16_t*>(a.y) + at, pack8(acc));
  }
}

struct ReturnGradArgs {
  const void* dy;         // [T, H]
  const uint16_t* rows;   // not read without d_w
  const int32_t* pair_rows;
  const float* w;         // optional
  uint16_t* d_rows;       // optional; may be rows
  float* d_w;             // [T, K], optional
  int64_t P;
  int T, H, K;
};

// LANES lanes per pick, a wave or 16 (rows of up to kNarrow columns): its row's dot product
// with the token's gradient in lane sums. A token's gradient is read K times, from the
// caches: 1.16 GB come from HBM for 8191 tokens, 1.04 GB are rows and gradients read once.
// A wave and 16 lanes per pick, top-4: 65317 x 72 86 and 32 us, 32768 x 256 49 and 29, x 512
// 56 and 54.
constexpr int kNarrow = 512;
template <int LANES, bool F32, bool NT>
__global__ __launch_bounds__(kRowThreads) void k_return_rows_grad(ReturnGradArgs a) {
  const int lane = threadIdx.x % LANES;
  int sub = threadIdx.x / LANES;
  if constexpr (LANES == 64) sub = __builtin_amdgcn_readfirstlane(sub);
  const int64_t pair = block_id() * (kRowThreads / LANES) + sub;
  if (pair >= a.P) return;
  const int64_t t = (uint32_t)pair / (uint32_t)a.K;   // P is below 2^28
  const uint32_t r = (uint32_t)a.pair_rows[pair];
  const bool ok = r < a.P;
  float dot = 0.f;
  if (ok) {
    const float w = a.w ? a.w[pair] : 1.f;
    const int64_t row = (int64_t)r * a.H;
    for (int c = 8 * lane; c < a.H; c += 8 * LANES) {
      float dy[8];
      load8<F32>(a.dy, t * a.H + c, dy);
      if (a.d_w) {
        float f[8];
        unpack8(load16_nt(a.rows + row + c), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(f[i], dy[i], dot);
      }
      if (a.d_rows) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dy[i] *= w;
        store_row<NT>(a.d_rows + row + c, pack8(dy));
      }
    }
  }
  if (a.d_w) {
    dot = row_sum<LANES>(dot);
    if (lane == 0) a.d_w[pair] = dot;
  }
}

// f<fp32, nontemporal>()
template <typename F>
void by_kind(bool f32, bool nt, F f) {
  if (f32) {
    if (nt) f(std::true_type{}, std::true_type{});
    else f(std::true_type{}, std::false_type{});
  } else {
    if (nt) f(std::false_type{}, std::true_type{});
    else f(std::false_type{}, std::false_type{});
  }
}

inline dim3 token_groups(int T, int H) { return grid_of_blocks(ceil_div((int64_t)T * (H / 8), kRowThreads)); }

}  // namespace

hipError_t launch_sort_rows(int T, int H, int K, const void* x, const uint8_t* x_s, const int32_t* pair_rows,
                            uint16_t* rows, hipStream_t s) {
  const SortArgs a{x, x_s, pair_rows, rows, (int64_t)T * K, T, H, K};
  const dim3 grid = token_groups(T, H), block(kRowThreads);
  if (x_s) hipLaunchKernelGGL((k_sort_rows<true, false>), grid, block, 0, s, a);
  else if (a.P * H > kCachedRows) hipLaunchKernelGGL((k_sort_rows<false, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_sort_rows<false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_return_rows(int T, int H, int K, const uint16_t* rows, const int32_t* pair_rows, const float* w,
                              const void* add, bool f32, void* y, hipStream_t s) {
  const ReturnArgs a{rows, pair_rows, w, add, y, (int64_t)T * K, T, H, K};
  const dim3 grid = token_groups(T, H), block(kRowThreads);
  by_kind(f32, a.P * H > kCachedRows, [&](auto f, auto nt) {
    hipLaunchKernelGGL((k_return_rows<decltype(f)::value, decltype(nt)::value>), grid, block, 0, s, a);
  });
  return hipGetLastError();
}

hipError_t launch_return_rows_grad(int T, int H, int K, const void* dy, bool f32, const uint16_t* rows,
                                   const int32_t* pair_rows, const float* w, uint16_t* d_rows, float* d_w,
                                   hipStream_t s) {
  const ReturnGradArgs a{dy, rows, pair_rows, w, d_rows, d_w, (int64_t)T * K, T, H, K};
  const dim3 block(kRowThreads);
  by_kind(f32, a.P * H > kCachedRows, [&](auto f, auto nt) {
    constexpr bool F = decltype(f)::value, N = decltype(nt)::value;
    auto go = [&](auto kernel, int lanes) {
      hipLaunchKernelGGL(kernel, grid_of_blocks(ceil_div(a.P, kRowThreads / lanes)), block, 0, s, a);
    };
    if (H <= kNarrow) go(k_return_rows_grad<16, F, N>, 16);
    else go(k_return_rows_grad<64, F, N>, 64);
  });
  return hipGetLastError();
}

}  // namespace moe

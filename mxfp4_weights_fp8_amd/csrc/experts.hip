// The experts' products on rows grouped by expert, and their gradients, in bf16 with fp32
// sums:  y[r] = W[e] x[r],  dx[r] = W[e]^T dy[r],  dW[e] = sum over e's rows of dy[r] x[r]^T
// for the rows r in [offsets[e], offsets[e + 1]). The offsets live on the device, so
// grids are sized by bounds and workgroups look up what is theirs.
//
// Few rows (a decode step): bound by streaming the weights of the experts that have rows,
// on k_expert_few. More rows: tiles (experts_tile.hip), along a list that one workgroup
// writes first.
#include "experts.h"
#include "linear.h"
#include "lane_reduce.h"
#include "rows.h"

#include <math.h>

namespace moe {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f mfma_bf16(const v4i a, const v4i b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// ------------------------------------------------------------------ few rows
// Unit u of the experts' rows in units of at most kFewRows; rows 0 past the last one. A
// wave looks it up: each lane counts the units of E / 64 neighbouring experts, a scan
// over the lanes finds the lane, a second one the expert.
constexpr int kFewRows = 64;
struct Unit {
  int expert, row0, rows;
};
__device__ __forceinline__ int scan_add(int v, int lane) {   // inclusive, over a wave
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    v += lane >= d ? o : 0;
  }
  return v;
}
__device__ __forceinline__ Unit find_unit(const int32_t* off, int E, int P, int u) {
  const int lane = threadIdx.x & 63, per = (E + 63) / 64;
  auto units = [&](const RowRange r) { return (r.hi - r.lo + kFewRows - 1) / kFewRows; };
  int n = 0, prev = off[min(lane * per, E)];
#pragma unroll 8
  for (int i = 1; i <= per; ++i) {   // experts past the last one have no rows
    const int next = off[min(lane * per + i, E)];
    n += units(rows_of(prev, next, P));
    prev = next;
  }
  const int end = scan_add(n, lane);
  const uint64_t past = __ballot(end > u);
  if (past == 0) return Unit{0, 0, 0};
  const int at = __ffsll((unsigned long long)past) - 1;
  int base = __shfl(end - n, at);
  const int e = at * per + lane;
  const bool mine = lane < per && e < E;
  const RowRange r = mine ? rows_of(off[e], off[e + 1], P) : RowRange{0, 0};
  const int m = units(r), stop = base + scan_add(m, lane);
  const int found = __ffsll((unsigned long long)__ballot(stop > u)) - 1;
  const int first = __shfl(stop - m, found), lo = __shfl(r.lo, found), hi = __shfl(r.hi, found);
  const int row0 = lo + (u - first) * kFewRows;
  return Unit{__builtin_amdgcn_readfirstlane(at * per + found), __builtin_amdgcn_readfirstlane(row0),
              __builtin_amdgcn_readfirstlane(min(kFewRows, hi - row0))};
}

// A workgroup owns 16 output columns of a unit; its waves take every waves-th step of 64
// of the contraction straight from memory into registers, kDepth steps' loads at a time,
// and add their sums through LDS in wave order. FT: 16-row fragments.
//
// 56 rows of 30 experts, 768 x 7168 (330 MB of weights) 74 us, 4.5 TB/s. The registers (94 per
// lane) leave room for five waves per SIMD: five workgroups of four waves share a CU, two of
// eight (78 us) or one of sixteen (88 us). A row's 128 bytes come by two loads of 64; with the
// nontemporal hint, which lets go of the line between them, 101 us.
constexpr int kFewWaves = 4;

template <int FT, bool F32>
__device__ __forceinline__ void few_rows(const ExpertArgs& a, const Unit& u, float* red) {
  constexpr int kDepth = 4 / FT;
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * 16, steps = a.D / 64;
  const uint16_t* w = a.w + u.expert * a.w_expert + (int64_t)(n0 + c) * a.ws + q * 8;
  const uint16_t* x[FT];
#pragma unroll
  for (int f = 0; f < FT; ++f) x[f] = a.x + (int64_t)(u.row0 + min(16 * f + c, u.rows - 1)) * a.D + q * 8;
  v4f acc[FT] = {};
  for (int s = wave; s < steps; s += waves * kDepth) {
    v4i wv[kDepth][2], xv[kDepth][FT][2];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int st = s + d * waves;
      if (st < steps) {   // wave-uniform
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          wv[d][h] = load16(w + st * 64 + 32 * h);
#pragma unroll
          for (int f = 0; f < FT; ++f) xv[d][f][h] = load16(x[f] + st * 64 + 32 * h);
        }
      }
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
      if (s + d * waves < steps) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int f = 0; f < FT; ++f) acc[f] = mfma_bf16(wv[d][h], xv[d][f][h], acc[f]);
      }
  }
  v4f* part = reinterpret_cast<v4f*>(red);
#pragma unroll
  for (int f = 0; f < FT; ++f) part[(wave * FT + f) * 64 + lane] = acc[f];
  __syncthreads();
  for (int i = threadIdx.x; i < FT * 64; i += blockDim.x) {
    v4f v = part[i];
    for (int k = 1; k < waves; ++k) v += part[k * FT * 64 + i];
    const int row = 16 * (i >> 6) + (i & 15), n = n0 + 4 * ((i & 63) >> 4);
    if (row < u.rows) {
      const int64_t at = (int64_t)(u.row0 + row) * a.O + n;
      if constexpr (F32) *reinterpret_cast<v4f*>(static_cast<float*>(a.y) + at) = v;
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) =
            make_uint2(bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]));
    }
  }
}

template <bool F32>
__global__ __launch_bounds__(64 * kFewWaves) void k_expert_few(ExpertArgs a) {
  __shared__ __attribute__((aligned(16))) float red[kFewWaves * 4 * 256];
  const Unit u = find_unit(a.off, a.E, a.P, blockIdx.y);
  if (u.rows == 0) return;
  if (u.rows <= 16) few_rows<1, F32>(a, u, red);
  else if (u.rows <= 32) few_rows<2, F32>(a, u, red);
  else few_rows<4, F32>(a, u, red);
}

// ------------------------------------------------------------------ the tile list
// list[0].x = number of row tiles, then {expert, first row, rows, 0} of each: an expert's
// rows in tiles of kTileRows, the last one shorter. Tiles of more than 128 rows come
// first, then those of more than 64, then the rest (the kernel's three sizes), experts in
// rising order in each: the short ones fill up the last round. together: a short tile
// stays behind its expert's other ones, whose weights it shares, which with many column
// tiles is worth more than an even last round (32K tokens, 384 experts, 7168 x 384 1731 us
// against 1819, dx of 768 x 7168 in 8K tokens 1056 against 1100; but 768 x 7168 2815
// against 2734).
// order: the experts by their number of rows, the most first (in classes of a quarter of
// an octave; within one by index).
// With 256 and 1024 threads, in us: 384 experts of one tile each right behind a product of theirs
// 3.4 and 4.3, behind other work 4.8 and 4.8, with the order 5.3 and 7.4; of three tiles each
// 6.7-7.3 and 5.7-6.3, with the order 8.7 and 8.8. (1024 threads for 4096 experts: 7, with the order 11.5.)
constexpr int kListPer = 4;     // experts per thread: 256 threads up to 1024 experts
constexpr int kClasses = 128;
constexpr int kTogether = 8;    // column tiles

template <int kListThreads>
__global__ __launch_bounds__(kListThreads) void k_expert_list(const int32_t* off, int E, int P, int4* list, int cap,
                                                              bool together, int32_t* order) {
  __shared__ int ends[kListPer * kListThreads];        // tall tiles up to and with expert e
  __shared__ int waves[3][kListThreads / 64];
  __shared__ int classes[kClasses];
  __shared__ int counts[kListPer * kListThreads / 64 * kClasses];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int kPer = kListPer;
  if (list) {
    // Each thread's kPer experts: tall tiles, and a last one of middle or small size.
    RowRange r[kPer];
    int tall[kPer], n[3] = {0, 0, 0}, disorder = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      const int lo = e < E ? off[e] : 0, hi = e < E ? off[e + 1] : 0;
      disorder |= lo < 0 || hi < lo || hi > P;
      r[i] = RowRange{lo, hi};
      const int rows = r[i].hi - r[i].lo, last = rows % kTileRows;
      const bool apart = last <= 128 && !(together && rows >= kTileRows);
      tall[i] = rows / kTileRows + (last > 0 && !apart);
      n[0] += tall[i];
      n[1] += apart && last > 64;
      n[2] += apart && last > 0 && last <= 64;
    }
    int at[3], total[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      at[k] = scan_add(n[k], lane);
      if (lane == 63) waves[k][wave] = at[k];
      at[k] -= n[k];
    }
    // Offsets that no plan gives: no tiles (what is counted here may then overflow).
    const bool sound = !__syncthreads_or(disorder);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      total[k] = 0;
#pragma unroll
      for (int w = 0; w < kListThreads / 64; ++w) {
        at[k] += w < wave ? waves[k][w] : 0;
        total[k] += waves[k][w];
      }
    }
    at[1] += total[0];
    at[2] += total[0] + total[1];
    auto write = [&](int t, int e, const RowRange& x, int k) {   // tile k of expert e at place t
      const int row0 = x.lo + k * kTileRows;
      if (sound && t < cap) list[1 + t] = make_int4(e, row0, min(kTileRows, x.hi - row0), 0);
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      at[0] += tall[i];
      ends[tid * kPer + i] = at[0];
      const int rows = r[i].hi - r[i].lo, last = rows - tall[i] * kTileRows;
      if (last > 0) write(last > 64 ? at[1]++ : at[2]++, tid * kPer + i, r[i], tall[i]);
    }
    __syncthreads();
    if (tid == 0) list[0] = make_int4(sound ? min(total[0] + total[1] + total[2], cap) : 0, 0, 0, 0);
    for (int t = tid; sound && t < min(total[0], cap); t += kListThreads) {
      int lo = 0, hi = E - 1;   // the first expert whose end is past t
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (ends[mid] > t) hi = mid;
        else lo = mid + 1;
      }
      write(t, lo, RowRange{off[lo], off[lo + 1]}, t - (lo ? ends[lo - 1] : 0));
    }
  }
  if (!order) return;
  // Class of n rows, 0 the largest; the rank of an expert is the experts of classes
  // before its own, those of its class in segments of 64 experts before its own, and
  // those before it in its segment, which the lanes of a wave find by comparing classes.
  auto class_of = [&](int v) {
    if (v == 0) return kClasses - 1;
    const int b = 31 - __clz(v), frac = b >= 2 ? (v >> (b - 2)) & 3 : 0;
    return kClasses - 2 - (4 * b + frac);   // b is at most 30
  };
  __syncthreads();
  const int segments = (E + 63) / 64;
  for (int i = tid; i < segments * kClasses; i += kListThreads) counts[i] = 0;
  __syncthreads();
  int cls[kPer], before[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * kListThreads + tid;
    const RowRange r = e < E ? rows_of(off[e], off[e + 1], P) : RowRange{0, 0};
    cls[i] = class_of(r.hi - r.lo);
    uint64_t same = __ballot(e < E);
#pragma unroll
    for (int b = 1; b < kClasses; b <<= 1) {
      const uint64_t set = __ballot((cls[i] & b) != 0);
      same &= (cls[i] & b) ? set : ~set;
    }
    before[i] = __popcll(same & (((uint64_t)1 << lane) - 1));
    if (e < E && before[i] == 0) counts[(e >> 6) * kClasses + cls[i]] = __popcll(same);
  }
  __syncthreads();
  if (tid < kClasses) {
    int s = 0;
    for (int g = 0; g < segments; ++g) {
      const int k = counts[g * kClasses + tid];
      counts[g * kClasses + tid] = s;
      s += k;
    }
    const int upto = scan_add(s, lane);
    classes[tid] = upto - s;
    if (tid == 63) waves[0][0] = upto;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * kListThreads + tid;
    if (e < E)
      order[classes[cls[i]] + (cls[i] >= 64 ? waves[0][0] : 0) + counts[(e >> 6) * kClasses + cls[i]] + before[i]] = e;
  }
}

// Which kernel: the least estimated time, in us, with as many experts at work as a mildly
// uneven router gives P picks. k_expert_few streams weights at 5.3 TB/s, pays for every
// workgroup of 16 columns (4.5 ns with all CUs at it), for its steps (their loads of x keep
// a CU busy for 0.08 to 0.25 us) and for its rows (110 TFLOP/s, partly hidden); the tiles
// stream at 5.2 TB/s behind the list, but a tile takes 0.75 us per step however few rows it
// has. k_expert_few and tiles (with an unsplit contraction), in us:
//   768 x 7168, 384 experts, 8 rows 13 and 76, 56 rows 78 and 135, 208 rows 156 and 160, 512
//   rows 319 and 327, 1363 rows 730 and 785, 5945 rows 1084 and 802
//   7168 x 384, 384 experts, 8 rows 11 and 14, 56 rows 68 and 41, 512 rows 429 and 170
//   4096 x 4096, 16 experts, 2 rows 15 and 44, 64 rows 90 and 120, 256 rows 141 and 129
//   1024 x 2048, 64 experts, 32 rows 14 and 28, 222 rows 54 and 46, 992 rows 80 and 53
//   512 x 256, 8 experts, 3 rows 7 and 11, 959 rows 7 and 16; 1024 x 512, 2048 rows 25 and 21
struct Estimate {
  double us;
  int splits;
};
// Experts at work, of E that P picks go to.
inline double at_work(double P, double E) { return fmax(1.0, E * (1.0 - exp(-0.65 * P / E))); }

// The tiles' product, its contraction of D split over workgroups where there are fewer
// tiles than CUs: each part at least 8 steps, joined at 4 TB/s. Unsplit and split: 8
// experts of 64 rows x 768 x 7168 65 and 31 us, of 200 x 1024 x 2048 49 and 35; as dx 8 of 128
// rows x 384 from 7168 columns 89 and 27.
inline Estimate tiles_estimate(double P, double E, int D, int O) {
  const double experts = at_work(P, E), steps = D / 64, rows = P / experts;
  const double tiles = fmax(experts, P / kTileRows) * (double)ceil_div(O, 32 * tile_fragments(O));
  const double step = 0.75 + 0.85 * fmin(1.0, rows / kTileRows);
  Estimate best{1e30, 1};
  for (int k = 1; k == 1 || (k <= steps / 8 && tiles * k <= 512); k += k < 8 ? 1 : k / 4) {
    const double t = 8 + fmax(2.0 * experts * D * O / 5.2e6, step * ceil(tiles * k / 256) * ceil(steps / k)) +
                     0.2 * steps / k + (k > 1 ? 4 + k * P * O * 8 / 4e6 : 0);
    if (t < best.us) best = Estimate{t, k};
  }
  return best;
}

inline bool few(const moe_expert_dims& d) {
  const double rows = d.P, matrix = (double)d.N * d.K, experts = at_work(rows, d.E);
  const double workgroups = (experts + rows / kFewRows) * (d.N / 16), per_expert = rows / experts;
  const double turn = per_expert > 32 ? 0.25 : per_expert > 16 ? 0.15 : 0.08;   // us of a workgroup's step
  const double t = 6 + fmax(fmax(2.0 * experts * matrix / 5.3e6, 0.0045 * workgroups),
                            turn * (d.K / 64) * ceil(workgroups / 256)) + 1.2 * rows * matrix / 1.1e8;
  return t <= tiles_estimate(rows, d.E, d.K, d.N).us;
}

// Splits of every expert's rows for the weights' gradient: as many as fill the CUs, where
// the weights are few, each at least 4 steps of an average expert. Unsplit and split: one
// expert of 65536 rows, 128 x 128 617 and 24 us, of 20000, 512 x 512 452 and 40, four of 5000,
// 256 x 256 122 and 26.
inline int wgrad_splits(const moe_expert_dims& d) {
  const double tiles = (double)d.E * ceil_div(d.N, 32 * tile_fragments(d.N)) * ceil_div(d.K, 32 * tile_fragments(d.K));
  const double steps = ceil((double)d.P / d.E / 64), elements = (double)d.E * d.N * d.K;
  double least = 1e30;
  int best = 1;
  for (int k = 1; k == 1 || (k <= steps / 4 && tiles * k <= 512); k += k < 8 ? 1 : k / 4) {
    const double t = 1.6 * ceil(tiles * k / 256) * ceil(steps / k) + (k > 1 ? 4 + k * elements * 8 / 4e6 : 0);
    if (t < least) {
      least = t;
      best = k;
    }
  }
  return best;
}

// out[i] = sum over the parts, of [P, O] results for the rows that experts have. A
// workgroup joins 256 elements, four per lane: each of its waves adds every waves-th part,
// eight loads on their way, then their sums are added in wave order.
constexpr int kJoinWaves = 16;
template <bool F32>
__global__ __launch_bounds__(64 * kJoinWaves) void k_expert_join(const float* parts, int splits, int64_t n, void* out,
                                                                 const int32_t* off, int E, int P, int O) {
  __shared__ v4f sums[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t at = 4 * (block_id() * 64 + lane);
  bool mine = at < n;
  if (off) {
    const RowRange r = rows_of(off[0], off[E], P);
    mine = at >= (int64_t)r.lo * O && at < (int64_t)r.hi * O;
  }
  v4f v{0.f, 0.f, 0.f, 0.f};
  if (mine) {
#pragma unroll 8
    for (int k = wave; k < splits; k += waves) v += *reinterpret_cast<const v4f*>(parts + k * n + at);
  }
  if (waves > 1) {
    sums[wave][lane] = v;
    __syncthreads();
    if (wave > 0) return;
    for (int w = 1; w < waves; ++w) v += sums[w][lane];
  }
  if (!mine) return;
  if constexpr (F32) *reinterpret_cast<v4f*>(static_cast<float*>(out) + at) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
        make_uint2(bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]));
}

void launch_join(const float* parts, int splits, int64_t n, void* out, bool f32, const int32_t* off, int E, int P, int O,
                 hipStream_t s) {
  const int waves = splits < 8 ? 1 : splits < 32 ? 4 : kJoinWaves;
  const dim3 grid = grid_of_blocks(ceil_div(n, 256)), block(64 * waves);
  if (f32) hipLaunchKernelGGL(k_expert_join<true>, grid, block, 0, s, parts, splits, n, out, off, E, P, O);
  else hipLaunchKernelGGL(k_expert_join<false>, grid, block, 0, s, parts, splits, n, out, off, E, P, O);
}

inline size_t list_bytes(const moe_expert_dims& d) {
  return align_up(sizeof(int4) * (size_t)(1 + expert_tiles_bound(d.P, d.E)), 256);
}
inline size_t order_bytes(const moe_expert_dims& d) { return align_up(sizeof(int32_t) * (size_t)d.E, 256); }
inline size_t parts_bytes(int splits, int64_t elements) { return splits > 1 ? sizeof(float) * splits * elements : 0; }

// O: the columns of the results that the tiles of the list are for.
void launch_list(const moe_expert_dims& d, const int32_t* off, int O, int4* list, int32_t* order, hipStream_t s) {
  auto go = [&](auto kernel, int threads) {
    hipLaunchKernelGGL(kernel, dim3(1), dim3(threads), 0, s, off, d.E, d.P, list, (int)expert_tiles_bound(d.P, d.E),
                       ceil_div(O, kTileRows) >= kTogether, order);
  };
  if (d.E <= 1024) go(k_expert_list<256>, 256);
  else go(k_expert_list<1024>, 1024);
}

// A product in tiles along the list, into parts where its contraction is split.
void launch_tiled(ExpertArgs a, bool w_trans, bool f32, float* parts, hipStream_t s) {
  a.splits = tiles_estimate(a.P, a.E, a.D, a.O).splits;
  if (a.splits == 1) return launch_expert_tiles(a, w_trans, f32, s);
  void* const y = a.y;
  a.y = parts;
  launch_expert_tiles(a, w_trans, true, s);
  launch_join(parts, a.splits, (int64_t)a.P * a.O, y, f32, a.off, a.E, a.P, a.O, s);
}

}  // namespace

size_t expert_linear_ws_bytes(const moe_expert_dims& d) {
  if (few(d)) return 0;
  return list_bytes(d) + parts_bytes(tiles_estimate(d.P, d.E, d.K, d.N).splits, (int64_t)d.P * d.N);
}

hipError_t launch_expert_linear(const moe_expert_dims& d, const uint16_t* x, const uint16_t* w, const int32_t* off,
                                void* y, void* ws, hipStream_t s) {
  const bool f32 = d.type == MOE_TYPE_F32;
  const ExpertArgs a{x, w, off, y, static_cast<const int4*>(ws), (int64_t)d.N * d.K, d.P, d.E, d.K, d.N, d.K, 1};
  if (few(d)) {
    const int64_t units = d.P / kFewRows + (d.P < d.E ? d.P : d.E);
    const int waves = d.K / 64 < kFewWaves ? d.K / 64 : kFewWaves;
    const dim3 grid((unsigned)(d.N / 16), (unsigned)units), block(64 * (unsigned)waves);
    if (f32) hipLaunchKernelGGL(k_expert_few<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_expert_few<false>, grid, block, 0, s, a);
  } else {
    launch_list(d, off, d.N, static_cast<int4*>(ws), nullptr, s);
    launch_tiled(a, false, f32, reinterpret_cast<float*>(static_cast<char*>(ws) + list_bytes(d)), s);
  }
  return hipGetLastError();
}

size_t expert_linear_grad_ws_bytes(const moe_expert_dims& d) {   // the two products run one after the other
  const size_t x = d.P ? parts_bytes(tiles_estimate(d.P, d.E, d.N, d.K).splits, (int64_t)d.P * d.K) : 0;
  const size_t w = parts_bytes(wgrad_splits(d), (int64_t)d.E * d.N * d.K);
  return order_bytes(d) + list_bytes(d) + (x > w ? x : w);
}

hipError_t launch_expert_linear_grad(const moe_expert_dims& d, const uint16_t* dy, const uint16_t* x, const uint16_t* w,
                                     const int32_t* off, uint16_t* dx, void* dw, void* ws, hipStream_t s) {
  int32_t* const order = static_cast<int32_t*>(ws);
  int4* const list = reinterpret_cast<int4*>(static_cast<char*>(ws) + order_bytes(d));
  float* const parts = reinterpret_cast<float*>(static_cast<char*>(ws) + order_bytes(d) + list_bytes(d));
  if (d.P == 0) dx = nullptr;
  if (!dx && !dw) return hipSuccess;
  launch_list(d, off, d.K, dx ? list : nullptr, dw ? order : nullptr, s);
  if (dx)   // [P, K] = dy [P, N] . w [E, N, K], contracted over N
    launch_tiled(ExpertArgs{dy, w, off, dx, list, (int64_t)d.N * d.K, d.P, d.E, d.N, d.K, d.K, 1}, true, false, parts, s);
  if (dw) {
    const bool f32 = d.type == MOE_TYPE_F32;
    const int splits = wgrad_splits(d);
    launch_expert_wgrad(ExpertGradArgs{dy, x, off, splits > 1 ? parts : dw, order, d.P, d.E, d.N, d.K, splits},
                        f32 || splits > 1, s);
    if (splits > 1) launch_join(parts, splits, (int64_t)d.E * d.N * d.K, dw, f32, nullptr, 0, 0, 0, s);
  }
  return hipGetLastError();
}

}  // namespace moe

// Dense bf16 product with bias, activation and residual in its epilogue:
//   y[m, n] = act(sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n]
// (the router's logits, or a projection back to the hidden size), accumulated in
// fp32 on v_mfma_f32_16x16x32_bf16 and rounded once.
//
// The weights are the MFMA's first operand, so D's rows are output columns and lane
// (c, q) = (l % 16, l / 16) holds columns 4q .. 4q+3 of token c: each lane stores
// four neighbouring outputs.
#include "linear.h"
#include "lane_reduce.h"

namespace moe {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f mfma_bf16(const v4i a, const v4i b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// ------------------------------------------------------------------ few rows
// At most 8 rows and few columns (a router's decode step): bound by latency, so the
// weights are spread over as many CUs as give each workgroup R columns, and every load
// of a wave is in flight at once. A lane multiplies 8 of a 512-long chunk of K (wave w
// takes chunks w, w + waves, ...) in fp32: R weights' and MT rows' 16 bytes give R MT
// sums, added over the lanes, then over the waves in order.
// 7 x 384 x 7168: 6.0 us (0.9 TB/s, latency), 24 workgroups of 16 columns on the matrix
// cores 12.3 us.
constexpr int kDotWaves = 16;

__device__ __forceinline__ void unpack8(const v4i raw, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float((uint32_t)raw[i] << 16);
    v[2 * i + 1] = __uint_as_float((uint32_t)raw[i] & 0xFFFF0000u);
  }
}

template <int MT, int R>
__global__ __launch_bounds__(64 * kDotWaves) void k_linear_dot(LinearArgs a) {
  __shared__ float red[kDotWaves][MT * R];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * R;
  float acc[MT][R] = {};
  for (int k = (wave * 64 + lane) * 8; k < a.C; k += waves * 512) {
    v4i wv[R], xv[MT];
#pragma unroll
    for (int r = 0; r < R; ++r) wv[r] = load16(a.w + min(n0 + r, a.N - 1) * a.ws + k);   // rows past the end: any valid row
#pragma unroll
    for (int m = 0; m < MT; ++m) xv[m] = load16(a.x + min(m, a.M - 1) * a.xs + k);
    float wf[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r) unpack8(wv[r], wf[r]);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float xf[8];
      unpack8(xv[m], xf);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[m][r] += xf[i] * wf[r][i];
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float s = row_sum<64>(acc[m][r]);
      if (lane == 0) red[wave][m * R + r] = s;
    }
  __syncthreads();
  if (threadIdx.x < MT * R) {
    float v[1] = {red[0][threadIdx.x]};
    for (int w = 1; w < waves; ++w) v[0] += red[w][threadIdx.x];
    const int m = threadIdx.x / R, n = n0 + threadIdx.x % R;
    finish<1>(a, m, n, v, load_residual<1>(a, m, n));
  }
}

// At most 64 rows: bound by reading the weights. A workgroup owns 16 output columns and
// one of a.splits shares of the contraction; its waves take every W-th step of 64 K,
// straight from memory into registers, and add their sums through LDS in wave order.
// 9 x 7168 x 7168 27 us, 3.8 TB/s; 64 x 384 x 7168 12.3 us per call, bound by the host.
constexpr int kSmallWaves = 16;

template <int FT>
__global__ __launch_bounds__(64 * kSmallWaves) void k_linear_small(LinearArgs a) {
  constexpr int kSmallDepth = 4 / FT;   // steps of loads in flight per wave (128 VGPRs at 16 waves)
  extern __shared__ __attribute__((aligned(16))) float red[];   // [wave][FT][64 lanes][4]
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * 16, split = blockIdx.y;
  const int first = a.C / 64 * split / a.splits, steps = a.C / 64 * (split + 1) / a.splits;
  const uint16_t* w = a.w + (int64_t)min(n0 + c, a.N - 1) * a.ws + q * 8;   // rows past the end: any valid row
  const uint16_t* x[FT];
#pragma unroll
  for (int f = 0; f < FT; ++f) x[f] = a.x + (int64_t)min(16 * f + c, a.M - 1) * a.xs + q * 8;
  v4f acc[FT] = {};
  for (int s = first + wave; s < steps; s += waves * kSmallDepth) {
    v4i wv[kSmallDepth][2], xv[kSmallDepth][FT][2];
#pragma unroll
    for (int d = 0; d < kSmallDepth; ++d) {
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
    for (int d = 0; d < kSmallDepth; ++d)
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
    const int f = i >> 6, l = i & 63;
    const int m = 16 * f + (l & 15), n = n0 + 4 * (l >> 4);
    float o[4] = {v[0], v[1], v[2], v[3]};
    if (a.splits == 1) finish<4>(a, m, n, o, load_residual<4>(a, m, n));
    else store_part<4>(a, split, m, n, o);
  }
}

// The parts of a split product, added in order, and the epilogue.
__global__ __launch_bounds__(256) void k_linear_join(LinearArgs a) {
  const int groups = (a.N + 3) / 4;
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (g >= (int64_t)a.M * groups) return;
  const int64_t m = g / groups;
  const int n = 4 * (int)(g - m * groups);
  const Residual<4> r = load_residual<4>(a, m, n);
  v4f v{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.splits; ++s) {
    const float* src = a.parts + ((int64_t)s * a.M + m) * a.N + n;
    if (a.N % 4 == 0) {
      v += *reinterpret_cast<const v4f*>(src);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.N) v[i] += src[i];
    }
  }
  float o[4] = {v[0], v[1], v[2], v[3]};
  finish<4>(a, m, n, o, r);
}

}  // namespace

// Rows that k_linear_dot is built for.
inline int dot_rows(int M) { return M == 1 ? 1 : M <= 4 ? 4 : 8; }

// Tile shape and splits of the contraction: the least estimated time. Measured with
// every CU busy, in 10 ns: a step of 64 takes `step` (two workgroups of the smallest
// tile share a CU), prologue and epilogue `fixed` per round of tiles, and joining the
// parts of a split product 4 us and its traffic at 4 TB/s. (8192^3: 256 x 256 tiles 851
// us, 128 x 128 971; 8191 x 7168 x 2048: 310 and 266; 4096 x 2048 x 7168: 256 x 256 split
// in two 112, 128 x 128 110, unsplit 256 x 256 168.)
LinearPlan linear_plan(int M, int N, int C, Layout l, bool plain, bool two) {
  // Few rows. The vector units (rows in ones, fours or eights) while their products take
  // less time than what kSmall pays for its parts. In us, kDot and kSmall: at 384 columns
  // 8 x 512 3.6 and 3.5, 8 x 1024 3.7 and 5.4, 8 x 7168 5.6 and 8.1, 8 x 16384 7.8 and 10.3; 8
  // rows x 1024 x 7168 8.8 and 9.5, x 1536 x 4096 7.5 and 8.3, x 2048 x 4096 8.9 and 8.7, x
  // 1536 x 7168 13.4 and 10.6; 4 x 384 x 256 3.0 and 2.8, 4 x 384 x 512 2.9 and 3.3, 4 x 1536
  // x 7168 8.0 and 10.0, 4 x 2048 x 7168 10.8 and 10.7; 1 x 384 x 128 2.4 and 2.5, 1 x 2048 x
  // 16384 11.9 and 17.0. From 2560 columns on kSmall needs no parts (8 x 2560 x 2048 6.4 and
  // 5.9). Above 16 rows kSmall while its workgroups' reads of x, M N K / 8 bytes, stay small:
  // 64 x 4096 x 2048 11.8 us against 15.8 us in tiles, 64 x 7168 x 7168 75 against 30.
  if (l == Layout::kRows && (M <= 16 || (M <= 64 && (int64_t)M * N * C <= 800000000))) {
    const int64_t tiles = ceil_div(N, 16), steps = C / 64;
    const int64_t rows = dot_rows(M);
    if (M <= 8 && N <= 2048 && C >= 128 * rows && rows * N * C <= 60000000) return LinearPlan{Path::kDot, 0, 0, 1};
    // fewer workgroups than CUs: split the contraction, at least 8 steps each
    int64_t splits = 256 / tiles;
    if (splits > steps / 8) splits = steps / 8;
    return LinearPlan{Path::kSmall, 0, 0, splits > 1 ? (int)splits : 1};
  }
  static const struct {
    int ft, fw, per_cu, step, fixed;
  } kShapes[] = {{8, 8, 1, 170, 2200}, {8, 6, 1, 145, 1500}, {6, 8, 1, 145, 1500}, {4, 4, 2, 98, 800}};
  const int64_t steps = ceil_div(C, 64) * (two ? 2 : 1);
  LinearPlan best{Path::kTiles, 0, 0, 1};
  int64_t least = -1;
  for (const auto& t : kShapes) {
    const int64_t tiles = ceil_div(M, 32 * t.ft) * ceil_div(N, 32 * t.fw), slots = 256 * t.per_cu;
    for (int64_t splits = 1; splits == 1 || (splits <= steps / 4 && tiles * splits <= 2 * slots);
         splits += splits < 4 ? 1 : splits / 4) {
      int64_t time = ceil_div(tiles * splits, slots) * (ceil_div(steps, splits) * t.step + t.fixed);
      if (splits > 1) time += 400 + splits * M * N * 8 / 40000;
      if (least < 0 || time < least) {
        least = time;
        best = LinearPlan{Path::kTiles, t.ft, t.fw, (int)splits};
      }
    }
  }
  // A contraction of up to 384 that needs no epilogue: rows kept in registers, once the
  // result is large enough for a pipeline that starts once. In us, rows kept and tiles, at
  // 384: 16384 x 1024 25 and 21, 4096 x 7168 33 and 35, 8192 x 7168 52 and 63, 16384 x 7168
  // 92 and 126, 32768 x 2048 56 and 70; at 128: 4096 x 7168 20 and 25, 16384 x 7168 49 and 76.
  // With x in two parts (and the kernel that makes them) at 384: 8192 x 2048 48 and 46, 4096 x
  // 7168 64 and 66, 16384 x 7168 199 and 230; at 128: 8192 x 2048 28 and 27, 4096 x 7168 34 and 38.
  if (C <= 384 && N % 8 == 0 && plain && l != Layout::kBothTrans && (int64_t)M * N >= 20000000)   // C is a multiple of 128
    return LinearPlan{Path::kShort, 0, 0, 1};
  return best;
}

size_t linear_plan_parts(int M, int N, const LinearPlan& p) {
  return p.splits > 1 ? sizeof(float) * (size_t)p.splits * M * N : 0;
}

size_t linear_parts_bytes(int M, int N, int K) {   // the larger of the two plans
  const size_t a = linear_plan_parts(M, N, linear_plan(M, N, K, Layout::kRows, false)),
               b = linear_plan_parts(M, N, linear_plan(M, N, K, Layout::kRows, true));
  return a > b ? a : b;
}

hipError_t launch_linear_plan(const LinearArgs& in, const LinearPlan& p, Layout l, hipStream_t s) {
  LinearArgs a = in;
  a.splits = p.splits;
  if (p.path == Path::kDot) {
    const int64_t chunks = ceil_div(a.C, 512);
    const dim3 block(64 * (unsigned)(chunks < kDotWaves ? chunks : kDotWaves));
    auto run = [&](auto kernel, int r) { hipLaunchKernelGGL(kernel, dim3((unsigned)ceil_div(a.N, r)), block, 0, s, a); };
    // Two columns per workgroup; four where two would come to more than 256 workgroups of
    // long rows (8 x 768 x 7168 8.1 us against 9.4, 8 x 768 x 4096 5.8 against 5.6).
    const int rows = dot_rows(a.M);
    if (rows == 1) run(k_linear_dot<1, 2>, 2);
    else if (rows == 4) run(k_linear_dot<4, 2>, 2);
    else if (a.N <= 512 || a.C <= 4096) run(k_linear_dot<8, 2>, 2);
    else run(k_linear_dot<8, 4>, 4);
    return hipGetLastError();
  }
  if (p.path == Path::kSmall) {
    const int steps = (int)ceil_div(a.C / 64, p.splits);
    const int waves = steps < kSmallWaves ? steps : kSmallWaves;
    const dim3 grid((unsigned)ceil_div(a.N, 16), p.splits), block(64 * waves);
    const int ft = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
    const size_t lds = (size_t)waves * ft * 1024;
    if (ft == 1) hipLaunchKernelGGL(k_linear_small<1>, grid, block, lds, s, a);
    else if (ft == 2) hipLaunchKernelGGL(k_linear_small<2>, grid, block, lds, s, a);
    else hipLaunchKernelGGL(k_linear_small<4>, grid, block, lds, s, a);
  } else if (p.path == Path::kShort) {
    launch_short(a, l, s);
  } else {
    launch_tiles(a, p, l, s);
  }
  if (p.splits > 1) {
    const int64_t n = (int64_t)a.M * ceil_div(a.N, 4);
    hipLaunchKernelGGL(k_linear_join, dim3((unsigned)ceil_div(n, 256)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_linear(const moe_linear_dims& d, const uint16_t* x, const uint16_t* w, const float* bias,
                         const void* res, void* y, float* z, float* parts, hipStream_t s) {
  const LinearArgs a{x, w, d.K, d.K, 0, bias, res, y, z, parts, d.M, d.N, d.K, d.K,
                     d.act, 1, d.type == MOE_TYPE_F32};
  const bool plain = !bias && !res && !z && d.act == MOE_ACT_NONE && d.type == MOE_TYPE_BF16;
  return launch_linear_plan(a, linear_plan(d.M, d.N, d.K, Layout::kRows, plain), Layout::kRows, s);
}

}  // namespace moe

// Dense bf16 product with bias, activation and residual in its epilogue:
//   y[m, n] = act(sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n]
// (the router's logits, or a projection back to the hidden size), accumulated in
// fp32 on v_mfma_f32_16x16x32_bf16 and rounded once.
//
// The weights are the MFMA's first operand, so D's rows are output columns and lane
// (c, q) = (l % 16, l / 16) holds columns 4q .. 4q+3 of token c: each lane stores
// four neighbouring outputs.
#include "linear.h"
#include "lds_copy.h"

namespace moe {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f mfma_bf16(const v4i a, const v4i b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// The epilogue of columns n .. n + 3 of row m (those below N), from their sums.
__device__ __forceinline__ void finish4(const LinearArgs& a, int64_t m, int n, v4f v) {
  if (m >= a.M || n >= a.N) return;
  const int64_t at = m * a.N + n;
  if (a.N % 4 == 0) {
    if (a.bias) v += *reinterpret_cast<const v4f*>(a.bias + n);
    if (a.z) *reinterpret_cast<v4f*>(a.z + at) = v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = activate(v[i], a.act);
    if (a.out_f32) {
      if (a.res) v += *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(a.res) + at);
      *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.y) + at) = v;
    } else {
      if (a.res) {
        const uint2 r = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(a.res) + at);
        v += v4f{__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                 __uint_as_float(r.y & 0xFFFF0000u)};
      }
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + at) =
          make_uint2(bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= a.N) break;
    float f = v[i] + (a.bias ? a.bias[n + i] : 0.f);
    if (a.z) a.z[at + i] = f;
    f = activate(f, a.act);
    if (a.out_f32) {
      if (a.res) f += reinterpret_cast<const float*>(a.res)[at + i];
      reinterpret_cast<float*>(a.y)[at + i] = f;
    } else {
      if (a.res) f += bf16_to_float(reinterpret_cast<const uint16_t*>(a.res)[at + i]);
      reinterpret_cast<uint16_t*>(a.y)[at + i] = (uint16_t)bf16_pack2(f, 0.f);
    }
  }
}

// ------------------------------------------------------------------ few rows
// At most 64 rows: bound by reading the weights (or by latency). A workgroup owns 16
// output columns; its waves take every W-th step of 64 K, straight from memory into
// registers, and add their sums through LDS in wave order. Lane (c, q) reads bytes
// 32q .. 32q+31 of its row's 128-byte step: as K is summed, the two operands only
// have to agree on which K a lane holds.
constexpr int kSmallWaves = 16;

template <int FT>
__global__ __launch_bounds__(64 * kSmallWaves) void k_linear_small(LinearArgs a) {
  constexpr int kSmallDepth = 4 / FT;   // steps of loads in flight per wave (128 VGPRs at 16 waves)
  extern __shared__ __attribute__((aligned(16))) float red[];   // [wave][FT][64 lanes][4]
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * 16, steps = a.K / 64;
  const uint16_t* w = a.w + (int64_t)min(n0 + c, a.N - 1) * a.K + q * 16;   // rows past the end: any valid row
  const uint16_t* x[FT];
#pragma unroll
  for (int f = 0; f < FT; ++f) x[f] = a.x + (int64_t)min(16 * f + c, a.M - 1) * a.K + q * 16;
  v4f acc[FT] = {};
  for (int s = wave; s < steps; s += waves * kSmallDepth) {
    v4i wv[kSmallDepth][2], xv[kSmallDepth][FT][2];
#pragma unroll
    for (int d = 0; d < kSmallDepth; ++d) {
      const int st = s + d * waves;
      if (st < steps) {   // wave-uniform
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          wv[d][h] = load16(w + st * 64 + 8 * h);
#pragma unroll
          for (int f = 0; f < FT; ++f) xv[d][f][h] = load16(x[f] + st * 64 + 8 * h);
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
    finish4(a, 16 * f + (l & 15), n0 + 4 * (l >> 4), v);
  }
}

// --------------------------------------------------------------------- tiles
// Tile: 32 FW columns x 128 rows, four waves in a 2 x 2 grid of 16 FW columns x 64
// rows each. Three LDS stages of 64 K (128-byte rows, 16-byte chunks XOR-swizzled by
// (row / 2) % 8), filled by direct-to-LDS copies of 8 rows per instruction; the copy
// of step k + 3 is issued while step k is multiplied and step k + 1's fragments are
// read. Rows past the tensors' ends and steps past the range are copied as zeros by
// the buffer resource's bounds check.
constexpr int kTileThreads = 256;
constexpr int kTileRows = 128;
constexpr int kBufs = 3;
constexpr int kXcds = 8;
constexpr int kGroup = 8;   // row tiles that share a pass over the column tiles

template <int FW>
__global__ __launch_bounds__(kTileThreads, 1) void k_linear_tile(LinearArgs a, int m_tiles, int n_tiles) {
  constexpr int FT = 4;
  constexpr int kCols = 32 * FW;
  constexpr int kStageA = kCols * 128, kStageB = kTileRows * 128;
  constexpr int kCopies = FW + FT;
  constexpr int kOutRow = kCols + 4;   // floats per row of the staged result: 16 rows apart in distinct banks
  constexpr int kStages = kBufs * (kStageA + kStageB);
  static_assert(kTileRows * kOutRow * 4 <= kStages, "the result tile fits the stages' LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kStages];
  uint8_t* const sA = smem;                       // [buf][row][128 B]
  uint8_t* const sB = smem + kBufs * kStageA;

  // Workgroups are dealt to the XCDs in turn; give each XCD a contiguous run of the
  // tile order (split, group of kGroup row tiles, column tile, row tile), so that the
  // tiles that share operand rows share an L2.
  const int tiles = m_tiles * n_tiles, total = tiles * a.splits;
  const int run = (total + kXcds - 1) / kXcds;
  const int id = (blockIdx.x % kXcds) * run + blockIdx.x / kXcds;
  if ((int)(blockIdx.x / kXcds) >= run || id >= total) return;
  const int split = id / tiles, tile = id % tiles;
  const int group = tile / (kGroup * n_tiles), in_group = tile % (kGroup * n_tiles);
  const int rows_in_group = min(kGroup, m_tiles - group * kGroup);
  const int mt = group * kGroup + in_group % rows_in_group, nt = in_group / rows_in_group;
  const int m0 = mt * kTileRows, n0 = nt * kCols;

  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int row_bytes = 2 * a.K;
  const int steps = a.K / 64;   // even
  // this split's steps: pairs dealt as evenly as they go
  const int pairs = steps / 2;
  const int k0 = 2 * (int)((int64_t)pairs * split / a.splits), k1 = 2 * (int)((int64_t)pairs * (split + 1) / a.splits);

  const v4i_s rw = rsrc4(a.w + (int64_t)n0 * a.K, (uint32_t)(min(kCols, a.N - n0) * row_bytes));
  const v4i_s rx = rsrc4(a.x + (int64_t)m0 * a.K, (uint32_t)(min(kTileRows, a.M - m0) * row_bytes));
  const int sw0 = ((lane & 7) ^ (lane >> 4)) << 4;
  const int sw1 = ((lane & 7) ^ (4 | (lane >> 4))) << 4;
  const int dA = (8 * FW * wave + (lane >> 3)) * row_bytes;
  const int dB = (8 * FT * wave + (lane >> 3)) * row_bytes;
  // copy instruction i of step st: FW of weights, then FT of tokens
  auto copy = [&](int buf, int st, int i) {
    const bool valid = st < k1;
    const int sw = (i & 1) ? sw1 : sw0;   // FW and FT are even, so i's parity is the row block's
    if (i < FW)
      dma16(rsrc_sized(rw, valid), lds_addr(sA + buf * kStageA + (8 * FW * wave + 8 * i) * 128), dA + 8 * i * row_bytes + sw + st * 128,
            0);
    else
      dma16(rsrc_sized(rx, valid), lds_addr(sB + buf * kStageB + (8 * FT * wave + 8 * (i - FW)) * 128),
            dB + 8 * (i - FW) * row_bytes + sw + st * 128, 0);
  };

  v4f acc[FW][FT];
#pragma unroll
  for (int i = 0; i < FW; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  const int off0 = c * 128 + ((q ^ (c >> 1)) << 4);
  const int off1 = c * 128 + (((4 + q) ^ (c >> 1)) << 4);
  const uint8_t* pA = sA + wn * FW * 2048;
  const uint8_t* pB = sB + wm * FT * 2048;
  struct Ops {
    v4i w[FW][2];
    v4i x[FT][2];
  };
  auto load_x = [&](Ops& o, int buf, int j) {
    o.x[j][0] = *reinterpret_cast<const v4i*>(pB + buf * kStageB + j * 2048 + off0);
    o.x[j][1] = *reinterpret_cast<const v4i*>(pB + buf * kStageB + j * 2048 + off1);
  };
  auto load_w = [&](Ops& o, int buf, int i) {
    o.w[i][0] = *reinterpret_cast<const v4i*>(pA + buf * kStageA + i * 2048 + off0);
    o.w[i][1] = *reinterpret_cast<const v4i*>(pA + buf * kStageA + i * 2048 + off1);
  };

#pragma unroll
  for (int b = 0; b < kBufs; ++b)
#pragma unroll
    for (int i = 0; i < kCopies; ++i) copy(b, k0 + b, i);
  wait_vmcnt<2 * kCopies>();
  __syncthreads();
  Ops opsA, opsB;
#pragma unroll
  for (int j = 0; j < FT; ++j) load_x(opsA, 0, j);
#pragma unroll
  for (int i = 0; i < FW; ++i) load_w(opsA, 0, i);

  // Step k: this wave's copies of step k + 1 have landed (the newest kCopies are step
  // k + 2's), and after the barrier everybody's have, and step k's stage is free.
  // FW groups of 2 FT MFMAs, each with a part of step k + 1's fragment reads and of
  // step k + 3's copies.
  auto step = [&](Ops& cur, Ops& nxt, int k) {
    const int buf = (k - k0) % kBufs, nbuf = (k - k0 + 1) % kBufs;
    wait_vmcnt<kCopies>();
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int p = 0; p < FW; ++p) {
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        acc[p][j] = mfma_bf16(cur.w[p][0], cur.x[j][0], acc[p][j]);
        acc[p][j] = mfma_bf16(cur.w[p][1], cur.x[j][1], acc[p][j]);
      }
      if (p < FT) load_x(nxt, nbuf, p);
      load_w(nxt, nbuf, p);
#pragma unroll
      for (int i = p * kCopies / FW; i < (p + 1) * kCopies / FW; ++i) copy(buf, k + 3, i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  for (int k = k0; k < k1; k += 2) {
    step(opsA, opsB, k);
    step(opsB, opsA, k + 1);
  }
  wait_vmcnt<0>();   // no copy may land in the result tile
  __syncthreads();

  // The tile goes through LDS, so that a wave's epilogue walks whole rows: 64 lanes
  // hold 256 neighbouring columns' sums of one row, or 128 of two.
  float* const out = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int j = 0; j < FT; ++j)
#pragma unroll
    for (int i = 0; i < FW; ++i)
      *reinterpret_cast<v4f*>(out + (64 * wm + 16 * j + c) * kOutRow + 16 * FW * wn + 16 * i + 4 * q) = acc[i][j];
  __syncthreads();
  constexpr int kGroups = kCols / 4;
#pragma unroll 1
  for (int g = tid; g < kTileRows * kGroups; g += kTileThreads) {
    const int r = g / kGroups, n = n0 + 4 * (g % kGroups);
    const int64_t m = m0 + r;
    const v4f v = *reinterpret_cast<const v4f*>(out + r * kOutRow + 4 * (g % kGroups));
    if (a.splits == 1) {
      finish4(a, m, n, v);
    } else if (m < a.M && n < a.N) {
      float* dst = a.parts + ((int64_t)split * a.M + m) * a.N + n;
      if (a.N % 4 == 0) {
        *reinterpret_cast<v4f*>(dst) = v;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (n + k < a.N) dst[k] = v[k];
      }
    }
  }
}

// The parts of a split product, added in order, and the epilogue.
__global__ __launch_bounds__(256) void k_linear_join(LinearArgs a) {
  const int groups = (a.N + 3) / 4;
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (g >= (int64_t)a.M * groups) return;
  const int64_t m = g / groups;
  const int n = 4 * (int)(g - m * groups);
  v4f v{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.splits; ++s) {
    const float* src = a.parts + ((int64_t)s * a.M + m) * a.N + n;
    if (a.N % 4 == 0) {
      v += *reinterpret_cast<const v4f*>(src);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < a.N) v[r] += src[r];
    }
  }
  finish4(a, m, n, v);
}

template <int FW>
void run_tiles(const LinearArgs& a, hipStream_t s) {
  const int m_tiles = (int)ceil_div(a.M, kTileRows), n_tiles = (int)ceil_div(a.N, 32 * FW);
  const int64_t total = (int64_t)m_tiles * n_tiles * a.splits;
  hipLaunchKernelGGL(k_linear_tile<FW>, dim3((unsigned)(ceil_div(total, kXcds) * kXcds)), dim3(kTileThreads), 0, s, a,
                     m_tiles, n_tiles);
}

}  // namespace

LinearPlan linear_plan(int M, int N, int K) {
  if (M <= 64) return LinearPlan{true, 0, 1};
  // tile width: the fewest column tiles' worth of padded work, wide tiles first
  int fw = 8;
  int64_t best = -1;
  for (int f : {8, 6, 4}) {
    const int64_t cols = ceil_div(N, 32 * f) * (32 * f + 32);   // + 32: the token fragments' share
    if (best < 0 || cols < best) {
      best = cols;
      fw = f;
    }
  }
  const int64_t tiles = ceil_div(M, kTileRows) * ceil_div(N, 32 * fw);
  int splits = 1;
  if (tiles < 192) {   // fewer tiles than CUs: split K, at least 4 steps each
    splits = (int)(256 / tiles);
    const int most = K / 256;
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
  }
  return LinearPlan{false, fw, splits};
}

size_t linear_parts_bytes(int M, int N, int K) {
  const LinearPlan p = linear_plan(M, N, K);
  return p.splits > 1 ? sizeof(float) * (size_t)p.splits * M * N : 0;
}

hipError_t launch_linear_plan(const LinearArgs& in, const LinearPlan& p, hipStream_t s) {
  LinearArgs a = in;
  a.splits = p.splits;
  if (p.small) {
    const int steps = a.K / 64;
    const int waves = steps < kSmallWaves ? steps : kSmallWaves;
    const dim3 grid((unsigned)ceil_div(a.N, 16)), block(64 * waves);
    const int ft = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
    const size_t lds = (size_t)waves * ft * 1024;
    if (ft == 1) hipLaunchKernelGGL(k_linear_small<1>, grid, block, lds, s, a);
    else if (ft == 2) hipLaunchKernelGGL(k_linear_small<2>, grid, block, lds, s, a);
    else hipLaunchKernelGGL(k_linear_small<4>, grid, block, lds, s, a);
    return hipGetLastError();
  }
  if (p.fw == 8) run_tiles<8>(a, s);
  else if (p.fw == 6) run_tiles<6>(a, s);
  else run_tiles<4>(a, s);
  if (p.splits > 1) {
    const int64_t n = (int64_t)a.M * ceil_div(a.N, 4);
    hipLaunchKernelGGL(k_linear_join, dim3((unsigned)ceil_div(n, 256)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_linear(const moe_linear_dims& d, const uint16_t* x, const uint16_t* w, const float* bias,
                         const void* res, void* y, float* z, float* parts, hipStream_t s) {
  const LinearArgs a{x, w, bias, res, y, z, parts, d.M, d.N, d.K, d.act, 1, d.type == MOE_TYPE_F32};
  return launch_linear_plan(a, linear_plan(d.M, d.N, d.K), s);
}

}  // namespace moe

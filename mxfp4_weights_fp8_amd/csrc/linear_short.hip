// The dense product with a short contraction (at most 384: the gradient of a router's
// input, contracted over its experts): bound by writing the result, and with square
// tiles by the copies into LDS.
//
// A workgroup keeps 256 rows of x in registers (128 of an x in two parts), 64 (32) per wave
// and the whole contraction (at C = 384 192 registers, in the AGPR file as the MFMAs'
// second operand), and walks a run of 128-column tiles. Only w goes through LDS: a ring
// of kRing one-step stages (64 x 128) that runs on across the tiles, so that the next
// tile's columns arrive during the epilogue. Per 256 x 128 outputs 96 KB are copied,
// against 4 x 192 KB for the same outputs in 128 x 128 tiles.
//
// Step g (tile g / KS, step g % KS): the MFMAs of its first half and the reads of its
// second; wait for this wave's copies of step g + 1 and barrier, which frees g's stage;
// the MFMAs of the second half, the reads of step g + 1's first half, the copies of
// step g + kRing, and the stores of a share of the previous tile's results, which lie in
// LDS as bf16. Stored all at once after their tile, they came from every CU at the same
// time: 16384 x 7168 x 384 103 us, spread over the steps 92 us (without any stores 81).
// The wait counts what was issued after the copies of g + 1, stores among them; loads
// and stores leave the counter in the order of their issue. Nothing else is loaded (no
// bias, residual or activation): the wait for a load would be a wait for every copy.
#include "lane_reduce.h"
#include "linear.h"
#include "linear_stage.h"

namespace moe {
namespace {

constexpr int kShortThreads = 256;
constexpr int kShortCols = 128;
constexpr int short_rows(bool two) { return two ? 128 : 256; }
constexpr int kRing = 5;
constexpr int kXcds = 8;

// acc += W X: acc and w in VGPRs, x in AGPRs. The compiler does not know that the
// statement is an MFMA: s_nop provides the wait states after a VALU write.
__device__ __forceinline__ void mma_x_agpr(v4f& acc, const v4i& w, const v4i& x) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(acc) : "v"(w), "a"(x));
#endif
}

// TWO: x in two parts; a fragment of w meets the high and the low part of half the rows.
template <int KS, bool WT, bool TWO>
__global__ __launch_bounds__(kShortThreads, 1) void k_linear_short(LinearArgs a, int m_tiles, int n_tiles, int per_cta,
                                                                    int total) {
  constexpr int P = TWO ? 2 : 1, FT = 4 / P, FW = 8;
  constexpr int kShortRows = short_rows(TWO), kWaveRows = 16 * FT;
  typedef Operand<kShortCols, WT> W;
  constexpr int kCopies = W::kCopies;
  constexpr int kOutRow = 2 * kShortCols + 16;   // bytes per staged row: 16 rows in distinct banks
  constexpr int kStores = kWaveRows / 4;         // of a wave per tile, 4 rows each
  constexpr int kLeastStores = kStores / KS;     // and step
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kRing * W::kBytes + 4 * kWaveRows * kOutRow];

  // (column run, row tile), each XCD a contiguous share: its L2 holds few column runs
  const int run = (total + kXcds - 1) / kXcds;
  const int id = (blockIdx.x % kXcds) * run + blockIdx.x / kXcds;
  if ((int)(blockIdx.x / kXcds) >= run || id >= total) return;
  const int m0 = id % m_tiles * kShortRows, t0 = id / m_tiles * per_cta, t1 = min(t0 + per_cta, n_tiles);

  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  W ow;
  ow.init(a.ws, wave, lane);
  FragReader<kShortCols, WT> rw;
  rw.init(lane);

  const int steps = (t1 - t0) * KS;
  int ct = t0, cs = 0, cbuf = 0, issued = 0;   // the copies' tile, step and stage
  ow.place(a.w, a.ws, ct * kShortCols, a.N, a.w_rows);
  auto next_rsrc = [&]() { return ow.rsrc(cs, issued < steps); };
  auto advance = [&]() {
    ++issued;
    cbuf = cbuf + 1 == kRing ? 0 : cbuf + 1;
    if (++cs == KS) {
      cs = 0;
      ++ct;
      ow.place(a.w, a.ws, min(ct, n_tiles - 1) * kShortCols, a.N, a.w_rows);
    }
  };
#pragma unroll 1
  for (int s = 0; s < kRing; ++s) {
    const v4i_s r = next_rsrc();
#pragma unroll
    for (int i = 0; i < kCopies; ++i) ow.copy(r, smem + cbuf * W::kBytes, wave, i);
    advance();
  }
  // x: lane (c, q) holds contraction 64 s + 32 h + 8q .. + 7 of rows 16 j + c; rows past
  // the end repeat the last one and are not stored
  v4i x[FT][P][KS][2];
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    const uint16_t* row = a.x + (int64_t)min(m0 + kWaveRows * wave + 16 * j + c, a.M - 1) * a.xs + 8 * q;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) x[j][p][s][h] = load16(row + p * a.x_low + 64 * s + 32 * h);
  }
#pragma unroll
  for (int j = 0; j < FT; ++j)
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) asm volatile("; in an AGPR from here" : "+a"(x[j][p][s][h]));
  wait_vmcnt<0>();
  __syncthreads();

  v4f acc[FW][FT];
#pragma unroll
  for (int i = 0; i < FW; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  v4i w0[FW], w1[FW];
#pragma unroll
  for (int i = 0; i < FW; ++i) w0[i] = rw.template read<0>(smem, i);

  // A tile's results wait in the wave's part of LDS as bf16 and are stored during the
  // next tile's steps. Every wave issues every store, those of rows or columns past the
  // end (and all of the first tile's) with an offset past the resource's size.
  uint8_t* const out = smem + kRing * W::kBytes + wave * kWaveRows * kOutRow;
  const uint8_t* const out_read = out + q * kOutRow + 16 * c;
  const int row_bytes = 2 * a.N;
  const rsrc_t ry = make_rsrc(static_cast<const char*>(a.y) + (int64_t)m0 * row_bytes,
                              (uint32_t)(min(kShortRows, a.M - m0) * row_bytes));   // at most 32 MB
  constexpr int kOutside = 1 << 30;
  int at = kOutside;   // this lane's offset in ry of the first store
  auto store = [&](int u, const v4i v) { buf_store16(ry, v, at + 4 * u * row_bytes); };
  int buf = 0;   // stage of step g
  for (int t = t0; t < t1; ++t) {
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      constexpr int kMost = (kStores + KS - 1) / KS;
      const int u0 = kStores * s / KS, u1 = kStores * (s + 1) / KS;
      const uint8_t* stage = smem + buf * W::kBytes;
      const int nbuf = buf + 1 == kRing ? 0 : buf + 1;
      const uint8_t* next = smem + nbuf * W::kBytes;
      v4i done[kMost];
#pragma unroll
      for (int i = 0; i < FW; ++i) {
        w1[i] = rw.template read<1>(stage, i);
        if (i < u1 - u0) done[i] = *reinterpret_cast<const v4i*>(out_read + 4 * (u0 + i) * kOutRow);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int j = 0; j < FT; ++j) mma_x_agpr(acc[i][j], w0[i], x[j][p][s][0]);
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_vmcnt<(kRing - 2) * (kCopies + kLeastStores)>();
      __syncthreads();
      __builtin_amdgcn_sched_barrier(0);
      const v4i_s r = next_rsrc();
#pragma unroll
      for (int i = 0; i < FW; ++i) {
        w0[i] = rw.template read<0>(next, i);
        if (i % 2 == 0 && i / 2 < kCopies) ow.copy(r, smem + cbuf * W::kBytes, wave, i / 2);
        if (i < u1 - u0) store(u0 + i, done[i]);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int j = 0; j < FT; ++j) mma_x_agpr(acc[i][j], w1[i], x[j][p][s][1]);
        __builtin_amdgcn_sched_barrier(0);
      }
      advance();
      buf = nbuf;
    }
    // The compiler does not see the MFMAs, so it inserts no wait states before the
    // accumulators are read: 64 of them here.
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#endif
    __builtin_amdgcn_sched_barrier(0);
    wave_sync();   // the tile before has been read
#pragma unroll
    for (int j = 0; j < FT; ++j)
#pragma unroll
      for (int i = 0; i < FW; ++i) {
        const v4f v = acc[i][j];
        *reinterpret_cast<uint2*>(out + (16 * j + c) * kOutRow + 2 * (16 * i + 4 * q)) =
            make_uint2(bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]));
        acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
      }
    wave_sync();
    const int n = t * kShortCols + 8 * c;
    at = n < a.N ? (kWaveRows * wave + q) * row_bytes + 2 * n : kOutside;
  }
#pragma unroll
  for (int u = 0; u < kStores; ++u) store(u, *reinterpret_cast<const v4i*>(out_read + 4 * u * kOutRow));
  wait_vmcnt<0>();   // no copy may be in flight when the workgroup's LDS is given away
}

template <int KS>
void run(const LinearArgs& a, bool w_trans, hipStream_t s) {
  const bool two = a.x_low != 0;   // only with w transposed
  const int m_tiles = (int)ceil_div(a.M, short_rows(two)), n_tiles = (int)ceil_div(a.N, kShortCols);
  const int per = short_tiles_per_cta(a.M, a.N, two);
  const int total = m_tiles * (int)ceil_div(n_tiles, per);
  const dim3 grid((unsigned)(ceil_div(total, kXcds) * kXcds)), block(kShortThreads);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, s, a, m_tiles, n_tiles, per, total); };
  if (two) go(k_linear_short<KS, true, true>);
  else if (w_trans) go(k_linear_short<KS, true, false>);
  else go(k_linear_short<KS, false, false>);
}

}  // namespace

// Column tiles per workgroup: as many as leave one workgroup per CU.
int short_tiles_per_cta(int M, int N, bool two) {
  const int64_t m_tiles = ceil_div(M, short_rows(two)), n_tiles = ceil_div(N, kShortCols);
  int64_t runs = 256 / m_tiles;
  runs = runs < 1 ? 1 : runs > n_tiles ? n_tiles : runs;
  return (int)ceil_div(n_tiles, runs);
}

void launch_short(const LinearArgs& a, Layout l, hipStream_t s) {
  const bool wt = l == Layout::kWTrans;
  if (a.C == 128) run<2>(a, wt, s);
  else if (a.C == 256) run<4>(a, wt, s);
  else run<6>(a, wt, s);
}

}  // namespace moe

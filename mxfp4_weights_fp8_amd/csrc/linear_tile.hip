// The tiled dense product on v_mfma_f32_16x16x32_bf16: tiles of 32 FT rows x 32 FW
// columns, four waves in a 2 x 2 grid of FT x FW fragments of 16 x 16 each, one wave
// per SIMD. The weights are the MFMA's first operand, so lane (c, q) = (l % 16, l / 16)
// of a result fragment holds columns 4q .. 4q+3 of row c.
//
// The accumulators (256 registers at 8 x 8) live in the AGPR file through inline-asm
// MFMAs with "+a" operands; the compiler's own choice copies them between the register
// files inside the loop.
//
// LDS: stages of 64 of the contraction index (one step), three for x and two for w,
// filled by direct-to-LDS copies. A step has two halves of 32:
//   half A: the MFMAs of the first half, the fragment reads of the second half into
//           the other register set, the copies of x of step s + 2;
//   wait for this wave's copies of step s + 1 (all but those of x of step s + 2) and
//   barrier: they have landed, and everybody has read step s to its end;
//   half B: the MFMAs of the second half, the fragment reads of the next step's first
//           half, the copies of w of step s + 2 into the stage of step s.
// One barrier per 2 FT FW MFMAs; x, which more often comes from HBM, is copied a step
// and a half ahead, w one step. Both operands' copies read at least 128 neighbouring
// bytes of a row: with stages of 32 (64-byte pieces) the copies' issue took most of the
// loop (32768 x 384 x 7168: 208 us).
//
// 32768 x 384 x 7168 to fp32 in 256 x 192 tiles 160 us, 1.13 PFLOP/s (one round of 256
// workgroups); 8191 x 7168 x 2048 with residual in 128 x 128 tiles 265 us, 0.91 PFLOP/s;
// 8192^3 851 us, 1.29 PFLOP/s. The library's product takes 187, 209 and 785 us. Without
// its copies 8192^3 takes 720 us, its MFMAs alone 652 us: bound by the issue of the copies
// and, where the contraction is short, by epilogues that all CUs reach together.
#include "linear.h"
#include "linear_stage.h"

namespace moe {
namespace {

constexpr int kTileThreads = 256;
constexpr int kXcds = 8;
constexpr int kGroup = 8;   // row tiles that share a pass over the column tiles

// acc += A B, acc in AGPRs. The compiler does not know that the statement is an MFMA
// and inserts no wait states after a VALU write of an operand: s_nop provides them.
__device__ __forceinline__ void mma_agpr(v4f& acc, const v4i& a, const v4i& b) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
#endif
}

// TWO: x in two parts. The steps of the contraction run twice, over x's high parts and
// then over its low ones, with the same w.
template <int FT, int FW, bool XT, bool WT, bool TWO>
__global__ __launch_bounds__(kTileThreads, 1) void k_linear_tile(LinearArgs a, int m_tiles, int n_tiles) {
  constexpr int kRows = 32 * FT, kCols = 32 * FW;
  constexpr int kXStages = 3, kWStages = 2;
  typedef Operand<kRows, XT> X;
  typedef Operand<kCols, WT> W;
  constexpr int kRing = kXStages * X::kBytes + kWStages * W::kBytes;
  constexpr int kOutRow = 16 * FW + 4;   // floats per row of a wave's staged result: 16 rows in distinct banks
  constexpr int kOut = 64 * kOutRow * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kRing > 4 * kOut ? kRing : 4 * kOut];
  uint8_t* const smem_w = smem + kXStages * X::kBytes;

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
  const int m0 = mt * kRows, n0 = nt * kCols;

  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  // this split's steps, dealt as evenly as they go
  const int part_steps = (a.C + 63) / 64, steps = TWO ? 2 * part_steps : part_steps;
  const int s0 = (int)((int64_t)steps * split / a.splits), s1 = (int)((int64_t)steps * (split + 1) / a.splits);

  X ox;
  W ow;
  ox.init(a.xs, wave, lane);
  ox.place(a.x, a.xs, m0, a.M, a.C);
  ow.init(a.ws, wave, lane);
  ow.place(a.w, a.ws, n0, a.N, a.w_rows);
  FragReader<kRows, XT> rx;
  FragReader<kCols, WT> rw;
  rx.init(lane);
  rw.init(lane);

  v4f acc[FW][FT];
#pragma unroll
  for (int i = 0; i < FW; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  struct Ops {
    v4i w[FW];
    v4i x[FT];
  };
  Ops ops[2];
  auto low = [&](int s) { return TWO && s >= part_steps; };
  auto rsrc_x = [&](int s) {
    return ox.rsrc(low(s) ? s - part_steps : s, s < s1, low(s) ? 2 * a.x_low : 0);
  };
  auto rsrc_w = [&](int s) { return ow.rsrc(low(s) ? s - part_steps : s, s < s1); };
  auto copy_x = [&](v4i_s r, int buf, int i) { ox.copy(r, smem + buf * X::kBytes, wave, i); };
  auto copy_w = [&](v4i_s r, int buf, int i) { ow.copy(r, smem_w + buf * W::kBytes, wave, i); };
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const v4i_s rw0 = rsrc_w(s0 + b), rx0 = rsrc_x(s0 + b);
#pragma unroll
    for (int i = 0; i < W::kCopies; ++i) copy_w(rw0, b, i);
#pragma unroll
    for (int i = 0; i < X::kCopies; ++i) copy_x(rx0, b, i);
  }
  wait_vmcnt<X::kCopies + W::kCopies>();
  __syncthreads();
#pragma unroll
  for (int j = 0; j < FT; ++j) ops[0].x[j] = rx.template read<0>(smem, FT * wm + j);
#pragma unroll
  for (int i = 0; i < FW; ++i) ops[0].w[i] = rw.template read<0>(smem_w, FW * wn + i);

  int xb = 0, wb = 0;   // stages of step s
  for (int s = s0; s < s1; ++s) {
    const int xb1 = xb + 1 == kXStages ? 0 : xb + 1, xb2 = xb1 + 1 == kXStages ? 0 : xb1 + 1;
    const v4i_s rx2 = rsrc_x(s + 2), rw2 = rsrc_w(s + 2);
    const uint8_t *px = smem + xb * X::kBytes, *pw = smem_w + wb * W::kBytes;
#pragma unroll
    for (int p = 0; p < FW; ++p) {   // half A
#pragma unroll
      for (int j = p * FT / FW; j < (p + 1) * FT / FW; ++j) ops[1].x[j] = rx.template read<1>(px, FT * wm + j);
      ops[1].w[p] = rw.template read<1>(pw, FW * wn + p);
#pragma unroll
      for (int i = p * X::kCopies / FW; i < (p + 1) * X::kCopies / FW; ++i) copy_x(rx2, xb2, i);
#pragma unroll
      for (int j = 0; j < FT; ++j) mma_agpr(acc[p][j], ops[0].w[p], ops[0].x[j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_vmcnt<X::kCopies>();
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    px = smem + xb1 * X::kBytes;
    pw = smem_w + (wb ^ 1) * W::kBytes;
#pragma unroll
    for (int p = 0; p < FW; ++p) {   // half B
#pragma unroll
      for (int j = p * FT / FW; j < (p + 1) * FT / FW; ++j) ops[0].x[j] = rx.template read<0>(px, FT * wm + j);
      ops[0].w[p] = rw.template read<0>(pw, FW * wn + p);
#pragma unroll
      for (int i = p * W::kCopies / FW; i < (p + 1) * W::kCopies / FW; ++i) copy_w(rw2, wb, i);
#pragma unroll
      for (int j = 0; j < FT; ++j) mma_agpr(acc[p][j], ops[1].w[p], ops[1].x[j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    xb = xb1;
    wb ^= 1;
  }
  wait_vmcnt<0>();   // no copy may land in the staged result
  // The compiler does not see the MFMAs, so it inserts no wait states before the
  // accumulators are read: 64 of them here.
  __builtin_amdgcn_sched_barrier(0);
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#endif
  __builtin_amdgcn_sched_barrier(0);
  __syncthreads();

  // Results, 64 rows of the wave at a time, through the wave's own part of LDS, so that
  // stores walk whole rows: 2 FW lanes hold 8 columns each of a row. Without activation
  // kAtOnce groups at a time, their residuals loaded ahead (four at a time left the
  // residuals' latency in the open: 8191 x 7168 x 2048 in 256 x 256 tiles 302 us).
  constexpr int kGroups = 2 * FW, kAtOnce = FW == 6 ? 6 : 8;
  float* const out = reinterpret_cast<float*>(smem + wave * kOut);
  const bool affine = a.splits == 1 && is_affine(a);
#pragma unroll
  for (int j0 = 0; j0 < FT; j0 += 4) {
    const int groups = 16 * (FT - j0 < 4 ? FT - j0 : 4) * kGroups;   // a multiple of 64 * kAtOnce
#pragma unroll
    for (int j = j0; j < j0 + 4 && j < FT; ++j)
#pragma unroll
      for (int i = 0; i < FW; ++i)
        *reinterpret_cast<v4f*>(out + (16 * (j - j0) + c) * kOutRow + 16 * i + 4 * q) = acc[i][j];
    __syncthreads();
    const int64_t mw = m0 + 16 * FT * wm + 16 * j0;
    const int nw = n0 + 16 * FW * wn;
    if (affine) {
      by_affine(a, [&](auto residual) {
        typedef decltype(residual) Res;
#pragma unroll 1
        for (int g0 = lane; g0 < groups; g0 += 64 * kAtOnce) {
          Res res[kAtOnce];
#pragma unroll
          for (int u = 0; u < kAtOnce; ++u)
            res[u].load(a, mw + (g0 + 64 * u) / kGroups, nw + 8 * ((g0 + 64 * u) % kGroups));
#pragma unroll
          for (int u = 0; u < kAtOnce; ++u) {
            const int r = (g0 + 64 * u) / kGroups, col = 8 * ((g0 + 64 * u) % kGroups);
            const float* src = out + r * kOutRow + col;
            finish_affine(a, mw + r, nw + col, *reinterpret_cast<const v4f*>(src),
                          *reinterpret_cast<const v4f*>(src + 4), res[u]);
          }
        }
      });
    } else {
#pragma unroll 1
      for (int g = lane; g < groups; g += 64) {
        const int r = g / kGroups, col = 8 * (g % kGroups);
        const v4f lo = *reinterpret_cast<const v4f*>(out + r * kOutRow + col);
        const v4f hi = *reinterpret_cast<const v4f*>(out + r * kOutRow + col + 4);
        float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        if (a.splits > 1) store_part<8>(a, split, mw + r, nw + col, v);
        else finish<8>(a, mw + r, nw + col, v, load_residual<8>(a, mw + r, nw + col));
      }
    }
    __syncthreads();
  }
}

template <int FT, int FW, bool XT, bool WT, bool TWO>
void run(const LinearArgs& a, hipStream_t s) {
  const int m_tiles = (int)ceil_div(a.M, 32 * FT), n_tiles = (int)ceil_div(a.N, 32 * FW);
  const int64_t total = (int64_t)m_tiles * n_tiles * a.splits;
  hipLaunchKernelGGL((k_linear_tile<FT, FW, XT, WT, TWO>), dim3((unsigned)(ceil_div(total, kXcds) * kXcds)),
                     dim3(kTileThreads), 0, s, a, m_tiles, n_tiles);
}

template <bool XT, bool WT, bool TWO>
void by_tile(const LinearArgs& a, const LinearPlan& p, hipStream_t s) {
  if (p.ft == 8 && p.fw == 8) run<8, 8, XT, WT, TWO>(a, s);
  else if (p.ft == 8) run<8, 6, XT, WT, TWO>(a, s);
  else if (p.ft == 6) run<6, 8, XT, WT, TWO>(a, s);
  else run<4, 4, XT, WT, TWO>(a, s);
}
template <bool XT>   // a gradient's layout: w transposed, x in one or two parts
void by_parts(const LinearArgs& a, const LinearPlan& p, hipStream_t s) {
  if (a.x_low) by_tile<XT, true, true>(a, p, s);
  else by_tile<XT, true, false>(a, p, s);
}

}  // namespace

void launch_tiles(const LinearArgs& a, const LinearPlan& p, Layout l, hipStream_t s) {
  if (l == Layout::kRows) by_tile<false, false, false>(a, p, s);
  else if (l == Layout::kWTrans) by_parts<false>(a, p, s);
  else by_parts<true>(a, p, s);
}

}  // namespace moe

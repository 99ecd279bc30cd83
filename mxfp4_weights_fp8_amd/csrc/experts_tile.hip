// The experts' products in tiles of 256 rows x 32 FW columns (an expert's last tile has
// fewer rows), and the weights' gradient in tiles of 32 FT x 32 FW, on
// v_mfma_f32_16x16x32_bf16: four waves in a 2 x 2 grid, one per SIMD, the accumulators in
// the AGPR file.
//
// One workgroup per CU walks its tiles as one run of steps of 64 of the contraction: the
// ring of LDS stages (two of the rows' operand A, three of the columns' B, filled by
// direct-to-LDS copies) goes on across the tiles, so that a tile's first steps arrive
// while the tile before is multiplied and stored. Contractions here are short: 6 to 12
// steps where an expert's inner size is contracted, 3 where its rows are.
//
// Step s, in two halves of 32:
//   half A: the first half's MFMAs, the second half's fragment reads, the copies of B of
//           step s + 2;
//   wait for this wave's copies of step s + 1, and barrier: they have landed, and
//           everybody has read step s to its end;
//   half B: the second half's MFMAs, the next step's first fragments, the copies of A of
//           step s + 2 into the stage of step s.
// B, an expert's weights, is copied half a step further ahead than A: it comes from HBM,
// for a few row tiles (384 experts of 50 rows, 768 x 7168: 798 us, 834 the other way
// round).
// Results go from the registers to memory (store_tile). The stores are in flight during the
// next tile's first step: its wait counts past them.
//
// One expert of 8192 rows, 8192 x 8192: 770 us, 1.43 PFLOP/s (the library's product 790-812).
// 262144 rows of 384 experts, 768 x 7168, of which 214784 fill tiles of 256: 2.68-2.76 ms;
// the full tiles alone 1.92 ms at 1.23 PFLOP/s, the others 0.98 ms at 5.1 TB/s of weights,
// and the two hardly overlap: a CU holds two steps in LDS, too few to hide a loaded HBM.
// MFMAs are busy 63 % of the time at the 1.75 GHz that the power leaves. dx of 64238 rows 1.08
// ms (4.8 TB/s), dw 1.31 ms: bound by reading (writing) 4.2 GB of weights; three steps
// of the contraction per tile of dw, then 128 KB of stores that the copies queue behind.
#include "experts.h"
#include "linear_stage.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kXcds = 8;
constexpr int kCus = 256;
constexpr int kGroup = 4;   // row tiles that share a pass over the column tiles
constexpr int kAStages = 2, kBStages = 3;

// acc += A B, or acc = A B (FIRST, which saves writing zeros: 5 % of a tile of three
// steps), acc in AGPRs. The compiler does not know that the statement is an MFMA and
// inserts no wait states after a VALU write of an operand: s_nop provides them.
template <bool FIRST>
__device__ __forceinline__ void mma_agpr(v4f& acc, const v4i& a, const v4i& b) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (FIRST) asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, 0" : "=a"(acc) : "v"(a), "v"(b));
  else asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
#endif
}
// ... nor before the accumulators are read: 64 of them.
__device__ __forceinline__ void mma_done() {
  __builtin_amdgcn_sched_barrier(0);
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#endif
  __builtin_amdgcn_sched_barrier(0);
}

// A scalar load: the pointer's values do not change during the launch.
typedef const __attribute__((address_space(4))) int32_t* const_ints;
__device__ __forceinline__ const_ints as_const(const void* p) { return (const_ints)(uintptr_t)p; }

// The quotient of two wave-uniform values, in a scalar register (the division itself is done
// by the vector unit).
__device__ __forceinline__ int uniform_div(int a, int b) { return __builtin_amdgcn_readfirstlane(a / b); }

// Where a wave stores its part of a tile: `base` the tile's first row, `rows` of them.
struct OutTile {
  rsrc_t r;
  int row_bytes, cols_left;   // columns from the tile's first one to the end
  template <bool F32>
  __device__ __forceinline__ void place(void* y, int64_t row0, int rows, int n0, int O) {
    constexpr int kSize = F32 ? 4 : 2;
    row_bytes = O * kSize;
    cols_left = O - n0;
    r = make_rsrc(static_cast<char*>(y) + row0 * row_bytes + n0 * kSize, (uint32_t)(rows * row_bytes - n0 * kSize));
  }
  __device__ __forceinline__ void put(const v4i v, int voff) const {
    typedef unsigned int v4u __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v), r, voff, 0, 2);   // nontemporal
  }
};
constexpr int kOutside = 1 << 30;   // past any tile: 256 rows of 64 K columns at most

// The accumulators acc[i][j], columns 16 i + 4q .. + 3 of row 16 j + c of the wave's part,
// which starts at row `m0` and column `n0` of the tile. A piece is the 16 bytes that a
// lane stores; four lanes (q) have 64 neighbouring bytes of a row. Lanes of neighbouring
// rows trade pieces that are 64 bytes apart, so that a store writes 128-byte lines whole:
// the gradient of 384 experts' 768 x 7168 weights from 64 rows each, nearly all stores,
// took 1125 us in half lines, 956 in whole ones, and 907 with these nontemporal. (Small
// results that the next kernel reads at once lose nothing by it: 8192 x 768 and its
// gated activation 40.1 us, 41.7 without; 65536 x 768 141 and 139.)
// Always FT FW stores (half of them in bf16); rows and columns past the end are dropped by
// the resource's bounds check.
template <int FT, int FW, int FTM, bool F32>
__device__ __forceinline__ void store_tile(const OutTile& o, v4f (&acc)[FW][FTM], int m0, int n0, int lane) {
  constexpr int kCols = F32 ? 4 : 8, kSize = F32 ? 4 : 2;   // of a piece
  constexpr int kFrags = F32 ? 1 : 2;                       // that a piece comes from
  const int c = lane & 15, q = lane >> 4;
  const bool odd = c & 1;
  int at = (m0 + c) * o.row_bytes + (n0 + kCols * q) * kSize, step = 16 * o.row_bytes;
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(at), "+s"(step));   // else every store's offset is kept in a register from tile to tile
#endif
  const int left = o.cols_left - n0 - kCols * q;
  // the piece of the fragments from i on
  auto piece = [&](int i, int j) {
    if constexpr (F32) {
      return __builtin_bit_cast(v4i, acc[i][j]);
    } else {
      v4f t0 = acc[i][j], t1 = acc[i + 1][j];
#if defined(__HIP_DEVICE_COMPILE__)
      asm volatile("" : "+v"(t0), "+v"(t1));   // here and not all at once, which takes registers that are not there
#endif
      v4i r;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // lane groups q of (f0, f1): (0 1 2 3, 0 1 2 3) -> (f0: 0 1, f1: 0 1; f0: 2 3, f1: 2 3)
        // -> (f0: 0 2, f1: 0 2; f0: 1 3, f1: 1 3): group q holds columns 8q .. 8q + 7 of 32
        const auto half = __builtin_amdgcn_permlane32_swap(bf16_pack2(t0[2 * h], t0[2 * h + 1]),
                                                           bf16_pack2(t1[2 * h], t1[2 * h + 1]), false, false);
        const auto quarter = __builtin_amdgcn_permlane16_swap(half[0], half[1], false, false);
        r[h] = (int)quarter[0];
        r[2 + h] = (int)quarter[1];
      }
      return r;
    }
  };
#pragma unroll
  for (int j = 0; j < FT; ++j) {
#pragma unroll
    for (int i = 0; i < FW; i += 2 * kFrags) {
      const v4i a = piece(i, j);
      const int col = 16 * i;
      if (i + kFrags < FW) {
        // rows c and c + 1 of an even lane and its neighbour: the even one stores the first
        // 64 bytes of both, the odd one the second
        const v4i b = piece(i + kFrags, j);
        v4i first, second;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int give = odd ? a[h] : b[h], got = __builtin_amdgcn_update_dpp(give, give, 0xB1, 0xF, 0xF, true);
          first[h] = odd ? got : a[h];
          second[h] = odd ? b[h] : got;
        }
        const int mine = at + kSize * col + (odd ? 64 - o.row_bytes : 0);   // of the even row
        const bool in = col + (odd ? 16 * kFrags : 0) < left;
        o.put(first, in ? mine : kOutside);
        o.put(second, in ? mine + o.row_bytes : kOutside);
      } else {
        o.put(a, col < left ? at + kSize * col : kOutside);
      }
    }
    at += step;
    __builtin_amdgcn_sched_barrier(0);   // a row's accumulators at a time in the other register file
  }
}

// A workgroup's view of the ring: FTM x FW fragments per wave at most, A the MFMA's second
// operand (rows of the result), B its first (columns).
template <int FTM, int FW, bool AT, bool BT, bool F32>
struct Stream {
  typedef Operand<32 * FTM, AT> A;
  typedef Operand<32 * FW, BT> B;
  static constexpr int kSmem = kAStages * A::kBytes + kBStages * B::kBytes;

  uint8_t* smem;
  int wave, lane, wm, wn;
  A oa;   // the tile that is copied
  B ob;
  FragReader<32 * FTM, AT> ra;
  FragReader<32 * FW, BT> rb;
  v4f acc[FW][FTM];
  v4i b[2][FW], a[2][FTM];
  int ab = 0, bb = 0;     // stages of the step that is multiplied
  int stores = 0;         // of the tile before: 1 if FTM's number of them, 0 if fewer or none

  __device__ __forceinline__ void init(uint8_t* lds, int64_t a_stride, int64_t b_stride) {
    smem = lds;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave & 1;
    wn = wave >> 1;
    oa.init(a_stride, wave, lane);
    ob.init(b_stride, wave, lane);
    ra.init(lane);
    rb.init(lane);
  }
  __device__ __forceinline__ uint8_t* stage_a(int i) const { return smem + i * A::kBytes; }
  __device__ __forceinline__ uint8_t* stage_b(int i) const { return smem + kAStages * A::kBytes + i * B::kBytes; }

  // Steps 0 and 1 on their way, step 0 landed. next(ra, rb): the resources of the next step.
  template <typename Next>
  __device__ __forceinline__ void start(Next next) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      v4i_s sa, sb;
      next(sa, sb);
#pragma unroll
      for (int i = 0; i < B::kCopies; ++i) ob.copy(sb, stage_b(k), wave, i);
#pragma unroll
      for (int i = 0; i < A::kCopies; ++i) oa.copy(sa, stage_a(k), wave, i);
    }
    wait_vmcnt<A::kCopies + B::kCopies>();
    __syncthreads();
  }

  // Step of a tile with FT row fragments per wave, its first half's fragments read.
  template <int FT, bool FIRST, typename Next>
  __device__ __forceinline__ void step(Next next) {
    const int bb1 = bb + 1 == kBStages ? 0 : bb + 1, bb2 = bb1 + 1 == kBStages ? 0 : bb1 + 1;
    v4i_s sa, sb;
    next(sa, sb);
    const uint8_t *pa = stage_a(ab), *pb = stage_b(bb);
#pragma unroll
    for (int p = 0; p < FW; ++p) {   // half A
#pragma unroll
      for (int j = p * FT / FW; j < (p + 1) * FT / FW; ++j) a[1][j] = ra.template read<1>(pa, FT * wm + j);
      b[1][p] = rb.template read<1>(pb, FW * wn + p);
#pragma unroll
      for (int i = p * B::kCopies / FW; i < (p + 1) * B::kCopies / FW; ++i) ob.copy(sb, stage_b(bb2), wave, i);
#pragma unroll
      for (int j = 0; j < FT; ++j) mma_agpr<FIRST>(acc[p][j], b[0][p], a[0][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // behind the copies that are waited for: this half's, and in a tile's first step the
    // stores of the tile before
    constexpr int kStores = F32 ? FTM * FW : FTM * FW / 2;
    constexpr int kPast = B::kCopies + kStores < 63 ? B::kCopies + kStores : 63;
    if (FIRST && stores) wait_vmcnt<kPast>();
    else wait_vmcnt<B::kCopies>();
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    pa = stage_a(ab ^ 1);
    pb = stage_b(bb1);
#pragma unroll
    for (int p = 0; p < FW; ++p) {   // half B
#pragma unroll
      for (int j = p * FT / FW; j < (p + 1) * FT / FW; ++j) a[0][j] = ra.template read<0>(pa, FT * wm + j);
      b[0][p] = rb.template read<0>(pb, FW * wn + p);
#pragma unroll
      for (int i = p * A::kCopies / FW; i < (p + 1) * A::kCopies / FW; ++i) oa.copy(sa, stage_a(ab), wave, i);
#pragma unroll
      for (int j = 0; j < FT; ++j) mma_agpr<false>(acc[p][j], b[1][p], a[1][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    ab ^= 1;
    bb = bb1;
    pin<FT>();
  }
  // The accumulators in AGPRs here: else the compiler copies them all to the other register
  // file, which spills, where the loop over the steps begins and ends.
  template <int FT>
  __device__ __forceinline__ void pin() {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int i = 0; i < FW; ++i)
#pragma unroll
      for (int j = 0; j < FT; ++j) asm volatile("; in an AGPR" : "+a"(acc[i][j]));
#endif
  }

  // One tile of `steps` (at least one) steps.
  template <int FT, typename Next>
  __device__ __forceinline__ void tile(int steps, Next next) {
#pragma unroll
    for (int j = 0; j < FT; ++j) a[0][j] = ra.template read<0>(stage_a(ab), FT * wm + j);
#pragma unroll
    for (int i = 0; i < FW; ++i) b[0][i] = rb.template read<0>(stage_b(bb), FW * wn + i);
    step<FT, true>(next);
    for (int s = 1; s < steps; ++s) step<FT, false>(next);
    mma_done();
    pin<FT>();
    stores = FT == FTM;
  }
  template <int FT>
  __device__ __forceinline__ void store(const OutTile& o) {
    store_tile<FT, FW, FTM, F32>(o, acc, 16 * FT * wm, 16 * FW * wn, lane);
  }
};

// Tiles in the order (group of kGroup row tiles, column tile, row tile), dealt to the XCDs
// in runs of as many as each has workgroups, so that the tiles that share operand rows
// and run at the same time share an L2, and so that every XCD has its share of the tall
// tiles, which come first, and of the short ones.
template <int FW, bool WT, bool F32>
__global__ __launch_bounds__(kThreads, 1) void k_expert_tile(ExpertArgs a) {
  typedef Stream<8, FW, false, WT, F32> S;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kSmem];
  const const_ints list = as_const(a.list);
  const int row_tiles = list[0], n_tiles = (a.O + 32 * FW - 1) / (32 * FW), steps = a.D / 64;
  const int tiles = row_tiles * n_tiles, end = tiles * a.splits, stride = gridDim.x;
  const int begin = blockIdx.x % kXcds * (stride / kXcds) + blockIdx.x / kXcds;
  if (begin >= end) return;

  struct Tile {
    int expert, row0, rows, n0, split, s0, s1;
  };
  auto tile_of = [&](int id) {
    const int split = uniform_div(id, tiles), in_split = id - split * tiles;
    const int group = uniform_div(in_split, kGroup * n_tiles), in = in_split - group * kGroup * n_tiles;
    const int in_group = min(kGroup, row_tiles - group * kGroup);
    const int nt = uniform_div(in, in_group), mt = group * kGroup + in - nt * in_group;
    return Tile{list[4 * mt + 4], list[4 * mt + 5], list[4 * mt + 6], nt * 32 * FW, split,
                uniform_div(steps * split, a.splits), uniform_div(steps * (split + 1), a.splits)};
  };

  S st;
  st.init(smem, a.D, a.ws);
  int at = begin, step = 0, stop = 0;   // what is copied next, up to which step
  auto place = [&]() {
    const Tile t = tile_of(min(at, end - 1));
    step = t.s0;
    stop = t.s1;
    st.oa.place(a.x, a.D, t.row0, t.row0 + t.rows, a.D);
    st.ob.place(a.w + t.expert * a.w_expert, a.ws, t.n0, a.O, a.D);
  };
  place();
  auto next = [&](v4i_s& sa, v4i_s& sb) {
    sa = st.oa.rsrc(step, at < end);
    sb = st.ob.rsrc(step, at < end);
    if (++step == stop) {
      at += stride;
      place();
    }
  };
  st.start(next);
  for (int id = begin; id < end; id += stride) {
    const Tile t = tile_of(id);
    OutTile o;
    o.place<F32>(static_cast<char*>(a.y) + (int64_t)t.split * a.P * a.O * 4, t.row0, t.rows, t.n0, a.O);   // split 0 in bf16
    auto go = [&](auto ft) {
      constexpr int FT = decltype(ft)::value;
      st.template tile<FT>(t.s1 - t.s0, next);
      st.template store<FT>(o);
    };
    if (t.rows > 128) go(std::integral_constant<int, 8>{});
    else if (t.rows > 64) go(std::integral_constant<int, 4>{});
    else go(std::integral_constant<int, 2>{});
  }
  wait_vmcnt<0>();   // no copy may be in flight when the workgroup's LDS is given away
}

// Every expert's tiles, in the same order (kGroup tiles of its N, column tile, tile of N),
// are split over four XCDs in runs, over eight where there are fewer than eight experts:
// enough for one expert of many rows, and a run still shares its operands' rows. Four and
// eight, in us: 384 experts, 768 x 7168, of 704 rows each 3014 and 3149, of a 32K chunk's 47 to
// 30133 rows 3613 and 3929 (two: 4107), 64 experts of up to 3418 rows, 1024 x 2048 293 and 300.
template <int FT, int FW, bool F32>
__global__ __launch_bounds__(kThreads, 1) void k_expert_wgrad(ExpertGradArgs a) {
  typedef Stream<FT, FW, true, true, F32> S;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kSmem];
  const int m_tiles = (a.N + 32 * FT - 1) / (32 * FT), n_tiles = (a.C + 32 * FW - 1) / (32 * FW);
  const int tiles = m_tiles * n_tiles, per = tiles * a.splits;   // of an expert
  const int parts = min(a.E < kXcds ? kXcds : kXcds / 2, per), len = (per + parts - 1) / parts;
  const int xcd = blockIdx.x % kXcds, stride = gridDim.x / kXcds;
  const int end = len * ((a.E * parts - xcd + kXcds - 1) / kXcds);   // this XCD's parts
  const const_ints off = as_const(a.off), order = as_const(a.order);

  struct Tile {
    int expert, m0, n0, lo, hi, steps, split;
  };
  // tile i of this XCD: part i / len of its parts; expert -1 where a part is short. Rows
  // [lo, hi), none where a split has no step: then its one step reads zeros.
  auto tile_of = [&](int i) {
    const int run = uniform_div(i, len), part = run * kXcds + xcd, at = uniform_div(part, parts);
    const int k = (part - at * parts) * len + i - run * len;
    if (i >= end || k >= per) return Tile{-1, 0, 0, 0, 0, 0, 0};
    const int e = order[at], split = uniform_div(k, tiles), t = k - split * tiles;
    const int group = uniform_div(t, kGroup * n_tiles), in = t - group * kGroup * n_tiles;
    const int in_group = min(kGroup, m_tiles - group * kGroup), nt = uniform_div(in, in_group);
    const int mt = group * kGroup + in - nt * in_group;
    const int lo = min(max(off[e], 0), a.P), hi = min(max(off[e + 1], lo), a.P);
    const int steps = (hi - lo + 63) / 64;
    const int s0 = uniform_div(steps * split, a.splits), s1 = uniform_div(steps * (split + 1), a.splits);
    return Tile{e, mt * 32 * FT, nt * 32 * FW, lo + 64 * s0, min(hi, lo + 64 * s1), max(s1 - s0, 1),
                split};
  };
  int id = blockIdx.x / kXcds;
  auto skip = [&](int& i) {   // to the next tile that there is
    Tile t = tile_of(i);
    while (t.expert < 0 && i < end) {
      i += stride;
      t = tile_of(i);
    }
    return t;
  };
  Tile now = skip(id);
  if (now.expert < 0) return;

  S st;
  st.init(smem, a.N, a.C);
  int at = id, step = 0;
  Tile copied = now;
  auto place = [&]() {
    st.oa.place(a.dy + (int64_t)copied.lo * a.N, a.N, copied.m0, a.N, copied.hi - copied.lo);
    st.ob.place(a.x + (int64_t)copied.lo * a.C, a.C, copied.n0, a.C, copied.hi - copied.lo);
  };
  place();
  auto next = [&](v4i_s& sa, v4i_s& sb) {
    sa = st.oa.rsrc(step, copied.expert >= 0);
    sb = st.ob.rsrc(step, copied.expert >= 0);
    if (copied.expert >= 0 && ++step == copied.steps) {
      step = 0;
      at += stride;
      copied = skip(at);
      if (copied.expert >= 0) place();
    }
  };
  st.start(next);
  while (now.expert >= 0) {
    OutTile o;
    o.place<F32>(static_cast<char*>(a.dw) + ((int64_t)now.split * a.E + now.expert) * a.N * a.C * (F32 ? 4 : 2), now.m0,
                 min(32 * FT, a.N - now.m0), now.n0, a.C);
    st.template tile<FT>(now.steps, next);
    st.template store<FT>(o);
    id += stride;
    now = skip(id);
  }
  wait_vmcnt<0>();
}

template <int FW, bool WT>
void run_tiles(const ExpertArgs& a, bool f32, hipStream_t s) {
  const int64_t most = expert_tiles_bound(a.P, a.E) * ceil_div(a.O, 32 * FW) * a.splits;
  const dim3 grid((unsigned)(most < kCus ? ceil_div(most, kXcds) * kXcds : kCus)), block(kThreads);
  if (f32) hipLaunchKernelGGL((k_expert_tile<FW, WT, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_expert_tile<FW, WT, false>), grid, block, 0, s, a);
}

template <int FT, int FW>
void run_wgrad(const ExpertGradArgs& a, bool f32, hipStream_t s) {
  if (f32) hipLaunchKernelGGL((k_expert_wgrad<FT, FW, true>), dim3(kCus), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((k_expert_wgrad<FT, FW, false>), dim3(kCus), dim3(kThreads), 0, s, a);
}

}  // namespace

// Columns of a tile: 256, unless 192 or 128 fill the last one so much better that more
// tiles cost less (a step of 64 of 256 columns takes 1.70 us, of 192 1.45, of 128 1.2).
int tile_fragments(int cols) {
  const int64_t t8 = 170 * ceil_div(cols, 256), t6 = 145 * ceil_div(cols, 192), t4 = 120 * ceil_div(cols, 128);
  return t8 <= t6 && t8 <= t4 ? 8 : t6 <= t4 ? 6 : 4;
}

void launch_expert_tiles(const ExpertArgs& a, bool w_trans, bool f32, hipStream_t s) {
  const int fw = tile_fragments(a.O);
  if (w_trans) {
    if (fw == 8) run_tiles<8, true>(a, f32, s);
    else if (fw == 6) run_tiles<6, true>(a, f32, s);
    else run_tiles<4, true>(a, f32, s);
  } else {
    if (fw == 8) run_tiles<8, false>(a, f32, s);
    else if (fw == 6) run_tiles<6, false>(a, f32, s);
    else run_tiles<4, false>(a, f32, s);
  }
}

void launch_expert_wgrad(const ExpertGradArgs& a, bool f32, hipStream_t s) {
  const int ft = tile_fragments(a.N), fw = tile_fragments(a.C);
  if (ft == 8) {
    if (fw == 8) run_wgrad<8, 8>(a, f32, s);
    else if (fw == 6) run_wgrad<8, 6>(a, f32, s);
    else run_wgrad<8, 4>(a, f32, s);
  } else if (ft == 6) {
    if (fw == 8) run_wgrad<6, 8>(a, f32, s);
    else if (fw == 6) run_wgrad<6, 6>(a, f32, s);
    else run_wgrad<6, 4>(a, f32, s);
  } else {
    if (fw == 8) run_wgrad<4, 8>(a, f32, s);
    else if (fw == 6) run_wgrad<4, 6>(a, f32, s);
    else run_wgrad<4, 4>(a, f32, s);
  }
}

}  // namespace moe

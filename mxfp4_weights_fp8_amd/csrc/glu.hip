// The gated activation between an expert's two products, with its input saved in 8 bits
// for the backward pass, and its gradient from what was saved:
//   z = (g, u), the two halves of a row's 2 I columns;  h = act(g) u
//   z_q, z_s: z as E4M3 codes with one E8M0 scale per 128 columns (the activation format
//   of the FFN: the smallest power of two with amax <= 448 * scale)
//   dg = dh u act'(g),  du = dh act(g),  and h once more, all at the values the codes
//   stand for (or at a z that was kept whole)
// Everything between load and store is fp32, each output is rounded once. HBM-bound: 16
// lanes own 128 gate columns and the 128 up columns of the same h, 8 each per lane, so a
// block's amax is a 16-lane butterfly. 262144 x 384: 147 us (5.5 TB/s), the gradient from
// codes 200 us (4.9 TB/s); with gelu 189 and 312 us, bound by erfcf; 128 x 512 3.3 us, bound by
// the launch. Rows from *live on (the plan's last offset) are neither read nor written.
#include "device_common.h"
#include "host_internal.h"
#include "lane_reduce.h"
#include "rows.h"
#include "linear.h"

#include <float.h>

namespace moe {
namespace {

constexpr int kGluThreads = 256;

struct GluArgs {
  const uint16_t* z;     // [R, 2I] bf16; null in the gradient from codes
  const uint16_t* dh;    // [R, I]
  const int32_t* live;   // optional
  uint16_t* h;           // [R, I], optional in the gradient; may be dh
  uint16_t* dz;          // [R, 2I]; may be z
  uint8_t* z_q;          // [R, 2I], read by the gradient
  uint8_t* z_s;          // [R, 2I / 128]
  int R, I, act;
};

// The 8 columns of h that a thread has: its row and column; row R where it has none.
struct Spot {
  int64_t row;
  int col;
};
__device__ __forceinline__ Spot spot_of(const GluArgs& a) {
  const int groups = a.I / 8;   // a multiple of 16: the 16 lanes of a block agree on the row
  const int64_t g0 = block_id() * kGluThreads, r0 = g0 / groups;
  const uint32_t in = (uint32_t)(g0 - r0 * groups) + threadIdx.x;
  const int rows = a.live ? min(max(*a.live, 0), a.R) : a.R;
  const int64_t row = r0 + in / (uint32_t)groups;
  return Spot{row < rows ? row : a.R, 8 * (int)(in % (uint32_t)groups)};
}

__device__ __forceinline__ void save8(const GluArgs& a, int64_t at, const float (&v)[8]) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  const int e = e8m0_exponent(row_max<16>(amax));
  const float inv = exp2_neg(e);
  *reinterpret_cast<uint2*>(a.z_q + at) =
      make_uint2(e4m3_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                 e4m3_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
  if ((threadIdx.x & 15) == 0) a.z_s[at / 128] = (uint8_t)(e + 127);
}

template <bool NT>
__global__ __launch_bounds__(kGluThreads) void k_glu(GluArgs a) {
  const Spot p = spot_of(a);
  if (p.row >= a.R) return;
  const int64_t gate = p.row * 2 * a.I + p.col, up = gate + a.I;
  float g[8], u[8];
  unpack8(load16_nt(a.z + gate), g);
  unpack8(load16_nt(a.z + up), u);
  if (a.z_q) {
    save8(a, gate, g);
    save8(a, up, u);
  }
  activate(g, a.act);
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] *= u[i];
  store_row<NT>(a.h + p.row * a.I + p.col, pack8(g));
}

template <bool CODES, bool NT>
__global__ __launch_bounds__(kGluThreads) void k_glu_grad(GluArgs a) {
  const Spot p = spot_of(a);
  if (p.row >= a.R) return;
  const int64_t gate = p.row * 2 * a.I + p.col, up = gate + a.I, at = p.row * a.I + p.col;
  float g[8], u[8], d[8];
  unpack8(load16_nt(a.dh + at), d);
  int scale = 0;
  if constexpr (CODES) {
    const int eg = a.z_s[gate / 128], eu = a.z_s[up / 128];
    decode8(*reinterpret_cast<const uint2*>(a.z_q + gate), eg - 127, g);
    decode8(*reinterpret_cast<const uint2*>(a.z_q + up), eu - 127, u);
    scale = max(eg, eu);
  } else {
    unpack8(load16_nt(a.z + gate), g);
    unpack8(load16_nt(a.z + up), u);
  }
  float dg[8], du[8], most = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    dg[i] = d[i] * u[i];
    most = fmaxf(most, fabsf(dg[i]));
    dg[i] *= activate_slope(g[i], a.act);
  }
  // What leaves fp32 on the way: dh u, where a gate's tail may take it back (relu: to zero), so
  // that the slope comes first; and 2^128, the code 256 under the largest scale of a finite
  // block, 2^120 (bf16 values from 1.9375 2^127 on), for which fp32's largest value stands.
  if (most > FLT_MAX || scale >= 120 + 127)
    for (int i = 0; i < 8; ++i) {
      if constexpr (CODES) {   // an infinity of z itself stays one
        g[i] = fabsf(g[i]) > FLT_MAX ? copysignf(FLT_MAX, g[i]) : g[i];
        u[i] = fabsf(u[i]) > FLT_MAX ? copysignf(FLT_MAX, u[i]) : u[i];
      }
      const float p = d[i] * u[i], slope = activate_slope(g[i], a.act);
      dg[i] = fabsf(p) > FLT_MAX ? d[i] * slope * u[i] : p * slope;
    }
  activate(g, a.act);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    du[i] = d[i] * g[i];
    u[i] *= g[i];
  }
  store_row<NT>(a.dz + gate, pack8(dg));
  store_row<NT>(a.dz + up, pack8(du));
  if (a.h) store_row<NT>(a.h + at, pack8(u));
}

inline bool past_cache(const GluArgs& a) { return (int64_t)a.R * 2 * a.I > kCachedRows; }
inline dim3 grid_of(const GluArgs& a) { return grid_of_blocks(ceil_div((int64_t)a.R * (a.I / 8), kGluThreads)); }

}  // namespace

hipError_t launch_glu(const moe_glu_dims& d, const uint16_t* z, const int32_t* live, uint16_t* h, uint8_t* z_q,
                      uint8_t* z_s, hipStream_t s) {
  const GluArgs a{z, nullptr, live, h, nullptr, z_q, z_s, d.R, d.I, d.act};
  if (past_cache(a)) hipLaunchKernelGGL(k_glu<true>, grid_of(a), dim3(kGluThreads), 0, s, a);
  else hipLaunchKernelGGL(k_glu<false>, grid_of(a), dim3(kGluThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_glu_grad(const moe_glu_dims& d, const uint16_t* dh, const uint16_t* z, const uint8_t* z_q,
                           const uint8_t* z_s, const int32_t* live, uint16_t* dz, uint16_t* h, hipStream_t s) {
  const GluArgs a{z, dh, live, h, dz, const_cast<uint8_t*>(z_q), const_cast<uint8_t*>(z_s), d.R, d.I, d.act};
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid_of(a), dim3(kGluThreads), 0, s, a); };
  if (past_cache(a)) z ? go(k_glu_grad<false, true>) : go(k_glu_grad<true, true>);
  else z ? go(k_glu_grad<false, false>) : go(k_glu_grad<true, false>);
  return hipGetLastError();
}

}  // namespace moe

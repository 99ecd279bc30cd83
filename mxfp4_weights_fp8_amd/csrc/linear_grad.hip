// Gradient of the dense product y = act(x w^T + b) + residual:
//   dz = dy act'(z),   dx = dz w,   dw = dz^T x,   db = sum over rows of dz
// (the residual's gradient is dy itself). The matrix cores take bf16: where dz is not bf16
// already (a bf16 dy without activation, or with relu, whose slopes are 0 and 1) it goes in
// as two bf16 values, its upper 16 bits and the rest rounded, together off by at most 2^-15
// of it (a rest below 2^-126 is lost). Rounded to one bf16 value, dz moved dx and dw by as
// much as their own rounding to bf16 does (router: 2.3e-3 of their norm instead of 1.7e-3).
// db is summed from the fp32 dz.
//
// Both products contract over the rows of an operand; the tiled kernel reads such
// operands transposed, as they lie. dz [M, N] goes to the workspace with its rows padded by
// zeros to a multiple of 128, in two parts the high row and then the low one.
// 16384 x 384 x 7168 (the router's) from an fp32 dy 372-386 us: dz 11, dx 179, dw 186 and 9 for
// joining its three parts, dbias 5; from a bf16 dy 240. Two parts cost twice the products' work:
// 8191 x 7168 x 2048 with silu 921 us, where one rounded part took 503.
#include "linear.h"

#include <type_traits>

namespace moe {
namespace {

struct DzArgs {
  const void* dy;
  const float* z;
  uint16_t* dz;       // [M, Np] or [M, 2, Np] (high, low), columns N .. Np - 1 zero
  float* db_parts;    // [ceil(M / 64), N]
  int M, N, Np, act;
};

// dz of 64 rows x 64 columns, and its column sums: a thread holds four columns of every
// 16th row. Without activation every load is on its way at once (VEC: N a multiple of 4,
// loads of four; one column per thread took 14.3 us of 16384 x 384); with one, rows follow
// each other, as four slopes fill the registers.
template <bool VEC, bool DY_F32, bool ACT, bool TWO>
__global__ __launch_bounds__(256) void k_linear_dz(DzArgs a) {
  __shared__ v4f sums[16][16];
  const int group = threadIdx.x & 15, sub = threadIdx.x >> 4;
  const int n = blockIdx.y * 64 + 4 * group;
  const int64_t m0 = (int64_t)blockIdx.x * 64 + sub;
  // columns past N are zeros
  auto load = [&](const void* p, bool f32, int64_t m) {
    v4f v{0.f, 0.f, 0.f, 0.f};
    const int64_t at = m * a.N + n;
    if constexpr (VEC) {
      if (n >= a.N) return v;
      if (f32) return *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(p) + at);
      const uint2 r = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + at);
      return v4f{__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                 __uint_as_float(r.y & 0xFFFF0000u)};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.N)
        v[i] = f32 ? reinterpret_cast<const float*>(p)[at + i] : bf16_to_float(reinterpret_cast<const uint16_t*>(p)[at + i]);
    return v;
  };
  auto store = [&](int64_t m, const v4f v) {
    if constexpr (TWO) {
      uint32_t hi[4];
      float lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hi[i] = __float_as_uint(v[i]) & 0xFFFF0000u;
        lo[i] = fabsf(v[i]) == INFINITY ? 0.f : v[i] - __uint_as_float(hi[i]);   // exact; NaN stays NaN
      }
      uint16_t* at = a.dz + m * 2 * a.Np + n;
      *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] >> 16 | hi[1], hi[2] >> 16 | hi[3]);
      *reinterpret_cast<uint2*>(at + a.Np) = make_uint2(bf16_pack2(lo[0], lo[1]), bf16_pack2(lo[2], lo[3]));
    } else {
      *reinterpret_cast<uint2*>(a.dz + m * a.Np + n) = make_uint2(bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]));
    }
  };
  v4f sum{0.f, 0.f, 0.f, 0.f};
  if constexpr (ACT) {
#pragma unroll 1
    for (int64_t m = m0; m < m0 + 64 && m < a.M; m += 16) {
      v4f dz = load(a.dy, DY_F32, m);
      const v4f z = load(a.z, true, m);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (VEC || n + i < a.N) dz[i] *= activate_slope(z[i], a.act);
      sum += dz;
      store(m, dz);
    }
  } else {
    constexpr int kTurns = 4;
    v4f dz[kTurns];
#pragma unroll
    for (int u = 0; u < kTurns; ++u) dz[u] = load(a.dy, DY_F32, min(m0 + 16 * u, (int64_t)a.M - 1));
#pragma unroll
    for (int u = 0; u < kTurns; ++u)
      if (m0 + 16 * u < a.M) {
        sum += dz[u];
        store(m0 + 16 * u, dz[u]);
      }
  }
  sums[sub][group] = sum;
  __syncthreads();
  const int c = threadIdx.x;
  if (c < 64 && blockIdx.y * 64 + c < a.N) {
    float s = sums[0][c >> 2][c & 3];
    for (int k = 1; k < 16; ++k) s += sums[k][c >> 2][c & 3];
    a.db_parts[(int64_t)blockIdx.x * a.N + blockIdx.y * 64 + c] = s;
  }
}

inline int pad128(int v) { return (v + 127) / 128 * 128; }
inline bool two_parts(const moe_linear_dims& d) {
  return d.type != MOE_TYPE_BF16 || (d.act != MOE_ACT_NONE && d.act != MOE_ACT_RELU);
}

struct GradWs {
  uint16_t* dz;
  float *db_parts, *parts;
};

size_t grad_ws_layout(const moe_linear_dims& d, void* base, GradWs* out) {
  const int M = d.M, N = d.N, K = d.K, Np = pad128(N);
  const bool two = two_parts(d);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + (bytes ? bytes : 1), 256);
    return o;
  };
  const size_t o_dz = take((two ? 4 : 2) * (size_t)M * Np), o_db = take(sizeof(float) * (size_t)ceil_div(M, 64) * N);
  const size_t px = linear_plan_parts(M, K, linear_plan(M, K, Np, Layout::kWTrans, true, two)),
               pw = linear_plan_parts(N, K, linear_plan(N, K, M, Layout::kBothTrans, true, two));
  const size_t o_parts = take(px > pw ? px : pw);
  if (out) {
    char* b = static_cast<char*>(base);
    out->dz = reinterpret_cast<uint16_t*>(b + o_dz);
    out->db_parts = reinterpret_cast<float*>(b + o_db);
    out->parts = reinterpret_cast<float*>(b + o_parts);
  }
  return off;
}

}  // namespace

size_t linear_grad_ws_bytes(const moe_linear_dims& d) { return grad_ws_layout(d, nullptr, nullptr); }

hipError_t launch_linear_grad(const moe_linear_dims& d, const void* dy, const uint16_t* x, const uint16_t* w,
                              const float* z, uint16_t* dx, uint16_t* dw, float* db, void* ws, hipStream_t s) {
  if (d.M == 0) {   // sums over no rows
    hipError_t err = dw ? launch_fill_zero(reinterpret_cast<int32_t*>(dw), (int64_t)d.N * d.K / 2, s) : hipSuccess;
    return err == hipSuccess && db ? launch_fill_zero(reinterpret_cast<int32_t*>(db), d.N, s) : err;
  }
  GradWs g;
  grad_ws_layout(d, ws, &g);
  const int Np = pad128(d.N), m_blocks = (int)ceil_div(d.M, 64);
  const bool one = m_blocks == 1 && db;   // the only part is the result: one launch less
  const DzArgs da{dy, z, g.dz, one ? db : g.db_parts, d.M, d.N, Np, d.act};
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(m_blocks, Np / 64), dim3(256), 0, s, da); };
  const bool two = two_parts(d);
  auto by_act = [&](auto vec, auto f32) {
    constexpr bool V = decltype(vec)::value, F = decltype(f32)::value;
    if (d.act == MOE_ACT_NONE) go(k_linear_dz<V, F, false, F>);
    else if (two) go(k_linear_dz<V, F, true, true>);
    else go(k_linear_dz<V, F, true, F>);   // relu of a bf16 dy
  };
  auto by_type = [&](auto vec) {
    if (d.type == MOE_TYPE_F32) by_act(vec, std::true_type{});
    else by_act(vec, std::false_type{});
  };
  if (d.N % 4 == 0) by_type(std::true_type{});
  else by_type(std::false_type{});
  hipError_t err = hipGetLastError();
  if (err == hipSuccess && db && !one) err = launch_sum_parts(g.db_parts, m_blocks, d.N, db, s);
  const int xs = two ? 2 * Np : Np, low = two ? Np : 0;
  if (err == hipSuccess && dx) {   // [M, K] = dz [M, Np] . w [N, K], contracted over N
    const LinearArgs a{g.dz, w, xs, d.K, low, nullptr, nullptr, dx, nullptr, g.parts, d.M, d.K, Np, d.N,
                       MOE_ACT_NONE, 1, false};
    err = launch_linear_plan(a, linear_plan(d.M, d.K, Np, Layout::kWTrans, true, two), Layout::kWTrans, s);
  }
  if (err == hipSuccess && dw) {   // [N, K] = dz [M, N] . x [M, K], contracted over M
    const LinearArgs a{g.dz, x, xs, d.K, low, nullptr, nullptr, dw, nullptr, g.parts, d.N, d.K, d.M, d.M,
                       MOE_ACT_NONE, 1, false};
    err = launch_linear_plan(a, linear_plan(d.N, d.K, d.M, Layout::kBothTrans, true, two), Layout::kBothTrans, s);
  }
  return err;
}

}  // namespace moe

// Gradient of the dense product y = act(x w^T + b) + residual:
//   dz = dy act'(z),   dx = dz w,   dw = dz^T x,   db = sum over rows of dz
// (the residual's gradient is dy itself). dz is rounded once to bf16, the matrix
// cores' operand type; db is summed from the fp32 dz.
//
// Both products contract over the rows of an operand; the tiled kernel reads such
// operands transposed, as they lie. dz [M, N] goes to the workspace with its rows
// padded by zeros to a multiple of 128. 16384 x 384 x 7168 (the router's): dz 8.7 us, 4.3
// TB/s, dbias 5 us, dx 109-112 us, dw 107-112 us and 8 us for joining its three parts.
#include "linear.h"

#include <type_traits>

namespace moe {
namespace {

struct DzArgs {
  const void* dy;
  const float* z;
  uint16_t* dz;       // [M, Np], columns N .. Np - 1 zero
  float* db_parts;    // [ceil(M / 64), N]
  int M, N, Np, act;
};

// dz of 64 rows x 64 columns, and its column sums: a thread holds four columns of every
// 16th row. Without activation every load is on its way at once (VEC: N a multiple of 4,
// loads of four; one column per thread took 14.3 us of 16384 x 384); with one, rows follow
// each other, as four slopes fill the registers.
template <bool VEC, bool DY_F32, bool ACT>
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
    *reinterpret_cast<uint2*>(a.dz + m * a.Np + n) = make_uint2(bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]));
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

struct GradWs {
  uint16_t* dz;
  float *db_parts, *parts;
};

size_t grad_ws_layout(int M, int N, int K, void* base, GradWs* out) {
  const int Np = pad128(N);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + (bytes ? bytes : 1), 256);
    return o;
  };
  const size_t o_dz = take(2 * (size_t)M * Np), o_db = take(sizeof(float) * (size_t)ceil_div(M, 64) * N);
  const size_t px = linear_plan_parts(M, K, linear_plan(M, K, Np, Layout::kWTrans, true)),
               pw = linear_plan_parts(N, K, linear_plan(N, K, M, Layout::kBothTrans, true));
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

size_t linear_grad_ws_bytes(int M, int N, int K) { return grad_ws_layout(M, N, K, nullptr, nullptr); }

hipError_t launch_linear_grad(const moe_linear_dims& d, const void* dy, const uint16_t* x, const uint16_t* w,
                              const float* z, uint16_t* dx, uint16_t* dw, float* db, void* ws, hipStream_t s) {
  if (d.M == 0) {   // sums over no rows
    hipError_t err = dw ? launch_fill_zero(reinterpret_cast<int32_t*>(dw), (int64_t)d.N * d.K / 2, s) : hipSuccess;
    return err == hipSuccess && db ? launch_fill_zero(reinterpret_cast<int32_t*>(db), d.N, s) : err;
  }
  GradWs g;
  grad_ws_layout(d.M, d.N, d.K, ws, &g);
  const int Np = pad128(d.N), m_blocks = (int)ceil_div(d.M, 64);
  const bool one = m_blocks == 1 && db;   // the only part is the result: one launch less
  const DzArgs da{dy, z, g.dz, one ? db : g.db_parts, d.M, d.N, Np, d.act};
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(m_blocks, Np / 64), dim3(256), 0, s, da); };
  auto by_act = [&](auto vec, auto f32) {
    if (d.act == MOE_ACT_NONE) go(k_linear_dz<decltype(vec)::value, decltype(f32)::value, false>);
    else go(k_linear_dz<decltype(vec)::value, decltype(f32)::value, true>);
  };
  auto by_type = [&](auto vec) {
    if (d.type == MOE_TYPE_F32) by_act(vec, std::true_type{});
    else by_act(vec, std::false_type{});
  };
  if (d.N % 4 == 0) by_type(std::true_type{});
  else by_type(std::false_type{});
  hipError_t err = hipGetLastError();
  if (err == hipSuccess && db && !one) err = launch_sum_parts(g.db_parts, m_blocks, d.N, db, s);
  if (err == hipSuccess && dx) {   // [M, K] = dz [M, Np] . w [N, K], contracted over N
    const LinearArgs a{g.dz, w, Np, d.K, nullptr, nullptr, dx, nullptr, g.parts, d.M, d.K, Np, d.N,
                       MOE_ACT_NONE, 1, false};
    err = launch_linear_plan(a, linear_plan(d.M, d.K, Np, Layout::kWTrans, true), Layout::kWTrans, s);
  }
  if (err == hipSuccess && dw) {   // [N, K] = dz [M, N] . x [M, K], contracted over M
    const LinearArgs a{g.dz, x, Np, d.K, nullptr, nullptr, dw, nullptr, g.parts, d.N, d.K, d.M, d.M,
                       MOE_ACT_NONE, 1, false};
    err = launch_linear_plan(a, linear_plan(d.N, d.K, d.M, Layout::kBothTrans, true), Layout::kBothTrans, s);
  }
  return err;
}

}  // namespace moe

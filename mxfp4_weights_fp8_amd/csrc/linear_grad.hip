// Gradient of the dense product y = act(x w^T + b) + residual:
//   dz = dy act'(z),   dx = dz w,   dw = dz^T x,   db = sum over rows of dz
// (the residual's gradient is dy itself). dz is rounded once to bf16, the matrix
// cores' operand type; db is summed from the fp32 dz.
//
// Both products contract over the rows of an operand; the tiled kernel reads such
// operands transposed, as they lie. dz [M, N] goes to the workspace with its rows
// padded by zeros to a multiple of 128.
#include "linear.h"

namespace moe {
namespace {

struct DzArgs {
  const void* dy;
  const float* z;
  uint16_t* dz;       // [M, Np], columns N .. Np - 1 zero
  float* db_parts;    // [ceil(M / 64), N]
  int M, N, Np, act;
  bool dy_f32;
};

// dz of 64 rows x 64 columns, and its column sums (16 rows per wave, then the waves).
__global__ __launch_bounds__(256) void k_linear_dz(DzArgs a) {
  __shared__ float sums[4][64];
  const int m0 = blockIdx.x * 64;
  const int c = threadIdx.x & 63, wave = threadIdx.x >> 6, n = blockIdx.y * 64 + c;
  float sum = 0.f;
  for (int r = wave; r < 64; r += 4) {
    const int m = m0 + r;
    if (m >= a.M) break;
    float v = 0.f;
    if (n < a.N) {
      const int64_t at = (int64_t)m * a.N + n;
      v = a.dy_f32 ? reinterpret_cast<const float*>(a.dy)[at]
                   : bf16_to_float(reinterpret_cast<const uint16_t*>(a.dy)[at]);
      if (a.act != MOE_ACT_NONE) v *= activate_slope(a.z[at], a.act);
    }
    sum += v;
    a.dz[(int64_t)m * a.Np + n] = (uint16_t)bf16_pack2(v, 0.f);
  }
  sums[wave][c] = sum;
  __syncthreads();
  if (wave == 0 && n < a.N)
    a.db_parts[(int64_t)blockIdx.x * a.N + n] = sums[0][c] + sums[1][c] + sums[2][c] + sums[3][c];
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
  const DzArgs da{dy, z, g.dz, g.db_parts, d.M, d.N, Np, d.act, d.type == MOE_TYPE_F32};
  hipLaunchKernelGGL(k_linear_dz, dim3(m_blocks, Np / 64), dim3(256), 0, s, da);
  hipError_t err = hipGetLastError();
  if (err == hipSuccess && db) err = launch_sum_parts(g.db_parts, m_blocks, d.N, db, s);
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

// Gradient of the dense product y = act(x w^T + b) + residual:
//   dz = dy act'(z),   dx = dz w,   dw = dz^T x,   db = sum over rows of dz
// (the residual's gradient is dy itself). dz is rounded once to bf16, the matrix
// cores' operand type; db is summed from the fp32 dz.
//
// Both products contract over the rows of an operand, while the tiled kernel reads
// operands whose contraction index runs along memory: dz, x and w are transposed
// into the workspace, padded with zeros to a multiple of 128.
#include "linear.h"

namespace moe {
namespace {

constexpr int kT = 64;   // transposed in tiles of 64 x 64

// Rows [r0, r0 + 64) x columns [c0, c0 + 64) of `in` to out[c][r], r < rows_padded
// (cols and rows_padded are multiples of 64);
// 64 x 66 halfwords of LDS: rows 33 dwords apart, so neighbouring rows lie in
// neighbouring banks.
__global__ __launch_bounds__(256) void k_transpose(const uint16_t* __restrict__ in, int rows, int cols,
                                                   int rows_padded, uint16_t* __restrict__ out) {
  __shared__ uint16_t tile[kT][kT + 2];
  const int r0 = blockIdx.x * kT, c0 = blockIdx.y * kT;
  for (int i = threadIdx.x; i < kT * kT / 2; i += 256) {
    const int r = i / (kT / 2), c = i % (kT / 2) * 2;
    uint32_t v = 0;
    if (r0 + r < rows) v = *reinterpret_cast<const uint32_t*>(in + (int64_t)(r0 + r) * cols + c0 + c);
    tile[r][c] = (uint16_t)v;
    tile[r][c + 1] = (uint16_t)(v >> 16);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kT * kT / 2; i += 256) {
    const int c = i / (kT / 2), r = i % (kT / 2) * 2;
    *reinterpret_cast<uint32_t*>(out + (int64_t)(c0 + c) * rows_padded + r0 + r) =
        (uint32_t)tile[r][c] | ((uint32_t)tile[r + 1][c] << 16);
  }
}

struct DzArgs {
  const void* dy;
  const float* z;
  uint16_t* dz;       // [M, Np], columns N .. Np - 1 zero
  uint16_t* dzt;      // [N, Mp], columns M .. Mp - 1 zero
  float* db_parts;    // [Mp / 64, N]
  int M, N, Mp, Np, act;
  bool dy_f32;
};

// dz of one 64 x 64 tile, as it is, transposed, and summed over its rows.
__global__ __launch_bounds__(256) void k_linear_dz(DzArgs a) {
  __shared__ uint16_t tile[kT][kT + 2];
  __shared__ float sums[4][kT];
  const int m0 = blockIdx.x * kT, n0 = blockIdx.y * kT;
  const int c = threadIdx.x & 63, wave = threadIdx.x >> 6, n = n0 + c;
  float sum = 0.f;
  for (int r = wave; r < kT; r += 4) {
    const int m = m0 + r;
    float v = 0.f;
    if (m < a.M && n < a.N) {
      const int64_t at = (int64_t)m * a.N + n;
      v = a.dy_f32 ? reinterpret_cast<const float*>(a.dy)[at]
                   : bf16_to_float(reinterpret_cast<const uint16_t*>(a.dy)[at]);
      if (a.act != MOE_ACT_NONE) v *= activate_slope(a.z[at], a.act);
    }
    sum += v;
    const uint16_t b = (uint16_t)bf16_pack2(v, 0.f);
    tile[r][c] = b;
    if (m < a.M && n < a.Np) a.dz[(int64_t)m * a.Np + n] = b;
  }
  sums[wave][c] = sum;
  __syncthreads();
  if (wave == 0 && n < a.N)
    a.db_parts[(int64_t)blockIdx.x * a.N + n] = sums[0][c] + sums[1][c] + sums[2][c] + sums[3][c];
  for (int i = threadIdx.x; i < kT * kT / 2; i += 256) {
    const int tc = i / (kT / 2), r = i % (kT / 2) * 2;
    if (n0 + tc < a.N)   // Mp is a multiple of 128, so every row of the tile is below it
      *reinterpret_cast<uint32_t*>(a.dzt + (int64_t)(n0 + tc) * a.Mp + m0 + r) =
          (uint32_t)tile[r][tc] | ((uint32_t)tile[r + 1][tc] << 16);
  }
}

inline int pad128(int v) { return (v + 127) / 128 * 128; }

struct GradWs {
  uint16_t *dz, *dzt, *wt, *xt;
  float *db_parts, *parts;
};

size_t grad_ws_layout(int M, int N, int K, void* base, GradWs* out) {
  const size_t Mp = pad128(M), Np = pad128(N);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + (bytes ? bytes : 1), 256);
    return o;
  };
  const size_t o_dz = take(2 * (size_t)M * Np), o_dzt = take(2 * (size_t)N * Mp), o_wt = take(2 * (size_t)K * Np),
               o_xt = take(2 * (size_t)K * Mp), o_db = take(sizeof(float) * (Mp / kT) * N);
  const size_t px = linear_parts_bytes(M, K, (int)Np), pw = linear_parts_bytes(N, K, (int)Mp);
  const size_t o_parts = take(px > pw ? px : pw);
  if (out) {
    char* b = static_cast<char*>(base);
    out->dz = reinterpret_cast<uint16_t*>(b + o_dz);
    out->dzt = reinterpret_cast<uint16_t*>(b + o_dzt);
    out->wt = reinterpret_cast<uint16_t*>(b + o_wt);
    out->xt = reinterpret_cast<uint16_t*>(b + o_xt);
    out->db_parts = reinterpret_cast<float*>(b + o_db);
    out->parts = reinterpret_cast<float*>(b + o_parts);
  }
  return off;
}

}  // namespace

size_t linear_grad_ws_bytes(int M, int N, int K) { return grad_ws_layout(M, N, K, nullptr, nullptr); }

hipError_t launch_linear_grad(const moe_linear_dims& d, const void* dy, const uint16_t* x, const uint16_t* w,
                              const float* z, uint16_t* dx, uint16_t* dw, float* db, void* ws, hipStream_t s) {
  if (d.M == 0) {   // sums over no rows; dw as N K / 2 zero words
    hipError_t err = dw ? launch_sum_parts(nullptr, 0, (int)((int64_t)d.N * d.K / 2), reinterpret_cast<float*>(dw), s)
                        : hipSuccess;
    return err == hipSuccess && db ? launch_sum_parts(nullptr, 0, d.N, db, s) : err;
  }
  GradWs g;
  grad_ws_layout(d.M, d.N, d.K, ws, &g);
  const int Mp = pad128(d.M), Np = pad128(d.N);
  const DzArgs da{dy, z, g.dz, g.dzt, g.db_parts, d.M, d.N, Mp, Np, d.act, d.type == MOE_TYPE_F32};
  hipLaunchKernelGGL(k_linear_dz, dim3(Mp / kT, Np / kT), dim3(256), 0, s, da);
  hipError_t err = hipGetLastError();
  if (err == hipSuccess && db) err = launch_sum_parts(g.db_parts, Mp / kT, d.N, db, s);
  if (err == hipSuccess && dx) {   // [M, K] = dz [M, Np] . wt [K, Np]
    hipLaunchKernelGGL(k_transpose, dim3(Np / kT, d.K / kT), dim3(256), 0, s, w, d.N, d.K, Np, g.wt);
    const LinearArgs a{g.dz, g.wt, nullptr, nullptr, dx, nullptr, g.parts, d.M, d.K, Np, MOE_ACT_NONE, 1, false};
    err = launch_linear_plan(a, linear_plan(d.M, d.K, Np), s);
  }
  if (err == hipSuccess && dw) {   // [N, K] = dzt [N, Mp] . xt [K, Mp]
    hipLaunchKernelGGL(k_transpose, dim3(Mp / kT, d.K / kT), dim3(256), 0, s, x, d.M, d.K, Mp, g.xt);
    const LinearArgs a{g.dzt, g.xt, nullptr, nullptr, dw, nullptr, g.parts, d.N, d.K, Mp, MOE_ACT_NONE, 1, false};
    err = launch_linear_plan(a, linear_plan(d.N, d.K, Mp), s);
  }
  return err;
}

}  // namespace moe

// Residual add + RMS norm with bf16 and 8-bit outputs, and its gradient.
//
//   h = x + res,  r = 1 / sqrt(mean_H(h^2) + eps),  y = h r w
//   x_q, x_s: y as E4M3 codes with one E8M0 scale per 128 columns (the operand of
//   the expert GEMMs: the smallest power of two with amax <= 448 * scale).
// The sum, the mean and y stay in fp32 from the loads on; each output is rounded
// once (h and y to bf16, the codes from the fp32 y and not from its bf16 rounding).
//
// HBM-bound: a row is read once and kept in registers between the sum of squares
// and the outputs. A lane's vector is 8 columns, so 16 lanes hold one 128-column
// block and its amax is a 16-lane butterfly.
#include "device_common.h"
#include "host_internal.h"
#include "lane_reduce.h"

namespace moe {
namespace {

__device__ __forceinline__ void unpack8(const v4i raw, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float((uint32_t)raw[i] << 16);
    v[2 * i + 1] = __uint_as_float((uint32_t)raw[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ v4i pack8(const float (&v)[8]) {
  v4i r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (int)bf16_pack2(v[2 * i], v[2 * i + 1]);
  return r;
}

// 8 norm weights of vector `vec`, bf16 or fp32.
template <bool WF32>
__device__ __forceinline__ void load_weight8(const void* w, int vec, float (&v)[8]) {
  if constexpr (WF32) {
    const v4f a = reinterpret_cast<const v4f*>(w)[2 * vec], b = reinterpret_cast<const v4f*>(w)[2 * vec + 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    unpack8(reinterpret_cast<const v4i*>(w)[vec], v);
  }
}

// Sum over a workgroup of WAVES waves of N values per thread, the same in every thread:
// lane reductions, then the waves' sums in wave order.
template <int WAVES, int N>
__device__ __forceinline__ void block_sum(float (&s)[N], float* red) {
#pragma unroll
  for (int n = 0; n < N; ++n) s[n] = row_sum<64>(s[n]);
  if constexpr (WAVES == 1) return;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int n = 0; n < N; ++n) red[(threadIdx.x >> 6) * N + n] = s[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    s[n] = red[n];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s[n] += red[w * N + n];
  }
}

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;   // optional
  const void* w;
  uint16_t* h;           // optional; may be res
  uint16_t* y;           // optional; may be x
  uint8_t* x_q;          // optional, with x_s
  uint8_t* x_s;
  int H;
  float eps;
};

// One workgroup per row; thread t holds vectors t, t + THREADS, ... (VPT of them, the
// last ones past H / 8 empty).
template <int THREADS, int VPT, bool WF32>
__global__ __launch_bounds__(THREADS) void k_add_norm(NormArgs a) {
  __shared__ float red[THREADS / 64];
  const int nv = a.H / 8, tid = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * a.H;
  float h[VPT][8], s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vec = tid + i * THREADS;
    if (vec < nv) {
      unpack8(load16_nt(a.x + row0 + vec * 8), h[i]);
      if (a.res) {
        float r[8];
        unpack8(load16_nt(a.res + row0 + vec * 8), r);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[i][k] += r[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s[0] += h[i][k] * h[i][k];
      if (a.h) *reinterpret_cast<v4i*>(a.h + row0 + vec * 8) = pack8(h[i]);
    }
  }
  block_sum<THREADS / 64>(s, red);
  const float r = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vec = tid + i * THREADS;
    if (vec < nv) {   // H is a multiple of 128: the 16 lanes of a block agree
      float w[8];
      load_weight8<WF32>(a.w, vec, w);
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        h[i][k] = h[i][k] * r * w[k];
        amax = fmaxf(amax, fabsf(h[i][k]));
      }
      if (a.y) *reinterpret_cast<v4i*>(a.y + row0 + vec * 8) = pack8(h[i]);
      if (a.x_q) {
        amax = row_max<16>(amax);
        const int e = e8m0_exponent(amax);
        const float inv = exp2_neg(e);
        *reinterpret_cast<uint2*>(a.x_q + row0 + vec * 8) =
            make_uint2(e4m3_pack4(h[i][0] * inv, h[i][1] * inv, h[i][2] * inv, h[i][3] * inv),
                       e4m3_pack4(h[i][4] * inv, h[i][5] * inv, h[i][6] * inv, h[i][7] * inv));
        if ((tid & 15) == 0) a.x_s[(row0 + vec * 8) / 128] = (uint8_t)(e + 127);
      }
    }
  }
}

// Threads per row: four vectors each at most, so that a short row does not leave most
// of a workgroup idle (64 threads up to H 2048); eight vectors above H 8192.
template <bool WF32>
hipError_t launch_fwd(const NormArgs& a, int T, hipStream_t s) {
  const int nv = a.H / 8;
  const dim3 grid((unsigned)T);
  if (nv <= 64) hipLaunchKernelGGL((k_add_norm<64, 1, WF32>), grid, dim3(64), 0, s, a);
  else if (nv <= 256) hipLaunchKernelGGL((k_add_norm<64, 4, WF32>), grid, dim3(64), 0, s, a);
  else if (nv <= 512) hipLaunchKernelGGL((k_add_norm<128, 4, WF32>), grid, dim3(128), 0, s, a);
  else if (nv <= 1024) hipLaunchKernelGGL((k_add_norm<256, 4, WF32>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_add_norm<256, 8, WF32>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

// Gradient. With n = h r and g = dy w:
//   dx = r (g - n mean_H(g n)) + dh,   dw = sum over rows of dy n.
// mean(g n) = r mean(g h), so one pass over a row gives both sums. Each workgroup
// walks rows b, b + gridDim, ..., the next row's values on their way while a row is
// reduced, and keeps its part of dw in registers; the parts go to the workspace as
// [gridDim, H] and k_sum_parts adds them in order.
struct NormGradArgs {
  const uint16_t* dy;
  const uint16_t* h;
  const void* w;
  const uint16_t* dh;   // optional; may be dx
  uint16_t* dx;         // may be dy
  float* parts;         // [gridDim, H]
  int T, H;
  float eps;
};

template <int THREADS, int VPT, bool WF32>
__global__ __launch_bounds__(THREADS) void k_add_norm_grad(NormGradArgs a) {
  __shared__ float red[2][2 * (THREADS / 64)];   // alternating, so one barrier per row is enough
  const int nv = a.H / 8, tid = threadIdx.x;
  float dw[VPT][8] = {};
  v4i rh[VPT], ry[VPT], rd[VPT];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = tid + i * THREADS;
      if (vec < nv && t < a.T) {
        rh[i] = load16_nt(a.h + t * a.H + vec * 8);
        ry[i] = load16_nt(a.dy + t * a.H + vec * 8);
        if (a.dh) rd[i] = load16_nt(a.dh + t * a.H + vec * 8);
      }
    }
  };
  load(blockIdx.x);
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    float h[VPT][8], g[VPT][8], o[VPT][8], s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = tid + i * THREADS;
      if (vec < nv) {
        unpack8(rh[i], h[i]);
        unpack8(ry[i], g[i]);
        if (a.dh) {
          unpack8(rd[i], o[i]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) o[i][k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) s[0] += h[i][k] * h[i][k];
      }
    }
    load(t + gridDim.x);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = tid + i * THREADS;
      if (vec < nv) {
        float w[8];
        load_weight8<WF32>(a.w, vec, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[1] += g[i][k] * w[k] * h[i][k];
      }
    }
    block_sum<THREADS / 64>(s, red[turn]);
    const float r = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
    const float c = r * r * (s[1] / (float)a.H);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = tid + i * THREADS;
      if (vec < nv) {
        float w[8];
        load_weight8<WF32>(a.w, vec, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          o[i][k] += r * (g[i][k] * w[k] - h[i][k] * c);
          dw[i][k] += g[i][k] * (h[i][k] * r);
        }
        *reinterpret_cast<v4i*>(a.dx + t * a.H + vec * 8) = pack8(o[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vec = tid + i * THREADS;
    if (vec < nv) {
      v4f* dst = reinterpret_cast<v4f*>(a.parts + (int64_t)blockIdx.x * a.H + vec * 8);
      dst[0] = v4f{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
      dst[1] = v4f{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
  }
}

// Two vectors per thread at most up to H 8192 (the row, the next row and dw in
// registers), four above.
template <bool WF32>
void launch_grad(const NormGradArgs& a, int ctas, hipStream_t s) {
  const int nv = a.H / 8;
  const dim3 grid((unsigned)ctas);
  if (nv <= 128) hipLaunchKernelGGL((k_add_norm_grad<64, 2, WF32>), grid, dim3(64), 0, s, a);
  else if (nv <= 256) hipLaunchKernelGGL((k_add_norm_grad<128, 2, WF32>), grid, dim3(128), 0, s, a);
  else if (nv <= 512) hipLaunchKernelGGL((k_add_norm_grad<256, 2, WF32>), grid, dim3(256), 0, s, a);
  else if (nv <= 1024) hipLaunchKernelGGL((k_add_norm_grad<512, 2, WF32>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((k_add_norm_grad<512, 4, WF32>), grid, dim3(512), 0, s, a);
}

// out[c] = sum over p of parts[p][c], c < n: 64 columns per workgroup; each of its 16
// waves adds every 16th part, eight at a time, then their sums are added in order.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void k_sum_parts(const float* __restrict__ parts, int n_parts, int n,
                                                               float* __restrict__ out) {
  __shared__ float red[kSumWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s[8] = {};
  if (c < n)
    for (int p = wave; p < n_parts; p += 8 * kSumWaves) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = p + u * kSumWaves < n_parts ? parts[(int64_t)(p + u * kSumWaves) * n + c] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s[u] += v[u];
    }
  red[wave][lane] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  __syncthreads();
  if (wave == 0 && c < n) {
    float sum = red[0][lane];
    for (int k = 1; k < kSumWaves; ++k) sum += red[k][lane];
    out[c] = sum;
  }
}

}  // namespace

hipError_t launch_add_norm(const uint16_t* x, const uint16_t* res, const void* w, bool w_f32, uint16_t* h,
                           uint16_t* y, uint8_t* x_q, uint8_t* x_s, int T, int H, float eps, hipStream_t s) {
  const NormArgs a{x, res, w, h, y, x_q, x_s, H, eps};
  return w_f32 ? launch_fwd<true>(a, T, s) : launch_fwd<false>(a, T, s);
}

// Workgroups of the gradient: about 16 waves per CU, at most a row each.
int norm_grad_parts(int T, int H) {
  const int most = H <= 1024 ? 4096 : H <= 2048 ? 2048 : H <= 4096 ? 1024 : 512;
  return T < most ? T : most;
}

hipError_t launch_add_norm_grad(const uint16_t* dy, const uint16_t* h, const void* w, bool w_f32, const uint16_t* dh,
                                uint16_t* dx, float* dw, float* parts, int T, int H, float eps, hipStream_t s) {
  const int n = norm_grad_parts(T, H);
  if (n > 0) {
    const NormGradArgs a{dy, h, w, dh, dx, parts, T, H, eps};
    if (w_f32) launch_grad<true>(a, n, s);
    else launch_grad<false>(a, n, s);
  }
  return launch_sum_parts(parts, n, H, dw, s);
}

hipError_t launch_sum_parts(const float* parts, int n_parts, int n, float* out, hipStream_t s) {
  hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)ceil_div(n, 64)), dim3(64 * kSumWaves), 0, s, parts,
                     n_parts, n, out);
  return hipGetLastError();
}

}  // namespace moe

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

namespace moe {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWaves = kNormThreads / 64;

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

// Sum over the workgroup of N values per thread, the same in every thread: lane
// butterflies, then the waves' sums in wave order.
template <int N>
__device__ __forceinline__ void block_sum(float (&s)[N], float* red) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) s[n] += __shfl_xor(s[n], m);
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int n = 0; n < N; ++n) red[(threadIdx.x >> 6) * N + n] = s[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    s[n] = red[n];
#pragma unroll
    for (int w = 1; w < kNormWaves; ++w) s[n] += red[w * N + n];
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

// One workgroup per row; thread t holds vectors t, t + 256, ... (VPT of them, the
// last ones past H / 8 empty).
template <int VPT, bool WF32>
__global__ __launch_bounds__(kNormThreads) void k_add_norm(NormArgs a) {
  __shared__ float red[kNormWaves];
  const int nv = a.H / 8, tid = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * a.H;
  float h[VPT][8], s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vec = tid + i * kNormThreads;
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
  block_sum(s, red);
  const float r = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vec = tid + i * kNormThreads;
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
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
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

template <bool WF32>
hipError_t add_norm_by_width(const NormArgs& a, int T, hipStream_t s) {
  const int vpt = (int)ceil_div(a.H / 8, kNormThreads);
  const dim3 grid((unsigned)T), block(kNormThreads);
  if (vpt <= 1) hipLaunchKernelGGL((k_add_norm<1, WF32>), grid, block, 0, s, a);
  else if (vpt <= 2) hipLaunchKernelGGL((k_add_norm<2, WF32>), grid, block, 0, s, a);
  else if (vpt <= 4) hipLaunchKernelGGL((k_add_norm<4, WF32>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_add_norm<8, WF32>), grid, block, 0, s, a);
  return hipGetLastError();
}

// Gradient. With n = h r and g = dy w:
//   dx = r (g - n mean_H(g n)) + dh,   dw = sum over rows of dy n.
// mean(g n) = r mean(g h), so one pass over a row gives both sums. Each workgroup
// walks rows b, b + gridDim, ... and keeps its part of dw in registers; the parts
// go to the workspace as [gridDim, H] and k_sum_parts adds them in order.
struct NormGradArgs {
  const uint16_t* dy;
  const uint16_t* h;
  const void* w;
  const uint16_t* dh;   // optional; may be dx
  uint16_t* dx;
  float* parts;         // [gridDim, H]
  int T, H;
  float eps;
};

template <int VPT, bool WF32>
__global__ __launch_bounds__(kNormThreads) void k_add_norm_grad(NormGradArgs a) {
  __shared__ float red[2][2 * kNormWaves];   // alternating, so one barrier per row is enough
  const int nv = a.H / 8, tid = threadIdx.x;
  float dw[VPT][8] = {};
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    const int64_t row0 = t * a.H;
    float h[VPT][8], dy[VPT][8], s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = tid + i * kNormThreads;
      if (vec < nv) {
        unpack8(load16_nt(a.h + row0 + vec * 8), h[i]);
        unpack8(load16_nt(a.dy + row0 + vec * 8), dy[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = tid + i * kNormThreads;
      if (vec < nv) {
        float w[8];
        load_weight8<WF32>(a.w, vec, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          s[0] += h[i][k] * h[i][k];
          s[1] += dy[i][k] * w[k] * h[i][k];
        }
      }
    }
    block_sum(s, red[turn]);
    const float r = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
    const float c = r * r * (s[1] / (float)a.H);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = tid + i * kNormThreads;
      if (vec < nv) {
        float w[8], o[8] = {};
        load_weight8<WF32>(a.w, vec, w);
        if (a.dh) unpack8(load16_nt(a.dh + row0 + vec * 8), o);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          o[k] += r * (dy[i][k] * w[k] - h[i][k] * c);
          dw[i][k] += dy[i][k] * (h[i][k] * r);
        }
        *reinterpret_cast<v4i*>(a.dx + row0 + vec * 8) = pack8(o);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vec = tid + i * kNormThreads;
    if (vec < nv) {
      v4f* dst = reinterpret_cast<v4f*>(a.parts + (int64_t)blockIdx.x * a.H + vec * 8);
      dst[0] = v4f{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
      dst[1] = v4f{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
  }
}

template <bool WF32>
void add_norm_grad_by_width(const NormGradArgs& a, int ctas, hipStream_t s) {
  const int vpt = (int)ceil_div(a.H / 8, kNormThreads);
  const dim3 grid((unsigned)ctas), block(kNormThreads);
  if (vpt <= 1) hipLaunchKernelGGL((k_add_norm_grad<1, WF32>), grid, block, 0, s, a);
  else if (vpt <= 2) hipLaunchKernelGGL((k_add_norm_grad<2, WF32>), grid, block, 0, s, a);
  else if (vpt <= 4) hipLaunchKernelGGL((k_add_norm_grad<4, WF32>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_add_norm_grad<8, WF32>), grid, block, 0, s, a);
}

// out[c] = sum over p of parts[p][c], c < n: 64 columns per workgroup; each of its 16
// waves adds every 16th part, four at a time, then their sums are added in order.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void k_sum_parts(const float* __restrict__ parts, int n_parts, int n,
                                                               float* __restrict__ out) {
  __shared__ float red[kSumWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < n)
    for (int p = wave; p < n_parts; p += 4 * kSumWaves) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (p + u * kSumWaves < n_parts) s[u] += parts[(int64_t)(p + u * kSumWaves) * n + c];
    }
  red[wave][lane] = (s[0] + s[1]) + (s[2] + s[3]);
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
  return w_f32 ? add_norm_by_width<true>(a, T, s) : add_norm_by_width<false>(a, T, s);
}

int norm_grad_parts(int T) { return T < 1024 ? T : 1024; }

hipError_t launch_add_norm_grad(const uint16_t* dy, const uint16_t* h, const void* w, bool w_f32, const uint16_t* dh,
                                uint16_t* dx, float* dw, float* parts, int T, int H, float eps, hipStream_t s) {
  const int n = norm_grad_parts(T);
  if (n > 0) {
    const NormGradArgs a{dy, h, w, dh, dx, parts, T, H, eps};
    if (w_f32) add_norm_grad_by_width<true>(a, n, s);
    else add_norm_grad_by_width<false>(a, n, s);
  }
  return launch_sum_parts(parts, n, H, dw, s);
}

hipError_t launch_sum_parts(const float* parts, int n_parts, int n, float* out, hipStream_t s) {
  hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)ceil_div(n, 64)), dim3(64 * kSumWaves), 0, s, parts,
                     n_parts, n, out);
  return hipGetLastError();
}

}  // namespace moe

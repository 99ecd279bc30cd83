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
// block and its amax is a 16-lane butterfly. 32768 x 7168 with residual and all outputs
// (2.1 GB) 380 us, 5.6 TB/s; 7 x 7168 5 us, bound by the launch.
#include "device_common.h"
#include "host_internal.h"
#include "lane_reduce.h"

#include <type_traits>

namespace moe {
namespace {

typedef int v2i __attribute__((ext_vector_type(2)));

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

// A row belongs to TPR threads: 16 lanes (H up to 512), a wave, or 128, 256 or 512
// threads; a workgroup holds 256 threads' worth of rows at least.
template <int TPR>
struct Rows {
  static constexpr int kThreads = TPR > 256 ? TPR : 256;
  static constexpr int kRows = kThreads / TPR;
  static constexpr int kWaves = TPR / 64;   // of a row, where it has more than one
};

// Sums over a row's threads of N values per thread, the same in all of them: lane
// reductions, then the waves' sums in wave order. red: this row's kWaves * N floats.
// With more than one wave per row every thread of the workgroup has to call it.
template <int TPR, int N>
__device__ __forceinline__ void sum_over_row(float (&s)[N], float* red) {
#pragma unroll
  for (int n = 0; n < N; ++n) s[n] = row_sum<(TPR < 64 ? 16 : 64)>(s[n]);
  if constexpr (TPR > 64) {
    constexpr int W = Rows<TPR>::kWaves;
    const int wave = (threadIdx.x % TPR) >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) red[wave * N + n] = s[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      s[n] = red[n];
#pragma unroll
      for (int w = 1; w < W; ++w) s[n] += red[w * N + n];
    }
  }
}

// Loads and stores of the row tensors. NT: nontemporal, for tensors that the 256 MB
// last-level cache does not hold from one kernel to the next. add_norm nontemporal and
// cached, in us, three sets of tensors in turn, and in brackets with the router's product
// behind it: at H 7168 8 M elements 16 and 13 (40 and 37), 16 M 31 and 36 (59 and 61), 32 M 55
// and 61 (98 and 105), 64 M 101 and 114 (180 and 189), 235 M 382 and 390; at H 1024 8 M 14 and
// 12 (31 and 27), 16 M 26 and 31 (49 and 50), 64 M 90 and 104 (167 and 180). Its gradient:
// 8 M 26 and 20, 16 M 36 and 35, 29 M 58 and 56, 32 M 61 and 62, 64 M 106 and 112; at H 1024
// 16 M 33 and 35, 32 M 53 and 58.
template <bool NT>
__device__ __forceinline__ v4i load_row(const uint16_t* p) {
  return NT ? load16_nt(p) : load16(p);
}
template <bool NT>
__device__ __forceinline__ void store_row(uint16_t* p, const v4i v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(p));
  else *reinterpret_cast<v4i*>(p) = v;
}
constexpr int64_t kCached = 16000000, kCachedGrad = 32000000;   // elements of a row tensor

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;   // optional
  const void* w;
  uint16_t* h;           // optional; may be res
  uint16_t* y;           // optional; may be x
  uint8_t* x_q;          // optional, with x_s
  uint8_t* x_s;
  int T, H;
  float eps;
};

// Thread t of a row holds vectors t, t + TPR, ... (VPT of them, the last ones past H / 8
// empty).
template <int TPR, int VPT, bool WF32, bool NT>
__global__ __launch_bounds__(Rows<TPR>::kThreads) void k_add_norm(NormArgs a) {
  __shared__ float red[Rows<TPR>::kRows][TPR / 64 + 1];
  const int nv = a.H / 8, tid = threadIdx.x % TPR, sub = Rows<TPR>::kRows == 1 ? 0 : threadIdx.x / TPR;
  const int64_t t = (int64_t)blockIdx.x * Rows<TPR>::kRows + sub;
  const int64_t row0 = t * a.H;
  const int mine = t < a.T ? nv : 0;   // vectors of this row
  float h[VPT][8], s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vec = tid + i * TPR;
    if (vec < mine) {
      unpack8(load_row<NT>(a.x + row0 + vec * 8), h[i]);
      if (a.res) {
        float r[8];
        unpack8(load_row<NT>(a.res + row0 + vec * 8), r);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[i][k] += r[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s[0] += h[i][k] * h[i][k];
      if (a.h) store_row<NT>(a.h + row0 + vec * 8, pack8(h[i]));
    }
  }
  sum_over_row<TPR>(s, red[sub]);
  const float r = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vec = tid + i * TPR;
    if (vec < mine) {   // H is a multiple of 128: the 16 lanes of a block agree
      float w[8];
      load_weight8<WF32>(a.w, vec, w);
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        h[i][k] = h[i][k] * r * w[k];
        amax = fmaxf(amax, fabsf(h[i][k]));
      }
      if (a.y) store_row<NT>(a.y + row0 + vec * 8, pack8(h[i]));
      if (a.x_q) {
        amax = row_max<16>(amax);
        const int e = e8m0_exponent(amax);
        const float inv = exp2_neg(e);
        const v2i q{(int)e4m3_pack4(h[i][0] * inv, h[i][1] * inv, h[i][2] * inv, h[i][3] * inv),
                    (int)e4m3_pack4(h[i][4] * inv, h[i][5] * inv, h[i][6] * inv, h[i][7] * inv)};
        *reinterpret_cast<v2i*>(a.x_q + row0 + vec * 8) = q;   // 8-byte pieces: left to the L2 to merge
        if ((tid & 15) == 0) a.x_s[(row0 + vec * 8) / 128] = (uint8_t)(e + 127);
      }
    }
  }
}

// Threads per row: four vectors each at most, so that short rows share a workgroup (32768
// x 128 on 64 threads per row 14.8 us); eight vectors above H 8192.
template <bool WF32, bool NT>
void launch_fwd(const NormArgs& a, hipStream_t s) {
  auto go = [&](auto kernel, int rows) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)ceil_div(a.T, rows)), dim3(256), 0, s, a);
  };
  const int nv = a.H / 8;
  if (nv <= 16) go(k_add_norm<16, 1, WF32, NT>, 16);
  else if (nv <= 64) go(k_add_norm<16, 4, WF32, NT>, 16);
  else if (nv <= 256) go(k_add_norm<64, 4, WF32, NT>, 4);
  else if (nv <= 512) go(k_add_norm<128, 4, WF32, NT>, 2);
  else if (nv <= 1024) go(k_add_norm<256, 4, WF32, NT>, 1);
  else go(k_add_norm<256, 8, WF32, NT>, 1);
}

// Gradient. With n = h r and g = dy w:
//   dx = r (g - n mean_H(g n)) + dh,   dw = sum over rows of dy n.
// mean(g n) = r mean(g h), so one pass over a row gives both sums. A row's threads
// walk every gridDim * kRows-th row, the next row's values on their way while a row is
// reduced, and keep their part of dw in registers; the parts of a workgroup are added
// through LDS, go to the workspace as [gridDim, H], and k_sum_parts adds them in order.
// 4099 x 7168 (235 MB) 51-53 us, 4.5 TB/s, and 5 us for the parts.
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

// Up to two vectors per thread 128 registers, so that 16 waves share a CU.
template <int TPR, int VPT, bool WF32, bool NT>
__global__ __launch_bounds__(Rows<TPR>::kThreads, VPT <= 2 ? 4 : 2) void k_add_norm_grad(NormGradArgs a) {
  constexpr int kRows = Rows<TPR>::kRows;
  __shared__ float red[2][kRows][2 * (TPR / 64) + 1];   // alternating, so one barrier per row is enough
  extern __shared__ float dw_rows[];                    // [kRows, H] where kRows > 1
  const int nv = a.H / 8, tid = threadIdx.x % TPR, sub = Rows<TPR>::kRows == 1 ? 0 : threadIdx.x / TPR;
  const int64_t stride = (int64_t)gridDim.x * kRows;
  float dw[VPT][8] = {};
  v4i rh[VPT], ry[VPT], rd[VPT];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = tid + i * TPR;
      if (vec < nv && t < a.T) {
        rh[i] = load_row<NT>(a.h + t * a.H + vec * 8);
        ry[i] = load_row<NT>(a.dy + t * a.H + vec * 8);
        if (a.dh) rd[i] = load_row<NT>(a.dh + t * a.H + vec * 8);
      }
    }
  };
  load((int64_t)blockIdx.x * kRows + sub);
  int turn = 0;
  // every row of a workgroup takes part in each turn, those past the end without vectors
  for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < a.T; t0 += stride, turn ^= 1) {
    const int64_t t = t0 + sub;
    const int mine = kRows == 1 || t < a.T ? nv : 0;
    v4i ch[VPT], cy[VPT], cd[VPT];   // this row, unpacked where it is used
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      ch[i] = rh[i];
      cy[i] = ry[i];
      cd[i] = rd[i];
      const int vec = tid + i * TPR;
      if (vec < mine) {
        float h[8];
        unpack8(ch[i], h);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[0] += h[k] * h[k];
      }
    }
    load(t + stride);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = tid + i * TPR;
      if (vec < mine) {
        float w[8], h[8], g[8];
        load_weight8<WF32>(a.w, vec, w);
        unpack8(ch[i], h);
        unpack8(cy[i], g);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[1] += g[k] * w[k] * h[k];
      }
    }
    sum_over_row<TPR>(s, red[turn][sub]);
    const float r = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
    const float c = r * r * (s[1] / (float)a.H);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = tid + i * TPR;
      if (vec < mine) {
        float w[8], h[8], g[8], o[8] = {};
        load_weight8<WF32>(a.w, vec, w);
        unpack8(ch[i], h);
        unpack8(cy[i], g);
        if (a.dh) unpack8(cd[i], o);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          o[k] += r * (g[k] * w[k] - h[k] * c);
          dw[i][k] += g[k] * (h[k] * r);
        }
        store_row<NT>(a.dx + t * a.H + vec * 8, pack8(o));
      }
    }
  }
  float* part = a.parts + (int64_t)blockIdx.x * a.H;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vec = tid + i * TPR;
    if (vec < nv) {
      v4f* dst = reinterpret_cast<v4f*>((kRows > 1 ? dw_rows + sub * a.H : part) + vec * 8);
      dst[0] = v4f{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
      dst[1] = v4f{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
  }
  if constexpr (kRows > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < a.H; c += Rows<TPR>::kThreads) {
      float v = dw_rows[c];
#pragma unroll
      for (int k = 1; k < kRows; ++k) v += dw_rows[k * a.H + c];
      part[c] = v;
    }
  }
}

// Rows of a workgroup by width: two vectors per thread at most up to H 8192 (the row,
// the next row and dw in registers), four above.
inline int grad_rows(int H) { return H <= 256 ? 16 : H <= 1024 ? 4 : H <= 2048 ? 2 : 1; }

template <bool WF32, bool NT>
void launch_grad(const NormGradArgs& a, int ctas, hipStream_t s) {
  const int nv = a.H / 8, rows = grad_rows(a.H);
  auto go = [&](auto kernel, int threads) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)ctas), dim3(threads), rows > 1 ? sizeof(float) * rows * a.H : 0, s, a);
  };
  if (nv <= 16) go(k_add_norm_grad<16, 1, WF32, NT>, 256);
  else if (nv <= 32) go(k_add_norm_grad<16, 2, WF32, NT>, 256);
  else if (nv <= 64) go(k_add_norm_grad<64, 1, WF32, NT>, 256);
  else if (nv <= 128) go(k_add_norm_grad<64, 2, WF32, NT>, 256);
  else if (nv <= 256) go(k_add_norm_grad<128, 2, WF32, NT>, 256);
  else if (nv <= 512) go(k_add_norm_grad<256, 2, WF32, NT>, 256);
  else if (nv <= 1024) go(k_add_norm_grad<512, 2, WF32, NT>, 512);
  else go(k_add_norm_grad<512, 4, WF32, NT>, 512);
}

// f<weights fp32, past the cache>()
template <typename F>
void by_kind(bool w_f32, bool nt, F f) {
  if (w_f32) {
    if (nt) f(std::true_type{}, std::true_type{});
    else f(std::true_type{}, std::false_type{});
  } else {
    if (nt) f(std::false_type{}, std::true_type{});
    else f(std::false_type{}, std::false_type{});
  }
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

__global__ __launch_bounds__(256) void k_fill_zero(int32_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

}  // namespace

hipError_t launch_add_norm(const uint16_t* x, const uint16_t* res, const void* w, bool w_f32, uint16_t* h,
                           uint16_t* y, uint8_t* x_q, uint8_t* x_s, int T, int H, float eps, hipStream_t s) {
  const NormArgs a{x, res, w, h, y, x_q, x_s, T, H, eps};
  by_kind(w_f32, (int64_t)T * H > kCached, [&](auto f, auto nt) { launch_fwd<decltype(f)::value, decltype(nt)::value>(a, s); });
  return hipGetLastError();
}

// Workgroups of the gradient: about 16 waves per CU, at most a turn of rows each.
int norm_grad_parts(int T, int H) {
  const int64_t most = H > 4096 ? 512 : 1024, turns = ceil_div(T, grad_rows(H));
  return (int)(turns < most ? turns : most);
}

hipError_t launch_add_norm_grad(const uint16_t* dy, const uint16_t* h, const void* w, bool w_f32, const uint16_t* dh,
                                uint16_t* dx, float* dw, float* parts, int T, int H, float eps, hipStream_t s) {
  const int n = norm_grad_parts(T, H);
  if (n > 0) {
    const NormGradArgs a{dy, h, w, dh, dx, n == 1 ? dw : parts, T, H, eps};   // one part is the result
    by_kind(w_f32, (int64_t)T * H > kCachedGrad,
            [&](auto f, auto nt) { launch_grad<decltype(f)::value, decltype(nt)::value>(a, n, s); });
  }
  return n == 1 ? hipGetLastError() : launch_sum_parts(parts, n, H, dw, s);
}

hipError_t launch_fill_zero(int32_t* p, int64_t n, hipStream_t s) {
  const int64_t ctas = ceil_div(n, 256);
  hipLaunchKernelGGL(k_fill_zero, dim3((unsigned)(ctas < 2048 ? ctas : 2048)), dim3(256), 0, s, p, n);
  return hipGetLastError();
}

hipError_t launch_sum_parts(const float* parts, int n_parts, int n, float* out, hipStream_t s) {
  hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)ceil_div(n, 64)), dim3(64 * kSumWaves), 0, s, parts,
                     n_parts, n, out);
  return hipGetLastError();
}

}  // namespace moe

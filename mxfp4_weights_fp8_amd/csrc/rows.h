// What the kernels that walk whole rows of activations share: vectors of 8 columns, and
// grids of more threads than one grid dimension takes.
#pragma once

#include "device_common.h"
#include "host_internal.h"

namespace moe {

__device__ __forceinline__ void unpack8(const v4i raw, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float((uint32_t)raw[i] << 16);
    v[2 * i + 1] = __uint_as_float((uint32_t)raw[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ v4i pack8(const float (&v)[8]) {
  return v4i{(int)bf16_pack2(v[0], v[1]), (int)bf16_pack2(v[2], v[3]), (int)bf16_pack2(v[4], v[5]),
             (int)bf16_pack2(v[6], v[7])};
}
// 8 E4M3 codes times 2^e in fp32 (exact for every scale that a finite block takes).
__device__ __forceinline__ void decode8(const uint2 q, int e, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int word = (int)(k ? q.y : q.x);
    v[4 * k] = __builtin_amdgcn_ldexpf(__builtin_amdgcn_cvt_f32_fp8(word, 0), e);
    v[4 * k + 1] = __builtin_amdgcn_ldexpf(__builtin_amdgcn_cvt_f32_fp8(word, 1), e);
    v[4 * k + 2] = __builtin_amdgcn_ldexpf(__builtin_amdgcn_cvt_f32_fp8(word, 2), e);
    v[4 * k + 3] = __builtin_amdgcn_ldexpf(__builtin_amdgcn_cvt_f32_fp8(word, 3), e);
  }
}

// Stores of rows. NT: nontemporal, for tensors that the caches do not hold until the next
// kernel reads them. A layer's forward and backward pass at hidden 7168, top-8, nontemporal
// and cached: 64 tokens 298 and 276 us, 256 (15 M elements of rows) 579 and 570, 512 872 and
// 891, 1024 1085 and 1115; the kernels alone at 32K tokens: rows by expert 777 and 806, back
// 716 and 777, the gradient at 8K 389 and 400.
constexpr int64_t kCachedRows = 16000000;   // elements
template <bool NT>
__device__ __forceinline__ void store_row(uint16_t* p, const v4i v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(p));
  else *reinterpret_cast<v4i*>(p) = v;
}

// A grid dimension holds fewer than 2^32 threads, a tensor of long rows more groups of 8
// columns than that: workgroups are counted over x and y.
inline dim3 grid_of_blocks(int64_t n) {
  const int64_t x = n < (1 << 20) ? n : 1 << 20;
  return dim3((unsigned)x, (unsigned)ceil_div(n, x));
}
__device__ __forceinline__ int64_t block_id() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

}  // namespace moe

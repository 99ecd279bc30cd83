// Staging the operands of the tiled dense products in LDS: the direct-to-LDS copies of
// one step (64 of the contraction index) and the fragment reads.
//
// An operand stored [rows, C] is staged as 128-byte rows, 16-byte chunks XORed by a
// function of the row (the 8 or 16 lanes that LDS serves together then hit every bank
// once), and a fragment is one ds_read_b128 per lane. One stored [C, rows] is staged as
// 64 rows of the contraction, and a fragment is two ds_read_b64_tr_b16: lane
// (4i + g, q) reads columns 4g .. 4g+3 of contraction row 8q + i (then 8q + 4 + i), and
// the transpose within 16 lanes leaves lane c with four contraction values of column c.
// The 16 rows of a read lie a multiple of 128 bytes apart, so 32-byte blocks are XORed
// by a function of the row that spreads them over the banks.
//
// Copies past an operand's end, or past this workgroup's share of the contraction, are
// zeros from the buffer resource's bounds check. A transposed operand's columns past
// its last one are the next row's values: they only reach outputs that are not stored.
#pragma once

#include "device_common.h"
#include "lds_copy.h"

namespace moe {

typedef short v4h __attribute__((ext_vector_type(4)));

// One operand's steps: ROWS tile rows (columns of the result for w).
template <int ROWS, bool TRANS>
struct Operand {
  static constexpr int kBytes = ROWS * 128;         // a stage
  static constexpr int kCopies = kBytes / 4096;     // per wave and step
  static constexpr int kRow = 2 * ROWS;             // bytes of a transposed stage's row
  static constexpr int kMask = kRow % 256 == 0 ? 7 : 3;   // 32-byte blocks that are XORed together

  const char* base;    // first byte of step 0
  int64_t step;        // bytes per step
  int64_t left;        // bytes from `base` to the operand's end (the tile's, for [rows, C])
  int row_bytes;
  int voff[kCopies];   // of this lane's 16 bytes, relative to the step

  // XOR of a transposed stage's blocks in contraction row r: the rows 8q + i of a read
  // differ in i = r % 4 and q
  __device__ static int xor_of(int r) {
    return kMask == 7 ? (r & 3) | ((r >> 3 & 1) << 2) : (r >> 1 & 1) | ((r >> 3 & 1) << 1);
  }
  // XOR of the chunks of row r
  __device__ static int chunk_xor(int r) { return (r >> 1 & 7) ^ ((r & 1) << 2); }

  // tile rows from `first` on, of `rows` (contraction index below C)
  __device__ void place(const uint16_t* p, int64_t stride, int first, int rows, int C) {
    if constexpr (TRANS) {
      base = reinterpret_cast<const char*>(p + first);
      left = (int64_t)C * row_bytes - 2 * first;
    } else {
      base = reinterpret_cast<const char*>(p + first * stride);
      left = (int64_t)min(ROWS, rows - first) * row_bytes;
    }
  }
  __device__ void init(int64_t stride, int wave, int lane) {
    row_bytes = (int)(2 * stride);
    step = TRANS ? (int64_t)64 * row_bytes : 128;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int b = (kCopies * wave + i) * 1024 + lane * 16;   // byte of the stage that this lane fills
      if constexpr (TRANS) {
        const int r = b / kRow, chunk = b % kRow / 16;
        voff[i] = r * row_bytes + ((chunk ^ (xor_of(r) << 1)) << 4);
      } else {
        const int r = b / 128, chunk = b % 128 / 16;
        voff[i] = r * row_bytes + ((chunk ^ chunk_xor(r)) << 4);
      }
    }
  }
  // the buffer resource of step s, `shift` bytes behind it; size 0 unless it is `wanted`
  __device__ v4i_s rsrc(int s, bool wanted, int shift = 0) const {
    const int64_t at = s * step + shift;
    int64_t bytes = left - at;
    const int64_t most = (int64_t)(TRANS ? 64 : ROWS) * row_bytes;   // keeps the size in 32 bits
    bytes = bytes < 0 ? 0 : bytes > most ? most : bytes;
    return rsrc4(base + at, wanted ? (uint32_t)bytes : 0u);
  }
  __device__ void copy(v4i_s r, uint8_t* stage, int wave, int i) const {
    dma16(r, lds_addr(stage + (kCopies * wave + i) * 1024), voff[i], 0);
  }
};

// A lane's view of the fragments of a stage: fragment f is 16 tile rows from 16 f on,
// half h the contraction index's 32 h .. 32 h + 31.
template <int ROWS, bool TRANS>
struct FragReader {
  int lane_off[2], x;
  __device__ void init(int lane) {
    const int c = lane & 15, q = lane >> 4;
    if constexpr (TRANS) {
      const int r = 8 * q + (c >> 2);
      lane_off[0] = r * 2 * ROWS + 8 * (c & 3);
      lane_off[1] = lane_off[0] + 32 * 2 * ROWS;
      x = Operand<ROWS, true>::xor_of(r);   // the same for r + 4 and r + 32
    } else {
      const int sw = Operand<ROWS, false>::chunk_xor(c);
      lane_off[0] = c * 128 + ((q ^ sw) << 4);
      lane_off[1] = c * 128 + (((4 + q) ^ sw) << 4);
      x = 0;
    }
  }
  template <int H>
  __device__ v4i read(const uint8_t* stage, int f) const {
    if constexpr (TRANS) {
      typedef __attribute__((address_space(3))) v4h* lds4;
      const uint8_t* p = stage + lane_off[H] + ((f ^ x) << 5);
      const v4h lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p);
      const v4h hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 4 * 2 * ROWS));
      const int2 a = __builtin_bit_cast(int2, lo), b = __builtin_bit_cast(int2, hi);
      return v4i{a.x, a.y, b.x, b.y};
    } else {
      return *reinterpret_cast<const v4i*>(stage + lane_off[H] + f * 2048);
    }
  }
};

}  // namespace moe

// Shared device helpers of the MXFP4 kernels (4-bit microscaling floats, gfx950).
//
// Format (Open Compute Project, "OCP Microscaling Formats (MX) Specification v1.0",
// sections 5.2 and 6.3): 32 consecutive input channels share one E8M0 scale byte b,
// 2^(b - 127), b = 255 meaning NaN; an element is e2m1: sign in bit 3, magnitude code
// 0..7 = 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Eight codes per uint32, the first channel in the
// lowest nibble.  The 32 codes of a block are 16 bytes: what one lane holds of a
// v_mfma_scale_f32_16x16x128_f8f6f4 operand, with the block's byte as its scale.
#pragma once

#include "internal.hpp"

namespace w4 {

constexpr int kMxBlock = 32;                 // channels per shared scale
// Longest K of the products: a tile of up to 256 rows of 2-byte activations stays
// below 2^31 bytes, the range of a buffer descriptor's 32-bit offsets used here.
constexpr int kMxMaxK = 1 << 21;
// Most rows and channels of the products: a tile's last row index is still an int.
constexpr int kMxMaxRows = 0x7FFFFFFF - 1023;
// Most threads along one dimension of a grid (its size in work items is a 32-bit field).
constexpr long long kMaxGridThreads = 0xFFFFFFFFLL;
// Most elements of one conversion: a thread takes eight.
constexpr long long kMxMaxElements = (kMaxGridThreads - 255) / 256 * 256 * 8;

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4;
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16p __attribute__((ext_vector_type(2)));

// fp32 with the scale byte as its exponent field: the conversion instructions read the
// scale from there (0 -> 2^-127, 255 -> NaN), checked on the GPU for all 256 bytes.
__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// The four pairs of one packed word as bf16, times the scale: exact (a 2-bit
// significand and a power of two), except that magnitudes past bf16's range (bytes 253
// and 254) become infinite.
__device__ __forceinline__ bf16x8 mx_expand(uint32_t w, float scale) {
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return __builtin_bit_cast(bf16x8, r);
}

// Position of chunk 0 in row r (0..15) of 256-byte LDS rows read as operands: lane (r, q) reads
// chunk 4 q + v of row r, 16 bytes, and an LDS pass takes lanes 0-3, 12-15, 20-27 (then 4-11,
// 16-19, 28-31, and the same of the upper half), so that rows 4-11 meet the other rows' chunk
// with bit 2 flipped: flipped back, the pass covers 16 positions.
__device__ __forceinline__ int mx_swizzle16(int r) { return r ^ ((((r >> 2) ^ (r >> 3)) & 1) << 2); }

// 16 bytes of e2m1 codes as a matrix operand (the upper half of the register group is
// not read for 4-bit elements).
__device__ __forceinline__ i32x8 mx_operand(u32x4 w) {
  return i32x8{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
}

}  // namespace w4

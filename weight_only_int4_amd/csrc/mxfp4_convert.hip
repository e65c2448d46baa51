// MXFP4 quantization of v = W diag(s) and its inverse.
//
// Per block of 32 channels: A = max |v|, shared byte = exponent field of A minus 2 (the
// largest e2m1 magnitude has exponent 2), at least 0; 255 if A is infinite or NaN.
// Codes are v / 2^(byte - 127) rounded to the nearest e2m1 value, ties to the even
// code, saturating at 6.  v is the bf16 weight, or the fp32 product with s.
//
// A block is four lanes of eight channels: 16-byte loads and 4-byte stores of
// consecutive lanes are consecutive in memory, the maximum is two quad permutes, and
// the rounding is the hardware's conversion (equal to the definition in the tests: every
// bf16 value at every scale, and fp32 values next to each border between magnitudes, at every
// scale and below).  A thread takes one chunk, no loop: bound by
// HBM traffic.  17408 x 5120 with s, 226 MB read and written: 38.6 us, 5.9 TB/s, from the caches where
// the weight fits them, 52.3 us (4.3 TB/s) from HBM (a large copy: 4.9 TB/s); the way back 32.4 and 42.7 us
// (5.3 TB/s).  16 x 2048 takes 2.2 us, as long as an empty kernel.
#include "mxfp4.hpp"

#pragma clang fp contract(off)

namespace w4 {
namespace {

// Maximum over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true));   // lane ^ 1
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true));   // lane ^ 2
}

template <bool SCALED>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const uint4* W, size_t chunks, int row_chunks, const float4* s,
                                                          uint32_t* codes, uint8_t* scales) {
  // chunks is a multiple of 4, so the lanes of a quad take the branch together
  const size_t c = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= chunks) return;
  const uint4 d = W[c];
  const uint32_t w[4] = {d.x, d.y, d.z, d.w};
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  if constexpr (SCALED) {
    const size_t k = c % (size_t)row_chunks;
    const float4 a = s[2 * k], b = s[2 * k + 1];
    v[0] *= a.x; v[1] *= a.y; v[2] *= a.z; v[3] *= a.w;
    v[4] *= b.x; v[5] *= b.y; v[6] *= b.z; v[7] *= b.w;
  }
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  const int e = (int)(quad_max(am) >> 23);
  const uint32_t byte = e == 255 ? 255u : (uint32_t)max(e - 2, 0);
  const float scale = mx_scale(byte);
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], scale, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], scale, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], scale, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], scale, 3);
  codes[c] = byte == 255u ? 0u : q;
  if ((threadIdx.x & 3) == 0) scales[c >> 2] = (uint8_t)byte;
}

__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint32_t* codes, const uint8_t* scales, size_t chunks,
                                                            uint4* W) {
  const size_t c = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= chunks) return;
  W[c] = __builtin_bit_cast(uint4, mx_expand(codes[c], mx_scale(scales[c >> 2])));
}

}  // namespace

int launch_mxfp4_quantize(const uint16_t* W, int N, int K, const float* s, uint32_t* codes, uint8_t* scales,
                          hipStream_t stream) {
  const size_t chunks = (size_t)N * (K / 8);
  const size_t blocks = (chunks + 255) / 256;   // kMxMaxElements bounds it
  const uint4* w = reinterpret_cast<const uint4*>(W);
  if (s)
    hipLaunchKernelGGL(mx_quantize_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, stream, w, chunks, K / 8,
                       reinterpret_cast<const float4*>(s), codes, scales);
  else
    hipLaunchKernelGGL(mx_quantize_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, stream, w, chunks, K / 8,
                       static_cast<const float4*>(nullptr), codes, scales);
  W4_CHECK_LAUNCH();
  return W4_OK;
}

int launch_mxfp4_dequantize(const uint32_t* codes, const uint8_t* scales, int N, int K, uint16_t* W,
                            hipStream_t stream) {
  const size_t chunks = (size_t)N * (K / 8);
  const size_t blocks = (chunks + 255) / 256;
  hipLaunchKernelGGL(mx_dequantize_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, codes, scales, chunks,
                     reinterpret_cast<uint4*>(W));
  W4_CHECK_LAUNCH();
  return W4_OK;
}

}  // namespace w4

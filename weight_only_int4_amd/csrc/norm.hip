// The residual's addition and the root-mean-square norm, out in bf16 (w4_rmsnorm) or as the
// int8 activations of the W4A8 linears (w4a8_rmsnorm).
//   h = bf16(x + residual), r = 1 / sqrt(mean h^2 + eps);  y = bf16((h r) w);
//   v = fp32(h w), t = max |v| fp32(1/127), codes = clamp(rint(v / t)), sx = t r.
// r > 0 is common to a row's values, so rint(127 y / max |y|) does not depend on it: taking
// the codes from v keeps them exact (v is, both factors having 8-bit significands), while r,
// whose last bit depends on the order of a sum, enters the scale alone.
//
// What bounds it: a few rows the launch (int8, 1 x 2,048: 3.1 us in the kernel, a round trip to memory and two
// barriers); many rows the memory (int8, 8,191 x 5,120 with a residual: 294 MB in 65 to 70 us, 4.5 to 4.2 TB/s; 4,096 x
// 2,048 in bf16: 67 MB in 11.6 to 12.2 us, part of it from the caches).
#include "serve.hpp"

#pragma clang fp contract(off)

namespace w4 {

namespace {

constexpr int kMostThreads = 1024;
constexpr float kStep = 1.0f / 127.0f;

__device__ __forceinline__ int row16_sum(int v) {
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// 2^e, e from -126 to 127
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// One workgroup per row of as many waves as CH chunks of 8 channels a thread leave work for (H = 5,120: five
// waves, two chunks), so that the row is read once, held, and no lane idles.
template <int CH, bool INT8>
__global__ __launch_bounds__(kMostThreads) void norm_kernel(const uint16_t* X, const uint16_t* R, int H,
                                                            const uint16_t* __restrict__ w, float eps, uint16_t* hout,
                                                            uint16_t* Y, int8_t* Xq, float* sx, int32_t* xsum) {
  __shared__ float red[2][kMostThreads / kWave];
  const size_t row = blockIdx.x;
  const int tid = threadIdx.x, threads = blockDim.x, waves = threads >> 6, chunks = H >> 3;
  uint4 hv[CH];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * threads;
    hv[i] = make_uint4(0u, 0u, 0u, 0u);
    if (c >= chunks) continue;
    hv[i] = *reinterpret_cast<const uint4*>(X + row * H + 8 * c);
    uint32_t* d = reinterpret_cast<uint32_t*>(&hv[i]);
    if (R) {
      const uint4 rv = *reinterpret_cast<const uint4*>(R + row * H + 8 * c);
      const uint32_t e[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bf16x2 s = {(__bf16)(__uint_as_float(d[q] << 16) + __uint_as_float(e[q] << 16)),
                          (__bf16)(__uint_as_float(d[q] & 0xFFFF0000u) + __uint_as_float(e[q] & 0xFFFF0000u))};
        d[q] = __builtin_bit_cast(uint32_t, s);
      }
      *reinterpret_cast<uint4*>(hout + row * H + 8 * c) = hv[i];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float a = __uint_as_float(d[q] << 16), b = __uint_as_float(d[q] & 0xFFFF0000u);
      ss = ss + a * a;
      ss = ss + b * b;
    }
  }
  auto row_sum = [&](float v) {
    v = wave_sum(v);
    if ((tid & 63) == 0) red[0][tid >> 6] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < waves; ++i) v = v + red[0][i];
    return v;
  };
  auto row_max = [&](uint32_t v) {            // of bit patterns of values without a sign: NaN counts as the largest
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, kWave));
    if ((tid & 63) == 0) red[1][tid >> 6] = __uint_as_float(v);
    __syncthreads();
    v = 0u;
    for (int i = 0; i < waves; ++i) v = max(v, __float_as_uint(red[1][i]));
    return v;
  };
  const float mean = row_sum(ss) / (float)H + eps;
  float r = 1.0f / sqrtf(mean);
  // Squares overflow from 2^64 on and lose bits below 2^-63 (at most 2^-149 each, which a mean of 2^-100 does not feel).
  // The sum of such a row is formed again, of its values times 2^-k, k from the largest of them and eps, and r is
  // then that of the scaled row.  The mean is the same in all threads.  (4,096 x 2,048 in bf16: 12.7 us without the
  // branch, 13.0 with it, not taken; int8 1 x 2,048: 3.7 and 3.8.)
  int k = 0;
  bool scaled = false;
  if (__builtin_expect(!(mean >= 0x1p-100f && mean < INFINITY), 0)) {
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      for (int q = 0; q < 4; ++q) {
        const uint32_t d = reinterpret_cast<const uint32_t*>(&hv[i])[q];
        top = max(top, max(d << 16 & 0x7FFF0000u, d & 0x7FFF0000u));
      }
    top = row_max(top);
    scaled = top < 0x7F800000u;
    if (scaled) {
      k = min(max((int)(__float_as_uint(fmaxf(__uint_as_float(top), sqrtf(eps))) >> 23) - 127, -126), 126);
      const float down = power_of_two(-k);
      ss = 0.0f;
#pragma unroll
      for (int i = 0; i < CH; ++i)
        for (int q = 0; q < 4; ++q) {
          const uint32_t d = reinterpret_cast<const uint32_t*>(&hv[i])[q];
          const float a = __uint_as_float(d << 16) * down, b = __uint_as_float(d & 0xFFFF0000u) * down;
          ss = ss + a * a;
          ss = ss + b * b;
        }
      r = 1.0f / sqrtf(row_sum(ss) / (float)H + eps * down * down);
    }
  }
  if constexpr (!INT8) {
    const float down = power_of_two(-k);      // 1 but for scaled rows
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * threads;
      if (c >= chunks) continue;
      const uint4 wv = *reinterpret_cast<const uint4*>(w + 8 * c);
      const uint32_t d[4] = {hv[i].x, hv[i].y, hv[i].z, hv[i].w}, e[4] = {wv.x, wv.y, wv.z, wv.w};
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float a = __uint_as_float(d[q] << 16) * down, b = __uint_as_float(d[q] & 0xFFFF0000u) * down;
        const bf16x2 y = {(__bf16)((a * r) * __uint_as_float(e[q] << 16)),
                          (__bf16)((b * r) * __uint_as_float(e[q] & 0xFFFF0000u))};
        o[q] = __builtin_bit_cast(uint32_t, y);
      }
      *reinterpret_cast<uint4*>(Y + row * H + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  } else {
    uint32_t top = 0u;                        // max |v|
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * threads;
      if (c >= chunks) continue;
      const uint4 wv = *reinterpret_cast<const uint4*>(w + 8 * c);
      const uint32_t d[4] = {hv[i].x, hv[i].y, hv[i].z, hv[i].w}, e[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        top = max(top, __float_as_uint(__uint_as_float(d[q] << 16) * __uint_as_float(e[q] << 16)) & 0x7FFFFFFFu);
        top = max(top, __float_as_uint(__uint_as_float(d[q] & 0xFFFF0000u) * __uint_as_float(e[q] & 0xFFFF0000u)) &
                           0x7FFFFFFFu);
      }
    }
    top = row_max(top);
    const bool finite = top < 0x7F800000u;
    const float step = __uint_as_float(top) * kStep, t = step > 0.0f ? step : 1.0f;     // (0: of a zero row, or by underflow)
    // Eight divisions a chunk are 75 us at 8,191 x 5,120, eight products 70.  v / t by the reciprocal is off by less
    // than 2^-15 (values to 127, three roundings of 2^-24), so where it lies 2^-14 or more from a half it rounds as the
    // quotient does; the others, and steps so small that the reciprocal might overflow, are divided.
    const float inv = 1.0f / t, far = t >= 0x1p-100f ? 1.0f : 0.0f;
    if (tid == 0) {
      // (a scaled row's r 2^-k in two factors: neither leaves the range where t r stays in it)
      const float product = scaled ? (t * power_of_two(-(k / 2))) * (r * power_of_two(k / 2 - k)) : t * r;
      sx[row] = finite ? product : __uint_as_float(0x7FC00000u);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * threads;
      int part = 0;
      if (c < chunks) {
        const uint4 wv = *reinterpret_cast<const uint4*>(w + 8 * c);
        const uint32_t d[4] = {hv[i].x, hv[i].y, hv[i].z, hv[i].w}, e[4] = {wv.x, wv.y, wv.z, wv.w};
        float v[8], q[8], near = far;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t x = (j & 1) ? (d[j >> 1] & 0xFFFF0000u) : (d[j >> 1] << 16);
          const uint32_t y = (j & 1) ? (e[j >> 1] & 0xFFFF0000u) : (e[j >> 1] << 16);
          v[j] = __uint_as_float(x) * __uint_as_float(y);
          const float z = v[j] * inv;
          q[j] = __builtin_rintf(z);
          near = fminf(near, 0.5f - fabsf(z - q[j]));
        }
        if (!(near > 0x1p-14f)) {
#pragma unroll
          for (int j = 0; j < 8; ++j) q[j] = fminf(fmaxf(__builtin_rintf(v[j] / t), -127.0f), 127.0f);
        }
        uint32_t packed[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t lo = __builtin_amdgcn_perm((uint32_t)(int)q[4 * p + 1], (uint32_t)(int)q[4 * p], 0x0C0C0400u);
          const uint32_t hi = __builtin_amdgcn_perm((uint32_t)(int)q[4 * p + 3], (uint32_t)(int)q[4 * p + 2], 0x04000C0Cu);
          packed[p] = finite ? lo | hi : 0u;
          part = __builtin_amdgcn_sdot4((int)packed[p], 0x01010101, part, false);
        }
        *reinterpret_cast<uint2*>(Xq + row * H + 8 * c) = make_uint2(packed[0], packed[1]);
      }
      part = row16_sum(part);                       // 16 lanes x 8 channels: one group
      if ((tid & 15) == 0 && c < chunks) xsum[row * (H >> 7) + (c >> 4)] = part;
    }
  }
}

template <int CH>
void launch(const NormArgs& a, hipStream_t st) {
  const int threads = ((a.H / 8 + CH - 1) / CH + kWave - 1) / kWave * kWave;
  if (a.Xq)
    hipLaunchKernelGGL((norm_kernel<CH, true>), dim3(a.T), dim3(threads), 0, st, a.X, a.residual, a.H, a.weight, a.eps,
                       a.h, a.Y, a.Xq, a.sx, a.xsum);
  else
    hipLaunchKernelGGL((norm_kernel<CH, false>), dim3(a.T), dim3(threads), 0, st, a.X, a.residual, a.H, a.weight, a.eps,
                       a.h, a.Y, a.Xq, a.sx, a.xsum);
}

}  // namespace

bool norm_fits(int T) { return (long long)T * kMostThreads <= kGridThreads; }

int launch_norm(const NormArgs& a, hipStream_t st) {
  // Few rows: as many threads as there are chunks, up to 1,024 (1 x 5,120: 4.1 us with 256 threads, 3.2; int8,
  // 16 x 17,408: 14.8 and 8.4).  Many: two chunks a thread (int8 with divisions, 8,191 x 5,120: 78 us with one, 71
  // with two, 75 with five, 82 with ten and one wave a row; 4,096 x 2,048: 13.3 with one, 12.5 with two).
  const int chunks = a.H / 8;
  if (chunks <= 1024 && a.T <= 512) launch<1>(a, st);
  else if (chunks <= 2048) launch<2>(a, st);
  else if (chunks <= 4096) launch<4>(a, st);
  else launch<8>(a, st);
  W4_CHECK_LAUNCH();
  return W4_OK;
}

}  // namespace w4

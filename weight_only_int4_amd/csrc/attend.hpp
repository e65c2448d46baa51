// Attention of one query by one wave, key by key: slow, and exact about what is not seen.  The
// attention kernels come back to it for rows whose result is not finite: there a matrix product may have
// multiplied a weight of 0 with an infinity or NaN in a value that the row does not see.  Rows that see one come here
// too.  A row of 64 keys takes 23 us, and a wave's rows go one after another: one NaN among 8,192 tokens of 16 heads of
// 128 makes a call of 0.25 ms one of 94, a decode step of 64 sequences of 2,000 tokens one of 1.0 where it takes 0.1.
#pragma once

#include <math.h>

#include "serve.hpp"

namespace w4 {

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
  return v;
}

// out = softmax(scale q . K) V over keys 0 .. n - 1; kv(key, k, v) gives a key's rows or NULL.
// 64 keys at a time, one per lane for the scores, then one after another for the product with V.
template <int HEAD, typename F>
__device__ void attend(const uint16_t* q, int n, float scale, F kv, uint16_t* out) {
  const int lane = threadIdx.x & 63;
  constexpr int PER = HEAD / kWave;                   // dims of a lane
  float m = -INFINITY, l = 0.0f, acc[PER] = {};
  bool any = false;
  for (int kb = 0; kb < n; kb += kWave) {
    const int key = kb + lane;
    const uint16_t *k = nullptr, *v = nullptr;
    if (key < n) kv(key, k, v);
    float s = -INFINITY;
    if (k) {
      s = 0.0f;
      for (int d = 0; d < HEAD; ++d) s = s + bf16_bits_to_f32(q[d]) * bf16_bits_to_f32(k[d]);
      s = s * scale;
    }
    any = any || __ballot(k != nullptr) != 0;
    const float mnew = fmaxf(m, wave_max(s));
    const float base = mnew == -INFINITY ? 0.0f : mnew;
    const float corr = expf(m - base);
    const float p = k ? expf(s - base) : 0.0f;
    l = l * corr + wave_sum(p);
    for (int i = 0; i < PER; ++i) acc[i] = acc[i] * corr;
    m = mnew;
    for (int j = 0; j < min(kWave, n - kb); ++j) {
      const uint16_t* vj = reinterpret_cast<const uint16_t*>(__shfl((unsigned long long)v, j, kWave));
      const float pj = __shfl(p, j, kWave);
      if (!vj) continue;
      for (int i = 0; i < PER; ++i) acc[i] = acc[i] + pj * bf16_bits_to_f32(vj[lane * PER + i]);
    }
  }
  for (int i = 0; i < PER; ++i) {
    const __bf16 o = any ? (__bf16)(acc[i] / l) : (__bf16)0.0f;
    out[lane * PER + i] = __builtin_bit_cast(uint16_t, o);
  }
}

}  // namespace w4

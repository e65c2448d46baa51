// Rotary embedding of new tokens' queries and keys, and the append of keys and values to the
// paged cache.
//   y_j = bf16(x_j cos - x_(j+h) sin), y_(j+h) = bf16(x_(j+h) cos + x_j sin), h half a head, at angle p base^(-j/h)
//
// What bounds it: the memory.  16 bytes a lane and turn, each pair of values rotated where it was read, both
// halves of a head by the same lane; 2,048 tokens of 8 sequences, 32 + 8 + 8 heads of 128: 46 us for 200 MB,
// 4.4 TB/s, of 4.85 that a large copy reaches.  Single tokens: the launch (16 sequences: 4.6 us).
#include <math.h>

#include "block_ops.hpp"
#include "serve.hpp"

#pragma clang fp contract(off)

namespace w4 {

namespace {

// cos / sin [P][half] of p base^(-2j / (2 half)), in fp64, stored fp32.
__global__ __launch_bounds__(256) void rope_table_kernel(long long items, int half, double base, float* cs, float* sn) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= items) return;
  const long long p = i / half;
  const int j = (int)(i - p * half);
  const double ang = (double)p * pow(base, -(double)j / half);
  cs[i] = (float)cos(ang);
  sn[i] = (float)sin(ang);
}

__device__ __forceinline__ void rotate8(const uint4& lo, const uint4& hi, const float* c, const float* s, uint4& ylo,
                                        uint4& yhi) {
  const uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
  uint32_t p[4], q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y0, y1, z0, z1;
    rope_rotate(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), c[2 * i], s[2 * i], y0, z0);
    rope_rotate(__uint_as_float(a[i] & 0xFFFF0000u), __uint_as_float(b[i] & 0xFFFF0000u), c[2 * i + 1], s[2 * i + 1],
                y1, z1);
    const bf16x2 y = {(__bf16)y0, (__bf16)y1}, z = {(__bf16)z0, (__bf16)z1};
    p[i] = __builtin_bit_cast(uint32_t, y);
    q[i] = __builtin_bit_cast(uint32_t, z);
  }
  ylo = make_uint4(p[0], p[1], p[2], p[3]);
  yhi = make_uint4(q[0], q[1], q[2], q[3]);
}

// One wave per token.  A unit is 8 pairs of a head (two 16-byte pieces, half a head apart): of
// the queries, then of the keys, then (without a turn) of the values.
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs g) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (t >= g.T) return;
  int b = t, n = 1, i = 0;
  if (g.offsets) {
    b = find_sequence(g.offsets, g.B, t);
    if (b < 0) return;
    const int first = held_offset(g.offsets[b], g.T);
    n = held_count(first, held_offset(g.offsets[b + 1], g.T));
    i = t - first;
  }
  const int p = held_position(g.lens[b], n, i, g.positions);
  if (p < 0) return;
  const int page_size = g.cache.page_size, n_kv = g.cache.n_kv, head = g.cache.head;
  const int shift = __builtin_ctz(page_size);
  const int entry = p >> shift, slot = p & (page_size - 1);
  const int page = entry < g.table_width ? held_page(g.table[(size_t)b * g.table_width + entry], g.cache.pages) : -1;
  const bool kept = page >= 0;
  const int per = head >> 4, half = head >> 1;             // units of a head, pairs of a head
  const int nq_units = g.n_q * per, nk_units = n_kv * per;
  const float* cs = g.cs + (size_t)p * half;
  const float* sn = g.sn + (size_t)p * half;
  for (int u = lane; u < nq_units + 2 * nk_units; u += kWave) {
    const bool is_q = u < nq_units, is_v = u >= nq_units + nk_units;
    const int v = is_q ? u : is_v ? u - nq_units - nk_units : u - nq_units;
    const int h = v / per, at = 8 * (v - h * per);
    const uint16_t* src = is_q ? g.Q + (size_t)t * g.q_stride
                               : is_v ? g.V + (size_t)t * g.v_stride : g.K + (size_t)t * g.k_stride;
    uint4 lo = *reinterpret_cast<const uint4*>(src + h * head + at);
    uint4 hi = *reinterpret_cast<const uint4*>(src + h * head + at + half);
    if (!is_v) rotate8(lo, hi, cs + at, sn + at, lo, hi);
    if (is_q || (!is_v && g.K_out)) {
      uint16_t* out = (is_q ? g.Q_out + (size_t)t * g.n_q * head : g.K_out + (size_t)t * n_kv * head) + h * head + at;
      *reinterpret_cast<uint4*>(out) = lo;
      *reinterpret_cast<uint4*>(out + half) = hi;
    }
    if (!is_q && kept) {
      uint16_t* out = (is_v ? g.cache.v : g.cache.k) + (((size_t)page * n_kv + h) * page_size + slot) * head + at;
      *reinterpret_cast<uint4*>(out) = lo;
      *reinterpret_cast<uint4*>(out + half) = hi;
    }
  }
}

}  // namespace

bool rope_table_fits(int positions, int head) { return (long long)positions * (head / 2) + 255 <= kGridThreads; }

int launch_rope_table(int positions, int head, double base, float* cs, float* sn, hipStream_t st) {
  const long long items = (long long)positions * (head / 2);
  hipLaunchKernelGGL(rope_table_kernel, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, st, items, head / 2, base,
                     cs, sn);
  W4_CHECK_LAUNCH();
  return W4_OK;
}

bool append_fits(int T) { return ((long long)T + 3) / 4 * 256 <= kGridThreads; }

int launch_kv_append(const AppendArgs& g, hipStream_t st) {
  hipLaunchKernelGGL(kv_append_kernel, dim3((unsigned)((g.T + 3LL) / 4)), dim3(256), 0, st, g);
  W4_CHECK_LAUNCH();
  return W4_OK;
}

}  // namespace w4

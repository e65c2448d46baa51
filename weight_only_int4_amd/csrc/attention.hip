// Causal attention of packed prompts and attention of single tokens over the paged cache: the
// plain kernels, one wave per (query, head).
#include <math.h>

#include "serve.hpp"

#pragma clang fp contract(off)

namespace w4 {

namespace {

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

template <int HEAD>
__global__ __launch_bounds__(256) void prompt_kernel(PromptArgs g) {
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= (long long)g.T * g.n_q) return;
  const int t = (int)(item / g.n_q), h = (int)(item - (long long)t * g.n_q);
  const int b = find_sequence(g.offsets, g.B, t);
  if (b < 0) return;
  const int first = token_offset(g.offsets, b, g.T);
  const size_t at = (size_t)(h / (g.n_q / g.n_kv)) * HEAD;
  attend<HEAD>(g.Q + (size_t)t * g.q_stride + (size_t)h * HEAD, t - first + 1, g.scale,
               [&](int key, const uint16_t*& k, const uint16_t*& v) {
                 k = g.K + (size_t)(first + key) * g.k_stride + at;
                 v = g.V + (size_t)(first + key) * g.v_stride + at;
               },
               g.O + ((size_t)t * g.n_q + h) * HEAD);
}

template <int HEAD>
__global__ __launch_bounds__(256) void decode_kernel(DecodeArgs g) {
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= (long long)g.B * g.n_q) return;
  const int b = (int)(item / g.n_q), h = (int)(item - (long long)b * g.n_q);
  const int n = min(max(g.lens[b], 0), g.max_len);
  const int kvh = h / (g.n_q / g.cache.n_kv);
  const int page_size = g.cache.page_size, shift = __builtin_ctz(page_size);
  attend<HEAD>(g.Q + (size_t)b * g.q_stride + (size_t)h * HEAD, n, g.scale,
               [&](int key, const uint16_t*& k, const uint16_t*& v) {
                 const size_t row = key < g.prefix_len ? 0 : (size_t)b * g.table_width;
                 const int page = g.table[row + (key >> shift)];
                 if (page < 0 || page >= g.cache.pages) return;
                 const size_t at =
                     (((size_t)page * g.cache.n_kv + kvh) * page_size + (key & (page_size - 1))) * HEAD;
                 k = g.cache.k + at;
                 v = g.cache.v + at;
               },
               g.O + ((size_t)b * g.n_q + h) * HEAD);
}

}  // namespace

size_t prompt_workspace_bytes(int T, int n_q, int n_kv, int head, int B) { return 0; }
bool prompt_fits(int T, int n_q) { return ((long long)T * n_q + 3) / 4 * 256 <= kGridThreads; }

int launch_prompt_attention(const PromptArgs& g, hipStream_t st) {
  const unsigned blocks = (unsigned)(((long long)g.T * g.n_q + 3) / 4);
  if (g.head == 64) hipLaunchKernelGGL(prompt_kernel<64>, dim3(blocks), dim3(256), 0, st, g);
  else hipLaunchKernelGGL(prompt_kernel<128>, dim3(blocks), dim3(256), 0, st, g);
  W4_CHECK_LAUNCH();
  return W4_OK;
}

size_t decode_workspace_bytes(int B, int n_q, const w4_kv_cache& cache, int max_len, int prefix_len) { return 0; }
bool decode_fits(int B, int n_q) { return ((long long)B * n_q + 3) / 4 * 256 <= kGridThreads; }

int launch_decode_attention(const DecodeArgs& g, hipStream_t st) {
  const unsigned blocks = (unsigned)(((long long)g.B * g.n_q + 3) / 4);
  if (g.cache.head == 64) hipLaunchKernelGGL(decode_kernel<64>, dim3(blocks), dim3(256), 0, st, g);
  else hipLaunchKernelGGL(decode_kernel<128>, dim3(blocks), dim3(256), 0, st, g);
  W4_CHECK_LAUNCH();
  return W4_OK;
}

}  // namespace w4

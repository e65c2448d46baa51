// Attention of single tokens over the paged cache: the plain kernel, one wave per (query, head).
#include "attend.hpp"

#pragma clang fp contract(off)

namespace w4 {

namespace {

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

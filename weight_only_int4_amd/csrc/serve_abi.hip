// C-ABI entry points of the serving operators: argument validation (host only, before any
// HIP call) and dispatch.  See include/w4a16.h for the contract.
#include <math.h>

#include "serve.hpp"

using namespace w4;

namespace {

inline bool misaligned(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int check_norm(const NormArgs& a, int multiple) {
  if (a.T < 0 || a.H <= 0 || a.H % multiple || a.H > 65536 || !norm_fits(a.T)) return W4_ERR_SHAPE;
  if (!(a.eps >= 0.0f) || isinf(a.eps)) return W4_ERR_VALUE;
  if (a.T == 0) return W4_OK;
  if (!a.X || !a.weight || (a.residual == nullptr) != (a.h == nullptr)) return W4_ERR_NULL;
  if (misaligned(a.X) || misaligned(a.residual) || misaligned(a.weight) || misaligned(a.h)) return W4_ERR_ALIGN;
  return W4_OK;
}

int check_heads(int n_q, int n_kv, int head) {
  if (head != 64 && head != 128) return W4_ERR_UNSUPPORTED;
  // a token's heads are addressed with int
  if (n_q <= 0 || n_kv <= 0 || n_q % n_kv || (long long)n_q * head > 0x7FFFFFFFLL) return W4_ERR_SHAPE;
  return W4_OK;
}

// one token of n heads every `stride` elements
int check_stride(long long stride, int n, int head) {
  return stride % 8 || stride < (long long)n * head || stride > kMaxStride ? W4_ERR_SHAPE : W4_OK;
}

int check_cache(const w4_kv_cache& c, int n_q) {
  if (int st = check_heads(n_q, c.n_kv, c.head)) return st;
  const int p = c.page_size;
  if (p != 16 && p != 32 && p != 64 && p != 128 && p != 256) return W4_ERR_UNSUPPORTED;
  return c.pages < 0 ? W4_ERR_SHAPE : W4_OK;
}

int check_workspace(const void* workspace, const size_t* bytes, size_t need) {
  return need > 0 && (!workspace || !bytes || *bytes < need) ? W4_ERR_WORKSPACE : W4_OK;
}

}  // namespace

extern "C" {

int w4_rmsnorm(const uint16_t* X, const uint16_t* residual, int T, int H, const uint16_t* weight, float eps, uint16_t* h,
               uint16_t* Y, void* stream) {
  const NormArgs a{X, residual, T, H, weight, eps, h, Y, nullptr, nullptr, nullptr};
  if (int st = check_norm(a, 8)) return st;
  if (T == 0) return W4_OK;
  if (!Y) return W4_ERR_NULL;
  if (misaligned(Y)) return W4_ERR_ALIGN;
  return launch_norm(a, static_cast<hipStream_t>(stream));
}

int w4a8_rmsnorm(const uint16_t* X, const uint16_t* residual, int T, int H, const uint16_t* weight, float eps,
                 uint16_t* h, int8_t* Xq, float* sx, int32_t* xsum, void* stream) {
  const NormArgs a{X, residual, T, H, weight, eps, h, nullptr, Xq, sx, xsum};
  if (int st = check_norm(a, kGroup)) return st;
  if (T == 0) return W4_OK;
  if (!Xq || !sx || !xsum) return W4_ERR_NULL;
  if (misaligned(Xq) || misaligned(sx) || misaligned(xsum)) return W4_ERR_ALIGN;
  return launch_norm(a, static_cast<hipStream_t>(stream));
}

int w4_rope_table(int positions, int head, double base, float* cs, float* sn, void* stream) {
  if (head != 64 && head != 128) return W4_ERR_UNSUPPORTED;
  if (positions < 0 || !rope_table_fits(positions, head)) return W4_ERR_SHAPE;
  if (!(base > 0.0) || isinf(base)) return W4_ERR_VALUE;
  if (positions == 0) return W4_OK;
  if (!cs || !sn) return W4_ERR_NULL;
  if (misaligned(cs) || misaligned(sn)) return W4_ERR_ALIGN;
  return launch_rope_table(positions, head, base, cs, sn, static_cast<hipStream_t>(stream));
}

int w4_kv_append(const uint16_t* Q, long long q_stride, const uint16_t* K, long long k_stride, const uint16_t* V,
                 long long v_stride, int T, int n_q, const int32_t* offsets, const int32_t* lens, int B,
                 const int32_t* table, int table_width, const float* cs, const float* sn, int positions,
                 const w4_kv_cache* cache, uint16_t* Q_out, uint16_t* K_out, void* stream) {
  if (!cache) return W4_ERR_NULL;
  if (int st = check_cache(*cache, n_q)) return st;
  if (T < 0 || B < 0 || table_width < 0 || positions < 0 || (!offsets && T != B) || !append_fits(T)) return W4_ERR_SHAPE;
  if (int st = check_stride(q_stride, n_q, cache->head)) return st;
  if (int st = check_stride(k_stride, cache->n_kv, cache->head)) return st;
  if (int st = check_stride(v_stride, cache->n_kv, cache->head)) return st;
  if (T == 0 || B == 0) return W4_OK;
  if (!Q || !K || !V || !lens || !Q_out) return W4_ERR_NULL;
  if ((table_width > 0 && !table) || (positions > 0 && (!cs || !sn)) || (cache->pages > 0 && (!cache->k || !cache->v)))
    return W4_ERR_NULL;
  if (misaligned(Q) || misaligned(K) || misaligned(V) || misaligned(offsets) || misaligned(lens) || misaligned(table) ||
      misaligned(cs) || misaligned(sn) || misaligned(cache->k) || misaligned(cache->v) || misaligned(Q_out) ||
      misaligned(K_out))
    return W4_ERR_ALIGN;
  return launch_kv_append(AppendArgs{Q, q_stride, K, k_stride, V, v_stride, T, n_q, offsets, lens, B, table, table_width,
                                     cs, sn, positions, *cache, Q_out, K_out},
                          static_cast<hipStream_t>(stream));
}

int w4_prompt_attention(const uint16_t* Q, long long q_stride, const uint16_t* K, long long k_stride, const uint16_t* V,
                        long long v_stride, int T, int n_q, int n_kv, int head, const int32_t* offsets, int B,
                        float scale, uint16_t* O, void* workspace, size_t* workspace_bytes, void* stream) {
  if (int st = check_heads(n_q, n_kv, head)) return st;
  if (T < 0 || B < 0 || !prompt_fits(T, n_q, n_kv, B)) return W4_ERR_SHAPE;
  const size_t need = prompt_workspace_bytes(T, n_q, n_kv, head, B);
  if (!workspace && workspace_bytes) {
    *workspace_bytes = need;
    return W4_OK;
  }
  if (int st = check_stride(q_stride, n_q, head)) return st;
  if (int st = check_stride(k_stride, n_kv, head)) return st;
  if (int st = check_stride(v_stride, n_kv, head)) return st;
  if (!(scale > 0.0f) || isinf(scale)) return W4_ERR_VALUE;
  if (int st = check_workspace(workspace, workspace_bytes, need)) return st;
  if (T == 0 || B == 0) return W4_OK;
  if (!Q || !K || !V || !offsets || !O) return W4_ERR_NULL;
  if (misaligned(Q) || misaligned(K) || misaligned(V) || misaligned(offsets) || misaligned(O) || misaligned(workspace))
    return W4_ERR_ALIGN;
  return launch_prompt_attention(
      PromptArgs{Q, q_stride, K, k_stride, V, v_stride, T, n_q, n_kv, head, offsets, B, scale, O, workspace},
      static_cast<hipStream_t>(stream));
}

int w4_decode_attention(const uint16_t* Q, long long q_stride, int B, int n_q, const w4_kv_cache* cache,
                        const int32_t* lens, const int32_t* table, int table_width, int max_len, int prefix_len,
                        float scale, uint16_t* O, void* workspace, size_t* workspace_bytes, void* stream) {
  if (!cache) return W4_ERR_NULL;
  if (int st = check_cache(*cache, n_q)) return st;
  if (B < 0 || max_len < 0 || prefix_len < 0 || prefix_len % cache->page_size ||
      !decode_fits(B, n_q, *cache, max_len, prefix_len))
    return W4_ERR_SHAPE;
  const size_t need = decode_workspace_bytes(B, n_q, *cache, max_len, prefix_len);
  if (!workspace && workspace_bytes) {
    *workspace_bytes = need;
    return W4_OK;
  }
  if (table_width < 0 || max_len > (long long)table_width * cache->page_size ||
      prefix_len > (long long)table_width * cache->page_size)
    return W4_ERR_SHAPE;
  if (int st = check_stride(q_stride, n_q, cache->head)) return st;
  if (!(scale > 0.0f) || isinf(scale)) return W4_ERR_VALUE;
  if (int st = check_workspace(workspace, workspace_bytes, need)) return st;
  if (B == 0) return W4_OK;
  if (!Q || !lens || !O) return W4_ERR_NULL;
  if ((table_width > 0 && !table) || (cache->pages > 0 && (!cache->k || !cache->v))) return W4_ERR_NULL;
  if (misaligned(Q) || misaligned(lens) || misaligned(table) || misaligned(cache->k) || misaligned(cache->v) ||
      misaligned(O) || misaligned(workspace))
    return W4_ERR_ALIGN;
  return launch_decode_attention(
      DecodeArgs{Q, q_stride, B, n_q, *cache, lens, table, table_width, max_len, prefix_len, scale, O, workspace},
      static_cast<hipStream_t>(stream));
}

}  // extern "C"

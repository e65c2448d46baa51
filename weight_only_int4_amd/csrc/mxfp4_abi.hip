// C-ABI entry points of the MXFP4 operators: argument validation (host only, before any
// HIP call) and dispatch.  See include/w4a16.h for the contract.
#include "mxfp4.hpp"

using namespace w4;

namespace {

inline bool misaligned(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int check_matrix(int N, int K) {
  return N < 0 || K <= 0 || K % kMxBlock ? W4_ERR_SHAPE : W4_OK;
}

int check_conversion(int N, int K) {
  if (int st = check_matrix(N, K)) return st;
  return (long long)N * K > kMxMaxElements ? W4_ERR_SHAPE : W4_OK;
}

// Shapes, size query, workspace, pointers: the order every workspace-taking call uses.
int run_gemm(const MxGemmArgs& g, size_t* workspace_bytes, void* stream) {
  if (int st = check_matrix(g.N, g.K)) return st;
  if (g.M < 0 || g.M > kMxMaxRows || g.N > kMxMaxRows || g.K > kMxMaxK) return W4_ERR_SHAPE;
  const MxPlan plan = plan_mxfp4_gemm(g.act_bits, g.M, g.K, g.N);
  if (!plan.fits) return W4_ERR_SHAPE;
  const size_t need = plan.workspace;
  if (!g.workspace && workspace_bytes) {
    *workspace_bytes = need;
    return W4_OK;
  }
  if (need > 0 && (!g.workspace || !workspace_bytes || *workspace_bytes < need)) return W4_ERR_WORKSPACE;
  if (g.M == 0 || g.N == 0) return W4_OK;
  if (g.act_bits == 16 ? !g.X : !g.Xq || !g.xscales) return W4_ERR_NULL;
  if (!g.qweight || !g.scales || !g.Y) return W4_ERR_NULL;
  if (misaligned(g.X) || misaligned(g.Xq) || misaligned(g.xscales) || misaligned(g.qweight) || misaligned(g.scales) ||
      misaligned(g.Y) || misaligned(g.workspace))
    return W4_ERR_ALIGN;
  return launch_mxfp4_gemm(plan, g, static_cast<hipStream_t>(stream));
}

}  // namespace

extern "C" {

int mxfp4_quantize(const uint16_t* W, int N, int K, const float* s, uint32_t* codes, uint8_t* scales, void* stream) {
  if (int st = check_conversion(N, K)) return st;
  if (N == 0) return W4_OK;
  if (!W || !codes || !scales) return W4_ERR_NULL;
  if (misaligned(W) || misaligned(s) || misaligned(codes) || misaligned(scales)) return W4_ERR_ALIGN;
  return launch_mxfp4_quantize(W, N, K, s, codes, scales, static_cast<hipStream_t>(stream));
}

int mxfp4_dequantize(const uint32_t* codes, const uint8_t* scales, int N, int K, uint16_t* W, void* stream) {
  if (int st = check_conversion(N, K)) return st;
  if (N == 0) return W4_OK;
  if (!codes || !scales || !W) return W4_ERR_NULL;
  if (misaligned(codes) || misaligned(scales) || misaligned(W)) return W4_ERR_ALIGN;
  return launch_mxfp4_dequantize(codes, scales, N, K, W, static_cast<hipStream_t>(stream));
}

int mxfp4_a16_gemm(const uint16_t* X, int M, int K, int N, const uint32_t* qweight, const uint8_t* scales, uint16_t* Y,
                   void* workspace, size_t* workspace_bytes, void* stream) {
  return run_gemm(MxGemmArgs{16, X, nullptr, nullptr, M, K, N, qweight, scales, Y, workspace}, workspace_bytes, stream);
}

int mxfp4_a4_gemm(const uint32_t* Xq, const uint8_t* xscales, int M, int K, int N, const uint32_t* qweight,
                  const uint8_t* scales, uint16_t* Y, void* workspace, size_t* workspace_bytes, void* stream) {
  return run_gemm(MxGemmArgs{4, nullptr, Xq, xscales, M, K, N, qweight, scales, Y, workspace}, workspace_bytes, stream);
}

}  // extern "C"

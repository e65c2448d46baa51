// Products with MXFP4 weights that read both operands straight into registers:
// Y = X W_hat^T with bf16 activations (ACT = 16) or MXFP4 activations (ACT = 4).
//
// A workgroup owns 16 CB output channels and up to 16 RB activation rows; its waves
// take the 128-channel steps of K in turn, each keeps its own fp32 tile, and the tiles
// meet in LDS once, at the end, added in wave order (results are the same bit for bit
// on every run).  The weights are the matrix instruction's row operand: lane (r, q)
// holds the 16 bytes of block q of the step in channel r, which is one MX block with
// one scale byte.
//   ACT = 16: each of the block's four words expands to eight bf16 (4 conversions,
//     scale included, exact), the operand of one v_mfma_f32_16x16x32_bf16 whose other
//     operand is the same 8 channels of an activation row: the lane's 64 bytes of
//     activations are the four operands as they stand.
//   ACT = 4: one v_mfma_scale_f32_16x16x128_f8f6f4 takes the block as it stands.
// Loads are range-checked buffer loads: rows past M and N and blocks past K read
// zeros and touch no memory.
#include <algorithm>

#include "mxfp4.hpp"

namespace w4 {
namespace {

struct MxStreamArgs {
  const uint16_t* X;      // ACT = 16: [M][K] bf16
  const uint32_t* Xq;     // ACT = 4: [M][K/8] codes
  const uint8_t* xs;      //          [M][K/32] scale bytes
  int M, K, N;
  const uint32_t* qweight;
  const uint8_t* scales;
  uint16_t* Y;
};

template <int ACT, int RB, int CB>
__global__ __launch_bounds__(512) void mx_stream_kernel(MxStreamArgs a) {
  constexpr int kRow = 16 * CB + 4;            // floats of an LDS row, padded against bank conflicts
  extern __shared__ float red[];               // [wave][16][kRow]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16 * CB, m0 = blockIdx.y * 16 * RB;
  const int KB = a.K / kMxBlock;
  const int nrows = min(16 * CB, a.N - n0), mrows = min(16 * RB, a.M - m0);
  const auto rw = make_rsrc(a.qweight + (size_t)n0 * (a.K / 8), (uint32_t)nrows * (uint32_t)(a.K / 2));
  const auto rs = make_rsrc(a.scales + (size_t)n0 * KB, (uint32_t)nrows * (uint32_t)KB);
  const auto rx = ACT == 16 ? make_rsrc(a.X + (size_t)m0 * a.K, (uint32_t)mrows * (uint32_t)a.K * 2u)
                            : make_rsrc(a.Xq + (size_t)m0 * (a.K / 8), (uint32_t)mrows * (uint32_t)(a.K / 2));
  const auto rxs = ACT == 16 ? rs : make_rsrc(a.xs + (size_t)m0 * KB, (uint32_t)mrows * (uint32_t)KB);

  constexpr int XV = ACT == 16 ? 4 : 1;        // 16-byte loads of an activation row per step
  f32x4 acc[RB][CB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const int steps = (KB + 3) / 4;
  for (int t = wave; t < steps; t += waves) {
    const int kb = 4 * t + q;
    const bool ok = kb < KB;
    u32x4 w[CB], x[RB][XV];
    uint32_t ws[CB], xsc[RB];
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      const uint32_t row = (uint32_t)(16 * j + r);
      w[j] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, ok ? row * (uint32_t)(a.K / 2) + 16u * kb : kOob, 0, 0));
      ws[j] = __builtin_amdgcn_raw_buffer_load_b8(rs, ok ? row * (uint32_t)KB + (uint32_t)kb : kOob, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const uint32_t row = (uint32_t)(16 * i + r);
      const uint32_t xo = row * (uint32_t)(ACT == 16 ? a.K * 2 : a.K / 2) + (ACT == 16 ? 64u : 16u) * kb;
#pragma unroll
      for (int v = 0; v < XV; ++v)
        x[i][v] = __builtin_bit_cast(u32x4,
                                     __builtin_amdgcn_raw_buffer_load_b128(rx, ok ? xo + 16u * v : kOob, 0, 0));
      if constexpr (ACT == 4)
        xsc[i] = __builtin_amdgcn_raw_buffer_load_b8(rxs, ok ? row * (uint32_t)KB + (uint32_t)kb : kOob, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      if constexpr (ACT == 16) {
        const float sc = mx_scale(ws[j]);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const bf16x8 wb = mx_expand(w[j][v], sc);
#pragma unroll
          for (int i = 0; i < RB; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, __builtin_bit_cast(bf16x8, x[i][v]), acc[i][j], 0,
                                                               0, 0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < RB; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(w[j]), mx_operand(x[i][0]), acc[i][j],
                                                                      4, 4, 0, (int)ws[j], 0, (int)xsc[i]);
      }
    }
  }

  // Tiles to LDS, 16 rows at a time: lane (c, q) holds row c, channels 16 j + 4 q .. + 3.
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    if (i) __syncthreads();
#pragma unroll
    for (int j = 0; j < CB; ++j)
      *reinterpret_cast<f32x4*>(&red[(wave * 16 + r) * kRow + 16 * j + 4 * q]) = acc[i][j];
    __syncthreads();
    for (int o = threadIdx.x; o < 64 * CB; o += blockDim.x) {
      const int row = o / (4 * CB), c = (o % (4 * CB)) * 4;
      f32x4 sum = *reinterpret_cast<const f32x4*>(&red[row * kRow + c]);
      for (int wv = 1; wv < waves; ++wv) {
        const f32x4 p = *reinterpret_cast<const f32x4*>(&red[(wv * 16 + row) * kRow + c]);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += p[e];
      }
      const int m = m0 + 16 * i + row, n = n0 + c;
      if (m < a.M) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < a.N) a.Y[(size_t)m * a.N + n + e] = __builtin_bit_cast(uint16_t, (__bf16)sum[e]);
      }
    }
  }
}

template <int ACT, int RB, int CB>
int launch_stream(const MxStreamArgs& a, hipStream_t stream) {
  const int steps = (a.K / kMxBlock + 3) / 4;
  const int waves = std::min(8, steps);
  const long long gx = (a.N + 16 * CB - 1) / (16 * CB), gy = (a.M + 16LL * RB - 1) / (16 * RB);
  if (gy > 65535) return W4_ERR_SHAPE;
  const size_t lds = (size_t)waves * 16 * (16 * CB + 4) * sizeof(float);
  hipLaunchKernelGGL((mx_stream_kernel<ACT, RB, CB>), dim3((unsigned)gx, (unsigned)gy), dim3(waves * 64), lds, stream, a);
  W4_CHECK_LAUNCH();
  return W4_OK;
}

}  // namespace

size_t mxfp4_gemm_workspace_bytes(int act_bits, int M, int K, int N) {
  (void)act_bits; (void)M; (void)K; (void)N;
  return 0;
}

int launch_mxfp4_gemm(const MxGemmArgs& g, hipStream_t stream) {
  MxStreamArgs a{g.X, g.Xq, g.xscales, g.M, g.K, g.N, g.qweight, g.scales, g.Y};
  if (g.act_bits == 16) {
    if (g.M <= 16) return launch_stream<16, 1, 1>(a, stream);
    if (g.M <= 32) return launch_stream<16, 2, 4>(a, stream);
    return launch_stream<16, 4, 4>(a, stream);
  }
  if (g.M <= 16) return launch_stream<4, 1, 1>(a, stream);
  if (g.M <= 32) return launch_stream<4, 2, 4>(a, stream);
  return launch_stream<4, 4, 4>(a, stream);
}

}  // namespace w4

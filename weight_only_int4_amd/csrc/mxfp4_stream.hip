// Products with MXFP4 weights that read both operands straight into registers:
// Y = X W_hat^T with bf16 activations (ACT = 16) or MXFP4 activations (ACT = 4), for the
// row counts at which the weights' bytes or plain latency are the bound.
//
// A workgroup owns CB tiles of 16 / SL output channels and up to 16 RB activation rows.
// Its waves take the steps of K in turn, each keeps its own fp32 tile, and the tiles meet
// in LDS once, at the end, added in wave order (results are the same bit for bit on
// every run).  Loads of the next step are issued before the current one is multiplied.
//
// The weights are the matrix instruction's row operand: lane (r, q) holds 16 bytes, one MX
// block with one scale byte.
//   ACT = 16: each of the block's four words expands to eight bf16 (4 conversions,
//     scale included, exact), the operand of one v_mfma_f32_16x16x32_bf16 whose other
//     operand is the same 8 channels of an activation row: the lane's 64 bytes of
//     activations are the four operands as they stand.
//   ACT = 4: one v_mfma_scale_f32_16x16x128_f8f6f4 takes the block as it stands.
// A step is SL slices of 128 channels of K for 16 / SL output channels: row operand r is
// channel r / SL in slice r % SL, column c of the other operand activation row c / SL in
// slice c % SL, and at the end the products of equal slices (r % SL == c % SL) are added.
// A load of weights then covers 16 / SL rows of 64 SL contiguous bytes: with SL = 1 every
// piece is half a cache line, which costs the L1 as much as a whole one, and there are
// SL times as many tiles to spread over the CUs.  The price, SL times the matrix
// instructions per row, is small change while the weights are the bound.
// bf16 activations are loaded in whole rows (16 lanes to the 256 bytes of a slice) and
// turned into operand order through 4 KB of LDS per wave: in operand order a load would be
// 64 pieces of 16 bytes, four times the cache lines.  Chunk k of column c is at position k ^
// mx_swizzle16(c), so that both sides are free of bank conflicts.
// Measured, with four weights in turn (Infinity Cache; from HBM, 24 in turn): M = 1, K = 5120, N = 17408
// 9.7 to 10.3 us (12.2 to 12.9, 3.7 to 3.9 TB/s of weights; a large copy reaches 4.9); M = 16 13.3 to 14.2 (18.6 to
// 19.0) with bf16 activations and 11.8 to 12.3 (15.4) with 4-bit ones, bound by what the busiest CU
// fetches (three workgroups, where 2.8 would be even); M = 1, K = N = 2048 2.8 (3.75), an empty kernel 2.5.
// Loads are range-checked buffer loads: rows past M and N and blocks past K read
// zeros and touch no memory.  A tile's first row is the scalar offset of the loads, which is not
// relied on to be part of the check: a tile that would end past the last row moves back to
// end there, and has some outputs (the same bits) in common with the tile before.
#include <algorithm>
#include <cfloat>

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
  float* partial;         // [splits][M][N] when K is split over blockIdx.z, else NULL
  int steps;              // steps of one split
  int col_groups;         // workgroups side by side along N; blockIdx.x counts them row group by row group
};

// Sum over the SL neighbouring lanes of a slice group (1, 2 or 4 lanes).
template <int SL>
__device__ __forceinline__ float slice_sum(float v) {
  if constexpr (SL >= 2)
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, true));   // lane ^ 1
  if constexpr (SL >= 4)
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, true));   // lane ^ 2
  return v;
}

constexpr int kMxStreamWaves = 4;              // at most, per workgroup
constexpr int kMxTurn = 4096;                  // bytes per wave that turn activations into operand order

template <int ACT, int SL, int RB, int CB>
__global__ __launch_bounds__(kMxStreamWaves * 64) void mx_stream_kernel(MxStreamArgs a) {
  constexpr int kCh = 16 / SL;                 // channels per tile, and activation rows per tile
  constexpr int kRow = kCh * CB + 4;           // floats of an LDS row, padded against bank conflicts
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  float* red = reinterpret_cast<float*>(lds);  // [wave][kCh][kRow], after the last step
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int n0 = (int)(blockIdx.x % (uint32_t)a.col_groups) * kCh * CB;
  const int m0 = (int)(blockIdx.x / (uint32_t)a.col_groups) * kCh * RB;
  const int KB = a.K / kMxBlock;
  const int nrows = min(kCh * CB, a.N - n0), mrows = min(kCh * RB, a.M - m0);
  const auto rw = make_rsrc(a.qweight + (size_t)n0 * (a.K / 8), (uint32_t)nrows * (uint32_t)(a.K / 2));
  const auto rs = make_rsrc(a.scales + (size_t)n0 * KB, (uint32_t)nrows * (uint32_t)KB);
  const auto rx = ACT == 16 ? make_rsrc(a.X + (size_t)m0 * a.K, (uint32_t)mrows * (uint32_t)a.K * 2u)
                            : make_rsrc(a.Xq + (size_t)m0 * (a.K / 8), (uint32_t)mrows * (uint32_t)(a.K / 2));
  const auto rxs = ACT == 16 ? rs : make_rsrc(a.xs + (size_t)m0 * KB, (uint32_t)mrows * (uint32_t)KB);
  const int t0 = blockIdx.z * a.steps, t1 = min((KB + 4 * SL - 1) / (4 * SL), t0 + a.steps);

  constexpr int XV = ACT == 16 ? 4 : 1;        // 16-byte loads of an activation tile per lane and step
  const uint32_t wo = (uint32_t)(r / SL) * (uint32_t)(a.K / 2), so = (uint32_t)(r / SL) * (uint32_t)KB;
  auto tile_row = [](int tile, int rows) { return max(0, min(tile * kCh, rows - kCh)); };   // of `rows` in all
  const int kq = 4 * (r % SL) + q;             // block of this lane's weights within a step
  // ACT = 16: load v of a tile covers columns 4 v + q, lane r its chunk r (8 channels);
  // ACT = 4: the lane's own column r and block q.
  uint32_t xo[XV];
  int xk[XV];
  const uint32_t xbytes = (uint32_t)(ACT == 16 ? a.K * 2 : a.K / 2);
#pragma unroll
  for (int v = 0; v < XV; ++v) {
    const int c = ACT == 16 ? 4 * v + q : r;
    xo[v] = (uint32_t)(c / SL) * xbytes + (ACT == 16 ? (uint32_t)(c % SL) * 256u + 16u * r : 16u * kq);
    xk[v] = ACT == 16 ? 4 * (c % SL) + r / 4 : kq;
  }

  int wrow[CB], xrow[RB];
#pragma unroll
  for (int j = 0; j < CB; ++j) wrow[j] = tile_row(j, nrows);
#pragma unroll
  for (int i = 0; i < RB; ++i) xrow[i] = tile_row(i, mrows);

  struct Step {
    u32x4 w[CB], x[RB][XV];
    uint32_t ws[CB], xs[RB];
  };
  auto load = [&](int t, Step& s) {
    const int left = t < t1 ? KB - 4 * SL * t : 0;       // blocks from this step on
    const uint32_t kb = 4u * SL * (uint32_t)t;
    const uint32_t wk = kq < left ? wo + 16u * (kb + kq) : kOob, sk = kq < left ? so + kb + kq : kOob;
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      s.w[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, wk, wrow[j] * (a.K / 2), 0));
      s.ws[j] = __builtin_amdgcn_raw_buffer_load_b8(rs, sk, wrow[j] * KB, 0);
    }
#pragma unroll
    for (int v = 0; v < XV; ++v) {
      const uint32_t o = xk[v] < left ? xo[v] + (ACT == 16 ? 64u : 16u) * kb : kOob;
#pragma unroll
      for (int i = 0; i < RB; ++i)
        s.x[i][v] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, o, xrow[i] * (int)xbytes, 0));
    }
    if constexpr (ACT == 4) {
#pragma unroll
      for (int i = 0; i < RB; ++i)
        s.xs[i] = __builtin_amdgcn_raw_buffer_load_b8(rxs, sk, xrow[i] * KB, 0);
    }
  };

  f32x4 acc[RB][CB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  unsigned char* turn = lds + wave * kMxTurn;
  auto multiply = [&](const Step& s) {
    if constexpr (ACT == 16) {
      // LDS operations of one wave complete in order: no barrier between the tiles
      bf16x8 x[RB][4];
#pragma unroll
      for (int i = 0; i < RB; ++i) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int c = 4 * v + q;
          *reinterpret_cast<u32x4*>(turn + c * 256 + ((r ^ mx_swizzle16(c)) * 16)) = s.x[i][v];
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int v = 0; v < 4; ++v)
          x[i][v] = *reinterpret_cast<const bf16x8*>(turn + r * 256 + (((4 * q + v) ^ mx_swizzle16(r)) * 16));
        __builtin_amdgcn_wave_barrier();
      }
#pragma unroll
      for (int j = 0; j < CB; ++j) {
        const float sc = mx_scale(s.ws[j]);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const bf16x8 wb = mx_expand(s.w[j][v], sc);
#pragma unroll
          for (int i = 0; i < RB; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, x[i][v], acc[i][j], 0, 0, 0);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < CB; ++j)
#pragma unroll
        for (int i = 0; i < RB; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(s.w[j]), mx_operand(s.x[i][0]),
                                                                      acc[i][j], 4, 4, 0, (int)s.ws[j], 0, (int)s.xs[i]);
    }
  };
  // two register sets take the steps in turn; loads past the end touch no memory
  Step s0, s1;
  load(t0 + wave, s0);
  for (int t = t0 + wave; t < t1; t += 2 * waves) {
    load(t + waves, s1);
    multiply(s0);
    if (t + waves >= t1) break;
    load(t + 2 * waves, s0);
    multiply(s1);
  }

  // Tiles to LDS, one row tile at a time.  Lane (c, q) of a tile holds column c and the tile's
  // rows 4 q .. 4 q + 3: channel (4 q + e) / SL of activation row c / SL, of use where
  // e % SL == c % SL.
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    __syncthreads();
    float* mine = red + (size_t)(wave * kCh + r / SL) * kRow;
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      const f32x4 v = acc[i][j];
      if constexpr (SL == 1) {
        *reinterpret_cast<f32x4*>(mine + 16 * j + 4 * q) = v;
      } else if constexpr (SL == 2) {
        const float e0 = slice_sum<2>(r & 1 ? v[1] : v[0]), e1 = slice_sum<2>(r & 1 ? v[3] : v[2]);
        if ((r & 1) == 0) *reinterpret_cast<float2*>(mine + 8 * j + 2 * q) = make_float2(e0, e1);
      } else {
        const float lo = r & 1 ? v[1] : v[0], hi = r & 1 ? v[3] : v[2];
        const float e0 = slice_sum<4>(r & 2 ? hi : lo);
        if ((r & 3) == 0) mine[4 * j + q] = e0;
      }
    }
    __syncthreads();
    constexpr int kQuads = kCh * CB / 4;       // groups of four channels per row
    for (int o = threadIdx.x; o < kCh * kQuads; o += blockDim.x) {
      const int row = o / kQuads, c = (o % kQuads) * 4;
      f32x4 sum = *reinterpret_cast<const f32x4*>(&red[row * kRow + c]);
      for (int wv = 1; wv < waves; ++wv) {
        const f32x4 p = *reinterpret_cast<const f32x4*>(&red[(wv * kCh + row) * kRow + c]);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += p[e];
      }
      const int m = m0 + xrow[i] + row, n = n0 + tile_row(c / kCh, nrows) + c % kCh;
      if (m >= a.M) continue;
      const size_t at = (size_t)m * a.N + n;
      const bool whole = n + 4 <= a.N;           // four outputs at once, aligned to one
      if (a.partial) {
        typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
        float* p = a.partial + (size_t)blockIdx.z * a.M * a.N + at;
        if (whole) *reinterpret_cast<f32x4_any*>(p) = f32x4_any{sum[0], sum[1], sum[2], sum[3]};
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (!whole && n + e < a.N) p[e] = sum[e];
      } else {
        typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
        typedef u16x4 u16x4_any __attribute__((aligned(2)));
        u16x4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __builtin_bit_cast(uint16_t, (__bf16)sum[e]);
        if (whole) *reinterpret_cast<u16x4_any*>(a.Y + at) = y;
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (!whole && n + e < a.N) a.Y[at + e] = y[e];
      }
    }
  }
}

template <int ACT, int SL, int RB, int CB>
int launch_stream(const MxStreamArgs& base, int waves, int splits, hipStream_t stream) {
  MxStreamArgs a = base;
  const int steps = (a.K / kMxBlock + 4 * SL - 1) / (4 * SL);
  a.steps = (steps + splits - 1) / splits;
  const int nc = 16 / SL * CB, mr = 16 / SL * RB;
  const long long gx = (a.N + nc - 1LL) / nc, gy = (a.M + mr - 1LL) / mr;   // mx_stream_fits
  a.col_groups = (int)gx;
  const size_t lds =
      std::max<size_t>((size_t)waves * (16 / SL) * (nc + 4) * sizeof(float), ACT == 16 ? waves * kMxTurn : 0);
  hipLaunchKernelGGL((mx_stream_kernel<ACT, SL, RB, CB>), dim3((unsigned)(gx * gy), 1, (unsigned)splits),
                     dim3(waves * 64), lds, stream, a);
  W4_CHECK_LAUNCH();
  return W4_OK;
}

template <int ACT, int SL, int RB>
int launch_cols(const MxStreamArgs& a, const MxStreamPlan& p, hipStream_t stream) {
  // what plan_mx_stream chooses from; the grid follows from the instance, so any would be right
  if constexpr (RB <= 2 && !(ACT == 16 && SL == 2))
    if (p.cols == 5) return launch_stream<ACT, SL, RB, 5>(a, p.waves, p.splits, stream);
  if constexpr (RB <= 2)
    if (p.cols == 4) return launch_stream<ACT, SL, RB, 4>(a, p.waves, p.splits, stream);
  switch (p.cols) {
    case 1: return launch_stream<ACT, SL, RB, 1>(a, p.waves, p.splits, stream);
    case 2: return launch_stream<ACT, SL, RB, 2>(a, p.waves, p.splits, stream);
    default: return launch_stream<ACT, SL, RB, 3>(a, p.waves, p.splits, stream);
  }
}

template <int ACT>
int launch_act(const MxStreamArgs& a, const MxStreamPlan& p, hipStream_t stream) {
  if (p.slices == 4) return launch_cols<ACT, 4, 1>(a, p, stream);
  if (p.slices == 2) {
    switch (p.rows) {
      case 1: return launch_cols<ACT, 2, 1>(a, p, stream);
      case 2: return launch_cols<ACT, 2, 2>(a, p, stream);
      default: return launch_cols<ACT, 2, 3>(a, p, stream);
    }
  }
  if constexpr (ACT == 16)                      // 4-bit activations: two slices up to 24 rows
    if (p.rows == 1) return launch_cols<ACT, 1, 1>(a, p, stream);
  switch (p.rows) {
    case 2: return launch_cols<ACT, 1, 2>(a, p, stream);
    case 3: return launch_cols<ACT, 1, 3>(a, p, stream);
    default: return launch_cols<ACT, 1, 4>(a, p, stream);
  }
}

}  // namespace

// Rules from a sweep of every plan over hidden-2048 to 27B-shaped linears, 1 to 333 rows, a
// few weights in turn, which the Infinity Cache holds (microseconds, chosen against the other side):
//  * Slices: 4 up to 4 rows, 2 up to 8, and up to 24 with 4-bit activations or long rows of weights: bf16, 16
//    rows, K = 5120, N = 17408 13.3 against 16.0 with one slice, K = 2048, N = 6144 5.1 against 4.7; 4 bits, 24
//    rows, K = N = 2048 4.7 against 5.4.  Their use is the piece of a row that one load takes (one
//    row, K = 5120, N = 17408: 64 bytes 19.4, 128 bytes 11.5, 256 bytes 9.95).
//  * Channel tiles per workgroup: what the busiest CU has to fetch decides, its workgroups' weights, past the
//    L2, at 39 bytes per nanosecond (half that in 64-byte pieces), and their activations at 100.  K = 5120,
//    N = 17408, 16 rows: three tiles (726 workgroups, three on a CU) 13.3, four (544, three) 14.9, two
//    (1088, five) 17.4, one (nine) 23; 4 bits five tiles 11.8, four 13.7, two 14.5; K = 17408, N = 5120, 16 rows:
//    three 15.7, four 18.0.  Beyond two row tiles, and with two slices of bf16 activations, five lack
//    registers or waves (K = 5120, N = 17408, 16 rows: 14.9 to 16.3).
//  * Above 24 rows a long K may be split over workgroups, with a second launch: M = 37, K = 6144, N = 2048 9.1
//    against 10.7, M = 32, K = 17408, N = 5120 20.4 against 28.
//  * Waves, which share K: about one for each SIMD and, with 4-bit activations, two (bf16, 726 workgroups 13.3 with
//    one, 14.5 with two; 214 workgroups 15.7 with four, 18.7 with two; 4 bits, 726: 12.1 with four, 15.7 with one).
MxStreamPlan plan_mx_stream(int act_bits, int M, int K, int N) {
  constexpr int kCus = 256;
  MxStreamPlan p{};
  p.slices = M <= 4 ? 4 : M <= 8 || (M <= 24 && (act_bits == 4 || K >= 4096)) ? 2 : 1;
  p.rows = std::min(4, (M * p.slices + 15) / 16);
  const int ch = 16 / p.slices;                 // channels per tile, and activation rows per tile
  const int steps = (K / kMxBlock + 4 * p.slices - 1) / (4 * p.slices);
  const long long row_groups = (M + (long long)ch * p.rows - 1) / (ch * p.rows);
  // microseconds of a workgroup: per channel tile, and for the activations and its start
  const double weights = ch * 0.53e-3 * K / (p.slices == 1 ? 20.0 : 39.0);
  const double activations = std::min(M, ch * p.rows) * (act_bits == 16 ? 2.0e-3 : 0.53e-3) * K / 100.0;
  const int most = p.rows > 2 ? 3 : act_bits == 16 && p.slices == 2 ? 4 : 5;
  double best = DBL_MAX;
  long long wgs = 0;
  for (int splits = 1; splits <= (M > 24 && steps >= 32 ? 4 : 1); splits *= 4)
    for (int cols = 1; cols <= most; ++cols) {
      const long long n = (N + (long long)ch * cols - 1) / (ch * cols) * row_groups * splits;
      double us = (double)((n + kCus - 1) / kCus) * ((cols * weights + activations) / splits + 0.2);
      if (splits > 1) us += 2.5 + splits * 2.7e-6 * M * N;
      if (us < best) {
        best = us;
        p.cols = cols;
        p.splits = splits;
        wgs = n;
      }
    }
  p.waves = act_bits == 16 ? (wgs <= 300 ? 4 : wgs <= 640 ? 2 : 1) : (wgs <= 768 ? 4 : wgs <= 1100 ? 2 : 1);
  // Two (four slices) or two and a half steps a wave at least.  4 bits, one / two / four waves: M = 333, K = 1056, N = 2047
  // (nine steps) 8.9 / 7.6 / 8.0; M = 16, K = 1536, N = 4096 (six) 5.2 / 4.2 / 4.3; M = 40, K = 512, N = 2048 (four) 3.7 /
  // 3.9 / 4.0; M = 100, K = 480, N = 2048 (four) 4.2 / 4.3 / 4.4; four slices, M = 2, K = N = 2048 (four) 3.9 / 3.4 / 3.2.  bf16:
  // M = 64, K = 768, N = 1024 (six) 6.6 / 5.7 / 6.2; M = 8, K = 512, N = 2048 (two) 2.9 / 2.8 / 2.9.  The other way round by at most
  // 0.4 us: bf16, M = 40, K = 512, N = 2048 4.6 / 4.2 / 4.5.
  while (p.waves > 1 && (p.slices == 4 ? 4 : 5) * p.waves * p.splits > 2 * steps) p.waves /= 2;
  return p;
}

bool mx_stream_fits(const MxStreamPlan& p, int M, int N) {
  const int nc = 16 / p.slices * p.cols, mr = 16 / p.slices * p.rows;
  return (N + nc - 1LL) / nc * ((M + mr - 1LL) / mr) * p.waves * 64 <= kMaxGridThreads;
}

int launch_mx_stream(const MxStreamPlan& p, const MxGemmArgs& g, hipStream_t stream) {
  MxStreamArgs a{g.X, g.Xq, g.xscales, g.M, g.K, g.N, g.qweight, g.scales, g.Y,
                 p.splits > 1 ? static_cast<float*>(g.workspace) : nullptr, 0, 0};
  const int st = g.act_bits == 16 ? launch_act<16>(a, p, stream) : launch_act<4>(a, p, stream);
  if (st || p.splits == 1) return st;
  const size_t MN = (size_t)g.M * g.N;
  return launch_split_reduce(a.partial, p.splits, MN, MN, g.Y, stream);
}

// The tiled form (stream against tile, microseconds): with 4-bit activations from 17 rows on (K = 2048, N = 6144:
// M = 20 5.8 against 5.4, M = 64 9.3 against 5.4; K = 5120, N = 17408: M = 16 11.8 against 14.3, M = 32 19.9 against 15.9),
// 33 on small weights (K = N = 2048: M = 20 4.9 against 5.4, M = 40 6.8 against 5.4).  With bf16 ones, whose
// expansion it shares among fewer rows, from 129 rows on and 10^9 products (K = 2048, N = 6144: M = 128 11.3 against
// 12.5, M = 200 16.5 against 14.3; K = 5120, N = 5120: 19.6 against 26.0, 32.9 against 31.2), 65 on wide weights
// (K = 5120, N = 17408: M = 64 32.3 against 33.2, M = 96 46.5 against 41.1; K = 1536, N = 9000: 9.5 against 9.6,
// 14.1 against 11.1).  Where scale rows have to be padded first, by another launch, from 33 rows on and 2 10^9
// products (weights from HBM; 4 bits, K = 2880, N = 201088: M = 4 65 against 110, M = 24 102 against 118, M = 33 132 against 121; K = 5152,
// N = 20000: M = 24 27.4 against 32.6, M = 33 32.8 against 33.1, M = 64 39.4 against 36.7; K = 2080, N = 8192: M = 64 9.2
// against 12.2, M = 128 12.5 against 13.2, M = 333 26.1 against 17.2; K = 1056, N = 8192: M = 128 7.6 against 8.3,
// M = 333 14.1 against 10.6; K = 17440, N = 5120: M = 24 24.4 against 31.8, M = 33 32.0 against 33.0).
bool mxfp4_use_tile(int act_bits, int M, int K, int N) {
  const double NK = (double)N * K, MNK = M * NK;
  if (act_bits == 16) return MNK >= 1e9 && M > (N >= 8192 ? 64 : 128);
  const int KB = K / kMxBlock;
  if (KB % 4 != 0 || KB < 16) return MNK >= 2e9 && M > 32;
  return M > (NK >= 8e6 ? 16 : 32);
}

MxPlan plan_mxfp4_gemm(int act_bits, int M, int K, int N) {
  MxPlan p{};
  p.fits = true;
  if (M == 0 || N == 0) return p;
  p.use_tile = mxfp4_use_tile(act_bits, M, K, N);
  if (p.use_tile) {
    p.tile = plan_mx_tile(act_bits, M, K, N);
    p.fits = mx_tile_fits(p.tile, act_bits, M, K, N);
    p.workspace = mx_tile_workspace_bytes(p.tile, act_bits, M, K, N);
  } else {
    p.stream = plan_mx_stream(act_bits, M, K, N);
    p.fits = mx_stream_fits(p.stream, M, N);
    p.workspace = p.stream.splits > 1 ? (size_t)p.stream.splits * M * N * sizeof(float) : 0;
  }
  return p;
}

int launch_mxfp4_gemm(const MxPlan& p, const MxGemmArgs& g, hipStream_t stream) {
  return p.use_tile ? launch_mx_tile(p.tile, g, stream) : launch_mx_stream(p.stream, g, stream);
}

}  // namespace w4

// Launch plan of the tiled MXFP4 products (mxfp4_gemm.hpp): tile shape, split of K, and
// the padded scale rows that the kernels need.
#include <algorithm>
#include <cfloat>

#include "mxfp4_gemm.hpp"

namespace w4 {
namespace {

// Scale rows padded to `to` bytes with zeros (a scale of 2^-127 for blocks whose codes
// are zero): the weights' rows, then the activations'.
__global__ __launch_bounds__(256) void mx_pad_scales_kernel(const uint8_t* w, int N, const uint8_t* x, int M, int kb,
                                                            uint8_t* wout, uint8_t* xout, int to) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, nw = (size_t)N * to;
  if (i >= nw + (size_t)M * to) return;
  const uint8_t* from = i < nw ? w : x;
  uint8_t* out = i < nw ? wout : xout;
  const size_t at = i < nw ? i : i - nw, row = at / to;
  const int b = (int)(at % to);
  out[at] = b < kb ? from[row * kb + b] : 0;
}

// A tile shape with what it costs: microseconds per workgroup (start, first copies, stores)
// and per stage of 128 channels, alone on its CU and with `occ` workgroups on every CU.
// Measured at M = 2048, K = 1024 / 2048 / 6144 with one full round of workgroups, and
// at M = 256, N = 1024, K = 1024 / 4096.
struct MxTile {
  int bm, bn, occ;
  float start, alone, full;
};
constexpr MxTile kTiles4[] = {{256, 256, 1, 7.0f, 0.87f, 0.87f}, {256, 192, 1, 5.5f, 0.67f, 0.67f},
                              {128, 128, 2, 3.0f, 0.36f, 0.54f}, {128, 64, 2, 2.0f, 0.27f, 0.37f},
                              {64, 64, 4, 1.5f, 0.25f, 0.45f}};
constexpr MxTile kTiles16[] = {{256, 192, 1, 6.0f, 2.48f, 2.48f}, {128, 128, 1, 3.2f, 0.88f, 0.97f},
                               {128, 64, 2, 2.4f, 0.62f, 1.03f}, {64, 64, 3, 1.7f, 0.50f, 1.16f}};
constexpr int kCus = 256;
// More than one round of the 256 x 192 tile is chained where K allows it: a further tile starts so many
// microseconds sooner.  (A single round keeps the other form, 41.0 us against 42.0 at K = 6144.)
constexpr int kChained = 1;
constexpr double kChainGain = 1.5;

double tile_cost(const MxTile& t, long long wgs, int stages) {
  const long long round = (long long)t.occ * kCus;
  auto slope = [&](long long n) {               // n <= round workgroups at once
    const long long per_cu = (n + kCus - 1) / kCus;
    return t.occ == 1 ? (double)t.full : t.alone + (t.full - t.alone) * (double)(per_cu - 1) / (t.occ - 1);
  };
  const long long rounds = wgs / round, rest = wgs % round;
  double us = rounds * (t.start + stages * slope(round));
  if (rest) us += t.start + stages * slope(rest);
  return us;
}

long long workgroups(const MxTile& t, int M, int N) { return ((M + t.bm - 1LL) / t.bm) * ((N + t.bn - 1LL) / t.bn); }

int padded_scale_row(int KB) { return KB % 4 == 0 && KB >= 16 ? 0 : std::max(16, (KB + 3) / 4 * 4); }

}  // namespace

MxTilePlan plan_mx_tile(int act_bits, int M, int K, int N) {
  const MxTile* tiles = act_bits == 4 ? kTiles4 : kTiles16;
  const int count = act_bits == 4 ? (int)(sizeof kTiles4 / sizeof *kTiles4) : (int)(sizeof kTiles16 / sizeof *kTiles16);
  const int KT = (K / kMxBlock + 3) / 4;
  MxTilePlan best{};
  double best_us = DBL_MAX;
  for (int i = 0; i < count; ++i) {
    const long long n = workgroups(tiles[i], M, N);
    for (int splits = 1; splits <= 16; splits *= 2) {
      const int per = (KT + splits - 1) / splits, stages = splits == 1 ? KT : (per + 3) / 4 * 4;
      const int actual = (KT + stages - 1) / stages;
      if (splits > 1 && actual < splits) break;
      double us = tile_cost(tiles[i], n * actual, stages);
      const bool chain = act_bits == 4 && i == kChained && splits == 1 && n > kCus && KT % 4 == 0 &&
                         M >= tiles[i].bm && N >= tiles[i].bn;
      if (chain) us -= kChainGain * (double)((n - 1) / kCus);
      // a split's partial outputs are written and read once, by another launch
      if (actual > 1) us += 3.0 + 8.0 * actual * M * N / 3.0e6;
      if (us < best_us) {
        best_us = us;
        best = MxTilePlan{i, actual, splits == 1 ? (KT + 3) / 4 * 4 : stages, chain};
      }
    }
  }
  return best;
}

// Workspace: padded scale rows of the weights and of the activations, partial outputs.
namespace {
struct MxTileLayout {
  size_t w, x, partial, total;
};
MxTileLayout tile_layout(const MxTilePlan& p, int act_bits, int M, int K, int N) {
  const int ss = padded_scale_row(K / kMxBlock);
  MxTileLayout l{};
  l.x = align_up((size_t)N * ss, 256);
  l.partial = l.x + (act_bits == 4 ? align_up((size_t)M * ss, 256) : 0);
  l.total = l.partial + (p.splits > 1 ? (size_t)p.splits * M * N * sizeof(float) : 0);
  return l;
}
}  // namespace

size_t mx_tile_workspace_bytes(const MxTilePlan& p, int act_bits, int M, int K, int N) {
  return tile_layout(p, act_bits, M, K, N).total;
}

bool mx_tile_fits(const MxTilePlan& p, int act_bits, int M, int K, int N) {
  const MxTile& t = act_bits == 4 ? kTiles4[p.tile] : kTiles16[p.tile];
  const long long padded = (N + (act_bits == 4 ? (long long)M : 0)) * padded_scale_row(K / kMxBlock);
  return workgroups(t, M, N) * 256 <= kMaxGridThreads && (padded + 255) / 256 * 256 <= kMaxGridThreads;
}

int launch_mx_tile(const MxTilePlan& p, const MxGemmArgs& g, hipStream_t stream) {
  const int KB = g.K / kMxBlock, ss = padded_scale_row(KB);
  const MxTileLayout l = tile_layout(p, g.act_bits, g.M, g.K, g.N);
  uint8_t* ws = static_cast<uint8_t*>(g.workspace);
  MxTileArgs a{};
  a.X = g.act_bits == 4 ? static_cast<const void*>(g.Xq) : g.X;
  a.xs = g.xscales;
  a.qweight = g.qweight;
  a.ws = g.scales;
  a.ss = KB;
  a.M = g.M;
  a.K = g.K;
  a.N = g.N;
  a.stages_per_split = p.stages;
  a.Y = g.Y;
  a.partial = p.splits > 1 ? reinterpret_cast<float*>(ws + l.partial) : nullptr;
  if (ss) {
    const int rows = g.act_bits == 4 ? g.M : 0;
    const size_t blocks = ((size_t)(g.N + (long long)rows) * ss + 255) / 256;   // mx_tile_fits
    hipLaunchKernelGGL(mx_pad_scales_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, g.scales, g.N, g.xscales, rows,
                       KB, ws + l.w, ws + l.x, ss);
    a.ws = ws + l.w;
    a.xs = ws + l.x;
    a.ss = ss;
  }
  a.tiles = (int)workgroups(g.act_bits == 4 ? kTiles4[p.tile] : kTiles16[p.tile], g.M, g.N);
  const dim3 grid((unsigned)a.tiles, (unsigned)p.splits), block(256);
  if (g.act_bits == 4) {
    switch (p.tile) {
      case 0: hipLaunchKernelGGL((mx_tile_a4_kernel<256, 256, false>), grid, block, 0, stream, a); break;
      case 1:
        if (p.chain) hipLaunchKernelGGL((mx_tile_a4_kernel<256, 192, true>), dim3(kCus), block, 0, stream, a);
        else hipLaunchKernelGGL((mx_tile_a4_kernel<256, 192, false>), grid, block, 0, stream, a);
        break;
      case 2: hipLaunchKernelGGL((mx_tile_a4_kernel<128, 128, false>), grid, block, 0, stream, a); break;
      case 3: hipLaunchKernelGGL((mx_tile_a4_kernel<128, 64, false>), grid, block, 0, stream, a); break;
      default: hipLaunchKernelGGL((mx_tile_a4_kernel<64, 64, false>), grid, block, 0, stream, a); break;
    }
  } else {
    switch (p.tile) {
      case 0: hipLaunchKernelGGL((mx_tile_a16_kernel<256, 192>), grid, block, 0, stream, a); break;
      case 1: hipLaunchKernelGGL((mx_tile_a16_kernel<128, 128>), grid, block, 0, stream, a); break;
      case 2: hipLaunchKernelGGL((mx_tile_a16_kernel<128, 64>), grid, block, 0, stream, a); break;
      default: hipLaunchKernelGGL((mx_tile_a16_kernel<64, 64>), grid, block, 0, stream, a); break;
    }
  }
  W4_CHECK_LAUNCH();
  if (p.splits > 1) {
    // its rounding is for numbers; a NaN stays one where its low 16 bits are zero, as those that come of bf16
    // NaNs and of NaN scales are (tested with every kind of bf16 NaN)
    const size_t MN = (size_t)g.M * g.N;
    return launch_split_reduce(a.partial, p.splits, MN, MN, g.Y, stream);
  }
  return W4_OK;
}

}  // namespace w4

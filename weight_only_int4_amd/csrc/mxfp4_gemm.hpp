// Tiled products with MXFP4 weights, Y = X W_hat^T, for row counts at which the
// matrix cores are the bound: MXFP4 activations (mx_tile_a4_kernel) or bf16 ones
// (mx_tile_a16_kernel).
//
// A workgroup of four waves (2 x 2, one per SIMD) owns BM rows x BN channels, a wave FM x FN
// tiles of 16 x 16 in accumulation registers.  K goes in stages of 128 channels that travel
// from global memory straight into LDS (global_load_lds, no registers).  The weights are
// the matrix instruction's row operand, so a lane ends with four consecutive channels
// of one output row.
//
// One wave per SIMD, so that a tile is as large as the registers allow: the LDS traffic of a
// product falls with the tile's side.  (256 x 192 takes 252 + 248 of the 512 registers; 256 x 256
// all of them and 24 bytes a lane of scratch besides.)  What two waves would overlap, the
// single one overlaps itself: between its matrix instructions it reads the next stage's
// fragments and issues copies.  Measured at M = 2048, K = 5120, N = 17408, 4-bit: eight waves in
// one phase 179 us, two waves per SIMD in opposite phases 152, this 104 to 112 (3.3 to 3.5 PFLOP/s).
//
// What bounds that: three rounds of 40 stages at 0.78 us (from K and N varied one at a time), 94 in
// all, and 18 for three starts, the stores and the launch.  A stage's matrix instructions alone take
// 0.51 us on random data; with inputs in the caches a stage takes 0.75, and 0.58 on zeros
// (power); from memory 0.73 to 0.78 whatever the data, so there it is the copies' arrival.
// The third round is 84 % full: 18432 channels, three full rounds, take 112 us, 17408 take 110.
//
// LDS layout: position p of a row holds its 16-byte chunk p ^ f(row), with f chosen for each
// row length so that every pass of a fragment read covers all 64 banks once (measured with
// bf16 activations: 7.8 M cycles of conflicts down to 1.5 M at M = 2048, K = 2048, N = 6144).
//
// Scale bytes are read 16 at a time (four stages of a row): an LDS read of one byte per
// lane costs nearly as much as one of 16 (2.9 against 3.5 ns per wave).  Lane (r, q) keeps
// byte q of each stage's dword, packed into one register.
//
// Rows past M or N re-read the last row (their outputs are not stored).  When K is not a
// multiple of 128, copies of the last stage clamp to the blocks that exist and the lanes
// of the missing ones zero their operands.  Rows of the scale arrays are multiples of
// four bytes, at least 16 long (the caller pads them with zeros otherwise).
#pragma once

#include "gemm_core.hpp"
#include "mxfp4.hpp"

namespace w4 {

struct MxTileArgs {
  const void* X;            // [M][K] bf16, or [M][K/8] codes
  const uint8_t* xs;        // [M][ss] scale bytes (MXFP4 activations)
  const uint32_t* qweight;  // [N][K/8]
  const uint8_t* ws;        // [N][ss]
  int ss;                   // bytes of a scale row: a multiple of 4, at least 16
  int M, K, N;
  int tiles;                // tiles of the output
  int stages_per_split;     // stages of blockIdx.y: [y, y + 1) * stages_per_split, a multiple of 4
  uint16_t* Y;              // [M][N], or
  float* partial;           // [splits][M][N] when not NULL
};

// Barrier that the compiler moves nothing across.
__device__ __forceinline__ void mx_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  lds_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// Byte q of each of four dwords, packed in order; sel = q | (q + 4) << 8 selects byte q
// of the second and of the first source of v_perm_b32.
__device__ __forceinline__ uint32_t pack_bytes(u32x4 d, uint32_t sel) {
  const uint32_t lo = __builtin_amdgcn_perm(d[1], d[0], sel), hi = __builtin_amdgcn_perm(d[3], d[2], sel);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// The tile's outputs: lane (c, q) of tile (i, j) holds row c, channels 4 q .. 4 q + 3, so
// a store straight from there writes 32-byte pieces.  bf16 rows go through `stage`, this
// wave's own kMxStage<FN> bytes of LDS (16 rows, padded by 16 bytes against bank
// conflicts), and leave in 16-byte pieces of whole rows.
template <int FN>
constexpr int kMxStage = 16 * (FN * 32 + 16);

// Where N is not a multiple of eight (WHOLE false) the pieces are not aligned, and the last one
// of a row goes element by element.  (Aligned pieces of one element instead: M = 2047, K = 1536, N = 17401 took
// 83 us against 48.)
template <int FM, int FN, bool WHOLE>
__device__ __forceinline__ void mx_store_rows(const MxTileArgs& a, const f32x4 (&acc)[FM][FN], int m1, int n1,
                                              unsigned char* stage) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
  typedef u16x8 u16x8_unaligned __attribute__((aligned(2)));
  constexpr int kRow = FN * 32 + 16, kPieces = FN * 2;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const bf16x4 b = {(__bf16)acc[i][j][0], (__bf16)acc[i][j][1], (__bf16)acc[i][j][2], (__bf16)acc[i][j][3]};
      *reinterpret_cast<bf16x4*>(stage + r * kRow + j * 32 + q * 8) = b;
    }
    __builtin_amdgcn_wave_barrier();            // LDS operations of one wave complete in order
#pragma unroll
    for (int p = lane; p < 16 * kPieces; p += 64) {
      const int row = p / kPieces, c = p % kPieces;
      const int m = m1 + 16 * i + row, n = n1 + 8 * c;
      if (m >= a.M || n >= a.N) continue;
      uint16_t* y = a.Y + (size_t)m * a.N + n;
      const u16x8 v = *reinterpret_cast<const u16x8*>(stage + row * kRow + c * 16);
      if (WHOLE) {
        *reinterpret_cast<u16x8*>(y) = v;
      } else if (n + 8 <= a.N) {
        *reinterpret_cast<u16x8_unaligned*>(y) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
          if (n + e < a.N) y[e] = v[e];
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// SPLIT: the launch may write partial outputs.
template <int FM, int FN, bool SPLIT>
__device__ __forceinline__ void mx_store_tile(const MxTileArgs& a, const f32x4 (&acc)[FM][FN], int m1, int n1,
                                              unsigned char* stage) {
  if (!SPLIT || !a.partial) {
    if ((a.N & 7) == 0) mx_store_rows<FM, FN, true>(a, acc, m1, n1, stage);
    else mx_store_rows<FM, FN, false>(a, acc, m1, n1, stage);
    return;
  }
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  float* part = a.partial + (size_t)blockIdx.y * a.M * a.N;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m1 + 16 * i + r;
    if (m >= a.M) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int n = n1 + 16 * j + 4 * q;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < a.N) part[(size_t)m * a.N + n + e] = acc[i][j][e];
    }
  }
}

// MXFP4 activations.  Four waves (2 x 2), one per SIMD, BM / 2 rows x BN / 2 channels each.
// CHAIN: a workgroup takes the tiles blockIdx.x + i gridDim.x in turn, and the copies run on from one tile
// to the next, so that a tile's outputs are stored while the next one's first stages arrive
// (needs stages in fours, and M >= BM and N >= BN).  Inputs from memory, M = 2048, N = 17408: K = 2048
// 56.7 us against 58.6, K = 5120 113.5 against 121.7; N = 17401: 116 against 127; M = 4096, K = 5120, N = 17408:
// 207 against 223.
template <int BM, int BN, bool CHAIN>
__global__ __launch_bounds__(256, 1) void mx_tile_a4_kernel(MxTileArgs a) {
  constexpr int W = 4;                          // waves
  static_assert(BM % 64 == 0 && BN % 64 == 0, "copies and scale copies cover 64 rows");
  constexpr int FM = BM / 32, FN = BN / 32, F = FM + FN, T = FM * FN;
  constexpr int kRows = BM + BN;                // activation rows, then channels
  constexpr int kSlot = kRows * 128, kScales = 2 * kSlot;
  constexpr int C = kRows / 8 / W;              // 1 KB copies (8 rows) per wave and pair of stages
  constexpr int CS = kRows / 16 / W;            // 1 KB copies (16 rows) per wave and 16 stages of scales
  // with CHAIN the outputs have LDS of their own: the slots belong to the next tile by then
  constexpr int kOut = CHAIN ? kScales + kRows * 64 : 0;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[kScales + kRows * 64 + (CHAIN ? W * kMxStage<FN> : 0)];
  constexpr int kEvery = T / C;                 // matrix instructions per copy
  static_assert(kEvery >= 1 && C * kEvery < 2 * T, "a pair's copies fit two steps");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int r = lane & 15, q = lane >> 4;
  const int MT = (a.M + BM - 1) / BM, NT = (a.N + BN - 1) / BN;
  const int KB = a.K / kMxBlock, KT = (KB + 3) / 4;
  const int kt0 = blockIdx.y * a.stages_per_split, kt1 = min(KT, kt0 + a.stages_per_split);
  const int n_stages = kt1 - kt0;
  const int rem = KB & 3;                       // blocks of the last stage, 0: all four
  const uint32_t smem_base = (uint32_t)(uintptr_t)smem;
  const uint32_t rowb = (uint32_t)a.K / 2u;

  // Stages travel in pairs, so that a row's piece is a whole 128-byte line (64-byte pieces
  // cost the L1 as much: 505 against 254 ns per 32 KB and CU).  Copy u of this wave is
  // unit wave + 4 u: rows 8 (wave + 4 u) + lane / 8, position lane % 8 holding chunk
  // (lane % 8) ^ ((row >> 1) & 7), the same for every u.
  // With CHAIN a tile at the edge moves back inside, so that one lane offset serves every copy (it
  // computes outputs that its neighbour has too, the same bits); otherwise rows past the
  // edge re-read the last one.
  constexpr int kOff = CHAIN ? 1 : C, kSoff = CHAIN ? 1 : CS;
  uint32_t off[kOff], soff[kSoff];
  const unsigned char *xb, *wb, *xsb, *wsb;
  int m0, n0;                                   // the tile that copies are made of
  auto is_x = [](int u) { return u < BM / 8 / W; };            // compile-time: activations first
  auto set_tile = [&](int tile) {
    int tm, tn;
    tile_coords(tile, MT, NT, tm, tn);
    m0 = CHAIN ? min(tm * BM, a.M - BM) : tm * BM;
    n0 = CHAIN ? min(tn * BN, a.N - BN) : tn * BN;
    xb = static_cast<const unsigned char*>(a.X) + (size_t)m0 * rowb;
    wb = reinterpret_cast<const unsigned char*>(a.qweight) + (size_t)n0 * rowb;
    xsb = a.xs + (size_t)m0 * a.ss;
    wsb = a.ws + (size_t)n0 * a.ss;
  };
  set_tile(blockIdx.x);
  if constexpr (CHAIN) {
    off[0] = (uint32_t)(wave * 8 + (lane >> 3)) * rowb;
    soff[0] = (uint32_t)(wave * 16 + (lane >> 2)) * (uint32_t)a.ss;
  } else {
    const int mlast = a.M - 1 - m0, nlast = a.N - 1 - n0;
#pragma unroll
    for (int u = 0; u < C; ++u) {
      const int row = (wave + W * u) * 8 + (lane >> 3) - (is_x(u) ? 0 : BM);
      off[u % kOff] = (uint32_t)min(row, is_x(u) ? mlast : nlast) * rowb;
    }
#pragma unroll
    for (int u = 0; u < CS; ++u) {
      const int row = (wave + W * u) * 16 + (lane >> 2) - (u < BM / 16 / W ? 0 : BM);
      soff[u % kSoff] = (uint32_t)min(row, u < BM / 16 / W ? mlast : nlast) * (uint32_t)a.ss;
    }
  }
  const int chunk = (lane & 7) ^ (((wave * 8 + (lane >> 3)) >> 1) & 7);
  // Copies of pair p of stages counted from kt0, into slot p % 2; past the end of the last tile
  // its last pair is copied again, into a slot that nothing reads any more.
  struct Src {
    const unsigned char *x, *w;
    uint32_t c;
  };
  auto source = [&](int pair) {
    const int kt = kt0 + 2 * min(pair, (n_stages - 1) >> 1);
    return Src{xb + (size_t)kt * 64, wb + (size_t)kt * 64, 16u * (uint32_t)min(chunk, min(8, KB - 4 * kt) - 1)};
  };
  auto copy = [&](const Src& s, int slot, int u) {
    const uint32_t rows = CHAIN ? W * 8 * (is_x(u) ? u : u - BM / 8 / W) : 0;
    lds_copy16(off[u % kOff] + rows * rowb + s.c, is_x(u) ? s.x : s.w, 
               smem_base + (uint32_t)(slot * kSlot + (wave + W * u) * 1024));
  };
  // A group's (four stages') first stage, moved back where the row ends before the group does.
  auto group_start = [&](int group) { return max(0, min(kt0 + 4 * group, KT - 4)); };
  // Scales of groups 4 b .. 4 b + 3: 64 bytes of a row, four lanes to a row, position p of row r
  // holding group 4 b + (p ^ ((r >> 2) & 3)).  (16 bytes of a row at a time would cost the L1 four
  // times the lines, a third of what the codes cost.)
  auto copy_scales = [&](int b) {
    const uint32_t c = 4u * (uint32_t)group_start(4 * b + ((lane & 3) ^ ((lane >> 4) & 3)));
#pragma unroll
    for (int u = 0; u < CS; ++u) {
      const bool x = u < BM / 16 / W;
      const uint32_t rows = CHAIN ? W * 16 * (x ? u : u - BM / 16 / W) : 0;
      lds_copy16(soff[u % kSoff] + rows * (uint32_t)a.ss + c, x ? xsb : wsb,
                 smem_base + (uint32_t)(kScales + (wave + W * u) * 1024));
    }
  };

  f32x4 acc[FM][FN];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  // fragment e: channels for e < FN, activation rows after; row 16 e' + r of this wave's
  // part ((row >> 1) & 7 does not depend on e'), chunk 4 h + q of the pair's stage h
  const uint32_t swz = (uint32_t)((q ^ ((r >> 1) & 7)) * 16);
  const uint32_t xfrag = (uint32_t)((wm * FM * 16 + r) * 128) + swz;
  const uint32_t wfrag = (uint32_t)((BM + wn * FN * 16 + r) * 128) + swz;
  const uint32_t xsrow = (uint32_t)(kScales + (wm * FM * 16 + r) * 64);
  const uint32_t wsrow = (uint32_t)(kScales + (BM + wn * FN * 16 + r) * 64);
  const uint32_t sel = (uint32_t)(q | ((q + 4) << 8)) | 0x0C0C0000u;

  u32x4 f[2][F];                                // fragments of this stage and the next
  uint32_t sc[F], scn[F];                       // packed scale bytes of four stages, and the next four
  auto read = [&](int buf, int j4, int e) {     // stage j4 of four: slot j4 / 2, half j4 % 2
    const uint32_t o = e < FN ? (wfrag ^ (uint32_t)(64 * (j4 & 1))) + e * 2048
                              : (xfrag ^ (uint32_t)(64 * (j4 & 1))) + (e - FN) * 2048;
    f[buf][e] = *reinterpret_cast<const u32x4*>(smem + (j4 >> 1) * kSlot + o);
  };
  auto read_scales = [&](int group, int e) {
    const uint32_t o = e < FN ? wsrow + e * 1024 : xsrow + (e - FN) * 1024;
    return *reinterpret_cast<const u32x4*>(smem + o + (uint32_t)(((group & 3) ^ ((r >> 2) & 3)) * 16));
  };
  auto shift_of = [&](int group) { return 8 * min(3, kt0 + 4 * group - group_start(group)); };

  // One stage; J = stage % 4 selects its slot, half and scale byte.  The stage's fragments are in
  // registers when it starts, and between the matrix instructions the wave reads the next
  // stage's (scales: the next four stages').  So a pair's slot is free when its second stage
  // starts: that step waits for the next pair, meets the other waves and refills the
  // slot, copies first, two stages before they are needed.
  // `ahead`: what is copied and read from here on belongs to the next tile (the last three of a
  // tile's stages).
  auto step = [&](auto jc, int s, bool ahead) {
    constexpr int J = decltype(jc)::value;
    constexpr int cur = J & 1, nxt = cur ^ 1;
    const int stage = s + J;
    if constexpr (cur == 1) {
      wait_vmcnt<0>();
      mx_barrier();
    }
    const int pair = (stage >> 1) + (cur == 1 ? 2 : 1);
    const Src src = source(ahead ? pair - (n_stages >> 1) : pair);
    if (rem != 0 && kt0 + stage == KT - 1 && q >= rem) {
#pragma unroll
      for (int j = 0; j < FN; ++j) f[cur][j] = u32x4{0, 0, 0, 0};
    }
    // Between the matrix instructions: a copy every kEvery of them, from the second step of
    // a pair on into the first step of the next (in a burst they would fill the memory
    // pipeline and hold back the wave's matrix instructions); reads one each.
    constexpr int kLag = 3;                     // a scale read is packed three operations later
    constexpr int kCopies = C + 1;              // the pair's, and every other pair scales
    constexpr int kReads = F + (J == 3 ? F + kLag : 0);
    constexpr int kPer = (kReads + T - 1) / T;  // more than one where the tile is small
    u32x4 raw[F];
    const int group = ahead ? 0 : (stage + 1) >> 2, shift = J == 3 ? shift_of(group) : 0;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int tc = cur == 1 ? t : T + t;      // matrix instructions since the pair's slot was free
      if (tc % kEvery == 0 && tc / kEvery < kCopies) {
        const int u = tc / kEvery;
        constexpr int slot = cur == 1 ? J >> 1 : (J >> 1) ^ 1;
        // the last group of the scales in LDS is in registers by now
        if (u == 0) { if (J == 1 && (ahead || ((stage + 3) & 15) == 0)) copy_scales(ahead ? 0 : (stage + 3) >> 4); }
        else copy(src, slot, u - 1);
      }
#pragma unroll
      for (int o = t * kPer; o < (t + 1) * kPer; ++o) {
        if (o < F) {
          read(nxt, (J + 1) % 4, o);
        } else if (o < kReads) {
          const int e = o - F;
          if (e >= kLag) scn[e - kLag] = pack_bytes(raw[e - kLag], sel) >> shift;
          if (e < F) raw[e] = read_scales(group, e);
        }
      }
      const int i = t / FN, j = t % FN;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(f[cur][j]), mx_operand(f[cur][FN + i]),
                                                                  acc[i][j], 4, 4, J, (int)sc[j], J, (int)sc[FN + i]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (J == 3) {
#pragma unroll
      for (int e = 0; e < F; ++e) sc[e] = scn[e];
    }
  };

  constexpr int kEarly = (T - 1) / kEvery < C ? (T - 1) / kEvery : C;
  int tile = blockIdx.x;
  copy_scales(0);
  {
    const Src p0 = source(0), p1 = source(1);
#pragma unroll
    for (int u = 0; u < C; ++u) copy(p0, 0, u);
    // of pair 1 the copies that a second step would have issued; the first step issues the rest
#pragma unroll
    for (int u = 0; u < kEarly; ++u) copy(p1, 1, u);
  }
  wait_vmcnt<kEarly>();
  mx_barrier();
#pragma unroll
  for (int e = 0; e < F; ++e) {
    read(0, 0, e);
    sc[e] = pack_bytes(read_scales(0, e), sel) >> shift_of(0);
  }
  for (;;) {
    const int next = tile + (int)gridDim.x;
    const bool more = CHAIN && next < a.tiles;
    const int m = m0 + wm * FM * 16, n = n0 + wn * FN * 16;
    clear();
    for (int s = 0; s < n_stages; s += 4) {
      const bool ahead = more && s + 4 >= n_stages;
      // the conditions also keep the compiler from moving a step's products into a later one
      step(std::integral_constant<int, 0>{}, s, false);
      if (ahead) set_tile(next);
      if (s + 1 < n_stages) step(std::integral_constant<int, 1>{}, s, ahead);
      if (s + 2 < n_stages) step(std::integral_constant<int, 2>{}, s, ahead);
      if (s + 3 < n_stages) step(std::integral_constant<int, 3>{}, s, ahead);
    }
    if constexpr (!CHAIN) {
      wait_vmcnt<0>();
      lds_barrier();                            // no copy and no read of the slots is left
    }
    mx_store_tile<FM, FN, !CHAIN>(a, acc, m, n, smem + kOut + wave * kMxStage<FN>);
    if (!more) break;
    tile = next;
  }
  wait_vmcnt<0>();                              // copies past the end
}

// bf16 activations.  Four waves (2 x 2), one per SIMD, BM / 2 rows x BN / 2 channels each.
// A stage of 128 channels is four steps of 32: step v multiplies word v of every MX block
// (channels 8 v .. 8 v + 7 of it), expanded to bf16, with chunk 4 q + v of the
// activation rows.  Two slots; a slot is free when the fragments of its last step are read.
// M = 2048, K = 2048, N = 6144: 40 to 44 us, 1.2 to 1.3 PFLOP/s: 16 stages of 2.0 us (1.9 on zeros), and
// 12 for the start, the stores and the launch; the matrix instructions alone, on random
// data, 31, and the expansion of the weights shares their issue slots.
template <int BM, int BN>
__global__ __launch_bounds__(256, 1) void mx_tile_a16_kernel(MxTileArgs a) {
  constexpr int W = 4;                          // waves
  static_assert(BM % 64 == 0 && BN % 64 == 0, "copies and scale copies cover 64 rows");
  constexpr int FM = BM / 32, FN = BN / 32, T = FM * FN;
  constexpr int kX = 0, kW = BM * 256, kSlot = kW + BN * 64;
  constexpr int kScales = 2 * kSlot;
  constexpr int CX = BM / 4 / W, CW = BN / 16 / W, C = CX + CW;   // 1 KB copies per wave and stage
  constexpr int kSUnits = BN / 32, CS = (kSUnits + W - 1) / W;    // 1 KB copies (32 rows) per wave and 8 stages of scales
  __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * kSlot + BN * 32];
  constexpr int kEvery = 2 * T / C;             // matrix instructions per copy: over two of the four steps
  static_assert(kEvery >= 1 && C * kEvery < 4 * T, "a stage's copies fit its steps");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int r = lane & 15, q = lane >> 4;
  int tm, tn;
  tile_coords(blockIdx.x, (a.M + BM - 1) / BM, (a.N + BN - 1) / BN, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int KB = a.K / kMxBlock, KT = (KB + 3) / 4;
  const int kt0 = blockIdx.y * a.stages_per_split, kt1 = min(KT, kt0 + a.stages_per_split);
  const int n_stages = kt1 - kt0;
  const int rem = KB & 3;                       // blocks of the last stage, 0: all four
  const uint32_t smem_base = (uint32_t)(uintptr_t)smem;
  const uint32_t xrowb = (uint32_t)a.K * 2u, wrowb = (uint32_t)a.K / 2u;
  const unsigned char* xb = static_cast<const unsigned char*>(a.X) + (size_t)m0 * xrowb;
  const unsigned char* wb = reinterpret_cast<const unsigned char*>(a.qweight) + (size_t)n0 * wrowb;
  const unsigned char* wsb = a.ws + (size_t)n0 * a.ss;
  const int mlast = a.M - 1 - m0, nlast = a.N - 1 - n0;

  // Activation copy u: rows 4 (wave + 4 u) + lane / 16, position lane % 16 holding chunk
  // (lane % 16) ^ mx_swizzle16(row & 15), and row & 15 is the same for every u.  Code copy u: rows
  // 16 (wave + 4 u) + lane / 4, position lane % 4 holding chunk (lane % 4) ^ ((row >> 2) & 3).
  uint32_t xoff[CX], woff[CW], soff[CS];
#pragma unroll
  for (int u = 0; u < CX; ++u) xoff[u] = (uint32_t)min((wave + W * u) * 4 + (lane >> 4), mlast) * xrowb;
#pragma unroll
  for (int u = 0; u < CW; ++u) woff[u] = (uint32_t)min((wave + W * u) * 16 + (lane >> 2), nlast) * wrowb;
#pragma unroll
  for (int u = 0; u < CS; ++u)
    soff[u] = (uint32_t)min(min(wave + W * u, kSUnits - 1) * 32 + (lane >> 1), nlast) * (uint32_t)a.ss;
  const int xchunk = (lane & 15) ^ mx_swizzle16((wave * 4 + (lane >> 4)) & 15), wchunk = (lane & 3) ^ ((lane >> 4) & 3);
  // Copies of a stage counted from kt0 into slot stage % 2; past the end the last stage is
  // copied again, into a slot that nothing reads any more.
  struct Src {
    const unsigned char *x, *w;
    uint32_t cx, cw;
  };
  auto source = [&](int stage) {
    const int kt = kt0 + min(stage, n_stages - 1);
    const int blocks = rem != 0 && kt == KT - 1 ? rem : 4;
    return Src{xb + (size_t)kt * 256, wb + (size_t)kt * 64, 16u * (uint32_t)min(xchunk, 4 * blocks - 1),
               16u * (uint32_t)min(wchunk, blocks - 1)};
  };
  auto copy = [&](const Src& s, uint32_t slot, int u) {
    if (u < CX) lds_copy16(xoff[u] + s.cx, s.x, smem_base + slot + (uint32_t)(kX + (wave + W * u) * 1024));
    else lds_copy16(woff[u - CX] + s.cw, s.w, smem_base + slot + (uint32_t)(kW + (wave + W * (u - CX)) * 1024));
  };
  // Groups of four stages as above; scales of groups 2 b and 2 b + 1, 32 bytes of a row, position
  // p of row r holding group 2 b + (p ^ ((r >> 3) & 1)).
  auto group_start = [&](int group) { return max(0, min(kt0 + 4 * group, KT - 4)); };
  auto copy_scales = [&](int b) {
    const uint32_t c = 4u * (uint32_t)group_start(2 * b + ((lane & 1) ^ ((lane >> 4) & 1)));
#pragma unroll
    for (int u = 0; u < CS; ++u)
      lds_copy16(soff[u] + c, wsb, smem_base + (uint32_t)(kScales + min(wave + W * u, kSUnits - 1) * 1024));
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint32_t xrow = (uint32_t)(kX + (wm * FM * 16 + r) * 256);
  const uint32_t wfrag = (uint32_t)(kW + (wn * FN * 16 + r) * 64 + ((q ^ ((r >> 2) & 3)) * 16));
  const uint32_t wsrow = (uint32_t)(kScales + (wn * FN * 16 + r) * 32);
  const uint32_t sel = (uint32_t)(q | ((q + 4) << 8)) | 0x0C0C0000u;

  bf16x8 x[2][FM];                              // activation fragments of this step and the next
  u32x4 w[FN], wn_[FN];                         // codes of this stage and the next
  uint32_t sc[FN], scn[FN];                     // packed scale bytes of four stages, and the next four
  auto read_x = [&](int buf, uint32_t slot, int v, int i) {
    x[buf][i] = *reinterpret_cast<const bf16x8*>(smem + slot + xrow + i * 4096 + (uint32_t)(((4 * q + v) ^ mx_swizzle16(r)) * 16));
  };
  auto read_w = [&](uint32_t slot, int j) { return *reinterpret_cast<const u32x4*>(smem + slot + wfrag + j * 1024); };
  auto read_scales = [&](int group, int j) {
    return *reinterpret_cast<const u32x4*>(smem + wsrow + j * 512 + (uint32_t)(((group & 1) ^ ((r >> 3) & 1)) * 16));
  };
  auto shift_of = [&](int group) { return 8 * min(3, kt0 + 4 * group - group_start(group)); };

  // One stage; J = stage % 4 selects the scale byte, J % 2 the slot.  The fragments of a step are read
  // during the step before.  The last step of a stage waits for the next stage's
  // copies, meets the other waves and starts refilling the slot; the copies go on into
  // the next stage's first steps.
  auto stage_steps = [&](auto jc, int s) {
    constexpr int J = decltype(jc)::value;
    constexpr uint32_t slot = (J & 1) * kSlot, other = kSlot - slot;
    const int stage = s + J;
    const bool last = rem != 0 && kt0 + stage == KT - 1;
    if (last && q >= rem) {
#pragma unroll
      for (int j = 0; j < FN; ++j) w[j] = u32x4{0, 0, 0, 0};
    }
    Src src = source(stage + 1);                // what the previous stage's last step began
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int cur = v & 1;
      if (v == 3) {
        wait_vmcnt<0>();
        mx_barrier();
        src = source(stage + 2);
      }
      if (last && q >= rem) {
        // the other operand of a missing block is zero too: infinities times zero are NaN
#pragma unroll
        for (int i = 0; i < FM; ++i) x[cur][i] = __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0});
      }
      u32x4 raw[FN];
      const int group = (stage + 1) >> 2, shift = J == 3 && v == 3 ? shift_of(group) : 0;
      bf16x8 wv[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) wv[j] = mx_expand(w[j][v], mx_scale((sc[j] >> (8 * J)) & 255u));
      // reads: the next step's activations; in the last step also the next stage's codes (and
      // at the end of four stages scales), packed a few operations later
      constexpr int kLag = 2;
      const int kReads = FM + (v == 3 ? FN + (J == 3 ? FN + kLag : 0) : 0);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int tc = v == 3 ? t : (v + 1) * T + t;      // matrix instructions since the slot was free
        if (tc % kEvery == 0 && tc / kEvery <= C) {
          const int u = tc / kEvery;
          // the last group of the scales in LDS is in registers by now
          if (u == 0) { if (J == 1 && ((stage + 3) & 7) == 0) copy_scales((stage + 3) >> 3); }
          else copy(src, v == 3 ? slot : other, u - 1);
        }
        const int per = (kReads + T - 1) / T;
#pragma unroll
        for (int o = t * per; o < (t + 1) * per && o < kReads; ++o) {
          if (o < FM) {
            if (v == 3) read_x(0, other, 0, o);
            else read_x(cur ^ 1, slot, v + 1, o);
          } else if (o < FM + FN) {
            wn_[o - FM] = read_w(other, o - FM);
          } else {
            const int e = o - FM - FN;
            if (e >= kLag) scn[e - kLag] = pack_bytes(raw[e - kLag], sel) >> shift;
            if (e < FN) raw[e] = read_scales(group, e);
          }
        }
        const int i = t / FN, j = t % FN;
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j], x[cur][i], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      w[j] = wn_[j];
      if constexpr (J == 3) sc[j] = scn[j];
    }
  };

  constexpr int kEarly = (T - 1) / kEvery < C ? (T - 1) / kEvery : C;
  copy_scales(0);
  {
    const Src s0 = source(0), s1 = source(1);
#pragma unroll
    for (int u = 0; u < C; ++u) copy(s0, 0, u);
    // of stage 1 the copies that a last step would have issued; the first stage issues the rest
#pragma unroll
    for (int u = 0; u < kEarly; ++u) copy(s1, kSlot, u);
  }
  wait_vmcnt<kEarly>();
  mx_barrier();
#pragma unroll
  for (int i = 0; i < FM; ++i) read_x(0, 0, 0, i);
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    w[j] = read_w(0, j);
    sc[j] = pack_bytes(read_scales(0, j), sel) >> shift_of(0);
  }
  for (int s = 0; s < n_stages; s += 4) {
    stage_steps(std::integral_constant<int, 0>{}, s);
    if (s + 1 < n_stages) stage_steps(std::integral_constant<int, 1>{}, s);
    if (s + 2 < n_stages) stage_steps(std::integral_constant<int, 2>{}, s);
    if (s + 3 < n_stages) stage_steps(std::integral_constant<int, 3>{}, s);
  }
  wait_vmcnt<0>();
  lds_barrier();                                // no copy and no read of the slots is left
  mx_store_tile<FM, FN, true>(a, acc, m0 + wm * FM * 16, n0 + wn * FN * 16, smem + wave * kMxStage<FN>);
}

}  // namespace w4

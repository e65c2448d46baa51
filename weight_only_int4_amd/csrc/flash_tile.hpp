// Attention of 32 queries a wave over tiles of 64 keys that the waves of a workgroup share, on the
// bf16 matrix cores: the walk of the prompt kernel and of the decode kernel's shared prefix.
//
// Scores come transposed, S^T = K Q^T (v_mfma_f32_32x32x16_bf16, keys as rows): lane (query l % 32,
// half h = l / 32) then holds 16 scores of its own query per 32 keys, so that maximum and sum need one
// exchange between halves, and its p, rounded to bf16, are the operand of O^T += V^T P^T as they
// stand: step s of 16 keys takes keys 16 s + 4 h + {0..3} and 8 more, and V^T is read in that
// order by the transposing LDS read.
//
// What bounds it: per tile and wave 32 matrix instructions of 32 cycles (head 128; 16 for head 64) and
// about 100 vector instructions of 4, of which 32 exp2 take 8, and every matrix instruction holds the vector
// ALU up for about 9; on random data the chip also lowers its clock (1 x 8192 tokens of 16 heads of 128: 249 us,
// 1.1 PFLOP/s of the 1.41 that a large matrix product reaches; on zeros 204).  Two waves a SIMD overlap the one with
// the other.  That is a long walk's; a short one is bound by what comes before and after its tiles, about 9 us of a
// workgroup at head 64 (12 x 2047 ragged, 32 heads: 96 us, of which the tiles would take 61).
// Measured and not kept: the weights of tile t + 1 woven between
// the matrix instructions of tile t in one wave (no change at head 128, where another 50 registers are no loss;
// 97 -> 119 us at head 64, where they cost waves), the two waves of a SIMD in opposite phases by a second barrier
// or by s_setprio (no change), 64 queries a wave with all 512 registers (1 x 8192: 395 us), tiles of 128 keys at
// head 64 (97 -> 110), a barrier every two tiles (267 -> 269 and 100 -> 104).
#pragma once

#include <math.h>

#include <type_traits>

#include "gemm_core.hpp"
#include "serve.hpp"

namespace w4 {

constexpr int kTile = 64;                     // keys of a tile
constexpr float kLog2e = 1.44269504088896340736f;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
typedef __attribute__((address_space(3))) bf16x8* lds_bf16x8;

// lds_copy16 that LDS reads may pass: for copies into slots that nobody reads before the next barrier.
// The five wait states are what a vector write to the base (v_readfirstlane, where the compiler comes by
// it that way) needs before a memory instruction reads it: the compiler does not look into the asm.
__device__ __forceinline__ void lds_copy16_free(uint32_t off, const void* base, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds));
}

template <int HEAD, int WAVES>
struct Flash {
  static constexpr int kSteps = HEAD / 16;    // matrix steps of a score
  static constexpr int kDb = HEAD / 32;       // 32-dim blocks of the output
  static constexpr int kRow = HEAD * 2;       // bytes of an LDS row
  static constexpr int kChunks = HEAD / 8;    // 16-byte pieces of a row
  static constexpr int kTileBytes = kTile * kRow;
  static constexpr int kSlots = 2;            // of K, and of V
  static constexpr int kLds = 2 * kSlots * kTileBytes;
  static constexpr int kCopies = kTileBytes / (WAVES * 1024);        // LDS copies (1 KB) of a wave per tile, K or V
  static constexpr int kPerCopy = 64 / kChunks;                      // rows of one copy
  static constexpr int kRowsApart = WAVES * kPerCopy;                // rows between a wave's copies
  static constexpr int kV = 4 * kDb, kK = 2 * kSteps;                // matrix steps of values, of scores
  static constexpr int kAhead = 4;
  // LDS rows hold their 16-byte pieces exchanged, so that reads meet distinct banks: piece c of
  // row r at c ^ k_swap(r) (score operand: 16 rows, one piece each) or c ^ v_swap(r) (transposing
  // read: 4 rows, 64 bytes each).
  static __device__ __forceinline__ int k_swap(int r) { return HEAD == 128 ? r & 15 : (r >> 1) & 7; }
  static __device__ __forceinline__ int v_swap(int r) { return HEAD == 128 ? (r & 3) * 4 : ((r >> 1) & 1) * 4; }

  uint32_t kaddr, vaddr, lds_k, lds_v;        // operands inside slot 0; copies' targets
  bf16x8 qf[kSteps], pf[4];                   // queries, weights of a tile
  f32x16 acc[kDb], s[2];                      // outputs, scores of 32 keys each
  float c, mref, mc, lsum;                    // exponent: c s + mc, mc = -c mref

  __device__ __forceinline__ void init(const unsigned char* smem, float scale) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l32 = lane & 31, h = lane >> 5;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const unsigned char*)smem;
    lds_k = lds0 + wave * 1024;
    lds_v = lds_k + kSlots * kTileBytes;
    // piece 2 st + h (4 db + ..) of the exchanged rows: one bit pattern away from the first
    kaddr = lds0 + l32 * kRow + 16 * (h ^ k_swap(l32));
    const int i = lane & 15, r = 4 * h + (i >> 2);
    vaddr = lds0 + kSlots * kTileBytes + r * kRow + 16 * ((2 * ((lane >> 4) & 1) + ((i & 3) >> 1)) ^ v_swap(r)) +
            8 * (i & 1);
    c = scale * kLog2e;
    mref = -INFINITY, mc = 0.0f, lsum = 0.0f;
#pragma unroll
    for (int db = 0; db < kDb; ++db) acc[db] = f32x16{};
  }

  // this lane's row of a copy, and its piece in K and in V rows
  static __device__ __forceinline__ int copy_row() {
    return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * kPerCopy + (threadIdx.x & 63) / kChunks;
  }
  static __device__ __forceinline__ uint32_t k_piece() { return 16 * ((threadIdx.x & 63) % kChunks ^ k_swap(copy_row())); }
  static __device__ __forceinline__ uint32_t v_piece() { return 16 * ((threadIdx.x & 63) % kChunks ^ v_swap(copy_row())); }

  __device__ __forceinline__ void load_q(const uint16_t* q) {
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
      qf[st] = *reinterpret_cast<const bf16x8*>(q + 8 * ((threadIdx.x & 63) >> 5) + 16 * st);
  }

  // score step i: keys 32 (i % 2) .., dims 16 (i / 2) ..
  __device__ __forceinline__ bf16x8 read_k(uint32_t base, int i) const {
    return *(lds_bf16x8)(uintptr_t)((base ^ (32 * (i / 2))) + i % 2 * 32 * kRow);
  }
  __device__ __forceinline__ void multiply_k(bf16x8 kf, int i) {
    s[i % 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[i / 2], i < 2 ? f32x16{} : s[i % 2], 0, 0, 0);
  }
  // value step i: keys 16 (i / kDb) .., dims 32 (i % kDb) ..
  __device__ __forceinline__ bf16x8 read_v(uint32_t base, int i) const {
    const uint32_t at = (base ^ (64 * (i % kDb))) + 16 * (i / kDb) * kRow;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(uintptr_t)at);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(uintptr_t)(at + 8 * kRow));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  __device__ __forceinline__ void multiply_v(bf16x8 vf, int i) {
    acc[i % kDb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[i / kDb], acc[i % kDb], 0, 0, 0);
  }

  // Raises the reference to the largest score (and scales what was summed with the old one).  A row that
  // has seen nothing keeps exponents of -infinity.
  __device__ __forceinline__ void raise() {
    float m = mref;
#pragma unroll
    for (int r = 0; r < 32; ++r) m = fmaxf(m, s[r >> 4][r & 15]);
    const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    m = fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
    const float corr = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((mref - m) * c);
    lsum *= corr;
#pragma unroll
    for (int db = 0; db < kDb; ++db) acc[db] *= corr;
    mref = m;
    mc = m == -INFINITY ? 0.0f : -m * c;
  }

  // The weights of a tile and their sum: of the rounded p, as the product with V has them.  (The dot products
  // keep the matrix unit for a while; additions in their place: 95 -> 116 us at head 64, no change at 128.)
  __device__ __forceinline__ float weights() {
    const bf16x2 ones = {(__bf16)1.0f, (__bf16)1.0f};
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const f32x16& x = s[k >> 1];
        const int r = 8 * (k & 1) + j;
        const bf16x2 p = {(__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(x[r], c, mc)),
                          (__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(x[r + 1], c, mc))};
        sum[j >> 1 & 1] = __builtin_amdgcn_fdot2_f32_bf16(p, ones, sum[j >> 1 & 1], false);
        pf[k][j] = p[0], pf[k][j + 1] = p[1];
      }
    return sum[0] + sum[1];
  }

  // Tiles 0 .. tiles - 1 of the workgroup (at least one); this wave takes the first `mine` of them, and
  // calls mask(t), which lays -infinity over scores that are not seen, for those from `masked` on (without
  // MANY: the last one at most).
  // copy(kv, t, j, lds): copy j of K's (0) or V's (1) tile t; per kv the tiles come in order, the last one
  // several times.
  // One barrier a tile, between its weights and its products (values of the tile, scores of the next):
  // behind it nobody reads K of tile t or V of tile t - 1 any more; the copies of K of tile t + 2 and V of
  // tile t + 1 are issued among the products and have to be there at the next.
  template <bool MANY, typename Copy, typename Mask>
  __device__ __forceinline__ void walk(int tiles, int mine, int masked, Copy copy, Mask mask) {
    int t = 0;
    auto to_k = [&](int slot, int j) { return lds_k + slot * kTileBytes + j * WAVES * 1024; };
    auto to_v = [&](int slot, int j) { return lds_v + slot * kTileBytes + j * WAVES * 1024; };
    auto copies = [&](int i) {                // copy i of a tile's, first K's, then V's
      if (i < kCopies) copy(0, min(t + 2, tiles - 1), i, to_k(t & 1, i));
      else copy(1, min(t + 1, tiles - 1), i - kCopies, to_v((t & 1) ^ 1, i - kCopies));
    };
    // The values of tile t and the scores of the next, in this order: operands are read four matrix
    // instructions ahead, copies go between.
    auto products = [&](auto with_values, auto with_scores, int slot) {
      constexpr int first = with_values ? 0 : kV, end = with_scores ? kV + kK : kV;
      const uint32_t vb = opaque_vgpr(vaddr + (t & 1) * kTileBytes), kb = opaque_vgpr(kaddr + slot * kTileBytes);
      bf16x8 ring[kAhead];
      auto read = [&](int i) {
        if (i < end) ring[i % kAhead] = i < kV ? read_v(vb, i) : read_k(kb, i - kV);
      };
#pragma unroll
      for (int i = first; i < first + kAhead; ++i) read(i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = first; i < end; ++i) {
        if (i < kV) multiply_v(ring[i % kAhead], i);
        else multiply_k(ring[i % kAhead], i - kV);
        read(i + kAhead);
        if (with_values && i % 2 == 1 && i / 2 < 2 * kCopies) copies(i / 2);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    auto turn = [&]() {                       // weights -> products
      wait_vmcnt<0>();
      lds_barrier();
    };
#pragma unroll
    for (int j = 0; j < kCopies; ++j) copy(0, 0, j, to_k(0, j));
#pragma unroll
    for (int j = 0; j < kCopies; ++j) copy(1, 0, j, to_v(0, j));
#pragma unroll
    for (int j = 0; j < kCopies; ++j) copy(0, min(1, tiles - 1), j, to_k(1, j));
    wait_vmcnt<0>();
    lds_barrier();
    if (mine > 0) {
      products(no, yes, 0);
      const int hot = MANY ? min(mine - 1, masked) : mine - 1;
      bool unset = false;                     // a row without a reference: its scores were all -infinity so far
      auto weigh = [&]() {
        float sum = weights();
        if (unset || __ballot(!(sum < 0x1p30f))) {
          asm volatile("");                   // a branch, not both ways and a choice
          raise();
          unset = __ballot(mref == -INFINITY) != 0;
          sum = weights();
        }
        lsum += sum;
      };
      if (hot > 0) {
        raise();
        unset = __ballot(mref == -INFINITY) != 0;
      }
      // Tiles without masks.  The reference is the first tile's maximum and stays while the p of a row sum to
      // less than 2^30: fp32 and bf16 lose nothing by that, and neither the maximum has to be found nor the
      // accumulators to be scaled.  (Values so large that it overflows come out infinite, and the callers
      // take such rows up again.)
      while (t < hot) {
        weigh();
        turn();
        products(yes, yes, (t & 1) ^ 1);
        ++t;
      }
      if constexpr (MANY) {                   // tiles with masks before the last
        for (; t < mine - 1; ++t) {
          mask(t);
          raise();
          lsum += weights();
          turn();
          products(yes, yes, (t & 1) ^ 1);
        }
      }
      if (t >= masked) mask(t);
      if (t == 0 || MANY) raise();
      weigh();
      turn();
      products(yes, no, 0);
      ++t;
    }
    for (; t < tiles; ++t) {
      turn();
#pragma unroll
      for (int i = 0; i < 2 * kCopies; ++i) copies(i);
    }
    wait_vmcnt<0>();                          // copies past the end
    // both halves' sums
    const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(lsum), __float_as_uint(lsum), false, false);
    lsum = __uint_as_float(both[0]) + __uint_as_float(both[1]);
  }
};

}  // namespace w4

// Causal attention of packed prompts with grouped heads on the bf16 matrix cores.
//   O_i = sum_{j <= i} p_ij V_j / l_i,  p_ij = exp(scale q_i . k_j - m_i),  l_i = sum_j p_ij
// in one pass over the keys with a running reference m and sum l.
//
// A workgroup of four or eight waves takes 32 queries a wave: 32 tokens of as many heads of a group as
// the group size lets it, twice, four times, .. as many tokens of fewer heads, and walks tiles of 64 keys
// that the waves share.  Scores come transposed, S^T = K Q^T (v_mfma_f32_32x32x16_bf16, keys as rows): lane
// (query l % 32, half h = l / 32) then holds 16 scores of its own query per 32 keys, so that maximum
// and sum need one exchange between halves, and its p, rounded to bf16, are the operand of
// O^T += V^T P^T as they stand: step s of 16 keys takes keys 16 s + 4 h + {0..3} and 8 more, and V^T
// is read in that order by the transposing LDS read.
#include <type_traits>

#include "attend.hpp"
#include "gemm_core.hpp"

#pragma clang fp contract(off)

namespace w4 {

namespace {

constexpr int kTile = 64;                     // keys of a tile
constexpr float kLog2e = 1.44269504088896340736f;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
typedef __attribute__((address_space(3))) bf16x8* lds_bf16x8;

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
// sum over the wave, in every lane (as a scalar)
__device__ __forceinline__ int wave_sum_int(int v) {
  v = dpp_add<0x111, 0xF>(v);                 // row_shr 1, 2, 4, 8
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);                 // row_bcast 15, 31
  v = dpp_add<0x143, 0xC>(v);
  return __builtin_amdgcn_readlane(v, 63);
}

// Query blocks of `size` tokens of all sequences, the longest walks first (block j of a sequence
// has j + 1 blocks of keys to see): the rank-th of them.  False: there are not that many.
__device__ __forceinline__ bool pick_block(const int32_t* offsets, int B, int T, int size, int rank, int& seq, int& block) {
  const int lane = threadIdx.x & 63;
  auto blocks = [&](int b) {
    return b < B ? max(0, token_offset(offsets, b + 1, T) - token_offset(offsets, b, T) + size - 1) / size : 0;
  };
  const int mine = blocks(lane);              // of the first 64 sequences: held
  auto from = [&](int j) {                    // blocks of index j and more
    int n = max(0, mine - j);
    for (int b = 64; b < B; b += 64) n += max(0, blocks(b + lane) - j);
    return wave_sum_int(n);
  };
  if (from(0) <= rank) return false;
  int lo = 0, hi = T / size + 1, above = 0;   // from(lo) > rank >= from(hi) = above
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1, n = from(mid);
    if (n > rank) lo = mid;
    else hi = mid, above = n;
  }
  block = lo;
  int k = rank - above;                       // the k-th sequence with more than lo blocks
  for (int b = 0; b < B; b += 64) {
    const bool has = (b ? blocks(b + lane) : mine) > lo;
    unsigned long long set = __ballot(has);
    const int n = __popcll(set);
    if (k < n) {
      while (k--) set &= set - 1;
      seq = b + __builtin_ctzll(set);
      return true;
    }
    k -= n;
  }
  return false;
}

// lds_copy16 that LDS reads may pass: for copies into slots that nobody reads before the next barrier.
// The five wait states are what a vector write to the base (v_readfirstlane, where the compiler comes by
// it that way) needs before a memory instruction reads it: the compiler does not look into the asm.
__device__ __forceinline__ void lds_copy16_free(uint32_t off, const void* base, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds));
}

template <int HEAD, int WAVES>
struct Prompt {
  static constexpr int kWaves = WAVES;
  static constexpr int kKb = kTile / 32;      // 32-key blocks of a tile
  static constexpr int kSteps = HEAD / 16;    // matrix steps of a score
  static constexpr int kDb = HEAD / 32;       // 32-dim blocks of the output
  static constexpr int kRow = HEAD * 2;       // bytes of an LDS row
  static constexpr int kChunks = HEAD / 8;    // 16-byte pieces of a row
  static constexpr int kTileBytes = kTile * kRow;
  static constexpr int kStages = 2;           // slots, of K and of V
  static constexpr int kCopies = kTileBytes / (kWaves * 1024);   // LDS copies (1 KB) of a wave per tile, K or V
  // LDS rows hold their 16-byte pieces exchanged, so that reads meet distinct banks: piece c of
  // row r at c ^ k_swap(r) (score operand: 16 rows, one piece each) or c ^ v_swap(r) (transposing
  // read: 4 rows, 64 bytes each).
  static __device__ __forceinline__ int k_swap(int r) { return HEAD == 128 ? r & 15 : (r >> 1) & 7; }
  static __device__ __forceinline__ int v_swap(int r) { return HEAD == 128 ? (r & 3) * 4 : ((r >> 1) & 1) * 4; }
};

template <int HEAD, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 2) void prompt_kernel(PromptArgs g, int heads, int groups) {
  using C = Prompt<HEAD, WAVES>;
  constexpr int kWaves = WAVES;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  // workgroup -> (query block, heads of a group): all heads of one rank first
  const int rank = blockIdx.x / groups, hg = blockIdx.x - rank * groups;
  const int size = kWaves * 32 / heads;               // tokens of a workgroup
  int seq, block;
  if (!pick_block(g.offsets, g.B, g.T, size, rank, seq, block)) return;
  seq = __builtin_amdgcn_readfirstlane(seq);
  block = __builtin_amdgcn_readfirstlane(block);
  const int first = __builtin_amdgcn_readfirstlane(token_offset(g.offsets, seq, g.T));
  const int n = __builtin_amdgcn_readfirstlane(token_offset(g.offsets, seq + 1, g.T)) - first;
  const int hq = hg * heads + wave % heads, kvh = hq / (g.n_q / g.n_kv);
  const int q0 = block * size + wave / heads * 32;            // the wave's first query
  const int wg_end = min(n, block * size + size);             // keys that the workgroup needs
  const int tiles = (wg_end + kTile - 1) / kTile;
  const int my_tiles = q0 < n ? (min(n, q0 + 32) + kTile - 1) / kTile : 0;

  // copies of a tile: this lane's row and piece
  constexpr int kPerCopy = 64 / C::kChunks;                   // rows of one copy
  const int row0 = wave * kPerCopy + lane / C::kChunks;
  const uint32_t kpiece = 16 * ((lane % C::kChunks) ^ C::k_swap(row0));
  const uint32_t vpiece = 16 * ((lane % C::kChunks) ^ C::v_swap(row0));
  const uint32_t kstep = (uint32_t)(2 * g.k_stride), vstep = (uint32_t)(2 * g.v_stride);
  const uint16_t* kbase = g.K + (size_t)first * g.k_stride + (size_t)kvh * HEAD;
  const uint16_t* vbase = g.V + (size_t)first * g.v_stride + (size_t)kvh * HEAD;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  // lane offsets of the copies in a whole tile, and in the sequence's last, whose rows past the end
  // repeat its last row
  constexpr int kRowsApart = kWaves * kPerCopy;               // rows between a wave's copies
  const int cut = n / kTile, rest = n - 1 - cut * kTile;      // tiles from `cut` on are not whole
  uint32_t koff[2][C::kCopies], voff[2][C::kCopies];
#pragma unroll
  for (int j = 0; j < C::kCopies; ++j) {
    const int r = row0 + j * kRowsApart, q = min(r, max(rest, 0));
    koff[0][j] = r * kstep + kpiece, koff[1][j] = q * kstep + kpiece;
    voff[0][j] = r * vstep + vpiece, voff[1][j] = q * vstep + vpiece;
  }
  const uint32_t lds_k = lds0 + wave * 1024, lds_v = lds_k + C::kStages * C::kTileBytes;
  auto copy_k = [&](int t, int slot, int j) {
    lds_copy16_free(t < cut ? koff[0][j] : koff[1][j], kbase + (size_t)(t * kTile) * g.k_stride,
                    lds_k + slot * C::kTileBytes + j * kWaves * 1024);
  };
  auto copy_v = [&](int t, int slot, int j) {
    lds_copy16_free(t < cut ? voff[0][j] : voff[1][j], vbase + (size_t)(t * kTile) * g.v_stride,
                    lds_v + slot * C::kTileBytes + j * kWaves * 1024);
  };

  // operand addresses inside a slot; piece 2 st + h (4 db + ..) of the exchanged rows: one bit
  // pattern away from the first
  const uint32_t kaddr = lds0 + l32 * C::kRow + 16 * (h ^ C::k_swap(l32));
  uint32_t vaddr;
  {
    const int i = lane & 15, r = 4 * h + (i >> 2);
    vaddr = lds0 + C::kStages * C::kTileBytes + r * C::kRow + 16 * ((2 * ((lane >> 4) & 1) + ((i & 3) >> 1)) ^ C::v_swap(r)) +
            8 * (i & 1);
  }

#pragma unroll
  for (int i = 0; i < C::kStages; ++i)
#pragma unroll
    for (int j = 0; j < C::kCopies; ++j) {
      copy_k(min(i, tiles - 1), i, j);
      if (i < C::kStages - 1) copy_v(min(i, tiles - 1), i, j);
    }
  bf16x8 qf[C::kSteps];
  {
    const uint16_t* qp = g.Q + (size_t)(first + min(q0 + l32, n - 1)) * g.q_stride + (size_t)hq * HEAD + 8 * h;
#pragma unroll
    for (int st = 0; st < C::kSteps; ++st) qf[st] = *reinterpret_cast<const bf16x8*>(qp + 16 * st);
  }
  const float c = g.scale * kLog2e;
  f32x16 acc[C::kDb];
#pragma unroll
  for (int db = 0; db < C::kDb; ++db) acc[db] = f32x16{};
  float mref = -INFINITY, lsum = 0.0f;
  typedef f32x16 Scores[C::kKb];              // of 32 keys each
  Scores s;
  auto read_k = [&](uint32_t base, int i) {   // operand of score step i: dims 16 (i / kKb) .., keys 32 (i % kKb) ..
    return *(lds_bf16x8)(uintptr_t)((base ^ (32 * (i / C::kKb))) + i % C::kKb * 32 * C::kRow);
  };
  auto multiply_k = [&](bf16x8 kf, int i) {
    s[i % C::kKb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[i / C::kKb], i < C::kKb ? f32x16{} : s[i % C::kKb], 0, 0, 0);
  };
  // Raises the reference to the tile's largest score.
  auto follow = [&]() {
    float m = s[0][0];
#pragma unroll
    for (int r = 1; r < 16 * C::kKb; ++r) m = fmaxf(m, s[r >> 4][r & 15]);
    const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    m = fmaxf(mref, fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1])));
    const float corr = __builtin_amdgcn_exp2f((mref - m) * c);
    lsum *= corr;
#pragma unroll
    for (int db = 0; db < C::kDb; ++db) acc[db] *= corr;
    mref = m;
  };
  // p of a tile, as operands, and their sum: of the rounded p, as the product with V has them
  bf16x8 pf[2 * C::kKb];
  const bf16x2 ones = {(__bf16)1.0f, (__bf16)1.0f};
  auto weights = [&]() {
    const float mc = -mref * c;
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 2 * C::kKb; ++k)
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const bf16x2 p = {(__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s[k >> 1][8 * (k & 1) + j], c, mc)),
                          (__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s[k >> 1][8 * (k & 1) + j + 1], c, mc))};
        sum[j >> 1 & 1] = __builtin_amdgcn_fdot2_f32_bf16(p, ones, sum[j >> 1 & 1], false);
        pf[k][j] = p[0], pf[k][j + 1] = p[1];
      }
    return sum[0] + sum[1];
  };
  auto read_v = [&](uint32_t base, int i) {   // operand of value step i: keys 16 (i / kDb) .., dims 32 (i % kDb) ..
    const uint32_t at = (base ^ (64 * (i % C::kDb))) + 16 * (i / C::kDb) * C::kRow;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(uintptr_t)at);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(uintptr_t)(at + 8 * C::kRow));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto multiply_v = [&](bf16x8 vf, int i) {
    acc[i % C::kDb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[i / C::kDb], acc[i % C::kDb], 0, 0, 0);
  };
  // One barrier a tile, between its weights and its products.  Among the products a wave issues its
  // copies of K of tile t + 2 and V of tile t + 1, whose slots nobody reads any more behind that barrier; they
  // have to be there at the next.
  constexpr int kBatch = 2 * C::kCopies;
  int t = 0, slot = 0;                        // tile, its slot
  auto turn = [&]() {                         // weights -> products
    wait_vmcnt<0>();
    lds_barrier();
  };
  auto copies = [&](int i) {                  // copy i of a tile's, first K's, then V's
    if (i < C::kCopies) copy_k(min(t + 2, tiles - 1), slot, i);
    else copy_v(min(t + 1, tiles - 1), slot ^ 1, i - C::kCopies);
  };
  auto close = [&]() {                        // products -> the next tile's weights
    ++t;
    slot ^= 1;
  };
  // The values of tile t and the scores of the next, in this order: operands are read four matrix
  // instructions ahead, copies go between.
  constexpr int kV = 2 * C::kKb * C::kDb, kK = C::kKb * C::kSteps, kAhead = 4;
  auto products = [&](auto with_values, auto with_scores, int kslot) {
    constexpr int v0 = with_values ? 0 : kV, end = with_scores ? kV + kK : kV;
    const uint32_t vbase_lds = opaque_vgpr(vaddr + slot * C::kTileBytes);
    const uint32_t kbase_lds = opaque_vgpr(kaddr + kslot * C::kTileBytes);
    bf16x8 ring[kAhead];
    auto read = [&](int i) {
      if (i < end) ring[i % kAhead] = i < kV ? read_v(vbase_lds, i) : read_k(kbase_lds, i - kV);
    };
#pragma unroll
    for (int i = v0; i < v0 + kAhead; ++i) read(i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = v0; i < end; ++i) {
      if (i < kV) multiply_v(ring[i % kAhead], i);
      else multiply_k(ring[i % kAhead], i - kV);
      read(i + kAhead);
      if (with_values && i % 2 == 1 && i / 2 < kBatch) copies(i / 2);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  wait_vmcnt<0>();
  lds_barrier();
  if (my_tiles > 0) {
    products(no, yes, 0);
    if (my_tiles > 1) follow();
    // Tiles whose keys all rows see.  The reference is the first tile's maximum and stays while the p
    // of a row sum to less than 2^30: fp32 and bf16 lose nothing by that, and neither the maximum has to be
    // found nor the accumulators to be scaled.  (Values so large that it overflows come out infinite, and are
    // taken up below.)
    while (t < my_tiles - 1) {
      float sum = weights();
      if (__ballot(!(sum < 0x1p30f))) {
        asm volatile("");                     // a branch, not both ways and a choice
        follow();
        sum = weights();
      }
      lsum += sum;
      turn();
      products(yes, yes, slot ^ 1);
      close();
    }
    // the tile that the diagonal or the sequence's end crosses
    const int end = min(q0 + l32, n - 1) - t * kTile - 4 * h;
#pragma unroll
    for (int kb = 0; kb < C::kKb; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (32 * kb + (r & 3) + 8 * (r >> 2) > end) s[kb][r] = -INFINITY;
    follow();
    lsum += weights();
    turn();
    products(yes, no, 0);
    close();
  }
  while (t < tiles) {
    turn();
#pragma unroll
    for (int i = 0; i < kBatch; ++i) copies(i);
    close();
  }
  wait_vmcnt<0>();                            // copies past the end
  if (my_tiles == 0) return;

  const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(lsum), __float_as_uint(lsum), false, false);
  const float inv = 1.0f / (__uint_as_float(both[0]) + __uint_as_float(both[1]));
  const int mine = q0 + l32;
  uint16_t* op = g.O + ((size_t)(first + min(mine, n - 1)) * g.n_q + hq) * HEAD + 8 * h;
  uint32_t bad = 0;
#pragma unroll
  for (int db = 0; db < C::kDb; ++db)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      // registers 4 i .. 4 i + 3: dims 8 i + 4 h ..; halves trade, so that a lane has 8 in a row
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bf16x2 p = {(__bf16)(acc[db][4 * i + 2 * e] * inv), (__bf16)(acc[db][4 * i + 2 * e + 1] * inv)};
        w[e] = __builtin_bit_cast(uint32_t, p);
        bad |= (w[e] & 0x7F807F80u) + 0x00800080u;
      }
      const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
      const auto y = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
      if (mine < n) *reinterpret_cast<uint4*>(op + 32 * db + 8 * i) = make_uint4(x[0], y[0], x[1], y[1]);
    }
  // rows with an infinity or NaN: once more, key by key
  const unsigned long long rows = __ballot((bad & 0x80008000u) != 0 && mine < n);
  uint32_t todo = (uint32_t)rows | (uint32_t)(rows >> 32);
  while (todo) {
    const int i = q0 + __builtin_ctz(todo);
    todo &= todo - 1;
    attend<HEAD>(g.Q + (size_t)(first + i) * g.q_stride + (size_t)hq * HEAD, i + 1, g.scale,
                 [&](int key, const uint16_t*& k, const uint16_t*& v) {
                   k = kbase + (size_t)key * g.k_stride;
                   v = vbase + (size_t)key * g.v_stride;
                 },
                 g.O + ((size_t)(first + i) * g.n_q + hq) * HEAD);
  }
}

// heads of a group that a workgroup takes: the more there are, the fewer tokens lie between its
// waves' ends
int heads_of(int group, int waves) {
  int heads = waves;
  while (group % heads) heads >>= 1;
  return heads;
}

// query blocks are at most this many (every sequence may have one that is not full)
long long most_blocks(int T, int B, int heads, int waves) { return (long long)T / (waves * 32 / heads) + B; }

template <int HEAD, int WAVES>
int launch(const PromptArgs& g, hipStream_t st) {
  using C = Prompt<HEAD, WAVES>;
  const int heads = heads_of(g.n_q / g.n_kv, WAVES), groups = g.n_q / heads;
  hipLaunchKernelGGL((prompt_kernel<HEAD, WAVES>), dim3((unsigned)(most_blocks(g.T, g.B, heads, WAVES) * groups)),
                     dim3(WAVES * 64), 2 * C::kTileBytes * C::kStages, st, g, heads, groups);
  W4_CHECK_LAUNCH();
  return W4_OK;
}

}  // namespace

size_t prompt_workspace_bytes(int T, int n_q, int n_kv, int head, int B) { return 0; }
bool prompt_fits(int T, int n_q, int n_kv, int B) {
  const int heads = heads_of(n_q / n_kv, 4);
  return most_blocks(T, B, heads, 4) * (n_q / heads) * 512 <= kGridThreads;
}

int launch_prompt_attention(const PromptArgs& g, hipStream_t st) {
  // eight waves share each key tile, four end sooner where there are few workgroups (8 x 512 tokens of 16
  // heads: 24.3 us with eight, 21.1 with four; 1 x 8192: 239 and 252)
  const bool wide = (long long)g.T * g.n_q >= 512 * 256;
  if (g.head == 64) return wide ? launch<64, 8>(g, st) : launch<64, 4>(g, st);
  return wide ? launch<128, 8>(g, st) : launch<128, 4>(g, st);
}

}  // namespace w4

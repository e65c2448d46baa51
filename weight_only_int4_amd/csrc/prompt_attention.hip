// Causal attention of packed prompts with grouped heads on the bf16 matrix cores.
//   O_i = sum_{j <= i} p_ij V_j / l_i,  p_ij = exp(scale q_i . k_j - m_i),  l_i = sum_j p_ij
// in one pass over the keys with a running reference m and sum l.
//
// A workgroup of eight waves, two per SIMD, takes 32 queries a wave: 32 tokens of eight heads of a
// group, 64 of four, 128 of two or 256 of one, as the group size divides, and walks tiles of 64 keys
// that the waves share.  Scores come transposed, S^T = K Q^T (v_mfma_f32_32x32x16_bf16, keys as rows): lane
// (query l % 32, half h = l / 32) then holds 16 scores of its own query per 32 keys, so that maximum
// and sum need one exchange between halves, and its p, rounded to bf16, are the operand of
// O^T += V^T P^T as they stand: step s of 16 keys takes keys 16 s + 4 h + {0..3} and 8 more, and V^T
// is read in that order by the transposing LDS read.
#include "attend.hpp"
#include "gemm_core.hpp"

#pragma clang fp contract(off)

namespace w4 {

namespace {

constexpr int kTile = 64;                     // keys of a tile
constexpr int kWaves = 8;
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

template <int HEAD>
struct Prompt {
  static constexpr int kSteps = HEAD / 16;    // matrix steps of a score
  static constexpr int kDb = HEAD / 32;       // 32-dim blocks of the output
  static constexpr int kRow = HEAD * 2;       // bytes of an LDS row
  static constexpr int kChunks = HEAD / 8;    // 16-byte pieces of a row
  static constexpr int kTileBytes = kTile * kRow;
  static constexpr int kStages = 3;           // slots, of K and of V
  static constexpr int kCopies = kTileBytes / (kWaves * 1024);   // LDS copies (1 KB) of a wave per tile, K or V
  // LDS rows hold their 16-byte pieces exchanged, so that reads meet distinct banks: piece c of
  // row r at c ^ k_swap(r) (score operand: 16 rows, one piece each) or c ^ v_swap(r) (transposing
  // read: 4 rows, 64 bytes each).
  static __device__ __forceinline__ int k_swap(int r) { return HEAD == 128 ? r & 15 : (r >> 1) & 7; }
  static __device__ __forceinline__ int v_swap(int r) { return HEAD == 128 ? (r & 3) * 4 : ((r >> 1) & 1) * 4; }
};

template <int HEAD>
__global__ __launch_bounds__(kWaves * 64, 2) void prompt_kernel(PromptArgs g, int heads, int groups) {
  using C = Prompt<HEAD>;
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
  const uint32_t koff = row0 * kstep + kpiece, voff = row0 * vstep + vpiece;
  constexpr int kRowsApart = kWaves * kPerCopy;               // rows between a wave's copies
  auto copy = [&](const uint16_t* base, long long stride, uint32_t step, uint32_t off, uint32_t piece, int t, uint32_t to) {
    const int kb = t * kTile;
    const uint16_t* from = base + (size_t)kb * stride;
    if (kb + kTile <= n) {
#pragma unroll
      for (int j = 0; j < C::kCopies; ++j)
        lds_copy16(off, from + (size_t)(j * kRowsApart) * stride, to + j * kWaves * 1024);
    } else {                                                  // rows past the sequence repeat its last
#pragma unroll
      for (int j = 0; j < C::kCopies; ++j)
        lds_copy16((uint32_t)min(row0 + j * kRowsApart, n - 1 - kb) * step + piece, from, to + j * kWaves * 1024);
    }
  };
  const uint32_t lds_k = lds0 + wave * 1024, lds_v = lds_k + C::kStages * C::kTileBytes;
  auto copy_k = [&](int t, int slot) { copy(kbase, g.k_stride, kstep, koff, kpiece, t, lds_k + slot * C::kTileBytes); };
  auto copy_v = [&](int t, int slot) { copy(vbase, g.v_stride, vstep, voff, vpiece, t, lds_v + slot * C::kTileBytes); };

  // operand addresses inside a slot; piece 2 st + h (4 db + ..) of the exchanged rows: one bit
  // pattern away from the first
  const uint32_t kaddr = lds0 + l32 * C::kRow + 16 * (h ^ C::k_swap(l32));
  uint32_t vaddr;
  {
    const int i = lane & 15, r = 4 * h + (i >> 2);
    vaddr = lds0 + C::kStages * C::kTileBytes + r * C::kRow + 16 * ((2 * ((lane >> 4) & 1) + ((i & 3) >> 1)) ^ C::v_swap(r)) +
            8 * (i & 1);
  }

  copy_k(0, 0);
  copy_k(min(1, tiles - 1), 1);
  copy_v(0, 0);
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
  typedef f32x16 Scores[2];                   // of 32 keys each
  Scores s;
  auto scores = [&](int slot) {
    s[0] = f32x16{}, s[1] = f32x16{};
    const uint32_t base = opaque_vgpr(kaddr + slot * C::kTileBytes);
#pragma unroll
    for (int st = 0; st < C::kSteps; ++st)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const bf16x8 kf = *(lds_bf16x8)(uintptr_t)((base ^ (32 * st)) + kb * 32 * C::kRow);
        s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[st], s[kb], 0, 0, 0);
      }
  };
  // Raises the reference to the tile's largest score.
  auto follow = [&]() {
    float m = s[0][0];
#pragma unroll
    for (int r = 1; r < 32; ++r) m = fmaxf(m, s[r >> 4][r & 15]);
    const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    m = fmaxf(mref, fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1])));
    const float corr = __builtin_amdgcn_exp2f((mref - m) * c);
    lsum *= corr;
#pragma unroll
    for (int db = 0; db < C::kDb; ++db) acc[db] *= corr;
    mref = m;
  };
  // p of a tile, as operands, and their sum: of the rounded p, as the product with V has them
  bf16x8 pf[4];
  const bf16x2 ones = {(__bf16)1.0f, (__bf16)1.0f};
  auto weights = [&]() {
    const float mc = -mref * c;
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const bf16x2 p = {(__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s[k >> 1][8 * (k & 1) + j], c, mc)),
                          (__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s[k >> 1][8 * (k & 1) + j + 1], c, mc))};
        sum[j >> 1 & 1] = __builtin_amdgcn_fdot2_f32_bf16(p, ones, sum[j >> 1 & 1], false);
        pf[k][j] = p[0], pf[k][j + 1] = p[1];
      }
    return sum[0] + sum[1];
  };
  auto values = [&](int slot) {
    const uint32_t base = opaque_vgpr(vaddr + slot * C::kTileBytes);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int db = 0; db < C::kDb; ++db) {
        const uint32_t at = (base ^ (64 * db)) + 16 * k * C::kRow;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(uintptr_t)at);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(uintptr_t)(at + 8 * C::kRow));
        const bf16x8 vf = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        acc[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[k], acc[db], 0, 0, 0);
      }
  };
  // The waves of a SIMD, w and w + 4, work in opposite phases: one turns scores into weights on the
  // vector ALU while the other multiplies (values of its tile, scores of its next).  A barrier ends
  // each phase; the late waves begin one phase later.  At the start of a weights phase a wave
  // issues its copies of K of tile t + 2 and V of tile t + 1, whose slots nobody reads any more; they have
  // to be there at the third barrier from the early waves', the second from the late waves' issue.
  const bool late = wave >= kWaves / 2;
  int t = 0, slot = 0, next = 1;              // tile, its slot, the next tile's
  auto open = [&]() {
    copy_k(min(t + 2, tiles - 1), 3 - slot - next);
    copy_v(min(t + 1, tiles - 1), next);
  };
  auto turn = [&]() {                         // weights -> products
    if (!late) wait_vmcnt<2 * C::kCopies>();
    lds_barrier();
  };
  auto close = [&]() {                        // products -> weights
    if (late) wait_vmcnt<0>();
    lds_barrier();
    ++t;
    const int after = 3 - slot - next;
    slot = next, next = after;
  };
  wait_vmcnt<0>();
  lds_barrier();
  if (late) lds_barrier();
  if (my_tiles > 0) {
    scores(0);
    if (my_tiles > 1) follow();
    // Tiles whose keys all rows see.  The reference is the first tile's maximum and stays while the p
    // of a row sum to less than 2^30: fp32 and bf16 lose nothing by that, and neither the maximum has to be
    // found nor the accumulators to be scaled.  (Values so large that it overflows come out infinite, and are
    // taken up below.)
    while (t < my_tiles - 1) {
      open();
      float sum = weights();
      if (__ballot(!(sum < 0x1p30f))) {
        asm volatile("");                     // a branch, not both ways and a choice
        follow();
        sum = weights();
      }
      lsum += sum;
      turn();
      values(slot);
      scores(next);
      close();
    }
    // the tile that the diagonal or the sequence's end crosses
    open();
    const int end = min(q0 + l32, n - 1) - t * kTile - 4 * h;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (32 * kb + (r & 3) + 8 * (r >> 2) > end) s[kb][r] = -INFINITY;
    follow();
    lsum += weights();
    turn();
    values(slot);
    close();
  }
  while (t < tiles) {
    open();
    turn();
    close();
  }
  if (!late) lds_barrier();
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
int heads_of(int group) { return group % 8 == 0 ? 8 : group % 4 == 0 ? 4 : group % 2 == 0 ? 2 : 1; }

// query blocks are at most this many (every sequence may have one that is not full)
long long most_blocks(int T, int B, int heads) { return (long long)T / (kWaves * 32 / heads) + B; }

}  // namespace

size_t prompt_workspace_bytes(int T, int n_q, int n_kv, int head, int B) { return 0; }
bool prompt_fits(int T, int n_q, int n_kv, int B) {
  const int heads = heads_of(n_q / n_kv);
  return most_blocks(T, B, heads) * (n_q / heads) * kWaves * 64 <= kGridThreads;
}

template <int HEAD>
static int launch(const PromptArgs& g, hipStream_t st) {
  const int heads = heads_of(g.n_q / g.n_kv), groups = g.n_q / heads;
  const size_t lds = 2 * Prompt<HEAD>::kTileBytes * Prompt<HEAD>::kStages;
  if (lds > 64 * 1024) {
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(prompt_kernel<HEAD>), hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)lds) != hipSuccess) {
      (void)hipGetLastError();
      return W4_ERR_HIP;
    }
  }
  hipLaunchKernelGGL(prompt_kernel<HEAD>, dim3((unsigned)(most_blocks(g.T, g.B, heads) * groups)), dim3(kWaves * 64), lds, st, g,
                     heads, groups);
  W4_CHECK_LAUNCH();
  return W4_OK;
}

int launch_prompt_attention(const PromptArgs& g, hipStream_t st) {
  return g.head == 64 ? launch<64>(g, st) : launch<128>(g, st);
}

}  // namespace w4

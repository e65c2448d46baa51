// Causal attention of packed prompts with grouped heads on the bf16 matrix cores.
//   O_i = sum_{j <= i} p_ij V_j / l_i,  p_ij = exp(scale q_i . k_j - m_i),  l_i = sum_j p_ij
// in one pass over the keys with a running reference m and sum l.
//
// A workgroup of four waves, one per SIMD, takes 64 queries a wave: 64 tokens of four heads of a
// group, 128 of two, or 256 of one, as the group size divides, and walks tiles of 64 keys that the
// waves share.  Scores come transposed, S^T = K Q^T (v_mfma_f32_32x32x16_bf16, keys as rows): lane
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
  static constexpr int kStage = 2 * kTileBytes;
  static constexpr int kStages = 3;
  static constexpr int kCopies = kTileBytes / 4096;   // LDS copies (1 KB) of a wave per tile, K or V
  // LDS rows hold their 16-byte pieces exchanged, so that reads meet distinct banks: piece c of
  // row r at c ^ k_swap(r) (score operand: 16 rows, one piece each) or c ^ v_swap(r) (transposing
  // read: 4 rows, 64 bytes each).
  static __device__ __forceinline__ int k_swap(int r) { return HEAD == 128 ? r & 15 : (r >> 1) & 7; }
  static __device__ __forceinline__ int v_swap(int r) { return HEAD == 128 ? (r & 3) * 4 : ((r >> 1) & 1) * 4; }
};

template <int HEAD>
__global__ __launch_bounds__(256, HEAD == 128 ? 1 : 2) void prompt_kernel(PromptArgs g, int heads, int groups) {
  using C = Prompt<HEAD>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  // workgroup -> (query block, heads of a group): all heads of one rank first
  const int rank = blockIdx.x / groups, hg = blockIdx.x - rank * groups;
  const int size = 256 / heads;               // tokens of a workgroup
  int seq, block;
  if (!pick_block(g.offsets, g.B, g.T, size, rank, seq, block)) return;
  seq = __builtin_amdgcn_readfirstlane(seq);
  block = __builtin_amdgcn_readfirstlane(block);
  const int first = token_offset(g.offsets, seq, g.T);
  const int n = token_offset(g.offsets, seq + 1, g.T) - first;
  const int hq = hg * heads + wave % heads, kvh = hq / (g.n_q / g.n_kv);
  const int q0 = block * size + wave / heads * 64;            // the wave's first query
  const int wg_end = min(n, block * size + size);             // keys that the workgroup needs
  const int tiles = (wg_end + kTile - 1) / kTile;
  const int my_tiles = q0 < n ? (min(n, q0 + 64) + kTile - 1) / kTile : 0;

  // copies of a tile: this lane's row and piece
  constexpr int kPerCopy = 64 / C::kChunks;                   // rows of one copy
  const int row0 = wave * kPerCopy + lane / C::kChunks;
  const uint32_t kpiece = 16 * ((lane % C::kChunks) ^ C::k_swap(row0));
  const uint32_t vpiece = 16 * ((lane % C::kChunks) ^ C::v_swap(row0));
  const uint32_t kstep = (uint32_t)(2 * g.k_stride), vstep = (uint32_t)(2 * g.v_stride);
  const uint16_t* kbase = g.K + (size_t)first * g.k_stride + (size_t)kvh * HEAD;
  const uint16_t* vbase = g.V + (size_t)first * g.v_stride + (size_t)kvh * HEAD;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  auto copy_tile = [&](int t, int slot) {
    const int kb = t * kTile, last = n - 1 - kb;              // rows past the sequence repeat its last
    const uint16_t* kt = kbase + (size_t)kb * g.k_stride;
    const uint16_t* vt = vbase + (size_t)kb * g.v_stride;
    const uint32_t at = __builtin_amdgcn_readfirstlane(lds0 + slot * C::kStage + wave * 1024);
#pragma unroll
    for (int j = 0; j < C::kCopies; ++j) {
      const uint32_t r = (uint32_t)min(row0 + j * 4 * kPerCopy, last);
      lds_copy16(r * kstep + kpiece, kt, at + j * 4096);
      lds_copy16(r * vstep + vpiece, vt, at + j * 4096 + C::kTileBytes);
    }
  };

  // operand addresses inside a stage
  uint32_t kaddr[C::kSteps], vaddr[C::kDb];
#pragma unroll
  for (int st = 0; st < C::kSteps; ++st)
    kaddr[st] = lds0 + l32 * C::kRow + 16 * ((2 * st + h) ^ C::k_swap(l32));
  {
    const int i = lane & 15, r = 4 * h + (i >> 2);
#pragma unroll
    for (int db = 0; db < C::kDb; ++db)
      vaddr[db] = lds0 + C::kTileBytes + r * C::kRow +
                  16 * ((4 * db + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1)) ^ C::v_swap(r)) + 8 * (i & 1);
  }

  copy_tile(0, 0);
  if (tiles > 1) copy_tile(1, 1);
  bf16x8 qf[2][C::kSteps];
#pragma unroll
  for (int qb = 0; qb < 2; ++qb) {
    const int t = min(q0 + 32 * qb + l32, n - 1);
    const uint16_t* qp = g.Q + (size_t)(first + t) * g.q_stride + (size_t)hq * HEAD + 8 * h;
#pragma unroll
    for (int st = 0; st < C::kSteps; ++st) qf[qb][st] = *reinterpret_cast<const bf16x8*>(qp + 16 * st);
  }
  const float c = g.scale * kLog2e, slack = 8.0f / c;
  f32x16 acc[2][C::kDb], s[2][2];
  float mref[2], lsum[2];
#pragma unroll
  for (int qb = 0; qb < 2; ++qb) {
    mref[qb] = -INFINITY, lsum[qb] = 0.0f;
#pragma unroll
    for (int db = 0; db < C::kDb; ++db) acc[qb][db] = f32x16{};
  }
  auto scores = [&](uint32_t stage, f32x16 (&out)[2][2]) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      out[0][kb] = f32x16{}, out[1][kb] = f32x16{};
#pragma unroll
      for (int st = 0; st < C::kSteps; ++st) {
        const bf16x8 kf = *(lds_bf16x8)(uintptr_t)(kaddr[st] + stage + kb * 32 * C::kRow);
        out[0][kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[0][st], out[0][kb], 0, 0, 0);
        out[1][kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[1][st], out[1][kb], 0, 0, 0);
      }
    }
  };
  wait_vmcnt<0>();
  lds_barrier();
  if (my_tiles > 0) scores(0, s);
  int slot = 0;
  for (int t = 0; t < tiles; ++t) {
    const int next = slot == C::kStages - 1 ? 0 : slot + 1;
    wait_vmcnt<0>();                          // tile t + 1 has arrived, and nobody reads tile t - 1 any more
    lds_barrier();
    if (t + 2 < tiles) copy_tile(t + 2, next == C::kStages - 1 ? 0 : next + 1);
    if (t < my_tiles) {
      if (t == my_tiles - 1) {                // the tile that the diagonal or the sequence's end crosses
#pragma unroll
        for (int qb = 0; qb < 2; ++qb) {
          const int last = min(q0 + 32 * qb + l32, n - 1) - t * kTile - 4 * h;
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (32 * kb + (r & 3) + 8 * (r >> 2) > last) s[qb][kb][r] = -INFINITY;
        }
      }
      float top[2];
#pragma unroll
      for (int qb = 0; qb < 2; ++qb) {
        float m = s[qb][0][0];
#pragma unroll
        for (int r = 1; r < 32; ++r) m = fmaxf(m, s[qb][r >> 4][r & 15]);
        const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
        top[qb] = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
      }
      // the reference stays while no score passes it by more than 8 in the exponent of 2: p <= 2^8
      // loses nothing in fp32 or bf16, and the accumulators are left alone
      if (__ballot(top[0] > mref[0] + slack || top[1] > mref[1] + slack)) {
#pragma unroll
        for (int qb = 0; qb < 2; ++qb) {
          const float m = fmaxf(mref[qb], top[qb]);
          const float corr = __builtin_amdgcn_exp2f((mref[qb] - m) * c);
          lsum[qb] *= corr;
#pragma unroll
          for (int db = 0; db < C::kDb; ++db) acc[qb][db] *= corr;
          mref[qb] = m;
        }
      }
      bf16x8 pf[2][4];
#pragma unroll
      for (int qb = 0; qb < 2; ++qb) {
        const float mc = -mref[qb] * c;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[qb][k >> 1][8 * (k & 1) + j], c, mc));
            lsum[qb] += p;
            pf[qb][k][j] = (__bf16)p;
          }
      }
      if (t + 1 < my_tiles) scores(next * C::kStage, s);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int db = 0; db < C::kDb; ++db) {
          const uint32_t at = vaddr[db] + slot * C::kStage + 16 * k * C::kRow;
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(uintptr_t)at);
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(uintptr_t)(at + 8 * C::kRow));
          const bf16x8 vf = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
          acc[0][db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[0][k], acc[0][db], 0, 0, 0);
          acc[1][db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[1][k], acc[1][db], 0, 0, 0);
        }
    }
    slot = next;
  }
  if (my_tiles == 0) return;

#pragma unroll
  for (int qb = 0; qb < 2; ++qb) {
    const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(lsum[qb]), __float_as_uint(lsum[qb]), false, false);
    const float inv = 1.0f / (__uint_as_float(x[0]) + __uint_as_float(x[1]));
    const int t = q0 + 32 * qb + l32;
    uint16_t* op = g.O + ((size_t)(first + min(t, n - 1)) * g.n_q + hq) * HEAD + 8 * h;
    uint32_t bad = 0;
#pragma unroll
    for (int db = 0; db < C::kDb; ++db)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        // registers 4 i .. 4 i + 3: dims 8 i + 4 h ..; halves trade, so that a lane has 8 in a row
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bf16x2 p = {(__bf16)(acc[qb][db][4 * i + 2 * e] * inv), (__bf16)(acc[qb][db][4 * i + 2 * e + 1] * inv)};
          w[e] = __builtin_bit_cast(uint32_t, p);
          bad |= (w[e] & 0x7F807F80u) + 0x00800080u;
        }
        const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        if (t < n) *reinterpret_cast<uint4*>(op + 32 * db + 8 * i) = make_uint4(a[0], b[0], a[1], b[1]);
      }
    // rows with an infinity or NaN: once more, key by key
    unsigned long long rows = __ballot((bad & 0x80008000u) != 0 && t < n);
    uint32_t todo = (uint32_t)rows | (uint32_t)(rows >> 32);
    while (todo) {
      const int i = q0 + 32 * qb + __builtin_ctz(todo);
      todo &= todo - 1;
      attend<HEAD>(g.Q + (size_t)(first + i) * g.q_stride + (size_t)hq * HEAD, i + 1, g.scale,
                   [&](int key, const uint16_t*& k, const uint16_t*& v) {
                     k = kbase + (size_t)key * g.k_stride;
                     v = vbase + (size_t)key * g.v_stride;
                   },
                   g.O + ((size_t)(first + i) * g.n_q + hq) * HEAD);
    }
  }
}

// heads of a group that a workgroup takes: all waves at the same 64 tokens where four divide it
// (they end together), else two or one
int heads_of(int group) { return group % 4 == 0 ? 4 : group % 2 == 0 ? 2 : 1; }

// query blocks are at most this many (every sequence may have one that is not full)
long long most_blocks(int T, int B, int heads) { return (long long)T / (256 / heads) + B; }

}  // namespace

size_t prompt_workspace_bytes(int T, int n_q, int n_kv, int head, int B) { return 0; }
bool prompt_fits(int T, int n_q, int n_kv, int B) {
  const int heads = heads_of(n_q / n_kv);
  return most_blocks(T, B, heads) * (n_q / heads) * 256 <= kGridThreads;
}

template <int HEAD>
static int launch(const PromptArgs& g, hipStream_t st) {
  const int heads = heads_of(g.n_q / g.n_kv), groups = g.n_q / heads;
  const size_t lds = Prompt<HEAD>::kStage * Prompt<HEAD>::kStages;
  if (lds > 64 * 1024) {
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(prompt_kernel<HEAD>), hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)lds) != hipSuccess) {
      (void)hipGetLastError();
      return W4_ERR_HIP;
    }
  }
  hipLaunchKernelGGL(prompt_kernel<HEAD>, dim3((unsigned)(most_blocks(g.T, g.B, heads) * groups)), dim3(256), lds, st, g,
                     heads, groups);
  W4_CHECK_LAUNCH();
  return W4_OK;
}

int launch_prompt_attention(const PromptArgs& g, hipStream_t st) {
  return g.head == 64 ? launch<64>(g, st) : launch<128>(g, st);
}

}  // namespace w4

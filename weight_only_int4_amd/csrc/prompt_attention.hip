// Causal attention of packed prompts with grouped heads on the bf16 matrix cores.
//   O_i = sum_{j <= i} p_ij V_j / l_i,  p_ij = exp(scale q_i . k_j - m_i),  l_i = sum_j p_ij
// in one pass over the keys with a running reference m and sum l.
//
// A workgroup of four or eight waves takes 32 queries a wave: 32 tokens of as many heads of a group as
// the group size lets it, twice, four times, .. as many tokens of fewer heads, and walks the keys as
// flash_tile.hpp has it.
#include "attend.hpp"
#include "flash_tile.hpp"

#pragma clang fp contract(off)

namespace w4 {

namespace {

constexpr int kCus = 256;

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
// has j + 1 blocks of keys to see): the rank-th of them.  Where two rounds of `round` ranks hold them
// all, the second goes the other way, so that a CU's two workgroups are a long and a short one.  False:
// there are not that many.
__device__ __forceinline__ bool pick_block(const int32_t* offsets, int B, int T, int size, int rank, int round, int& block, int& first,
                                           int& length) {
  const int lane = threadIdx.x & 63;
  auto range = [&](int b, int& at, int& n) {
    at = b < B ? held_offset(offsets[b], T) : 0;
    n = b < B ? held_count(at, held_offset(offsets[b + 1], T)) : 0;
  };
  auto blocks = [&](int b) {
    int at, n;
    range(b, at, n);
    return (n + size - 1) / size;
  };
  constexpr int kHeld = 4;                    // blocks of the first 256 sequences: held
  int mine[kHeld], at, n;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) mine[i] = 64 * i < B ? blocks(64 * i + lane) : 0;
  auto from = [&](int j) {                    // blocks of index j and more
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) sum += max(0, mine[i] - j);
#pragma unroll 4
    for (int b = 64 * kHeld; b < B; b += 64) sum += max(0, blocks(b + lane) - j);
    return wave_sum_int(sum);
  };
  const int total = from(0);
  if (total <= rank) return false;
  if (total <= 2 * round && rank >= round) rank = total - 1 - (rank - round);
  int lo = 0, hi = T / size + 1, above = 0;   // from(lo) > rank >= from(hi) = above
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1, n = from(mid);
    if (n > rank) lo = mid;
    else hi = mid, above = n;
  }
  block = lo;
  int k = rank - above;                       // the k-th sequence with more than lo blocks
  for (int b = 0; b < B; b += 64) {
    range(b + lane, at, n);
    unsigned long long set = __ballot((n + size - 1) / size > lo);
    const int count = __popcll(set);
    if (k < count) {
      while (k--) set &= set - 1;
      first = __builtin_amdgcn_readlane(at, __builtin_ctzll(set));
      length = __builtin_amdgcn_readlane(n, __builtin_ctzll(set));
      return true;
    }
    k -= count;
  }
  return false;
}

template <int HEAD, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 2) void prompt_kernel(PromptArgs g, int heads, int groups) {
  using F = Flash<HEAD, WAVES>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  // workgroup -> (query block, heads of a group): all heads of one rank first
  const int rank = blockIdx.x / groups, hg = blockIdx.x - rank * groups;
  const int size = WAVES * 32 / heads;               // tokens of a workgroup
  int block, first, n;
  if (!pick_block(g.offsets, g.B, g.T, size, rank, WAVES == 4 ? kCus / groups : 0, block, first, n)) return;
  block = __builtin_amdgcn_readfirstlane(block);
  first = __builtin_amdgcn_readfirstlane(first);
  n = __builtin_amdgcn_readfirstlane(n);
  const int hq = hg * heads + wave % heads, kvh = hq / (g.n_q / g.n_kv);
  const int q0 = block * size + wave / heads * 32;            // the wave's first query
  const int wg_end = min(n, block * size + size);             // keys that the workgroup needs
  const int tiles = (wg_end + kTile - 1) / kTile;
  const int my_tiles = q0 < n ? (min(n, q0 + 32) + kTile - 1) / kTile : 0;

  F f;
  f.init(smem, g.scale);
  f.load_q(g.Q + (size_t)(first + min(q0 + l32, n - 1)) * g.q_stride + (size_t)hq * HEAD);
  const uint16_t* kbase = g.K + (size_t)first * g.k_stride + (size_t)kvh * HEAD;
  const uint16_t* vbase = g.V + (size_t)first * g.v_stride + (size_t)kvh * HEAD;
  // lane offsets of the copies in a whole tile, and in the sequence's last, whose rows past the end
  // repeat its last row
  const int cut = n / kTile, rest = max(n - 1 - cut * kTile, 0);     // tiles from `cut` on are not whole
  const uint32_t kstep = (uint32_t)(2 * g.k_stride), vstep = (uint32_t)(2 * g.v_stride);
  uint32_t koff[2][F::kCopies], voff[2][F::kCopies];
#pragma unroll
  for (int j = 0; j < F::kCopies; ++j) {
    const int r = F::copy_row() + j * F::kRowsApart, q = min(r, rest);
    koff[0][j] = r * kstep + F::k_piece(), koff[1][j] = q * kstep + F::k_piece();
    voff[0][j] = r * vstep + F::v_piece(), voff[1][j] = q * vstep + F::v_piece();
  }
  // tiles come in order: their addresses are steps from one to the next
  const size_t kpitch = (size_t)kTile * g.k_stride, vpitch = (size_t)kTile * g.v_stride;
  int kt = 0, vt = 0;
  f.template walk<false>(
      tiles, my_tiles, my_tiles - 1,
      [&](int kv, int t, int j, uint32_t lds) {
        const bool rest = t >= cut;
        if (kv == 0) {
          kbase += t > kt ? kpitch : 0, kt = t;
          lds_copy16_free(rest ? koff[1][j] : koff[0][j], kbase, lds);
        } else {
          vbase += t > vt ? vpitch : 0, vt = t;
          lds_copy16_free(rest ? voff[1][j] : voff[0][j], vbase, lds);
        }
      },
      [&](int t) {                            // the diagonal, or the sequence's end
        const int end = min(q0 + l32, n - 1) - t * kTile - 4 * h;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (32 * kb + (r & 3) + 8 * (r >> 2) > end) f.s[kb][r] = -INFINITY;
      });
  if (my_tiles == 0) return;

  const float inv = 1.0f / f.lsum;
  const int mine = q0 + l32;
  uint16_t* op = g.O + ((size_t)(first + min(mine, n - 1)) * g.n_q + hq) * HEAD + 8 * h;
  uint32_t bad = 0;
#pragma unroll
  for (int db = 0; db < F::kDb; ++db)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      // registers 4 i .. 4 i + 3: dims 8 i + 4 h ..; halves trade, so that a lane has 8 in a row
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bf16x2 p = {(__bf16)(f.acc[db][4 * i + 2 * e] * inv), (__bf16)(f.acc[db][4 * i + 2 * e + 1] * inv)};
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
                   k = g.K + (size_t)(first + key) * g.k_stride + (size_t)kvh * HEAD;
                   v = g.V + (size_t)(first + key) * g.v_stride + (size_t)kvh * HEAD;
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
int launch(const PromptArgs& g, hipStream_t stream) {
  const int heads = heads_of(g.n_q / g.n_kv, WAVES), groups = g.n_q / heads;
  constexpr int kLds = Flash<HEAD, WAVES>::kLds;
  static std::atomic<int> state[64];          // 0 not yet, 1 done, -1 failed (per device)
  if (int st = allow_lds(reinterpret_cast<const void*>(prompt_kernel<HEAD, WAVES>), kLds, state)) return st;
  hipLaunchKernelGGL((prompt_kernel<HEAD, WAVES>), dim3((unsigned)(most_blocks(g.T, g.B, heads, WAVES) * groups)),
                     dim3(WAVES * 64), kLds, stream, g, heads, groups);
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
  // heads: 24.3 us with eight, 21.1 with four; 1 x 8192: 239 and 252).  The rule looks at the rows alone: many
  // sequences shorter than 256 tokens by the heads of a group leave waves of the eight without queries.
  const bool wide = (long long)g.T * g.n_q >= 512 * 256;
  if (g.head == 64) return wide ? launch<64, 8>(g, st) : launch<64, 4>(g, st);
  return wide ? launch<128, 8>(g, st) : launch<128, 4>(g, st);
}

}  // namespace w4

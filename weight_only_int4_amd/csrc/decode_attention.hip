// Attention of single tokens over the paged cache, a prefix common to the batch read once.
//
// The keys are split: the prefix into chunks that all sequences' queries of a key/value head see together
// (as many rows as the batch has sequences times the group), each sequence's own tokens into chunks of their
// own.  Every chunk gives, per row, a reference m, the sum l of p = exp(scale (s - m)) and sum p V in fp32; a
// second kernel joins a row's chunks: O = sum_c w_c O_c / sum_c w_c l_c, w_c = exp(scale (m_c - max m)).  (m is no
// more than the largest score, and less by as much as p may grow: to 2^8 in 16 rows' chunks, to sums of 2^30 in 128 rows'.)
// Chunk sizes follow from what the host knows, so a captured graph serves any lengths.
//
// What bounds it: long lengths the memory (64 sequences of 2,000 tokens behind 8,192, 32 heads on 8: 302 MB from
// it and 64 us in the chunks, 4.7 TB/s); short ones the way of one chunk from the lengths over the table, keys,
// scores and values to LDS and out, 5 us, and a second launch of 4 (16 sequences of 512 behind 2,048: 9.5 and 4.4).
#include "attend.hpp"
#include "flash_tile.hpp"

#pragma clang fp contract(off)

namespace w4 {

namespace {

constexpr float kSlack = 8.0f;                // a reference lags the maximum by at most 2^8: fp32 and bf16 lose nothing by it

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4_t;

constexpr int kWideRows = 128;                // rows of a prefix tile of four waves

// Everything a workgroup needs of a row: where its query lies and how far it sees.
struct Row {
  int b, hq, limit;
};

struct Kernel {
  DecodeArgs g;
  DecodePlan p;
  float* stats;               // NULL: one chunk in all, the output is written at once
  float* part;
};

// Page numbers of the 64 table entries from `base` on, one per lane: 1,024 keys, 16 a page or more.
struct Pages {
  int pages, base, held;
  __device__ __forceinline__ Pages(const int32_t* row, int width, int pages, int base) : pages(pages), base(base) {
    const int e = base + (threadIdx.x & 63);
    held = e < width ? row[e] : -1;
  }
  // page of a (wave-uniform) entry, -1 if there is none
  __device__ __forceinline__ int operator()(int entry) const {
    return held_page(__builtin_amdgcn_readlane(held, entry - base), pages);
  }
};

typedef const __attribute__((address_space(1))) char* global_bytes;
typedef const __attribute__((address_space(1))) u32x4* global_u32x4;

// One row once more, key by key.
template <int HEAD>
__device__ __forceinline__ void again(const DecodeArgs& g, int b, int hq) {
  const int n = held_length(g.lens[b], g.max_len), kvh = hq / (g.n_q / g.cache.n_kv);
  const int page_size = g.cache.page_size, shift = __builtin_ctz(page_size);
  attend<HEAD>(g.Q + (size_t)b * g.q_stride + (size_t)hq * HEAD, n, g.scale,
               [&](int key, const uint16_t*& k, const uint16_t*& v) {
                 const size_t row = key < g.prefix_len ? 0 : (size_t)b * g.table_width;
                 const int page = held_page(g.table[row + (key >> shift)], g.cache.pages);
                 if (page < 0) return;
                 const size_t at = (((size_t)page * g.cache.n_kv + kvh) * page_size + (key & (page_size - 1))) * HEAD;
                 k = g.cache.k + at;
                 v = g.cache.v + at;
               },
               g.O + ((size_t)b * g.n_q + hq) * HEAD);
}

// One chunk of keys [key0, end) for up to 16 rows; the waves take its tiles of 32 keys in turn,
// each by itself: K straight into registers as the operand of S^T = K Q^T
// (v_mfma_f32_16x16x32_bf16), V through LDS, from where the transposing read gives the operand of
// O^T += V^T P^T; the next tile's loads run meanwhile.
template <int HEAD, int WAVES>
__device__ void narrow_chunk(const Kernel& k, const Row& row, bool live, int kvh, const int32_t* table_row, int key0,
                             int end, int split, unsigned char* smem) {
  constexpr int kSteps = HEAD / 32, kDb = HEAD / 16, kRowB = 2 * HEAD, kChunks = HEAD / 8;
  constexpr int kRowsPer = 64 / kChunks, kLoads = 32 / kRowsPer;      // V rows of one load, loads of a tile
  const DecodeArgs& g = k.g;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, qd = lane >> 4;
  const int page_size = g.cache.page_size, shift = __builtin_ctz(page_size);
  const size_t page_elems = (size_t)g.cache.n_kv * page_size * HEAD;
  const size_t head_off = (size_t)kvh * page_size * HEAD;
  unsigned char* vlds = smem + wave * 32 * kRowB;
  const int first = key0 + wave * 32;
  const Pages pages(table_row, g.table_width, g.cache.pages, first >> shift);     // before the length is known

  bf16x8 qf[kSteps];
  {
    const uint16_t* qp = g.Q + (size_t)row.b * g.q_stride + (size_t)row.hq * HEAD + 8 * qd;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) qf[st] = *reinterpret_cast<const bf16x8*>(qp + 32 * st);
  }
  const float c = g.scale * kLog2e;
  f32x4_t acc[kDb];
#pragma unroll
  for (int db = 0; db < kDb; ++db) acc[db] = f32x4_t{};
  float mref = -INFINITY, lsum = 0.0f;

  // V rows in LDS: piece c of row r at c ^ swap(r): a transposing read takes 8 rows, 32 bytes each
  auto swap = [](int r) { return HEAD == 128 ? (r & 7) * 2 : ((r >> 1) & 3) * 2; };
  const int vrow = lane / kChunks, vpiece = lane % kChunks;
  uint32_t vwrite[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int r = vrow + j * kRowsPer;
    vwrite[j] = r * kRowB + 16 * (vpiece ^ swap(r));
  }
  const int tr = 4 * qd + (l16 >> 2);
  const uint32_t vread = tr * kRowB + 16 * (((l16 & 3) >> 1) ^ swap(tr)) + 8 * (l16 & 1);

  bf16x8 kf[2][kSteps];
  u32x4 vf[kLoads];
  int missing = 0, missing_next = 0;          // bits: the tile's 16-key halves that have no page
  // byte offsets into 16 rows of a page; the chunk's last 16 may end early: their rows past the end
  // repeat the last one in V (K's scores are masked)
  const uint32_t koff = l16 * kRowB + 16 * qd, voff = vrow * kRowB + 16 * vpiece;
  const int final16 = (end - 1) & ~15;
  uint32_t vfinal[kLoads / 2];
#pragma unroll
  for (int j = 0; j < kLoads / 2; ++j) vfinal[j] = min(vrow + j * kRowsPer, (end - 1) & 15) * kRowB + 16 * vpiece;
  auto load_tile = [&](int kb) {              // kb < end
    missing_next = 0;
    global_bytes kp[2], vp[2];
    bool final_half[2];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int k0 = min(kb + 16 * a, final16);
      final_half[a] = k0 == final16;
      const int page = pages(k0 >> shift);
      if (page < 0) missing_next |= 1 << a;
      const size_t at = 2 * ((size_t)max(page, 0) * page_elems + head_off + (size_t)(k0 & (page_size - 1)) * HEAD);
      kp[a] = (global_bytes)g.cache.k + at;
      vp[a] = (global_bytes)g.cache.v + at;
#pragma unroll
      for (int st = 0; st < kSteps; ++st)
        kf[a][st] = __builtin_bit_cast(bf16x8, *(global_u32x4)(kp[a] + (koff + 64 * st)));
    }
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int j = 0; j < kLoads / 2; ++j)
        vf[a * (kLoads / 2) + j] = *(global_u32x4)(vp[a] + (final_half[a] ? vfinal[j] : voff + j * kRowsPer * kRowB));
  };
  const bool work = first < end && g.cache.pages > 0;
  if (work) {
    load_tile(first);
    for (int kb = first; kb < end; kb += 32 * WAVES) {
      missing = missing_next;
      f32x4_t s[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        s[a] = f32x4_t{};
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
          s[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[a][st], qf[st], s[a], 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < kLoads; ++j) *reinterpret_cast<u32x4*>(vlds + vwrite[j]) = vf[j];
      if (kb + 32 * WAVES < end) load_tile(kb + 32 * WAVES);
      const int last = min(end, row.limit) - kb - 4 * qd;       // keys from here on are not this row's
      if (__ballot(last < 32 - 4 * qd) || missing) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (16 * a + r >= last || (missing >> a & 1)) s[a][r] = -INFINITY;
      }
      float top = s[0][0];
#pragma unroll
      for (int r = 1; r < 8; ++r) top = fmaxf(top, s[r >> 2][r & 3]);
      if (__ballot((top - mref) * c > kSlack)) {
        top = fmaxf(top, __shfl_xor(top, 16, kWave));
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        const float m = fmaxf(mref, top);
        const float corr = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((mref - m) * c);
        lsum *= corr;
#pragma unroll
        for (int db = 0; db < kDb; ++db) acc[db] *= corr;
        mref = m;
      }
      const float mc = mref == -INFINITY ? 0.0f : -mref * c;
      bf16x8 pf;
      const bf16x2 ones = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
      for (int r = 0; r < 8; r += 2) {        // the sum is of the rounded p, as the product with V has them
        const bf16x2 p = {(__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s[r >> 2][r & 3], c, mc)),
                          (__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s[r >> 2][(r & 3) + 1], c, mc))};
        lsum = __builtin_amdgcn_fdot2_f32_bf16(p, ones, lsum, false);
        pf[r] = p[0], pf[r + 1] = p[1];
      }
#pragma unroll
      for (int db = 0; db < kDb; ++db) {
        unsigned char* at = vlds + (vread ^ (32 * db));
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)at);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at + 16 * kRowB));
        const bf16x8 v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        acc[db] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, pf, acc[db], 0, 0, 0);
      }
    }
  }
  lsum += __shfl_xor(lsum, 16, kWave);
  lsum += __shfl_xor(lsum, 32, kWave);

  // the waves' results meet in LDS: [wave][row][HEAD + 4], then m and l
  constexpr int kPad = HEAD + 4;
  float* o = reinterpret_cast<float*>(smem);
  float* ml = o + WAVES * 16 * kPad;
  __syncthreads();
#pragma unroll
  for (int db = 0; db < kDb; ++db)
    *reinterpret_cast<f32x4_t*>(o + (wave * 16 + l16) * kPad + 16 * db + 4 * qd) = acc[db];
  if (qd == 0) ml[wave * 32 + l16] = mref, ml[wave * 32 + 16 + l16] = lsum;
  __syncthreads();
  if (threadIdx.x >= 256) return;
  const int i = threadIdx.x >> 4, d = (threadIdx.x & 15) * (HEAD / 16);
  float m = ml[i];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) m = fmaxf(m, ml[w * 32 + i]);
  float l = 0.0f, sum[HEAD / 16] = {};
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    // (a wave without a reference has the factor 0; it is multiplied like the others, see join_kernel)
    const float mw = ml[w * 32 + i], f = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((mw - m) * c);
    l += f * ml[w * 32 + 16 + i];
#pragma unroll
    for (int e = 0; e < HEAD / 16; ++e) sum[e] += f * o[(w * 16 + i) * kPad + d + e];
  }
  // thread group i of 16 writes row i; its numbers are lane i's
  const int b = __shfl(row.b, i, kWave), hq = __shfl(row.hq, i, kWave);
  const bool on = __shfl((int)live, i, kWave) != 0;
  const size_t r = (size_t)b * g.n_q + hq;
  if (k.stats) {
    if (!on) return;
    float* out = k.part + ((size_t)split * k.p.rows + r) * HEAD + d;
#pragma unroll
    for (int e = 0; e < HEAD / 16; e += 4)
      *reinterpret_cast<float4*>(out + e) = make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
    if ((threadIdx.x & 15) == 0)
      *reinterpret_cast<float2*>(k.stats + 2 * ((size_t)split * k.p.rows + r)) = make_float2(m, l);
    return;
  }
  // all there is: the output itself; rows that see nothing, or that are not finite, once more, key by key
  uint32_t w[HEAD / 32], bad = on && m == -INFINITY ? 0x80008000u : 0u;
#pragma unroll
  for (int e = 0; e < HEAD / 32; ++e) {
    const bf16x2 y = {(__bf16)(sum[2 * e] / l), (__bf16)(sum[2 * e + 1] / l)};
    w[e] = __builtin_bit_cast(uint32_t, y);
    bad |= on ? (w[e] & 0x7F807F80u) + 0x00800080u : 0u;
  }
  uint16_t* out = g.O + r * HEAD + d;
  if (on) {
    if constexpr (HEAD == 128) *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
  }
  const unsigned long long rows = __ballot((bad & 0x80008000u) != 0);
#pragma unroll 1
  for (int j = 0; j < 4; ++j)                 // a wave's four rows, 16 lanes each
    if (rows >> (16 * j) & 0xFFFF) again<HEAD>(g, __shfl(b, 16 * j, kWave), __shfl(hq, 16 * j, kWave));
}

// One chunk of the prefix, keys [key0, end), for up to 128 rows of the batch: four waves of 32 rows
// that share the key tiles (flash_tile.hpp).
template <int HEAD>
__device__ void wide_chunk(const Kernel& k, int tile, int kvh, int key0, int end, int split, unsigned char* smem) {
  using F = Flash<HEAD, 4>;
  const DecodeArgs& g = k.g;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int rows = g.B * k.p.group, i = tile * kWideRows + wave * 32 + l32, r = min(i, rows - 1);
  const int b = r / k.p.group, hq = kvh * k.p.group + r - b * k.p.group;
  const int limit = min(end, held_length(g.lens[b], g.max_len));
  const int page_size = g.cache.page_size, shift = __builtin_ctz(page_size);
  const size_t page_elems = (size_t)g.cache.n_kv * page_size * HEAD, head_off = (size_t)kvh * page_size * HEAD;
  // the chunk's pages, one per lane (at most 64: 1,024 keys, 16 a page or more)
  const int entry0 = key0 >> shift, entries = ((end - 1) >> shift) - entry0 + 1;
  const int held = lane < entries ? g.table[entry0 + lane] : 0;
  const bool missing = __ballot(lane < entries && held_page(held, g.cache.pages) < 0) != 0;
  int least = limit;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) least = min(least, __shfl_xor(least, off, kWave));
  const int tiles = (end - key0 + kTile - 1) / kTile;
  const int masked = missing ? 0 : max(__builtin_amdgcn_readfirstlane(least) - key0, 0) / kTile;
  const int mine = g.cache.pages > 0 && tile * kWideRows + wave * 32 < rows ? tiles : 0;

  F f;
  f.init(smem, g.scale);
  f.load_q(g.Q + (size_t)b * g.q_stride + (size_t)hq * HEAD);
  // Keys past the end and keys without a page are masked; what is copied for them is some other
  // page's rows, or rows of the same.
  const int row0 = F::copy_row();
  const uint32_t koff = (row0 & 15) * F::kRow + F::k_piece(), voff = (row0 & 15) * F::kRow + F::v_piece();
  auto page_of = [&](int key) {               // of a wave-uniform key of the chunk
    return held_page(__builtin_amdgcn_readlane(held, (key >> shift) - entry0), g.cache.pages);
  };
  if (g.cache.pages > 0)
    f.template walk<true>(
        tiles, mine, masked,
        [&](int kv, int t, int j, uint32_t lds) {
          const int first = key0 + t * kTile + ((wave * F::kPerCopy + j * F::kRowsApart) & ~15);     // 16 keys of one page
          const int key = min(first, (end - 1) & ~15);
          const uint16_t* from = (kv ? g.cache.v : g.cache.k) + (size_t)max(page_of(key), 0) * page_elems + head_off +
                                 (size_t)(key & (page_size - 1)) * HEAD;
          lds_copy16_free(kv ? voff : koff, from, lds);
        },
        [&](int t) {
          const int last = limit - key0 - t * kTile - 4 * h;
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int key = key0 + t * kTile + 32 * kb + 16 * half;
              const bool none = key >= end || page_of(key) < 0;
#pragma unroll
              for (int q = 0; q < 8; ++q)
                if (none || 32 * kb + 16 * half + (q & 3) + 8 * (q >> 2) >= last) f.s[kb][8 * half + q] = -INFINITY;
            }
        });
  if (i >= rows) return;
  const size_t row = (size_t)split * k.p.rows + (size_t)b * g.n_q + hq;
  float* out = k.part + row * HEAD + 4 * h;
#pragma unroll
  for (int db = 0; db < F::kDb; ++db)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<float4*>(out + 32 * db + 8 * q) =
          make_float4(f.acc[db][4 * q], f.acc[db][4 * q + 1], f.acc[db][4 * q + 2], f.acc[db][4 * q + 3]);
  if (h == 0) *reinterpret_cast<float2*>(k.stats + 2 * row) = make_float2(f.mref, f.lsum);
}

template <int HEAD, int WAVES>
constexpr int narrow_lds() {
  return WAVES * 16 * (HEAD + 4) * 4 + WAVES * 32 * 4;     // the join is larger than the V tiles (32 rows a wave)
}

template <int HEAD, int WAVES, bool WIDE>
constexpr int chunk_lds() {
  return WIDE ? std::max(Flash<HEAD, 4>::kLds, narrow_lds<HEAD, WAVES>()) : narrow_lds<HEAD, WAVES>();
}

template <int HEAD, int WAVES, bool WIDE>
__global__ __launch_bounds__(WAVES * 64, 2) void chunk_kernel(Kernel k) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const DecodeArgs& g = k.g;
  const DecodePlan& p = k.p;
  const int l16 = threadIdx.x & 15;
  int id = blockIdx.x;
  const int per_tile = g.cache.n_kv * p.p_splits;
  if (id < per_tile * p.p_tiles) {
    // prefix: row tile, chunk, key/value head (where the chunks of all heads are a multiple of 8, one chunk's row
    // tiles are on one XCD)
    const int tile = id / per_tile;
    id -= tile * per_tile;
    const int split = id / g.cache.n_kv, kvh = id - split * g.cache.n_kv;
    const int key0 = split * p.p_chunk, end = min(key0 + p.p_chunk, p.prefix);
    if constexpr (WIDE) {
      wide_chunk<HEAD>(k, tile, kvh, key0, end, split, smem);
    } else {
      const int rows = g.B * p.group, i = tile * 16 + l16, r = min(i, rows - 1);
      const int b = r / p.group;
      const Row row{b, kvh * p.group + r - b * p.group, held_length(g.lens[b], g.max_len)};
      narrow_chunk<HEAD, WAVES>(k, row, i < rows, kvh, g.table, key0, end, split, smem);
    }
    return;
  }
  id -= per_tile * p.p_tiles;
  // own tokens: chunk, row tile, sequence, key/value head
  const int kvh = id % g.cache.n_kv;
  id /= g.cache.n_kv;
  const int b = id % g.B;
  id /= g.B;
  const int tile = id % p.o_tiles, split = id / p.o_tiles;
  const int n = held_length(g.lens[b], g.max_len);
  const int key0 = p.prefix + split * p.o_chunk, end = min(key0 + p.o_chunk, n);
  if (k.stats && key0 >= end) return;
  const int i = tile * 16 + l16;
  const Row row{b, kvh * p.group + min(i, p.group - 1), n};
  narrow_chunk<HEAD, WAVES>(k, row, i < p.group, kvh, g.table + (size_t)b * g.table_width, key0, end, p.p_splits + split, smem);
}

// One wave per row: joins its chunks, 16 bytes a lane, so that 64 / (head / 4) chunks are read at once.
// Chunks of weight 0 are multiplied too: 0 times the infinity or NaN of a value that the row sees is NaN, as in one
// chunk, and one that it does not see goes when the row is computed once more.
template <int HEAD>
__global__ __launch_bounds__(256) void join_kernel(Kernel k) {
  constexpr int kLanes = HEAD / 4, kAtOnce = 64 / kLanes;
  const DecodeArgs& g = k.g;
  const DecodePlan& p = k.p;
  const size_t r = (size_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= p.rows) return;
  const int lane = threadIdx.x & 63, sub = lane / kLanes, d = 4 * (lane % kLanes);
  const int b = (int)(r / g.n_q), hq = (int)(r - (size_t)b * g.n_q);
  const int n = held_length(g.lens[b], g.max_len);
  const int own = n > p.prefix ? (n - p.prefix + p.o_chunk - 1) / p.o_chunk : 0;
  const int live = n > 0 ? p.p_splits + own : 0;
  const float c = g.scale * kLog2e;
  float m = -INFINITY;
  for (int s = lane; s < live; s += 64) m = fmaxf(m, k.stats[2 * ((size_t)s * p.rows + r)]);
  m = wave_max(m);
  float l = 0.0f;
  f32x4_t o = {};
  if (m != -INFINITY) {
    for (int s0 = 0; s0 < live; s0 += 64) {
      float f = 0.0f;
      if (s0 + lane < live) {
        const float2 v = *reinterpret_cast<const float2*>(k.stats + 2 * ((size_t)(s0 + lane) * p.rows + r));
        f = __builtin_amdgcn_exp2f((v.x - m) * c);      // without a v.x 0: nothing seen, or scores of NaN or -infinity alone
        l += f * v.y;
      }
      const int count = min(64, live - s0);
      for (int s1 = 0; s1 < count; s1 += 8 * kAtOnce) {
        f32x4_t x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int s = min(s1 + u * kAtOnce + sub, count - 1);
          x[u] = *reinterpret_cast<const f32x4_t*>(k.part + ((size_t)(s0 + s) * p.rows + r) * HEAD + d);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int s = s1 + u * kAtOnce + sub;
          const float fs = __shfl(f, min(s, 63), kWave);
          if (s < count) o += fs * x[u];
        }
      }
    }
    l = wave_sum(l);
  }
#pragma unroll
  for (int off = kLanes; off < 64; off *= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], off, kWave);
  const bf16x2 y0 = {(__bf16)(o[0] / l), (__bf16)(o[1] / l)}, y1 = {(__bf16)(o[2] / l), (__bf16)(o[3] / l)};
  const uint2 w = make_uint2(__builtin_bit_cast(uint32_t, y0), __builtin_bit_cast(uint32_t, y1));
  // nothing seen, or an infinity or NaN: once more, key by key
  const uint32_t bad = ((w.x & 0x7F807F80u) + 0x00800080u) | ((w.y & 0x7F807F80u) + 0x00800080u);
  if (m == -INFINITY || __ballot((bad & 0x80008000u) != 0)) {
    again<HEAD>(g, b, hq);
    return;
  }
  if (sub == 0) *reinterpret_cast<uint2*>(g.O + r * HEAD + d) = w;
}

// Chunks are as long as 256 workgroups make them, between 128 keys (four waves' tiles) and 1,024: fewer chunks
// have less to join (9 sequences of up to 1,214 tokens behind 11,136: 21.1 us, with 512 workgroups 22.2).
int chunk_of(long long work) { return (int)std::min(1024LL, std::max(128LL, (work / 256 + 127) / 128 * 128)); }

}  // namespace

DecodePlan plan_decode(int B, int n_q, const w4_kv_cache& cache, int max_len, int prefix_len) {
  DecodePlan p{};
  p.group = n_q / cache.n_kv;
  p.rows = (size_t)B * n_q;
  p.prefix = B > 1 ? std::min(prefix_len, max_len) : 0;      // (a single sequence shares with nobody)
  const int own = max_len - p.prefix;
  p.o_tiles = (p.group + 15) / 16;
  const long long o_work = (long long)own * B * cache.n_kv * p.o_tiles;
  // One chunk holds everything: eight waves take it, and there is nothing to join.  (One sequence of 500
  // tokens, 8 key/value heads: 9.9 us this way, 9.3 in four chunks and a join; of 380: 8.8 and 9.3; 250: 7.7 and 9.2.)
  if (p.prefix == 0 && own <= std::max(384, chunk_of(o_work))) {
    p.direct = true;
    p.o_chunk = 1024, p.o_splits = p.splits = 1;
    return p;
  }
  if (p.prefix > 0) {
    const long long rows = (long long)B * p.group;
    // Sixteen rows at a time read the prefix once per sixteen, from the L2; past 64 MB of that the shared walk is
    // faster (32 sequences x 4 heads: 1,024 tokens 16.3 us narrow, 17.7 wide; 2,048: 18.7 and 18.4; 4,096: 21.8 and
    // 20.7; 64 sequences under 8,192: 105 and 71).
    p.wide = rows > 64 && (double)rows / 16 * p.prefix * cache.n_kv * cache.head * 4 > 64 << 20;
    p.p_tiles = (int)(p.wide ? (rows + kWideRows - 1) / kWideRows : (rows + 15) / 16);
    const long long p_work = (long long)p.prefix * p.p_tiles * cache.n_kv;
    // wide: a workgroup per CU, or longer walks on fewer of them while the own tokens are many enough to be read
    // beside them (a workgroup per CU, and this; 8 key/value heads of 128, group 4: 64 sequences of up to 2,000 tokens
    // behind 8,192 71.6 and 64.4 us, of 1,000 51.2 and 47.4, 128 of 1,000 behind 4,096 75.0 and 66.8, 200 of 700 behind
    // 2,048 81.5 and 74.4, 100 of 500 behind 8,192 47.0 and 47.4, 48 of 3,000 behind 12,288 79.5 and 80.0; heads of 64
    // 40.7 and 39.3; but 2 heads, group 8, 128 of 1,500 behind 6,144 39.9 and 43.5; twice or half the divisor changes
    // nothing)
    const long long along = (long long)std::min(1024.0, (double)o_work / p.o_tiles * cache.head / 45000);
    p.p_chunk = p.wide ? (int)std::min(1024LL, std::max(256LL, (std::max(p_work / 256, along) + 63) / 64 * 64))
                       : chunk_of(p_work + o_work);
    p.o_chunk = p.wide ? chunk_of(o_work) : p.p_chunk;
    p.p_splits = (p.prefix + p.p_chunk - 1) / p.p_chunk;
  } else {
    p.o_chunk = chunk_of(o_work);
  }
  p.o_splits = (own + p.o_chunk - 1) / p.o_chunk;
  p.splits = p.p_splits + p.o_splits;
  p.stats_bytes = align_up((size_t)p.splits * p.rows * 8, 256);
  p.bytes = p.stats_bytes + (size_t)p.splits * p.rows * cache.head * 4;
  return p;
}

namespace {

long long chunk_blocks(const DecodePlan& p, int B, int n_kv) {
  return (long long)p.p_tiles * p.p_splits * n_kv + (long long)p.o_tiles * p.o_splits * n_kv * B;
}

}  // namespace

size_t decode_workspace_bytes(int B, int n_q, const w4_kv_cache& cache, int max_len, int prefix_len) {
  return B == 0 ? 0 : plan_decode(B, n_q, cache, max_len, prefix_len).bytes;
}

// Rows below 2^31 and lengths to 2^30 keep the plan's numbers within 64 bits and a chunk's last key within an int;
// the grid's limit then keeps splits x rows below 2^31.

bool decode_fits(int B, int n_q, const w4_kv_cache& cache, int max_len, int prefix_len) {
  if ((long long)B * n_q > 0x7FFFFFFFLL || max_len > 1 << 30 || prefix_len > 1 << 30) return false;
  const DecodePlan p = plan_decode(B, n_q, cache, max_len, prefix_len);
  return chunk_blocks(p, B, cache.n_kv) * 512 <= kGridThreads && (long long)((p.rows + 3) / 4) * 256 <= kGridThreads;
}

template <int HEAD, int WAVES, bool WIDE>
static int launch_chunks(const Kernel& k, hipStream_t st) {
  const long long blocks = chunk_blocks(k.p, k.g.B, k.g.cache.n_kv);
  constexpr int kLds = chunk_lds<HEAD, WAVES, WIDE>();
  static std::atomic<int> state[64];          // 0 not yet, 1 done, -1 failed (per device)
  if (int rc = allow_lds(reinterpret_cast<const void*>(chunk_kernel<HEAD, WAVES, WIDE>), kLds, state)) return rc;
  hipLaunchKernelGGL((chunk_kernel<HEAD, WAVES, WIDE>), dim3((unsigned)blocks), dim3(WAVES * 64), kLds, st, k);
  return W4_OK;
}

template <int HEAD>
static int launch(const DecodeArgs& g, hipStream_t st) {
  Kernel k{g, plan_decode(g.B, g.n_q, g.cache, g.max_len, g.prefix_len), nullptr, nullptr};
  if (!k.p.direct) {
    k.stats = static_cast<float*>(g.workspace);
    k.part = reinterpret_cast<float*>(static_cast<char*>(g.workspace) + k.p.stats_bytes);
  }
  if (int rc = k.p.direct ? launch_chunks<HEAD, 8, false>(k, st)
               : k.p.wide ? launch_chunks<HEAD, 4, true>(k, st)
                          : launch_chunks<HEAD, 4, false>(k, st))
    return rc;
  if (!k.p.direct)
    hipLaunchKernelGGL(join_kernel<HEAD>, dim3((unsigned)((k.p.rows + 3) / 4)), dim3(256), 0, st, k);
  W4_CHECK_LAUNCH();
  return W4_OK;
}

int launch_decode_attention(const DecodeArgs& g, hipStream_t st) {
  return g.cache.head == 64 ? launch<64>(g, st) : launch<128>(g, st);
}

}  // namespace w4

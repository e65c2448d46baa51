// Shared parts of the serving operators: norm, rotary append to the paged cache, prompt and
// single-token attention.  See include/w4a16.h for what each computes.
#pragma once

#include <atomic>

#include "held.hpp"
#include "internal.hpp"

namespace w4 {

// Most threads along one dimension of a grid (its size in work items is a 32-bit field).
constexpr long long kGridThreads = 0xFFFFFFFFLL;

// Most elements from one token to the next: 64 tokens stay below 2^32 bytes, the range of a
// copy's 32-bit offset.
constexpr long long kMaxStride = 1LL << 24;

// The sequence that token t of a packed batch belongs to, or -1: the last b with
// offsets[b] <= t, if t < offsets[b + 1].  All 64 lanes of the wave take part, with the same t:
// each step asks 64 places at once, so up to 4,096 sequences take two round trips.
__device__ __forceinline__ int find_sequence(const int32_t* offsets, int B, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int i = lane * step;
    const bool before = i < n && offsets[lo + i] <= t;
    const int c = __popcll(__ballot(before));
    if (c == 0) return -1;                         // (of ascending offsets only the first can lie behind t)
    const int skip = min((c - 1) * step, n - 1);
    lo += skip;
    n = min(step, n - skip);
  }
  return offsets[lo] <= t && t < offsets[lo + 1] ? lo : -1;
}

// Asks once per device for more than 64 KB of dynamic LDS for a kernel.
inline int allow_lds(const void* kernel, int bytes, std::atomic<int> (&state)[64]) {
  if (bytes <= 64 * 1024) return W4_OK;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return W4_ERR_HIP;
  int done = state[dev].load(std::memory_order_relaxed);
  if (done == 0) {
    done = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) == hipSuccess ? 1 : -1;
    state[dev].store(done, std::memory_order_relaxed);
  }
  return done == 1 ? W4_OK : W4_ERR_HIP;
}

}  // namespace w4

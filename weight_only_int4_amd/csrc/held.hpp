// What device arrays may say is held in range by these, before it becomes an address: packed offsets,
// lengths and page numbers cannot be seen by the host.  Plain functions, for host and device.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define W4_HELD __host__ __device__ __forceinline__
#else
#define W4_HELD inline
#endif

namespace w4 {

// token offset, in [0, T]
W4_HELD int held_offset(int32_t v, int T) { return v < 0 ? 0 : v > T ? T : v; }

// tokens of a sequence between two held offsets, at least 0
W4_HELD int held_count(int first, int next) { return next > first ? next - first : 0; }

// length of a cached sequence, in [0, max_len]
W4_HELD int held_length(int32_t v, int max_len) { return v < 0 ? 0 : v > max_len ? max_len : v; }

// page number, or -1 where the cache has no such page
W4_HELD int held_page(int32_t v, int pages) { return (uint32_t)v < (uint32_t)pages ? v : -1; }

// position of new token i of n of a sequence that is then `len` long, or -1 where it lies before 0 or past `positions`
W4_HELD int held_position(int32_t len, int n, int i, int positions) {
  const int64_t p = (int64_t)len - n + i;
  return p >= 0 && p < positions ? (int)p : -1;
}

}  // namespace w4

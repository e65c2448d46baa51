// The functions that hold device arrays' contents in range, over edge values: every result lies where the
// kernels may follow it, and values that are in range come back as they are.  Exit status 0: all hold.
#include <stdio.h>

#include "../weight_only_int4_amd/csrc/held.hpp"

using namespace w4;

int main() {
  const int32_t edges[] = {INT32_MIN, INT32_MIN + 1, -65536, -2, -1, 0, 1, 2, 15, 16, 17, 4095, 4096, 65535, 1 << 24, INT32_MAX - 1, INT32_MAX};
  const int sizes[] = {0, 1, 2, 16, 4096, 65536, INT32_MAX};
  long bad = 0, seen = 0;
  auto check = [&](bool ok, const char* what, long a, long b) {
    ++seen;
    if (!ok && bad++ < 10) printf("%s(%ld, %ld)\n", what, a, b);
  };
  for (int32_t v : edges)
    for (int n : sizes) {
      const int o = held_offset(v, n), l = held_length(v, n), p = held_page(v, n);
      check(o >= 0 && o <= n && (v < 0 || v > n || o == v), "held_offset", v, n);
      check(l >= 0 && l <= n && (v < 0 || v > n || l == v), "held_length", v, n);
      check(p == -1 || (p >= 0 && p < n && p == v), "held_page", v, n);
      check((p >= 0) == (v >= 0 && v < n), "held_page", v, n);
      for (int32_t w : edges) {
        const int a = held_offset(v, n), b = held_offset(w, n), c = held_count(a, b);
        check(c >= 0 && (c == 0 || a + c == b) && a + c <= n, "held_count", v, w);
        for (int i = 0; i <= 65535; i = 2 * i + 1) {
          const int q = held_position(v, c, i, n);
          const long want = (long)v - c + i;
          check(q == (want >= 0 && want < n ? want : -1), "held_position", v, i);
        }
      }
    }
  printf("%ld of %ld failed\n", bad, seen);
  return bad != 0 || seen < 1000;
}

// Host-side check of grid.h for the counts of workgroups (of 256 threads) on stdin:
// the launches follow one another, cover every workgroup once, and are ones that
// HIP takes.  Prints "ok <counts>" or the first failure.
#include <cstdio>

#include "../orthogonal_reparameterized_poetx_amd/csrc/grid.h"

int main() {
  long long n, seen = 0;
  while (std::scanf("%lld", &n) == 1) {
    long long at = 0;
    bool ok = true;
    poetx::launches(n, [&](int64_t first, uint32_t number) {
      ok = ok && first == at && number >= 1 && number * 256ll < 1ll << 32;
      at += number;
    });
    if (!ok || at != n) {
      std::printf("FAIL %lld workgroups\n", n);
      return 1;
    }
    ++seen;
  }
  std::printf("ok %lld\n", seen);
  return 0;
}

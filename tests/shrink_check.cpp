// Host-side check of the LDS layout of the adapters' shrink (shrink.h, the same
// functions the kernel calls): for every largest rank of a set, every rank of
// an adapter, every group of ranks that a workgroup may get (groups reach
// the end of the padding to whole matrix steps) and both element sizes, a group
// with ranks has pieces, each piece's place lies inside the weights' part of
// LDS, and so does every value the products read; a group without has none.
// Prints "ok <groups>" or the first failure.
#include <cstdio>

#include "../orthogonal_reparameterized_poetx_amd/csrc/shrink.h"

using namespace poetx;

int main() {
  long long groups = 0;
  for (int el = 8; el >= 4; el -= 4)
    for (int rmax = 1; rmax <= 256; ++rmax)
      for (int r = 1; r <= rmax; ++r) {
        const int rp = rmax <= 16 ? 16 : (r + 31) / 32 * 32;   // the adapter's padded ranks
        for (int rt = 1; rt <= 4; rt *= 2)
          for (int rank0 = 0; rank0 < rp; rank0 += 16 * rt, ++groups) {
            const RankGroup g = rank_group(r, rank0, rt, el);
            const int es = 16 / el, rows = shrink_rb(rt) / es;   // rows of B in a chunk: its columns
            const int have = r > rank0 ? (r - rank0 < 16 * rt ? r - rank0 : 16 * rt) : 0;
            bool ok = g.ranks == have && (have == 0) == (g.pieces == 0) && g.pieces >= 0;
            // the last piece of the last row; 16 bytes each
            ok = ok && (have == 0 || ((rows - 1) * g.ld + g.pieces * el) * es <= shrink_w(rt, es));
            ok = ok && g.pieces * el <= g.ld && g.ld >= 0 && (rows * g.pieces <= 16 * rt * shrink_rb(rt) / 16);
            if (!ok) {
              std::printf("FAIL el %d largest rank %d rank %d tiles %d from rank %d: ranks %d pieces %d ld %d\n", el, rmax,
                          r, rt, rank0, g.ranks, g.pieces, g.ld);
              return 1;
            }
          }
      }
  std::printf("ok %lld\n", groups);
  return 0;
}

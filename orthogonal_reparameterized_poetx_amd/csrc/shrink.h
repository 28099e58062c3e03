// How a workgroup of the adapters' shrink lays its operands out in LDS, shared
// by the kernel and by a host-side check.  Plain C++ (no HIP types).
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define POETX_HD __host__ __device__
#else
#define POETX_HD
#endif

namespace poetx {

constexpr int AD_T = 32;          // tokens of a tile
constexpr int SHRINK_WAVES = 4;
constexpr int TURN_LDS = 16 * 1024;   // bytes a transpose may take
// a chunk: bytes of a row; LDS bytes of a row of x or A, of x, of the weights
constexpr int shrink_rb(int rt) { return rt == 1 ? 1024 : 512; }
constexpr int shrink_row(int rt) { return shrink_rb(rt) + 16; }
constexpr int shrink_x(int rt) { return AD_T * shrink_row(rt); }
constexpr int shrink_w(int rt, int es) {
  const int byA = 16 * rt * shrink_row(rt), byB = shrink_rb(rt) / es * (16 * rt + (es == 4 ? 4 : 0)) * es;
  return byA > byB ? byA : byB;
}
constexpr int shrink_lds(int rt, int es) {
  const int most = shrink_x(rt) + shrink_w(rt, es);
  return most > TURN_LDS ? most : TURN_LDS;
}

// A workgroup's ranks rank0 .. rank0 + 16 rt of an adapter of rank r, and B's rows
// of them in LDS: pieces of el elements (16 bytes) a row, rows ld elements apart.
// The ranks are padded to whole matrix steps of 32, so a group of 16 may lie wholly
// in the padding: it has no ranks and no pieces.  (Larger groups begin at multiples
// of 32, and the last 32 of the padded ranks hold one of the adapter's.)
struct RankGroup { int ranks, pieces, ld; };
POETX_HD inline RankGroup rank_group(int r, int rank0, int rt, int el) {
  const int left = r - rank0, ranks = rt == 1 && left < 0 ? 0 : left < 16 * rt ? left : 16 * rt;
  const int pieces = (ranks + el - 1) / el;
  return RankGroup{ranks, pieces, pieces * el + (el == 4 ? 4 : 0)};
}

}  // namespace poetx

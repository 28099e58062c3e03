// Low-rank adapters of many requests beside one shared projection, forward
// and backward (include/poetx.h has the contract).  With T = s A x per token:
//   forward   y += B T
//   backward  U = s B^T dy,  dx += A^T U,  dA = sum U x^T,  dB = sum dy T^T
// The work is two kinds of product: "shrink", width -> rank (T from x, U from
// dy), and "expand", rank -> width (y from T, dx from U), plus the two
// gradients, sums of outer products over an adapter's tokens.  Every one of
// them reads or updates the activations once against a rank of a few dozen:
// HBM bounds them, not the matrix units.
//
// Tokens go in tiles of 32 of one segment.  Segment i owns the tile indices
// from start_i / 32 + i on, which are enough for its tiles whatever its length,
// so that a tile finds its segment by a search and no launch has to lay the
// tiles out first.
#include "../../include/poetx.h"
#include "common.h"
#include "host.h"

namespace poetx {

constexpr int AD_T = 32;          // tokens of a tile
constexpr int AD_MAX_RANK = 256;

struct AdEntry {
  const void* A;
  const void* B;
  float* dA;
  float* dB;
  int32_t r;
  float scale;
  int32_t rp;      // rank padded to whole MFMA steps
  int32_t row0;    // sum of rp over the adapters before this one
  int32_t pad[4];
};

struct AdSegs {
  const int32_t* start;   // [nseg + 1]
  const int32_t* which;   // [nseg]
  int32_t nseg, count;
  int32_t N;
};

struct AdTile {
  int t0, rows, adapter;   // rows == 0: nothing to do
};

__device__ __forceinline__ int clamp_token(int t, int N) { return t < 0 ? 0 : t > N ? N : t; }

// tile w of the launch: a 64-way search of the segment whose tiles it is
// among, by the whole wave; the result is the same in every lane.  Whatever
// the segment arrays hold, t0 and t0 + rows lie within [0, N] and the adapter
// is one of the set's.
__device__ __forceinline__ AdTile find_tile(const AdSegs& g, int w) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = g.nseg;
  for (;;) {
    const int step = (len + 63) >> 6;
    const int s = lo + lane * step;
    const bool in = lane * step < len;
    const int a = in ? clamp_token(g.start[s], g.N) : 0;
    const int b = in && step == 1 ? clamp_token(g.start[s + 1], g.N) : 0;
    const int ad = in && step == 1 ? g.which[s] : -1;
    const int k = __popcll(__ballot(in && a / AD_T + s <= w));
    if (k == 0) return AdTile{0, 0, 0};
    if (step == 1) {
      const int a0 = __builtin_amdgcn_readlane(a, k - 1), b0 = __builtin_amdgcn_readlane(b, k - 1);
      const int which = __builtin_amdgcn_readlane(ad, k - 1);
      const int64_t t0 = a0 + (int64_t)(w - (a0 / AD_T + lo + k - 1)) * AD_T;
      if (t0 >= b0 || which < 0 || which >= g.count) return AdTile{0, 0, 0};
      return AdTile{(int)t0, (int)(b0 - t0 < AD_T ? b0 - t0 : AD_T), which};
    }
    lo += (k - 1) * step;
    len = len - (k - 1) * step < step ? len - (k - 1) * step : step;
  }
}

// ---- element types.  A fragment is 16 bytes of a row: EL elements; the four
// lane groups of a wave hold KF = 4 EL elements of the contraction.  bf16: one
// 16x16x32 MFMA; fp32: four 16x16x4 MFMAs, element e of every group in MFMA e.
template <typename E> struct El;
template <> struct El<uint16_t> {
  static constexpr int EL = 8, KF = 32;
  static __device__ __forceinline__ f32x4 mma(uint4 a, uint4 b, f32x4 c) {
    return mfma16(as_bf16x8(a), as_bf16x8(b), c);
  }
};
template <> struct El<float> {
  static constexpr int EL = 4, KF = 16;
  static __device__ __forceinline__ f32x4 mma(uint4 a, uint4 b, f32x4 c) {
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
  }
};

// elements k .. k + EL of a row of `width`, zeros past its end
template <typename E, bool VEC>
__device__ __forceinline__ uint4 load_frag(const E* row, int k, int width) {
  constexpr int EL = El<E>::EL;
  if (VEC || k + EL <= width) {
    if (VEC) return k < width ? ldg16(row + k) : make_uint4(0, 0, 0, 0);
    E e[EL];
#pragma unroll
    for (int i = 0; i < EL; ++i) e[i] = row[k + i];
    return __builtin_bit_cast(uint4, e);
  }
  E e[EL];
#pragma unroll
  for (int i = 0; i < EL; ++i) e[i] = k + i < width ? row[k + i] : E(0);
  return __builtin_bit_cast(uint4, e);
}

// ---- shrink: T[rank][token] of each tile, fp32 [rpmax][32]
struct ShrinkJob {
  const void* X;      // [N][width], rows ldx apart
  const void* W;      // null: each adapter's A; else the padded rows [row0 + rank][ldw]
  float* T;
  int64_t ldx, ldw;
  int width;
};
struct ShrinkArgs {
  ShrinkJob job[2];
  AdSegs seg;
  const AdEntry* table;
  int rpmax;
};

template <typename E, int RT, bool VEC>
__global__ __launch_bounds__(512) void adapter_shrink_kernel(const ShrinkArgs a) {
  constexpr int EL = El<E>::EL, KF = El<E>::KF, WAVES = 8;
  __shared__ float red[WAVES][512];
  const int w = blockIdx.x;
  const AdTile tile = find_tile(a.seg, w);
  if (tile.rows == 0) return;
  const ShrinkJob& J = a.job[blockIdx.y];
  const AdEntry ad = a.table[tile.adapter];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int rt_n = (ad.rp + 15) >> 4;
  const E* X = static_cast<const E*>(J.X);
  const E* x[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int t = 16 * s + l16;
    x[s] = X + (int64_t)(tile.t0 + (t < tile.rows ? t : 0)) * J.ldx;
  }
  const E* W = J.W ? static_cast<const E*>(J.W) + (int64_t)ad.row0 * J.ldw : static_cast<const E*>(ad.A);
  const int64_t ldw = J.W ? J.ldw : J.width;
  f32x4 acc[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  // a step is two fragments: lane group g holds 2 EL neighbouring elements
  for (int k0 = wave * 2 * KF; k0 < J.width; k0 += WAVES * 2 * KF) {
    const int k = k0 + g * 2 * EL;
    uint4 xf[2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) xf[s][h] = load_frag<E, VEC>(x[s], k + h * EL, J.width);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      if (i < rt_n) {
        const int rank = 16 * i + l16;
        const E* wr = W + (int64_t)(rank < ad.r ? rank : 0) * ldw;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 wf = load_frag<E, VEC>(wr, k + h * EL, J.width);
          acc[i][0] = El<E>::mma(wf, xf[0][h], acc[i][0]);
          acc[i][1] = El<E>::mma(wf, xf[1][h], acc[i][1]);
        }
      }
    }
  }
  float* T = J.T + (int64_t)w * a.rpmax * AD_T;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    if (i < rt_n) {
#pragma unroll
      for (int s = 0; s < 2; ++s) *reinterpret_cast<f32x4*>(&red[wave][s * 256 + lane * 4]) = acc[i][s];
      __syncthreads();
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < WAVES; ++q) v += red[q][tid];
      const int rank = 16 * i + 4 * ((tid >> 6) & 3) + (tid & 3), t = 16 * (tid >> 8) + ((tid >> 2) & 15);
      T[rank * AD_T + t] = rank < ad.r && t < tile.rows ? v * ad.scale : 0.f;
      __syncthreads();
    }
  }
}

// ---- expand: Y[t][j] += sum_k T[k][t] W[j][k]
struct ExpandArgs {
  void* Y;
  int64_t ldy;
  int width, cols;      // cols: columns of a workgroup
  const void* W;        // null: each adapter's B (rows of r); else the padded rows, adapter a's from row0 * width on, rows of rp
  const float* T;
  AdSegs seg;
  const AdEntry* table;
  int rpmax;
};

// 8 (bf16) fp32 values as bf16 pairs: hi, and lo = value - hi, which keep 16 bits of the value
__device__ __forceinline__ void split8(const float f[8], uint4& hi, uint4& lo) {
  bf16x8 h, l;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bf16 x, y;
    split_bf16(f[e], x, y);
    h[e] = x;
    l[e] = y;
  }
  hi = as_u4(h);
  lo = as_u4(l);
}

template <typename E, int RT, bool VECY, bool VECW>
__global__ __launch_bounds__(256) void adapter_expand_kernel(const ExpandArgs a) {
  constexpr int EL = El<E>::EL, KF = El<E>::KF;
  constexpr bool BF = EL == 8;
  constexpr bool PACK = BF && RT == 1;   // 16 ranks: hi and lo side by side in one MFMA
  constexpr int NK = PACK ? 1 : RT * 16 / KF;
  constexpr int NP = BF && !PACK ? 2 : 1;
  const AdTile tile = find_tile(a.seg, blockIdx.x);
  if (tile.rows == 0) return;
  const AdEntry ad = a.table[tile.adapter];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const float* T = a.T + (int64_t)blockIdx.x * a.rpmax * AD_T;
  const int nk = PACK ? 1 : ad.rp / KF;
  // column of fragment c, element k: kk * KF + kc + e
  const int kc = PACK ? 8 * (g & 1) : g * EL;
  uint4 tf[NK][2][NP];
#pragma unroll
  for (int kk = 0; kk < NK; ++kk) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float f[8];
#pragma unroll
      for (int e = 0; e < EL; ++e) f[e] = kk >= nk ? 0.f : T[(kk * KF + kc + e) * AD_T + 16 * s + l16];
      if constexpr (BF) {
        uint4 hi, lo;
        split8(f, hi, lo);
        if constexpr (PACK) {
          const bool first = g < 2;
          tf[kk][s][0] = make_uint4(first ? hi.x : lo.x, first ? hi.y : lo.y, first ? hi.z : lo.z, first ? hi.w : lo.w);
        } else {
          tf[kk][s][0] = hi;
          tf[kk][s][NP - 1] = lo;
        }
      } else {
        tf[kk][s][0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                  __float_as_uint(f[3]));
      }
    }
  }
  const E* W = a.W ? static_cast<const E*>(a.W) + (int64_t)ad.row0 * a.width : static_cast<const E*>(ad.B);
  const int ldw = a.W ? ad.rp : ad.r;
  const int c0 = blockIdx.y * a.cols, c1 = c0 + a.cols < a.width ? c0 + a.cols : a.width;
  for (int jb = c0 + wave * 64; jb < c1; jb += 256) {
    // row of MFMA c, index 4 g' + q, is column jb + 16 g' + 4 c + q: a lane then holds 16 neighbouring columns
    f32x4 acc[4][2];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      acc[c][0] = acc[c][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      int j = jb + 16 * (l16 >> 2) + 4 * c + (l16 & 3);
      j = j < a.width ? j : a.width - 1;
      const E* wr = W + (int64_t)j * ldw;
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        if (kk < nk) {
          const uint4 wf = load_frag<E, VECW>(wr, kk * KF + kc, ldw);
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int p = 0; p < NP; ++p) acc[c][s] = El<E>::mma(wf, tf[kk][s][p], acc[c][s]);
        }
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int t = 16 * s + l16;
      if (t >= tile.rows) continue;
      E* y = static_cast<E*>(a.Y) + (int64_t)(tile.t0 + t) * a.ldy;
      const int j0 = jb + 16 * g;
#pragma unroll
      for (int h = 0; h < 16 / EL; ++h) {
        const int j = j0 + h * EL;
        float v[EL];
#pragma unroll
        for (int e = 0; e < EL; ++e) v[e] = acc[(h * EL + e) >> 2][s][e & 3];
        if (VECY) {
          if (j >= a.width) continue;
          const uint4 o = ldg16(y + j);
          const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
          uint32_t n[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if constexpr (BF)
              n[q] = pack2(f32_to_bits(__uint_as_float(ow[q] << 16) + v[2 * q]),
                           f32_to_bits(__uint_as_float(ow[q] & 0xffff0000u) + v[2 * q + 1]));
            else
              n[q] = __float_as_uint(__uint_as_float(ow[q]) + v[q]);
          }
          stg16(y + j, make_uint4(n[0], n[1], n[2], n[3]));
        } else {
#pragma unroll
          for (int e = 0; e < EL; ++e)
            if (j + e < a.width) {
              if constexpr (BF) y[j + e] = f32_to_bits(bits_to_f32(y[j + e]) + v[e]);
              else y[j + e] += v[e];
            }
        }
      }
    }
  }
}

// ---- the tiles of each adapter, one adapter after another, for the gradients:
// list entry {t0, rows, adapter, tile index}, offs[a] the first entry of
// adapter a; and the transposed, rank-padded adapters: Bt [rank][mp] and
// At [column][rp], which make U a shrink and dx an expand.
struct PrepArgs {
  AdSegs seg;
  const AdEntry* table;
  int4* list;
  int32_t* offs;
  void *Bt, *At;
  int m, n, mp, cap, tw;   // cap: entries of list; tw: rows of B or columns of A a transpose takes at a time
};

__device__ __forceinline__ int tiles_of(const AdSegs& g, int s, int& a, int& t0, int& t1) {
  t0 = clamp_token(g.start[s], g.N);
  t1 = clamp_token(g.start[s + 1], g.N);
  a = g.which[s];
  return a >= 0 && a < g.count && t1 > t0 ? (t1 - t0 + AD_T - 1) / AD_T : 0;
}

template <typename E>
__global__ __launch_bounds__(256) void adapter_prep_kernel(const PrepArgs p) {
  extern __shared__ char lds_raw[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if ((int)blockIdx.x < p.seg.count) {
    int* cnt = reinterpret_cast<int*>(lds_raw);   // [4] sums of the waves
    const int me = blockIdx.x;
    int before = 0;
    for (int s = tid; s < p.seg.nseg; s += 256) {
      int a, t0, t1;
      const int k = tiles_of(p.seg, s, a, t0, t1);
      if (k && a < me) before += k;
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) before += __shfl_xor(before, o);
    if (lane == 0) cnt[wave] = before;
    __syncthreads();
    int pos = cnt[0] + cnt[1] + cnt[2] + cnt[3];
    __syncthreads();
    // (segments that overlap, against the contract, could fill more than the list)
    if (tid == 0) p.offs[me] = pos < p.cap ? pos : p.cap;
    for (int s0 = 0; s0 < p.seg.nseg; s0 += 256) {
      int a = -1, t0 = 0, t1 = 0, k = 0;
      if (s0 + tid < p.seg.nseg) k = tiles_of(p.seg, s0 + tid, a, t0, t1);
      if (a != me) k = 0;
      int inc = k;   // inclusive sum over the wave
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 63) cnt[wave] = inc;
      __syncthreads();
      int at = pos + inc - k;
      for (int q = 0; q < wave; ++q) at += cnt[q];
      pos += cnt[0] + cnt[1] + cnt[2] + cnt[3];
      __syncthreads();
      for (int i = 0; i < k; ++i) {
        const int t = t0 + i * AD_T;
        if (at + i < p.cap) p.list[at + i] = make_int4(t, t1 - t < AD_T ? t1 - t : AD_T, me, t0 / AD_T + s0 + tid + i);
      }
    }
    if (tid == 0 && me == p.seg.count - 1) p.offs[p.seg.count] = pos < p.cap ? pos : p.cap;
    return;
  }
  // transposes
  E* lds = reinterpret_cast<E*>(lds_raw);
  const int tw = p.tw, bt = (p.m + tw - 1) / tw, at = (p.n + tw - 1) / tw;
  int b = blockIdx.x - p.seg.count;
  const AdEntry ad = p.table[b / (bt + at)];
  b %= bt + at;
  if (b < bt) {
    const int j0 = b * tw, rows = p.m - j0 < tw ? p.m - j0 : tw;
    const E* B = static_cast<const E*>(ad.B) + (int64_t)j0 * ad.r;
    for (int i = tid; i < rows * ad.r; i += 256) lds[(i / ad.r) * (ad.r + 1) + i % ad.r] = B[i];
    __syncthreads();
    E* out = static_cast<E*>(p.Bt) + (int64_t)ad.row0 * p.mp + j0;
    const int cols = p.mp - j0 < tw ? p.mp - j0 : tw;
    for (int i = tid; i < ad.rp * tw; i += 256) {
      const int rank = i / tw, j = i % tw;
      if (j < cols) out[(int64_t)rank * p.mp + j] = rank < ad.r && j < rows ? lds[j * (ad.r + 1) + rank] : E(0);
    }
  } else {
    const int i0 = (b - bt) * tw, cols = p.n - i0 < tw ? p.n - i0 : tw;
    const E* A = static_cast<const E*>(ad.A) + i0;
    for (int i = tid; i < ad.r * tw; i += 256) {
      const int rank = i / tw, c = i % tw;
      if (c < cols) lds[c * (ad.r + 1) + rank] = A[(int64_t)rank * p.n + c];
    }
    __syncthreads();
    E* out = static_cast<E*>(p.At) + (int64_t)ad.row0 * p.n + (int64_t)i0 * ad.rp;
    for (int i = tid; i < cols * ad.rp; i += 256) {
      const int c = i / ad.rp, rank = i % ad.rp;
      out[i] = rank < ad.r ? lds[c * (ad.r + 1) + rank] : E(0);
    }
  }
}

// ---- outer products: part[slot][rank][col] = sum over a run's tokens of T[rank][t] X[t][col]
struct OuterJob {
  const void* X;
  const float* T;
  float* part;
  int64_t ldx;
  int width;
};
struct OuterArgs {
  OuterJob job[2];
  const int4* list;
  const int32_t* offs;
  int count, rpmax, run, groups;   // run: list entries of a workgroup; groups of 64 ranks
};

// Wave: one slab of columns (16 lanes x EL), every list entry of the run.
// Lane (g, c) loads EL neighbouring columns of its tokens; the MFMA for
// element e takes column EL c + e as its row c.  bf16: eight tokens a lane
// (8 g + i), gathered into operands of eight tokens by byte permutes; fp32:
// MFMA step i takes token 4 i + g.  Partial sums of one adapter within a run
// go to slot run + adapter (each run begins where the one before it ended, so
// no two pairs share a slot); a second kernel adds an adapter's slots in order.
template <typename E, int RT, bool VEC>
__global__ __launch_bounds__(256) void adapter_outer_kernel(const OuterArgs a) {
  constexpr int EL = El<E>::EL;
  constexpr bool BF = EL == 8;
  const int jz = blockIdx.z / a.groups, grp = blockIdx.z % a.groups;
  const OuterJob& J = a.job[jz];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int cb = (blockIdx.x * 4 + wave) * 16 * EL;
  if (cb >= J.width) return;
  const int col = cb + l16 * EL;
  const int total = a.offs[a.count];
  int e0 = blockIdx.y * a.run, e1 = e0 + a.run;
  if (e1 > total) e1 = total;
  if (e0 >= e1) return;
  f32x4 acc[EL][RT];
  auto clear = [&]() {
#pragma unroll
    for (int e = 0; e < EL; ++e)
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[e][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  auto flush = [&](int adapter) {
    float* P = J.part + (int64_t)(blockIdx.y + adapter) * a.rpmax * J.width;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int rank = grp * 64 + 16 * i + l16;
      if (rank >= a.rpmax) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = cb + (4 * g + q) * EL;
        float* dst = P + (int64_t)rank * J.width + c;
        if (VEC) {
          if (c < J.width) {
#pragma unroll
            for (int h = 0; h < EL / 4; ++h)
              *reinterpret_cast<f32x4*>(dst + 4 * h) =
                  f32x4{acc[4 * h][i][q], acc[4 * h + 1][i][q], acc[4 * h + 2][i][q], acc[4 * h + 3][i][q]};
          }
        } else {
#pragma unroll
          for (int e = 0; e < EL; ++e)
            if (c + e < J.width) dst[e] = acc[e][i][q];
        }
      }
    }
  };
  clear();
  int cur = -1;
  for (int p = e0; p < e1; ++p) {
    const int4 en = a.list[p];
    if (en.z != cur) {
      if (cur >= 0) {
        flush(cur);
        clear();
      }
      cur = en.z;
    }
    const E* X = static_cast<const E*>(J.X) + (int64_t)en.x * J.ldx;
    const float* T = J.T + (int64_t)en.w * a.rpmax * AD_T;
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = BF ? 8 * g + i : 4 * i + g;
      // past the tile's end T is zero, but 0 x NaN is not
      x[i] = t < en.y ? load_frag<E, VEC>(X + (int64_t)t * J.ldx, col, J.width) : make_uint4(0, 0, 0, 0);
    }
    if constexpr (BF) {
      uint4 op[8];   // operand e: column e of the lane, eight tokens
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = c == 0 ? x[i].x : c == 1 ? x[i].y : c == 2 ? x[i].z : x[i].w;
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = __builtin_amdgcn_perm(d[2 * i + 1], d[2 * i], 0x05040100u);
          hi[i] = __builtin_amdgcn_perm(d[2 * i + 1], d[2 * i], 0x07060302u);
        }
        op[2 * c] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        op[2 * c + 1] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int rank = grp * 64 + 16 * i + l16;
        const float* tr = T + (rank < a.rpmax ? rank : 0) * AD_T + 8 * g;
        const f32x4 f0 = *reinterpret_cast<const f32x4*>(tr), f1 = *reinterpret_cast<const f32x4*>(tr + 4);
        const float f[8] = {f0[0], f0[1], f0[2], f0[3], f1[0], f1[1], f1[2], f1[3]};
        uint4 h, l;
        split8(f, h, l);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          acc[e][i] = El<E>::mma(op[e], h, acc[e][i]);
          acc[e][i] = El<E>::mma(op[e], l, acc[e][i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int rank = grp * 64 + 16 * i + l16;
        const float* tr = T + (rank < a.rpmax ? rank : 0) * AD_T + g;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const float f = tr[4 * s];
          acc[0][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[s].x), f, acc[0][i], 0, 0, 0);
          acc[1][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[s].y), f, acc[1][i], 0, 0, 0);
          acc[2][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[s].z), f, acc[2][i], 0, 0, 0);
          acc[3][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[s].w), f, acc[3][i], 0, 0, 0);
        }
      }
    }
  }
  flush(cur);
}

struct ReduceArgs {
  const float* part[2];
  const int32_t* offs;
  const AdEntry* table;
  int width[2];          // n (dA), m (dB)
  int rpmax, run, accumulate;
};

// dA [r][n] and dB [m][r] of every adapter; zero where it had no token
__global__ __launch_bounds__(256) void adapter_reduce_kernel(const ReduceArgs a) {
  const int ad = blockIdx.y, job = blockIdx.z, width = a.width[job];
  const AdEntry e = a.table[ad];
  float* out = job ? e.dB : e.dA;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (!out || i >= (int64_t)e.r * width) return;
  const int rank = (int)(i / width), col = (int)(i % width);
  const int o0 = a.offs[ad], o1 = a.offs[ad + 1];
  float v = 0.f;
  if (o1 > o0) {
    const int q1 = (o1 - 1) / a.run;
    const float* p = a.part[job] + (int64_t)rank * width + col;
    for (int q = o0 / a.run; q <= q1; ++q) v += p[(int64_t)(q + ad) * a.rpmax * width];
  }
  float* dst = job ? out + (int64_t)col * e.r + rank : out + i;
  *dst = a.accumulate ? *dst + v : v;
}

}  // namespace poetx

using namespace poetx;

namespace {

constexpr int64_t kMaxAdapterDim = 32768;
constexpr int kMaxAdapters = 65535, kMaxSegs = 1 << 20;
enum { LAY_A16 = 1, LAY_B16 = 2 };   // poetx_adapters.layout

// ranks in whole MFMA steps: 16, or multiples of 32 for all adapters of a set with a rank over 16
int pad_rank(int r, int rmax) { return rmax <= 16 ? 16 : (r + 31) / 32 * 32; }
int rank_tiles(int rmax) {
  const int rp = pad_rank(rmax, rmax);
  return rp <= 16 ? 1 : rp <= 32 ? 2 : rp <= 64 ? 4 : rp <= 128 ? 8 : 16;
}
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check_dims(int64_t m, int64_t n, int32_t dtype) {
  if (m < 1 || m > kMaxAdapterDim || n < 1 || n > kMaxAdapterDim)
    return host_fail(POETX_ESHAPE, "m=%lld n=%lld out of range [1, %lld]", (long long)m, (long long)n,
                     (long long)kMaxAdapterDim);
  if (dtype != POETX_F32 && dtype != POETX_BF16) return host_fail(POETX_EDTYPE, "unsupported dtype %d", (int)dtype);
  return POETX_OK;
}

int check_adapters(const poetx_adapters* s, bool table) {
  if (!s) return host_fail(POETX_EINVAL, "set is NULL");
  const int rc = check_dims(s->m, s->n, s->dtype);
  if (rc) return rc;
  if (s->reserved || s->count < 0 || s->count > kMaxAdapters || s->max_rank < 0 || s->max_rank > AD_MAX_RANK ||
      s->rows < 0 || (s->layout & ~(LAY_A16 | LAY_B16)) || (s->count > 0) != (s->max_rank > 0))
    return host_fail(POETX_EINVAL, "set was not made by poetx_adapter_table");
  if (s->flags & ~POETX_ACCUMULATE_GRAD) return host_fail(POETX_EINVAL, "unknown flags 0x%x", s->flags);
  if (table && s->count > 0 && (!s->table || (reinterpret_cast<uintptr_t>(s->table) & (kWsAlign - 1))))
    return host_fail(POETX_EINVAL, "set->table is NULL or not %zu-byte aligned", kWsAlign);
  return POETX_OK;
}

int check_tokens(int64_t N, int32_t nseg, const int32_t* start, const int32_t* which) {
  if (N < 0 || N >= (int64_t(1) << 31) - AD_T) return host_fail(POETX_ESHAPE, "N=%lld out of range", (long long)N);
  if (nseg < 0 || nseg > kMaxSegs) return host_fail(POETX_ESHAPE, "nseg=%d out of range [0, %d]", (int)nseg, kMaxSegs);
  if (nseg > 0 && (!start || !which)) return host_fail(POETX_EINVAL, "NULL segment array");
  return POETX_OK;
}

// one activation matrix: pointer and row stride
int check_rows(const char* name, const void* p, int64_t ld, int64_t width, int32_t dtype) {
  if (!p) return host_fail(POETX_EINVAL, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & (dtype == POETX_F32 ? 3 : 1))
    return host_fail(POETX_EINVAL, "%s not aligned to its type", name);
  if (ld < width || ld > (int64_t(1) << 31))
    return host_fail(POETX_ESHAPE, "row stride of %s: %lld, width %lld", name, (long long)ld, (long long)width);
  return POETX_OK;
}

struct AdPlan {
  int64_t tiles;           // tile indices of a call
  int rpmax, mp, run, runs, slots, groups;
  float *T, *U, *part[2];
  void *Bt, *At;
  int4* list;
  int32_t* offs;
  size_t bytes;
};

AdPlan plan_adapters(const poetx_adapters* s, int64_t N, int32_t nseg, bool bwd, void* ws) {
  AdPlan p{};
  const bool f32 = s->dtype == POETX_F32;
  const size_t es = f32 ? 4 : 2;
  p.tiles = N / AD_T + nseg;
  p.rpmax = pad_rank(s->max_rank, s->max_rank);
  size_t off = 0;
  auto take = [&](size_t bytes) -> char* {
    off = (off + kWsAlign - 1) / kWsAlign * kWsAlign;
    char* q = ws ? static_cast<char*>(ws) + off : nullptr;
    off += bytes;
    return q;
  };
  const size_t tbytes = (size_t)p.tiles * p.rpmax * AD_T * sizeof(float);
  p.T = reinterpret_cast<float*>(take(tbytes));
  if (bwd) {
    p.U = reinterpret_cast<float*>(take(tbytes));
    p.mp = (int)((s->m + 7) / 8 * 8);
    p.Bt = take((size_t)s->rows * p.mp * es);
    p.At = take((size_t)s->rows * s->n * es);
    p.list = reinterpret_cast<int4*>(take((size_t)p.tiles * sizeof(int4)));
    p.offs = reinterpret_cast<int32_t*>(take((size_t)(s->count + 1) * sizeof(int32_t)));
    // runs of tiles: about 1024 workgroups over both gradients
    p.groups = (p.rpmax + 63) / 64;
    const int64_t slab = 4 * 16 * (f32 ? 4 : 8);
    const int64_t x = ((s->m + slab - 1) / slab + (s->n + slab - 1) / slab) * p.groups;
    int64_t runs = 1024 / x;
    if (runs < 1) runs = 1;
    if (runs > p.tiles) runs = p.tiles > 0 ? p.tiles : 1;
    p.run = (int)((p.tiles + runs - 1) / runs);
    if (p.run < 1) p.run = 1;
    p.runs = (int)((p.tiles + p.run - 1) / p.run);
    p.slots = p.runs + s->count;
    p.part[0] = reinterpret_cast<float*>(take((size_t)p.slots * p.rpmax * s->n * sizeof(float)));
    p.part[1] = reinterpret_cast<float*>(take((size_t)p.slots * p.rpmax * s->m * sizeof(float)));
  }
  p.bytes = off + kWsAlign;
  return p;
}

AdSegs segs_of(const poetx_adapters* s, const int32_t* start, const int32_t* which, int32_t nseg, int64_t N) {
  return AdSegs{start, which, nseg, s->count, (int32_t)N};
}

template <typename E, int RT, bool VEC>
void shrink(const ShrinkArgs& a, int64_t tiles, int jobs, hipStream_t s) {
  hipLaunchKernelGGL((adapter_shrink_kernel<E, RT, VEC>), dim3((unsigned)tiles, jobs), dim3(512), 0, s, a);
}
template <typename E>
void launch_shrink(const ShrinkArgs& a, int64_t tiles, int jobs, int rt, bool vec, hipStream_t s) {
#define POETX_RT(R) case R: vec ? shrink<E, R, true>(a, tiles, jobs, s) : shrink<E, R, false>(a, tiles, jobs, s); break;
  switch (rt) { POETX_RT(1) POETX_RT(2) POETX_RT(4) POETX_RT(8) POETX_RT(16) }
#undef POETX_RT
}

template <typename E, int RT>
void expand(const ExpandArgs& a, dim3 grid, bool vecy, bool vecw, hipStream_t s) {
  if (vecy && vecw) hipLaunchKernelGGL((adapter_expand_kernel<E, RT, true, true>), grid, dim3(256), 0, s, a);
  else if (vecy) hipLaunchKernelGGL((adapter_expand_kernel<E, RT, true, false>), grid, dim3(256), 0, s, a);
  else if (vecw) hipLaunchKernelGGL((adapter_expand_kernel<E, RT, false, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((adapter_expand_kernel<E, RT, false, false>), grid, dim3(256), 0, s, a);
}
template <typename E>
void launch_expand(ExpandArgs a, int64_t tiles, int rt, bool vecw, hipStream_t s) {
  const size_t es = sizeof(E);
  const bool vecy = al16(a.Y) && a.ldy * es % 16 == 0 && a.width * es % 16 == 0;
  // columns of a workgroup: enough workgroups to fill the chip, then as many columns as there are
  int64_t parts = (2048 + tiles - 1) / tiles;
  const int64_t most = (a.width + 255) / 256;
  if (parts > most) parts = most;
  a.cols = (int)((most + parts - 1) / parts * 256);
  const dim3 grid((unsigned)tiles, (unsigned)((a.width + a.cols - 1) / a.cols));
  switch (rt) {
    case 1: expand<E, 1>(a, grid, vecy, vecw, s); break;
    case 2: expand<E, 2>(a, grid, vecy, vecw, s); break;
    case 4: expand<E, 4>(a, grid, vecy, vecw, s); break;
    case 8: expand<E, 8>(a, grid, vecy, vecw, s); break;
    case 16: expand<E, 16>(a, grid, vecy, vecw, s); break;
  }
}

template <typename E, int RT>
void outer(const OuterArgs& a, dim3 grid, bool vec, hipStream_t s) {
  if (vec) hipLaunchKernelGGL((adapter_outer_kernel<E, RT, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((adapter_outer_kernel<E, RT, false>), grid, dim3(256), 0, s, a);
}

template <typename E>
int forward_impl(const poetx_adapters* set, const AdSegs& seg, const void* X, int64_t ldx, void* Y, int64_t ldy,
                 const AdPlan& p, hipStream_t s) {
  const size_t es = sizeof(E);
  const int rt = rank_tiles(set->max_rank);
  const AdEntry* table = static_cast<const AdEntry*>(set->table);
  const double flops = 2.0 * seg.N * set->max_rank;
  {
    HostTimer tm(s, "adapter_shrink", flops * set->n, (double)seg.N * set->n * es);
    ShrinkArgs a{};
    a.job[0] = ShrinkJob{X, nullptr, p.T, ldx, 0, (int)set->n};
    a.seg = seg;
    a.table = table;
    a.rpmax = p.rpmax;
    const bool vec = al16(X) && ldx * es % 16 == 0 && set->n * es % 16 == 0 && (set->layout & LAY_A16);
    launch_shrink<E>(a, p.tiles, 1, rt, vec, s);
  }
  {
    HostTimer tm(s, "adapter_expand", flops * set->m, 2.0 * seg.N * set->m * es);
    ExpandArgs a{};
    a.Y = Y; a.ldy = ldy; a.width = (int)set->m; a.T = p.T; a.seg = seg; a.table = table; a.rpmax = p.rpmax;
    launch_expand<E>(a, p.tiles, rt, (set->layout & LAY_B16) != 0, s);
  }
  return host_check_launch("adapters forward");
}

template <typename E>
int backward_impl(const poetx_adapters* set, const AdSegs& seg, const void* X, int64_t ldx, const void* dY,
                  int64_t lddy, void* dX, int64_t lddx, const AdPlan& p, hipStream_t s) {
  const size_t es = sizeof(E);
  const int rt = rank_tiles(set->max_rank);
  const int m = (int)set->m, n = (int)set->n;
  const AdEntry* table = static_cast<const AdEntry*>(set->table);
  const double flops = 2.0 * seg.N * set->max_rank;
  const bool xvec = al16(X) && ldx * es % 16 == 0 && n * es % 16 == 0;
  const bool yvec = al16(dY) && lddy * es % 16 == 0 && m * es % 16 == 0;
  {
    HostTimer tm(s, "adapter_prep", 0.0, 2.0 * set->rows * (m + n) * es);
    const int tw = set->max_rank > 96 ? 32 : 64;   // at most 33 KB of LDS
    PrepArgs a{seg, table, p.list, p.offs, p.Bt, p.At, m, n, p.mp, (int)p.tiles, tw};
    const unsigned grid = (unsigned)(set->count * (1 + (m + tw - 1) / tw + (n + tw - 1) / tw));
    const size_t lds = (size_t)tw * (set->max_rank + 1) * sizeof(E);
    hipLaunchKernelGGL(adapter_prep_kernel<E>, dim3(grid), dim3(256), lds < 64 ? 64 : lds, s, a);
  }
  if (p.tiles > 0) {
    {
      HostTimer tm(s, "adapter_shrink", flops * (m + n), (double)seg.N * (m + n) * es);
      ShrinkArgs a{};
      a.job[0] = ShrinkJob{X, nullptr, p.T, ldx, 0, n};
      a.job[1] = ShrinkJob{dY, p.Bt, p.U, lddy, p.mp, m};
      a.seg = seg;
      a.table = table;
      a.rpmax = p.rpmax;
      launch_shrink<E>(a, p.tiles, 2, rt, xvec && yvec && (set->layout & LAY_A16), s);
    }
    {
      HostTimer tm(s, "adapter_outer", 2 * flops * (m + n), (double)seg.N * (m + n) * es);
      OuterArgs a{};
      a.job[0] = OuterJob{X, p.U, p.part[0], ldx, n};
      a.job[1] = OuterJob{dY, p.T, p.part[1], lddy, m};
      a.list = p.list; a.offs = p.offs; a.count = set->count; a.rpmax = p.rpmax; a.run = p.run; a.groups = p.groups;
      const int slab = 4 * 16 * El<E>::EL, wide = m > n ? m : n;
      const dim3 grid((unsigned)((wide + slab - 1) / slab), (unsigned)p.runs, (unsigned)(2 * p.groups));
      if (rt == 1) outer<E, 1>(a, grid, xvec && yvec, s);
      else if (rt == 2) outer<E, 2>(a, grid, xvec && yvec, s);
      else outer<E, 4>(a, grid, xvec && yvec, s);
    }
    if (dX) {
      HostTimer tm(s, "adapter_expand", flops * n, 2.0 * seg.N * n * es);
      ExpandArgs a{};
      a.Y = dX; a.ldy = lddx; a.width = n; a.W = p.At; a.T = p.U; a.seg = seg; a.table = table; a.rpmax = p.rpmax;
      launch_expand<E>(a, p.tiles, rt, true, s);
    }
  }
  {
    HostTimer tm(s, "adapter_reduce", 0.0, 0.0);
    ReduceArgs a{};
    a.part[0] = p.part[0]; a.part[1] = p.part[1];
    a.offs = p.offs; a.table = table; a.width[0] = n; a.width[1] = m; a.rpmax = p.rpmax; a.run = p.run;
    a.accumulate = (set->flags & POETX_ACCUMULATE_GRAD) != 0;
    const int64_t most = (int64_t)set->max_rank * (m > n ? m : n);
    hipLaunchKernelGGL(adapter_reduce_kernel, dim3((unsigned)((most + 255) / 256), (unsigned)set->count, 2), dim3(256),
                       0, s, a);
  }
  return host_check_launch("adapters backward");
}

}  // namespace

extern "C" {

size_t poetx_adapter_table_bytes(int32_t count) {
  if (count < 0 || count > kMaxAdapters) {
    host_fail(POETX_ESHAPE, "count=%d out of range [0, %d]", (int)count, kMaxAdapters);
    return 0;
  }
  return (size_t)(count > 0 ? count : 1) * sizeof(AdEntry);
}

int poetx_adapter_table(const poetx_adapter* adapters, int32_t count, int64_t m, int64_t n, int32_t dtype,
                        void* host_table, size_t bytes, poetx_adapters* set) {
  int rc = check_dims(m, n, dtype);
  if (rc) return rc;
  const size_t need = poetx_adapter_table_bytes(count);
  if (need == 0) return POETX_ESHAPE;
  if ((count > 0 && !adapters) || !host_table || !set) return host_fail(POETX_EINVAL, "NULL argument");
  if (bytes < need) return host_fail(POETX_EWORKSPACE, "table has %zu bytes, needs %zu", bytes, need);
  const uintptr_t am = dtype == POETX_F32 ? 3 : 1;
  const int el = dtype == POETX_F32 ? 4 : 8;
  AdEntry* t = static_cast<AdEntry*>(host_table);
  int64_t rows = 0;
  int32_t rmax = 0;
  uint32_t layout = LAY_A16 | LAY_B16;
  for (int32_t i = 0; i < count; ++i) {
    const poetx_adapter& a = adapters[i];
    if (a.r < 1 || a.r > AD_MAX_RANK)
      return host_fail(POETX_ESHAPE, "adapter %d: rank %d out of range [1, %d]", (int)i, (int)a.r, AD_MAX_RANK);
    if (!a.A || !a.B) return host_fail(POETX_EINVAL, "adapter %d: NULL matrix", (int)i);
    if (((reinterpret_cast<uintptr_t>(a.A) | reinterpret_cast<uintptr_t>(a.B)) & am) ||
        ((reinterpret_cast<uintptr_t>(a.dA) | reinterpret_cast<uintptr_t>(a.dB)) & 3))
      return host_fail(POETX_EINVAL, "adapter %d: pointer not aligned to its type", (int)i);
    if (a.r > rmax) rmax = a.r;
    if (!al16(a.A) || n % el) layout &= ~LAY_A16;
    if (!al16(a.B) || a.r % el) layout &= ~LAY_B16;
  }
  for (int32_t i = 0; i < count; ++i) {
    const poetx_adapter& a = adapters[i];
    const int rp = pad_rank(a.r, rmax);
    t[i] = AdEntry{a.A, a.B, a.dA, a.dB, a.r, a.scale, rp, (int32_t)rows, {0, 0, 0, 0}};
    rows += rp;
  }
  *set = poetx_adapters{m, n, dtype, count, rmax, 0, layout, 0, rows, nullptr};
  return POETX_OK;
}

size_t poetx_adapters_workspace_bytes(const poetx_adapters* set, int64_t N, int32_t nseg, int op) {
  int32_t dummy = 0;
  if (check_adapters(set, false) || check_tokens(N, nseg, &dummy, &dummy)) return 0;
  if (op != POETX_OP_FORWARD && op != POETX_OP_BACKWARD) {
    host_fail(POETX_EINVAL, "op=%d", op);
    return 0;
  }
  return plan_adapters(set, N, nseg, op == POETX_OP_BACKWARD, nullptr).bytes;
}

int poetx_adapters_forward(const poetx_adapters* set, const int32_t* seg_start, const int32_t* seg_adapter,
                           int32_t nseg, const void* X, int64_t ldx, int64_t N, void* Y, int64_t ldy, void* ws,
                           size_t ws_bytes, void* stream) {
  int rc = check_adapters(set, true);
  if (rc) return rc;
  if ((rc = check_tokens(N, nseg, seg_start, seg_adapter))) return rc;
  if (N == 0 || nseg == 0 || set->count == 0) return POETX_OK;
  if ((rc = check_rows("X", X, ldx, set->n, set->dtype)) || (rc = check_rows("Y", Y, ldy, set->m, set->dtype)))
    return rc;
  const AdPlan p = plan_adapters(set, N, nseg, false, ws);
  if ((rc = host_check_ws(ws, ws_bytes, p.bytes))) return rc;
  const AdSegs seg = segs_of(set, seg_start, seg_adapter, nseg, N);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return set->dtype == POETX_F32 ? forward_impl<float>(set, seg, X, ldx, Y, ldy, p, s)
                                 : forward_impl<uint16_t>(set, seg, X, ldx, Y, ldy, p, s);
}

int poetx_adapters_backward(const poetx_adapters* set, const int32_t* seg_start, const int32_t* seg_adapter,
                            int32_t nseg, const void* X, int64_t ldx, const void* dY, int64_t lddy, int64_t N,
                            void* dX, int64_t lddx, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_adapters(set, true);
  if (rc) return rc;
  if ((rc = check_tokens(N, nseg, seg_start, seg_adapter))) return rc;
  if (set->count == 0) return POETX_OK;
  if (N == 0) nseg = 0;
  if (nseg > 0) {
    if ((rc = check_rows("X", X, ldx, set->n, set->dtype)) || (rc = check_rows("dY", dY, lddy, set->m, set->dtype)) ||
        (dX && (rc = check_rows("dX", dX, lddx, set->n, set->dtype))))
      return rc;
  }
  const AdPlan p = plan_adapters(set, nseg > 0 ? N : 0, nseg, true, ws);
  if ((rc = host_check_ws(ws, ws_bytes, p.bytes))) return rc;
  const AdSegs seg = segs_of(set, seg_start, seg_adapter, nseg, N);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return set->dtype == POETX_F32 ? backward_impl<float>(set, seg, X, ldx, dY, lddy, dX, lddx, p, s)
                                 : backward_impl<uint16_t>(set, seg, X, ldx, dY, lddy, dX, lddx, p, s);
}

}  // extern "C"

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
#include "global.h"
#include "host.h"
#include "shrink.h"

namespace poetx {

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
    const bool in = lane * step < len;
    const int s = lo + (in ? lane * step : 0);
    const int a = clamp_token(g.start[s], g.N), b = clamp_token(g.start[s + 1], g.N), ad = g.which[s];
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

// what an expand needs of a tile, written by the shrink before it
struct AdInfo {
  int32_t t0, rows;   // rows == 0: nothing to do
  const void* W;      // rows of ldw: the adapter's B, or its part of At
  int32_t ldw, pad[3];
};

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

// 16 bytes that lie within a row
template <bool VEC, bool NT>
__device__ __forceinline__ uint4 load_whole(const void* p) {
  return !VEC ? gld16_u(p) : NT ? __builtin_bit_cast(uint4, gld_nt<u32x4>(p)) : gld16(p);
}

// Elements k .. k + EL of a row of `width`, zeros past its end.  VEC: rows of
// whole 16-byte pieces, and the load is all.  Otherwise the piece may start at
// any element (global loads of 16 bytes need no alignment beyond the element's):
// load_frag loads what lies before `end`, the end of the matrix; rest_frag then
// loads the matrix's last elements one by one; cut_frag clears what lies past the
// row.  Three steps, so that all loads of a lane are on their way before one of
// them is waited for.  NT: past the caches.
template <typename E, bool VEC, bool NT = false>
__device__ __forceinline__ uint4 load_frag(const E* row, int k, int width, const E* end) {
  return k < width && (VEC || row + k + El<E>::EL <= end) ? load_whole<VEC, NT>(row + k) : make_uint4(0, 0, 0, 0);
}
template <typename E, bool VEC>
__device__ __forceinline__ void rest_frag(uint4& v, const E* row, int k, int width, const E* end) {
  constexpr int EL = El<E>::EL;
  if (VEC || k >= width || row + k + EL <= end) return;
  E e[EL];
#pragma unroll
  for (int i = 0; i < EL; ++i) e[i] = k + i < width ? gld(row + k + i) : E(0);
  v = __builtin_bit_cast(uint4, e);
}
template <typename E, bool VEC>
__device__ __forceinline__ void cut_frag(uint4& v, int left) {
  if (VEC || left >= El<E>::EL) return;
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (El<E>::EL == 8) w[q] = left >= 2 * q + 2 ? w[q] : left == 2 * q + 1 ? w[q] & 0xffffu : 0u;
    else w[q] = left > q ? w[q] : 0u;
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
}

// the three at once: what the expand's few pieces of B want (64 tokens of 64 requests,
// ranks 16 to 64, 2048 -> 5632: 20.7 us against 21.5 us in three steps; the shrink's
// chunks of the same sets 14.3 us in three steps against 15.7 us at once)
template <typename E, bool VEC>
__device__ __forceinline__ uint4 load_cut(const E* row, int k, int width, const E* end) {
  constexpr int EL = El<E>::EL;
  if (VEC) return load_frag<E, VEC>(row, k, width, end);
  uint4 v = make_uint4(0, 0, 0, 0);
  if (k >= width) return v;
  if (row + k + EL <= end) {
    v = gld16_u(row + k);
    cut_frag<E, VEC>(v, width - k);
  } else {
    rest_frag<E, VEC>(v, row, k, width, end);
  }
  return v;
}

// ---- shrink: T of each tile, fp32, as the expand's lanes hold it ("frags"):
// [step kk][half s][lane][EL], the value of rank kk KF + EL (lane / 16) + e and
// token 16 s + lane % 16 (bf16 sets of rank 16: [half][lane < 32][8]).
// A workgroup takes a tile, RT rank tiles and a part of the width, which goes
// through LDS in chunks: rows of a KiB (or half) are read whole, and each wave
// multiplies a quarter of the chunk's columns; at the end the waves' sums are
// added.  Who reads T adds the parts.  Reading the operands of the products
// straight from memory, 16 rows of 64 bytes an instruction, took 1.4 to 1.7 times
// as long (rows a power of two apart lie in the same channel of the caches, and
// all workgroups ask for the same columns at once): 8192 rows of 11008 47.8 us
// against 33.3 us, the rows read in order (without products).  Now: x and dy of
// 8192 x (4096 + 11008) 50 us, 4.9 TB/s (HBM); with few tokens the chain of segment
// search, table, chunk and sums, 7 us.
struct ShrinkJob {
  const void* X;      // [N][width], rows ldx apart
  float* T;           // [parts][tiles][rpmax * 32]
  int64_t ldx;
  int width, parts;
  int useB;           // weights: each adapter's A [rank][width] or B [width][rank]
};
struct ListArgs {     // see build_list
  int4* list;
  int2* offs;
  int cap, ordered;
};
struct TurnArgs {     // see turn_a
  void* At;
  int n, per, tw;     // per: workgroups of an adapter; tw: columns a workgroup turns
};
struct ShrinkArgs {
  ShrinkJob job[2];
  AdSegs seg;
  const AdEntry* table;
  AdInfo* info;       // of each tile, for the expand
  ListArgs lists;     // extra workgroups after the tiles': count lists, then count * turn.per transposes
  TurnArgs turn;
  int rpmax, tiles, pw, groups;   // pw: columns of a part; groups: rank groups of RT tiles
};                                // grid.x: rank groups of the parts of the jobs; grid.y, z: tiles, then the extra work

// the tiles of each adapter, one adapter after another, for the gradients:
// entry {t0, rows, adapter, tile index}; offs[a]: the first entry of adapter a, and its
// index; or (ordered) how many adapters before it have tokens
__device__ __forceinline__ int tiles_of(const AdSegs& g, int s, int& a, int& t0, int& t1) {
  t0 = clamp_token(g.start[s], g.N);
  t1 = clamp_token(g.start[s + 1], g.N);
  a = g.which[s];
  return a >= 0 && a < g.count && t1 > t0 ? (t1 - t0 + AD_T - 1) / AD_T : 0;
}

// LDS: a word a wave, and with an order a bit for each adapter
template <int THREADS>
__device__ __forceinline__ void build_list(const AdSegs& g, const ListArgs& p, int me, int* cnt) {
  constexpr int WAVES = THREADS / 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int before = 0;
  unsigned* seen = reinterpret_cast<unsigned*>(cnt + WAVES);   // those before this one that have tokens
  const int words = p.ordered ? (me + 31) / 32 : 0;
  int order = me;
  if (p.ordered) {
    for (int q = tid; q < words; q += THREADS) seen[q] = 0u;
    __syncthreads();
  }
  for (int s = tid; s < g.nseg; s += THREADS) {
    int a, t0, t1;
    const int k = tiles_of(g, s, a, t0, t1);
    if (k && a < me) {
      before += k;
      if (p.ordered) atomicOr(&seen[a >> 5], 1u << (a & 31));
    }
  }
  if (p.ordered) {
    __syncthreads();
    int n = 0;
    for (int q = tid; q < words; q += THREADS) n += __popc(seen[q]);
#pragma unroll
    for (int o = 32; o; o >>= 1) n += __shfl_xor(n, o);
    if (lane == 0) cnt[wave] = n;
    __syncthreads();
    order = 0;
    for (int q = 0; q < WAVES; ++q) order += cnt[q];
    __syncthreads();
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) before += __shfl_xor(before, o);
  if (lane == 0) cnt[wave] = before;
  __syncthreads();
  int pos = 0;
  for (int q = 0; q < WAVES; ++q) pos += cnt[q];
  __syncthreads();
  // (segments that overlap, against the contract, could fill more than the list)
  if (tid == 0) p.offs[me] = make_int2(pos < p.cap ? pos : p.cap, order);
  for (int s0 = 0; s0 < g.nseg; s0 += THREADS) {
    int a = -1, t0 = 0, t1 = 0, k = 0;
    if (s0 + tid < g.nseg) k = tiles_of(g, s0 + tid, a, t0, t1);
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
    for (int q = 0; q < WAVES; ++q) pos += cnt[q];
    __syncthreads();
    for (int i = 0; i < k; ++i) {
      const int t = t0 + i * AD_T;
      if (at + i < p.cap) p.list[at + i] = make_int4(t, t1 - t < AD_T ? t1 - t : AD_T, me, t0 / AD_T + s0 + tid + i);
    }
  }
  if (tid == 0 && me == g.count - 1) p.offs[g.count] = make_int2(pos < p.cap ? pos : p.cap, 0);
}

__device__ __forceinline__ i16x4 ds_read_tr16a(const uint16_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(i16x4, const_cast<uint16_t*>(p)));
}

// At [column][rp] of each adapter, the ranks past r zero: with it dx is an expand
// like y.  Workgroups of the shrink's launch do it beside the tiles, in whole rows of
// its grid (with one to a row, the others empty, the backward of 2001 x 2048, rank
// 64, took 42.9 us instead of 39.8 us).
template <typename E>
__device__ __forceinline__ void turn_a(const AdEntry* table, const TurnArgs& p, int b, char* lds_raw) {
  E* lds = reinterpret_cast<E*>(lds_raw);
  const AdEntry ad = table[b / p.per];
  const int tid = threadIdx.x, tw = p.tw, c0 = b % p.per * tw, cols = p.n - c0 < tw ? p.n - c0 : tw;
  const int lane = tid & (tw - 1), row = tid / tw, rows = blockDim.x / tw;
  const E* A = static_cast<const E*>(ad.A) + c0;
  // a row of LDS: one column of A, its ranks; padded so that rows of whole matrix steps begin in different banks
  const int ld = ad.r + (sizeof(E) == 2 ? 2 + (ad.r & 1) : 1);
  if (lane < cols)
#pragma unroll 4
    for (int r = row; r < ad.r; r += rows) lds[lane * ld + r] = gld(A + (int64_t)r * p.n + lane);
  __syncthreads();
  E* out = static_cast<E*>(p.At) + (int64_t)ad.row0 * p.n + (int64_t)c0 * ad.rp;
  const int total = cols * ad.rp;
  int c = tid / ad.rp, r = tid % ad.rp;
  const int dc = blockDim.x / ad.rp, dr = blockDim.x % ad.rp;
  for (int i = tid; i < total; i += blockDim.x) {
    out[i] = r < ad.r ? lds[c * ld + r] : E(0);
    c += dc;
    r += dr;
    if (r >= ad.rp) { r -= ad.rp; ++c; }
  }
}

template <typename E, int RT, bool VEC, bool NT, bool USEB>
__device__ __forceinline__ void shrink_body(const ShrinkArgs& a, const ShrinkJob& J, const AdTile& tile, int w,
                                            int group, int part, char* lds) {
  constexpr int EL = El<E>::EL, KF = El<E>::KF, ES = sizeof(E), THREADS = 64 * SHRINK_WAVES;
  constexpr int RB = shrink_rb(RT), CW = RB / ES, LD = shrink_row(RT) / ES, PR = RB / 16;   // PR: pieces of a row
  constexpr int NX = AD_T * PR / THREADS, NW = 16 * RT * PR / THREADS;                    // pieces of a thread
  constexpr int NF = CW / SHRINK_WAVES / KF;                                              // fragments of a wave
  const AdEntry ad = a.table[tile.adapter];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int rank0 = group * RT * 16;
  if (rank0 >= (RT == 1 ? ad.r : ad.rp)) {
    if (rank0 >= ad.rp) return;
    // padding alone: zeros, which the expand multiplies, for 16 ranks of 32 tokens: EL ranks
    // of 16 tokens side by side
    float* T = J.T + ((int64_t)part * a.tiles + w) * a.rpmax * AD_T;
#pragma unroll 1
    for (int i = tid; i < 16 * AD_T; i += THREADS) {
      const int rank = rank0 + i / AD_T, t = i % AD_T;
      T[((rank / KF * 2 + t / 16) * 64 + rank % KF / EL * 16 + t % 16) * EL + rank % EL] = 0.f;
    }
    return;
  }
  const int rt_n = (ad.rp - rank0) >> 4;   // rank tiles of this adapter from rank0 on
  const RankGroup group_of = rank_group(ad.r, rank0, RT, EL);
  const E* X = static_cast<const E*>(J.X) + (int64_t)tile.t0 * J.ldx;
  const E* xend = static_cast<const E*>(J.X) + (int64_t)(a.seg.N - 1) * J.ldx + J.width;
  const E* W = static_cast<const E*>(USEB ? ad.B : ad.A);
  const E* wend = W + (int64_t)ad.r * J.width;
  E* lx = reinterpret_cast<E*>(lds);
  E* lw = reinterpret_cast<E*>(lds + shrink_x(RT));
  // B: rows of the chunk, the ranks rank0 .. rank0 + rw in rc pieces, ldb elements apart
  const int rw = group_of.ranks, rc = group_of.pieces, ldb = group_of.ld;
  int brow[USEB ? NW : 1], bcol[USEB ? NW : 1];
  if constexpr (USEB) {
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int c = i * THREADS + tid;
      brow[i] = c / rc;
      bcol[i] = (c - brow[i] * rc) * EL;
    }
  }
  f32x4 acc[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint4 xr[NX], wr[NW];
  auto load = [&](int k0) {   // the chunk from column k0 on
    const bool whole = k0 + CW <= J.width;
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int c = i * THREADS + tid, row = c / PR, k = k0 + c % PR * EL;
      const E* x = X + (int64_t)(row < tile.rows ? row : 0) * J.ldx;
      xr[i] = whole ? load_whole<VEC, NT>(x + k) : load_frag<E, VEC, NT>(x, k, J.width, xend);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      if constexpr (USEB) {
        const int j = k0 + brow[i];
        wr[i] = brow[i] < CW && j < J.width ? load_frag<E, VEC>(W + (int64_t)j * ad.r + rank0, bcol[i], rw, wend)
                                            : make_uint4(0, 0, 0, 0);
      } else {
        const int c = i * THREADS + tid, rank = rank0 + c / PR, k = k0 + c % PR * EL;
        const E* r = W + (int64_t)(rank < ad.r ? rank : 0) * J.width;
        wr[i] = whole ? load_whole<VEC, false>(r + k) : load_frag<E, VEC>(r, k, J.width, wend);
      }
    }
    if (VEC) return;
    if (!whole) {
#pragma unroll
      for (int i = 0; i < NX; ++i) {
        const int c = i * THREADS + tid, row = c / PR;
        rest_frag<E, VEC>(xr[i], X + (int64_t)(row < tile.rows ? row : 0) * J.ldx, k0 + c % PR * EL, J.width, xend);
      }
    }
    if (USEB ? k0 + CW + EL > J.width : !whole) {
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        if constexpr (USEB) {
          const int j = k0 + brow[i];
          if (brow[i] < CW && j < J.width) rest_frag<E, VEC>(wr[i], W + (int64_t)j * ad.r + rank0, bcol[i], rw, wend);
        } else {
          const int c = i * THREADS + tid, rank = rank0 + c / PR;
          rest_frag<E, VEC>(wr[i], W + (int64_t)(rank < ad.r ? rank : 0) * J.width, k0 + c % PR * EL, J.width, wend);
        }
      }
    }
  };
  const int k_end = (part + 1) * a.pw < J.width ? (part + 1) * a.pw : J.width;
  int k0 = part * a.pw;
  load(k0);
  for (;;) {
    if (!VEC && k0 + CW > J.width) {   // of a piece of B past its ranks only sums that are dropped take anything
#pragma unroll
      for (int i = 0; i < NX; ++i) cut_frag<E, VEC>(xr[i], J.width - k0 - (i * THREADS + tid) % PR * EL);
#pragma unroll
      for (int i = 0; i < NW; ++i)
        if (!USEB) cut_frag<E, VEC>(wr[i], J.width - k0 - (i * THREADS + tid) % PR * EL);
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int c = i * THREADS + tid;
      *reinterpret_cast<uint4*>(lx + c / PR * LD + c % PR * EL) = xr[i];
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int c = i * THREADS + tid;
      if constexpr (USEB) {
        if (brow[i] < CW) *reinterpret_cast<uint4*>(lw + brow[i] * ldb + bcol[i]) = wr[i];
      } else {
        *reinterpret_cast<uint4*>(lw + c / PR * LD + c % PR * EL) = wr[i];
      }
    }
    __syncthreads();
    k0 += CW;
    const bool more = k0 < k_end;
    if (more) load(k0);   // on its way while this chunk is multiplied
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int kf = (wave * NF + f) * KF;   // of the chunk
      uint4 xf[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) xf[s] = *reinterpret_cast<const uint4*>(lx + (16 * s + l16) * LD + kf + g * EL);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        if (i < rt_n) {
          uint4 wf;
          if constexpr (!USEB) {
            wf = *reinterpret_cast<const uint4*>(lw + (16 * i + l16) * LD + kf + g * EL);
          } else if constexpr (ES == 2) {
            // 16 lanes read 4 rows of 16 ranks and get 4 rows of their own rank
            // (past the pieces: another's, whose sums are dropped)
            const int col = 16 * i + 4 * (l16 & 3) < ldb ? 16 * i + 4 * (l16 & 3) : 0;
            const uint16_t* src = lw + (kf + 8 * g + (l16 >> 2)) * ldb + col;
            const i16x4 p = ds_read_tr16a(src), q = ds_read_tr16a(src + 4 * ldb);
            typedef short i16x8 __attribute__((ext_vector_type(8)));
            wf = __builtin_bit_cast(uint4, i16x8{p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]});
          } else {
            const int col = 16 * i + l16 < ldb ? 16 * i + l16 : 0;
            const E* src = lw + (kf + 4 * g) * ldb + col;
            wf = make_uint4(__builtin_bit_cast(uint32_t, src[0]), __builtin_bit_cast(uint32_t, src[ldb]),
                            __builtin_bit_cast(uint32_t, src[2 * ldb]), __builtin_bit_cast(uint32_t, src[3 * ldb]));
          }
          acc[i][0] = El<E>::mma(wf, xf[0], acc[i][0]);
          acc[i][1] = El<E>::mma(wf, xf[1], acc[i][1]);
        }
      }
    }
    __syncthreads();
    if (!more) break;
  }
  float* red = reinterpret_cast<float*>(lds);
  float* T = J.T + ((int64_t)part * a.tiles + w) * a.rpmax * AD_T;
  const int lanes = a.rpmax < KF ? 16 * (a.rpmax / EL) : 64;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    if (i < rt_n) {
#pragma unroll
      for (int s = 0; s < 2; ++s) *reinterpret_cast<f32x4*>(&red[wave * 512 + s * 256 + lane * 4]) = acc[i][s];
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < SHRINK_WAVES; ++q) v += red[q * 512 + s * 256 + tid];
        const int rank = rank0 + 16 * i + 4 * (tid >> 6) + (tid & 3), c = (tid >> 2) & 15;
        v = rank < ad.r && 16 * s + c < tile.rows ? v * ad.scale : 0.f;
        const int kk = rank / KF, gg = rank % KF / EL, e = rank % EL;
        T[((kk * 2 + s) * lanes + gg * 16 + c) * EL + e] = v;
      }
      __syncthreads();
    }
  }
}

constexpr int TILES_Y = 32768;   // tiles along the grid's second dimension

template <typename E, int RT, bool VEC, bool NT>
__global__ __launch_bounds__(64 * SHRINK_WAVES) void adapter_shrink_kernel(const ShrinkArgs a) {
  __shared__ __align__(16) char lds[shrink_lds(RT, sizeof(E))];
  const int64_t w = (int64_t)blockIdx.z * TILES_Y + blockIdx.y;
  if (w >= a.tiles) {
    const int64_t x = (w - a.tiles) * gridDim.x + blockIdx.x;
    if (!a.lists.list) return;
    if (x < a.seg.count) build_list<64 * SHRINK_WAVES>(a.seg, a.lists, (int)x, reinterpret_cast<int*>(lds));
    else if (a.turn.At && x - a.seg.count < (int64_t)a.seg.count * a.turn.per)
      turn_a<E>(a.table, a.turn, (int)(x - a.seg.count), lds);
    return;
  }
  const AdTile tile = find_tile(a.seg, (int)w);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    AdInfo in{tile.t0, tile.rows, nullptr, 0, {0, 0, 0}};
    if (tile.rows) {
      const AdEntry ad = a.table[tile.adapter];
      in.W = a.turn.At ? static_cast<const E*>(a.turn.At) + (int64_t)ad.row0 * a.turn.n : static_cast<const E*>(ad.B);
      in.ldw = a.turn.At ? ad.rp : ad.r;
    }
    a.info[w] = in;
  }
  if (tile.rows == 0) return;
  int x = blockIdx.x;
  const int n0 = a.job[0].parts * a.groups;
  const ShrinkJob& J = a.job[x >= n0];
  if (x >= n0) x -= n0;
  const int part = x / a.groups, group = x % a.groups;
  if (J.useB) shrink_body<E, RT, VEC, NT, true>(a, J, tile, (int)w, group, part, lds);
  else shrink_body<E, RT, VEC, NT, false>(a, J, tile, (int)w, group, part, lds);
}

// ---- expand: Y[t][j] += sum_k T[k][t] W[j][k], W = each adapter's B, or (dx) At
struct ExpandArgs {
  void* Y;
  int64_t ldy;
  int width;
  const float* T;       // frags [parts][tiles][rpmax * 32], the parts to be added
  const AdInfo* info;
  int rpmax, tiles, parts, cols;   // cols: column groups; the grid's x past them: sums
  // (backward) sums of the parts in the order [rank][32 tokens], for the gradients
  const float* F[2];
  float* rows[2];
  int fparts[2];
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

// the lanes' 8 rows of 8 bf16 (x[i]: row i) as 8 operands of 8 rows (op[e]: column e)
__device__ __forceinline__ void transpose8(const uint4 x[8], uint4 op[8]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t d[8], lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = c == 0 ? x[i].x : c == 1 ? x[i].y : c == 2 ? x[i].z : x[i].w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __builtin_amdgcn_perm(d[2 * i + 1], d[2 * i], 0x05040100u);
      hi[i] = __builtin_amdgcn_perm(d[2 * i + 1], d[2 * i], 0x07060302u);
    }
    op[2 * c] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    op[2 * c + 1] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

// exchanges a's lanes 32..63 with b's lanes 0..31
__device__ __forceinline__ void swap32(uint4& a, uint4& b) {
  uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const auto r = __builtin_amdgcn_permlane32_swap(x[q], y[q], false, false);
    x[q] = r[0];
    y[q] = r[1];
  }
  a = make_uint4(x[0], x[1], x[2], x[3]);
  b = make_uint4(y[0], y[1], y[2], y[3]);
}

// y + v for EL elements
template <typename E>
__device__ __forceinline__ uint4 add_frag(uint4 y, const float* v) {
  const uint32_t w[4] = {y.x, y.y, y.z, y.w};
  uint32_t n[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (sizeof(E) == 2)
      n[q] = pack2(f32_to_bits(__uint_as_float(w[q] << 16) + v[2 * q]),
                   f32_to_bits(__uint_as_float(w[q] & 0xffff0000u) + v[2 * q + 1]));
    else
      n[q] = __float_as_uint(__uint_as_float(w[q]) + v[q]);
  }
  return make_uint4(n[0], n[1], n[2], n[3]);
}

// A workgroup takes one tile and four waves' columns; column groups of a tile
// follow one another in the grid.  Small workgroups in the order of the memory
// are what in-place updates of Y want: runs of four tiles a workgroup, with W kept
// in registers and the next tile's Y fetched ahead, took 48.6 us where one
// tile a workgroup takes 40.4 us, 4.6 TB/s (8192 x 5632, rank 16; 128 columns a wave,
// a workgroup's T a sixteenth of the Y it moves; with 64 columns 43.0 us, with 32 46.9 us).
// The update of Y alone, without T and W, takes 38.8 us.
// The MFMA's rows are the wave's columns, in an order that gives each lane EL
// neighbouring columns of a token, and the four lanes of a token neighbouring
// 16-byte pieces.
// MFMAs across a wave's columns, 16 columns each:
constexpr int expand_nc(int rt, bool narrow) { return narrow && rt < 16 ? 2 : rt == 1 ? 8 : 4; }

// T's operands of contraction step kk from LDS; PACK: lane groups 0, 1 hold half
// 0 of the tile's tokens, 2, 3 half 1
template <typename E, int RT>
struct Operands {
  static constexpr int EL = El<E>::EL, KF = El<E>::KF;
  static constexpr bool BF = EL == 8, PACK = BF && RT == 1;   // PACK: 16 ranks, hi and lo side by side in one MFMA
  static constexpr int NK = PACK ? 1 : RT * 16 / KF, NP = BF && !PACK ? 2 : 1;
  // element e of step kk: rank kk KF + rank0 + e
  static __device__ __forceinline__ int rank0(int g) { return PACK ? 8 * (g & 1) : g * EL; }
  static __device__ __forceinline__ void load(const float* tl, int kk, int lane, uint4 (&tf)[2][NP]) {
#pragma unroll
    for (int s = 0; s < (PACK ? 1 : 2); ++s) {
      const float* src = tl + ((kk * 2 + s) * 64 + lane) * EL;
      if constexpr (BF) {
        const f32x4 f0 = *reinterpret_cast<const f32x4*>(src), f1 = *reinterpret_cast<const f32x4*>(src + 4);
        const float f[8] = {f0[0], f0[1], f0[2], f0[3], f1[0], f1[1], f1[2], f1[3]};
        uint4 hi, lo;
        split8(f, hi, lo);
        if constexpr (PACK) {
          // lanes < 32: hi of a half, lanes >= 32: its lo
          tf[0][0] = hi;
          tf[1][0] = lo;
          swap32(tf[0][0], tf[1][0]);
        } else {
          tf[s][0] = hi;
          tf[s][NP - 1] = lo;
        }
      } else {
        tf[s][0] = *reinterpret_cast<const uint4*>(src);
      }
    }
  }
};

// a wave's columns of a tile of Y: column of MFMA c, the pieces as read ahead,
// and the update; y[s]: the lane's token of half s at its first column, `left`
// columns before the width's end
template <typename E, int NC, bool VECY>
struct Columns {
  static constexpr int EL = El<E>::EL, CP = EL / 4, NH = NC / CP;   // CP: MFMAs of a piece, NH: pieces of a lane and token
  E* y[2];
  int left, rows, l16;
  uint4 old[2][NH];
  static __device__ __forceinline__ int col(int c, int l16) {
    return (c / CP) * 4 * EL + (l16 >> 2) * EL + 4 * (c % CP) + (l16 & 3);
  }
  __device__ __forceinline__ void init(void* Y, int64_t ldy, int t0, int rows_, int jb, int width, int lane) {
    l16 = lane & 15;
    rows = rows_;
    const int j = jb + (lane >> 4) * EL;
    left = width - j;
#pragma unroll
    for (int s = 0; s < 2; ++s) y[s] = static_cast<E*>(Y) + (int64_t)(t0 + 16 * s + l16) * ldy + j;
    if (VECY) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int h = 0; h < NH; ++h)
          if (h * 4 * EL < left && 16 * s + l16 < rows) old[s][h] = gld16(y[s] + h * 4 * EL);
    }
  }
  __device__ __forceinline__ void add(const f32x4 (&acc)[NC][2]) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (16 * s + l16 >= rows) continue;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        E* o = y[s] + h * 4 * EL;
        const int n = left - h * 4 * EL;
        float v[EL];
#pragma unroll
        for (int e = 0; e < EL; ++e) v[e] = acc[h * CP + (e >> 2)][s][e & 3];
        if (VECY) {
          if (n > 0) gst16(o, add_frag<E>(old[s][h], v));
        } else if (n >= EL) {
          gst16_u(o, add_frag<E>(gld16_u(o), v));
        } else {
#pragma unroll
          for (int e = 0; e < EL; ++e)
            if (e < n) {
              if constexpr (EL == 8) o[e] = f32_to_bits(bits_to_f32(o[e]) + v[e]);
              else o[e] += v[e];
            }
        }
      }
    }
  }
};

template <typename E, int RT, bool NARROW, bool VECY, bool VECW>
__global__ __launch_bounds__(256) void adapter_expand_kernel(const ExpandArgs a) {
  using Op = Operands<E, RT>;
  constexpr int EL = El<E>::EL, KF = El<E>::KF, NK = Op::NK, NC = expand_nc(RT, NARROW);
  constexpr int KU = RT <= 4 ? NK : 1;   // contraction steps whose W is in flight together
  __shared__ __align__(16) float tl[RT * 512];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int64_t w = (int64_t)blockIdx.z * TILES_Y + blockIdx.y;
  if (w >= a.tiles) return;
  const AdInfo in = a.info[w];
  if (in.rows == 0) return;
  // T, its parts added: two floats a thread and rank tile
  const int job = (int)blockIdx.x - a.cols;   // >= 0: a sum for the gradients
  const int64_t size = (int64_t)a.rpmax * AD_T;
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  f32x2 t[RT];
  {
    const float* T = (job >= 0 ? a.F[job] : a.T) + w * size + tid * 2;
    const int parts = job >= 0 ? a.fparts[job] : a.parts;
#pragma unroll
    for (int i = 0; i < RT; ++i)
      t[i] = 16 * i < a.rpmax ? *reinterpret_cast<const f32x2*>(T + i * 512) : f32x2{0.f, 0.f};
    // four parts' loads at a time
    for (int p = 1; p < parts; p += 4) {
      f32x2 q[4][RT];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < RT; ++i)
          if (p + k < parts && 16 * i < a.rpmax)
            q[k][i] = *reinterpret_cast<const f32x2*>(T + (p + k) * a.tiles * size + i * 512);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < RT; ++i)
          if (p + k < parts) t[i] += q[k][i];
    }
  }
  if (job >= 0) {
    float* rows = a.rows[job] + w * size;
    const int lanes = Op::PACK ? 32 : 64;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = i * 512 + tid * 2 + h;
        const int e = k % EL, ln = k / EL % lanes, s = k / EL / lanes & 1, kk = k / EL / lanes >> 1;
        if (16 * i < a.rpmax) rows[(kk * KF + (ln >> 4) * EL + e) * AD_T + 16 * s + (ln & 15)] = t[i][h];
      }
    return;
  }
  const int jb = (blockIdx.x * 4 + wave) * 16 * NC;
  const int kc = Op::rank0(g);
  const E* W = static_cast<const E*>(in.W);
  const E* wend = W + (int64_t)a.width * in.ldw;
  Columns<E, NC, VECY> out;
  out.init(a.Y, a.ldy, in.t0, in.rows, jb, a.width, lane);
  uint4 wf[KU][NC];
  auto load_w = [&](int k0) {
#pragma unroll
    for (int u = 0; u < KU; ++u)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        int j = jb + out.col(c, l16);
        j = j < a.width ? j : a.width - 1;
        wf[u][c] = load_cut<E, VECW>(W + (int64_t)j * in.ldw, (k0 + u) * KF + kc, in.ldw, wend);
      }
  };
  load_w(0);
#pragma unroll
  for (int i = 0; i < RT; ++i) *reinterpret_cast<f32x2*>(&tl[i * 512 + tid * 2]) = t[i];
  __syncthreads();
  if (jb >= a.width) return;
  f32x4 acc[NC][2];
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c][0] = acc[c][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int k0 = 0; k0 < NK; k0 += KU) {
    if (k0 > 0) {
      if (k0 * KF >= in.ldw) break;
      load_w(k0);
    }
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      // steps past the adapter's ranks: W is zero, T was never written
      if (k0 + u > 0 && (k0 + u) * KF >= in.ldw) continue;
      uint4 tf[2][Op::NP];
      Op::load(tl, k0 + u, lane, tf);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int p = 0; p < Op::NP; ++p) acc[c][s] = El<E>::mma(wf[u][c], tf[s][p], acc[c][s]);
    }
  }
  out.add(acc);
}

// ---- the forward in one launch, for few tokens and ranks up to 32: every
// workgroup forms T of its tile itself (A then is read once for each 512 columns
// of Y) and adds its columns.  What the second launch costs, some 4 us, is
// more than those reads as long as they are few.
struct SmallArgs {
  const void* X;
  void* Y;
  int64_t ldx, ldy;
  int n, m, tiles;
  AdSegs seg;
  const AdEntry* table;
};
constexpr int SMALL_WAVES = 8, SMALL_COLS = SMALL_WAVES * 64;

template <typename E, int RT, bool VEC>
__global__ __launch_bounds__(64 * SMALL_WAVES) void adapter_small_kernel(const SmallArgs a) {
  using Op = Operands<E, RT>;
  constexpr int EL = El<E>::EL, KF = El<E>::KF, NK = Op::NK, NC = 4, STEP = 2 * KF, U = 4 / RT;
  __shared__ __align__(16) float red[SMALL_WAVES][RT * 512];
  __shared__ __align__(16) float tl[RT * 512];
  const int64_t w = (int64_t)blockIdx.z * TILES_Y + blockIdx.y;
  if (w >= a.tiles) return;
  const AdTile tile = find_tile(a.seg, (int)w);
  if (tile.rows == 0) return;
  const AdEntry ad = a.table[tile.adapter];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int jb = blockIdx.x * SMALL_COLS + wave * 64;
  // what the end needs, on its way while T is formed
  Columns<E, NC, VEC> out;
  out.init(a.Y, a.ldy, tile.t0, jb < a.m ? tile.rows : 0, jb, a.m, lane);
  uint4 wf[NK][NC];
  {
    const E* W = static_cast<const E*>(ad.B);
#pragma unroll
    for (int u = 0; u < NK; ++u)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        int j = jb + out.col(c, l16);
        j = j < a.m ? j : a.m - 1;
        wf[u][c] = load_frag<E, VEC>(W + (int64_t)j * ad.r, u * KF + Op::rank0(g), ad.r, W + (int64_t)a.m * ad.r);
      }
    if (!VEC && jb + 64 + EL > a.m) {
#pragma unroll
      for (int u = 0; u < NK; ++u)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          int j = jb + out.col(c, l16);
          j = j < a.m ? j : a.m - 1;
          rest_frag<E, VEC>(wf[u][c], W + (int64_t)j * ad.r, u * KF + Op::rank0(g), ad.r, W + (int64_t)a.m * ad.r);
        }
    }
  }
  const E* A = static_cast<const E*>(ad.A);
  const E* aend = A + (int64_t)ad.r * a.n;
  const E* x[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int t = 16 * s + l16;
    x[s] = static_cast<const E*>(a.X) + (int64_t)(tile.t0 + (t < tile.rows ? t : 0)) * a.ldx;
  }
  const E* xend = static_cast<const E*>(a.X) + (int64_t)(a.seg.N - 1) * a.ldx + a.n;
  const int halves = tile.rows > 16 ? 2 : 1;
  f32x4 sum[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i) sum[i][0] = sum[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * STEP; k0 < a.n; k0 += SMALL_WAVES * STEP * U) {
    uint4 xf[U][2][2], af[U][RT][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = k0 + u * SMALL_WAVES * STEP + h * KF + g * EL;
        xf[u][0][h] = load_frag<E, VEC>(x[0], k, a.n, xend);
        xf[u][1][h] = make_uint4(0, 0, 0, 0);
        if (halves == 2) xf[u][1][h] = load_frag<E, VEC>(x[1], k, a.n, xend);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const int rank = 16 * i + l16;
          af[u][i][h] = load_frag<E, VEC>(A + (int64_t)(rank < ad.r ? rank : 0) * a.n, k, a.n, aend);
        }
      }
    if (!VEC && k0 + ((U - 1) * SMALL_WAVES + 1) * STEP > a.n) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = k0 + u * SMALL_WAVES * STEP + h * KF + g * EL;
          rest_frag<E, VEC>(xf[u][0][h], x[0], k, a.n, xend);
          if (halves == 2) rest_frag<E, VEC>(xf[u][1][h], x[1], k, a.n, xend);
#pragma unroll
          for (int s = 0; s < 2; ++s) cut_frag<E, VEC>(xf[u][s][h], a.n - k);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const int rank = 16 * i + l16;
            rest_frag<E, VEC>(af[u][i][h], A + (int64_t)(rank < ad.r ? rank : 0) * a.n, k, a.n, aend);
            cut_frag<E, VEC>(af[u][i][h], a.n - k);
          }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int s = 0; s < 2; ++s) sum[i][s] = El<E>::mma(af[u][i][h], xf[u][s][h], sum[i][s]);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int s = 0; s < 2; ++s) *reinterpret_cast<f32x4*>(&red[wave][i * 512 + s * 256 + lane * 4]) = sum[i][s];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < SMALL_WAVES; ++q) v += red[q][i * 512 + tid];
    const int rank = 16 * i + 4 * ((tid >> 6) & 3) + (tid & 3), s = tid >> 8, c = (tid >> 2) & 15;
    v = rank < ad.r && 16 * s + c < tile.rows ? v * ad.scale : 0.f;
    const int kk = rank / KF, gg = rank % KF / EL, e = rank % EL, lanes = Op::PACK ? 32 : 64;
    tl[((kk * 2 + s) * lanes + gg * 16 + c) * EL + e] = v;
  }
  __syncthreads();
  f32x4 acc[NC][2];
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c][0] = acc[c][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int kk = 0; kk < NK; ++kk) {
    uint4 tf[2][Op::NP];
    Op::load(tl, kk, lane, tf);
#pragma unroll
    for (int c = 0; c < NC; ++c) cut_frag<E, VEC>(wf[kk][c], ad.r - kk * KF - Op::rank0(g));
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int p = 0; p < Op::NP; ++p) acc[c][s] = El<E>::mma(wf[kk][c], tf[s][p], acc[c][s]);
  }
  out.add(acc);
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
  const int2* offs;
  int count, rpmax, run, slabs, slabs0, groups;   // run: list entries of a workgroup; slabs0: slabs of job 0; groups of 16 ranks
  int N;
};

// A workgroup takes a slab of columns (16 lanes x EL), 16 ranks and a run of
// list entries, every fourth a wave; the waves' sums of one adapter are added
// in LDS.  (With 64 ranks a workgroup x is read once, but one wave fills a
// SIMD's registers: rank 64, 2001 tokens 27.6 us against 17.3 us.)
// Lane (g, c) loads EL neighbouring columns of its tokens; the MFMA for element
// e takes column EL c + e as its row c.  bf16: eight tokens a lane (8 g + i),
// gathered into operands of eight tokens by byte permutes; fp32: MFMA step i
// takes token 4 i + g.  Sums of an adapter within a run go to slot run + adapter
// (a run begins where the one before it ended, so no two pairs share a
// slot), counted among those with tokens where the set has more than the batch
// has segments; a second kernel adds an adapter's slots in order.  A slot is written
// and read as fp32, rank x (n + m): with a run for each wave those bytes
// outweighed the activations (the same case: 32.8 us).  8192 x (4096 + 11008), rank
// 16: 54 us, 4.5 TB/s, HBM; 2001 x 4096, rank 64: 15 us.
template <typename E, bool VEC, bool NT>
__global__ __launch_bounds__(256) void adapter_outer_kernel(const OuterArgs a) {
  constexpr int EL = El<E>::EL, COLS = 16 * EL, LD = COLS + 4;
  constexpr bool BF = EL == 8;
  __shared__ __align__(16) float red[4][16 * LD];
  // the rank groups of eight slabs follow one another, those of a slab eight
  // workgroups apart: on the same eighth of the chip, whose cache gives them x again
  const int octet = blockIdx.x / (8 * a.groups), in = blockIdx.x % (8 * a.groups);
  int bx = octet * 8 + in % 8;
  const int rank0 = in / 8 * 16;
  if (bx >= a.slabs) return;
  const int jz = bx >= a.slabs0;
  if (jz) bx -= a.slabs0;
  const OuterJob& J = a.job[jz];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int cb = bx * COLS, col = cb + l16 * EL;
  const int total = a.offs[a.count].x;
  int e0 = blockIdx.y * a.run, e1 = e0 + a.run;
  if (e1 > total) e1 = total;
  const E* xend = static_cast<const E*>(J.X) + (int64_t)(a.N - 1) * J.ldx + J.width;
  const bool whole = cb + COLS <= J.width;
  auto load = [&](uint4 (&x)[8], const int4& en) {
    const E* X = static_cast<const E*>(J.X) + (int64_t)en.x * J.ldx;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = BF ? 8 * g + i : 4 * i + g;
      // past the tile's end T is zero, but 0 x NaN is not
      const E* row = X + (int64_t)t * J.ldx;
      x[i] = make_uint4(0, 0, 0, 0);
      if (t < en.y) x[i] = whole ? load_whole<VEC, NT>(row + col) : load_frag<E, VEC, NT>(row, col, J.width, xend);
    }
    if (VEC || whole) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = BF ? 8 * g + i : 4 * i + g;
      if (t < en.y) rest_frag<E, VEC>(x[i], X + (int64_t)t * J.ldx, col, J.width, xend);
    }
  };
  while (e0 < e1) {
    const int adapter = a.list[e0].z;
    const int own = a.offs[adapter + 1].x, end = own < e1 ? own : e1;
    f32x4 acc[EL];
#pragma unroll
    for (int e = 0; e < EL; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint4 x[8], nx[8];
    int p = e0 + wave;
    int4 en = make_int4(0, 0, 0, 0);
    if (p < end) {
      en = a.list[p];
      load(x, en);
    }
    while (p < end) {
      int4 en2 = en;
      if (p + 4 < end) {
        en2 = a.list[p + 4];
        load(nx, en2);   // on its way while this tile is multiplied
      }
      const float* T = J.T + ((int64_t)en.w * a.rpmax + rank0 + l16) * AD_T;
      if constexpr (BF) {
        const f32x4 f0 = *reinterpret_cast<const f32x4*>(T + 8 * g), f1 = *reinterpret_cast<const f32x4*>(T + 8 * g + 4);
        const float f[8] = {f0[0], f0[1], f0[2], f0[3], f1[0], f1[1], f1[2], f1[3]};
        // three bf16 values keep all 24 bits of T: the gradients are fp32
        float rest[8];
        uint4 h, l, l2, none;
        split8(f, h, l);
        const bf16x8 hb = as_bf16x8(h), lb = as_bf16x8(l);
#pragma unroll
        for (int e = 0; e < 8; ++e) rest[e] = f[e] - (float)hb[e] - (float)lb[e];
        split8(rest, l2, none);
        uint4 op[8];   // operand e: column e of the lane, eight tokens
        transpose8(x, op);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          acc[e] = El<E>::mma(op[e], h, acc[e]);
          acc[e] = El<E>::mma(op[e], l, acc[e]);
          acc[e] = El<E>::mma(op[e], l2, acc[e]);
        }
      } else {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const float f = T[4 * s + g];
          acc[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[s].x), f, acc[0], 0, 0, 0);
          acc[1] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[s].y), f, acc[1], 0, 0, 0);
          acc[2] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[s].z), f, acc[2], 0, 0, 0);
          acc[3] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[s].w), f, acc[3], 0, 0, 0);
        }
      }
      p += 4;
      en = en2;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = nx[i];
    }
    // the waves' sums; element e of lane (g, rank l16), row q: column (4 g + q) EL + e
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < EL; e += 4)
        *reinterpret_cast<f32x4*>(&red[wave][l16 * LD + (4 * g + q) * EL + e]) =
            f32x4{acc[e][q], acc[e + 1][q], acc[e + 2][q], acc[e + 3][q]};
    __syncthreads();
    const int slot = blockIdx.y + a.offs[adapter].y;
    float* P = J.part + ((int64_t)slot * a.rpmax + rank0) * J.width + cb;
    const int c = tid % COLS;
#pragma unroll
    for (int r = tid / COLS; r < 16; r += 256 / COLS) {
      const float v = (red[0][r * LD + c] + red[1][r * LD + c]) + (red[2][r * LD + c] + red[3][r * LD + c]);
      if (cb + c < J.width) P[(int64_t)r * J.width + c] = v;
    }
    __syncthreads();
    e0 = end;
  }
}

struct ReduceArgs {
  const float* part[2];
  const int2* offs;
  const AdEntry* table;
  int width[2];          // n (dA), m (dB)
  int rpmax, run, accumulate;
};

// dA [r][n] and dB [m][r] of every adapter; zero where it had no token.  A
// workgroup takes 64 columns and 16 ranks; dB turns through LDS.  The slots come out
// of the caches: 4 to 5 us, the launch for the most part.
__global__ __launch_bounds__(256) void adapter_reduce_kernel(const ReduceArgs a) {
  __shared__ float turn[64][17];
  const int ad = blockIdx.y, job = blockIdx.z & 1, rank0 = (blockIdx.z >> 1) * 16, width = a.width[job];
  const AdEntry e = a.table[ad];
  float* out = job ? e.dB : e.dA;
  const int col = blockIdx.x * 64 + (threadIdx.x & 63);
  if (!out || rank0 >= e.r || (int)blockIdx.x * 64 >= width) return;
  const int o0 = a.offs[ad].x, o1 = a.offs[ad + 1].x;
  const int q0 = o0 / a.run, q1 = o1 > o0 ? (o1 - 1) / a.run : q0 - 1;
  const int64_t stride = (int64_t)a.rpmax * width;
  const int rank = rank0 + (threadIdx.x >> 6) * 4;   // four ranks a thread
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (col < width) {
    const float* p = a.part[job] + (q0 + a.offs[ad].y) * stride + (int64_t)rank * width + col;
#pragma unroll 4
    for (int q = q0; q <= q1; ++q, p += stride)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += p[i * width];   // (ranks past r: padding of the slot)
  }
  if (job == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (rank + i < e.r && col < width) {
        float* dst = out + (int64_t)(rank + i) * width + col;
        gst(dst, a.accumulate ? gld(dst) + v[i] : v[i]);
      }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) turn[threadIdx.x & 63][rank - rank0 + i] = v[i];
  __syncthreads();
  const int ranks = e.r - rank0 < 16 ? e.r - rank0 : 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = threadIdx.x + 256 * i, c = k >> 4, rr = k & 15;
    const int j = blockIdx.x * 64 + c;
    if (rr < ranks && j < width) {
      float* dst = out + (int64_t)j * e.r + rank0 + rr;
      gst(dst, a.accumulate ? gld(dst) + turn[c][rr] : turn[c][rr]);
    }
  }
}

__global__ __launch_bounds__(256) void adapter_list_kernel(const AdSegs seg, const ListArgs lists) {
  __shared__ int cnt[4];
  build_list<256>(seg, lists, blockIdx.x, cnt);
}

}  // namespace poetx

using namespace poetx;

namespace {

constexpr int64_t kMaxAdapterDim = 32768;
constexpr int kMaxAdapters = 65535, kMaxSegs = 1 << 20;
enum { LAY_A16 = 1, LAY_B16 = 2 };   // poetx_adapters.layout

// ranks in whole MFMA steps: 16, or multiples of 32 for all adapters of a set with a rank over 16
int pad_rank(int r, int rmax) { return rmax <= 16 ? 16 : (r + 31) / 32 * 32; }
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
  int rpmax, run, runs, slots, slabs[2];
  int rt, rgroups, pw;     // shrink: rank tiles of a workgroup, their groups, columns of a part
  int parts[2];            // of x and of dy
  float *F[2], *T, *U, *part[2];   // frags of T and U, their sums in rows, the gradients' partial sums
  void* At;
  AdInfo* info;
  int4* list;
  int2* offs;
  int ordered;         // see ListArgs
  size_t bytes;
};

int ceil_rt(int t) { return t <= 1 ? 1 : t <= 2 ? 2 : t <= 4 ? 4 : t <= 8 ? 8 : 16; }

AdPlan plan_adapters(const poetx_adapters* s, int64_t N, int32_t nseg, bool bwd, void* ws) {
  AdPlan p{};
  const bool f32 = s->dtype == POETX_F32;
  p.tiles = N / AD_T + nseg;
  p.rpmax = pad_rank(s->max_rank, s->max_rank);
  // the shrink's parts: 1024 columns; with very many workgroups 2048, with few
  // 512; where these are too few still, the ranks are shared out as well
  // (x is then read again).  Measured with parts of 512, 1024, 1536, 2048, 2560
  // columns, before later steps: 4099 x 5632 (rank 32) 33.2, 28.8, 27.4, 34.2, 34.9 us,
  // 8192 x 2048 -> 5632 58.8, 55.4, 58.0, 57.6, 57.8 us, backward of 2001 x 2048 (rank 64)
  // 49.2, 45.5, 50.3, 50.0, 49.7 us, of 8192 x 4096 -> 11008 170, 154, 151, 153, 152 us.
  const int rt_all = p.rpmax / 16;
  p.rt = rt_all < 4 ? ceil_rt(rt_all) : 4;
  auto groups = [&](int rt) { return (rt_all + rt - 1) / rt; };
  const int64_t parts1k = p.tiles * (s->n + (bwd ? s->m : 0)) / 1024;
  p.pw = parts1k > 2048 ? 2048 : parts1k < 128 ? 512 : 1024;
  p.parts[0] = (int)((s->n + p.pw - 1) / p.pw);
  p.parts[1] = bwd ? (int)((s->m + p.pw - 1) / p.pw) : 0;
  while (p.rt > 1 && p.tiles * groups(p.rt) * (p.parts[0] + p.parts[1]) < 512) p.rt /= 2;
  p.rgroups = groups(p.rt);
  size_t off = 0;
  auto take = [&](size_t bytes) -> char* {
    off = (off + kWsAlign - 1) / kWsAlign * kWsAlign;
    char* q = ws ? static_cast<char*>(ws) + off : nullptr;
    off += bytes;
    return q;
  };
  const size_t tbytes = (size_t)p.tiles * p.rpmax * AD_T * sizeof(float);
  p.info = reinterpret_cast<AdInfo*>(take((size_t)p.tiles * sizeof(AdInfo)));
  p.F[0] = reinterpret_cast<float*>(take(p.parts[0] * tbytes));
  if (bwd) {
    p.F[1] = reinterpret_cast<float*>(take(p.parts[1] * tbytes));
    p.T = reinterpret_cast<float*>(take(tbytes));
    p.U = reinterpret_cast<float*>(take(tbytes));
    p.At = take((size_t)s->rows * s->n * (f32 ? 4 : 2));
    p.list = reinterpret_cast<int4*>(take((size_t)p.tiles * sizeof(int4)));
    p.offs = reinterpret_cast<int2*>(take((size_t)(s->count + 1) * sizeof(int2)));
    p.ordered = s->count > nseg;
    // runs of tiles: about 512 workgroups over both gradients
    const int64_t cols = f32 ? 64 : 128;
    p.slabs[0] = (int)((s->n + cols - 1) / cols);
    p.slabs[1] = (int)((s->m + cols - 1) / cols);
    const int64_t run = p.tiles * (p.slabs[0] + p.slabs[1]) * rt_all / 512;
    p.run = (int)(run < 1 ? 1 : run);
    p.runs = (int)((p.tiles + p.run - 1) / p.run);
    p.slots = p.runs + (s->count < nseg ? s->count : nseg);
    p.part[0] = reinterpret_cast<float*>(take((size_t)p.slots * p.rpmax * s->n * sizeof(float)));
    p.part[1] = reinterpret_cast<float*>(take((size_t)p.slots * p.rpmax * s->m * sizeof(float)));
  }
  p.bytes = off + kWsAlign;
  return p;
}

// Activations of this many bytes are read past the caches: they would not
// survive beside the rest in the 256 MiB that the memory side holds.  Measured:
// 8192 x 2048 -> 5632 (126 MB) 53.2 us instead of 55.4, backward of 8192 x 4096 ->
// 11008 (314 MB) 139.5 us instead of 152.6; 4099 x 5632 -> 2048 (63 MB) 30.4 us instead of 28.8,
// backward of 2001 x 2048 (25 MB) 52.8 us instead of 50.0.
constexpr int64_t STREAM_BYTES = 96ll << 20;
bool streams(const poetx_adapters* s, int64_t N) {
  return N * (s->n + s->m) * (s->dtype == POETX_F32 ? 4 : 2) > STREAM_BYTES;
}

// x workgroups of each of `count` tiles (or more)
dim3 tile_grid(int64_t x, int64_t count) {
  return dim3((unsigned)x, (unsigned)(count < TILES_Y ? count : TILES_Y), (unsigned)((count + TILES_Y - 1) / TILES_Y));
}

AdSegs segs_of(const poetx_adapters* s, const int32_t* start, const int32_t* which, int32_t nseg, int64_t N) {
  return AdSegs{start, which, nseg, s->count, (int32_t)N};
}

template <typename E>
void launch_shrink(ShrinkArgs a, const AdPlan& p, int64_t extra, bool vec, bool nt, hipStream_t s) {
  a.rpmax = p.rpmax;
  a.tiles = (int)p.tiles;
  a.info = p.info;
  a.pw = p.pw;
  a.groups = p.rgroups;
  const int64_t x = (p.parts[0] + p.parts[1]) * p.rgroups;
  const dim3 grid = tile_grid(x, p.tiles + (extra + x - 1) / x);
  const dim3 block(64 * SHRINK_WAVES);
#define POETX_RT(R) \
  case R: \
    if (vec && nt) hipLaunchKernelGGL((adapter_shrink_kernel<E, R, true, true>), grid, block, 0, s, a); \
    else if (vec) hipLaunchKernelGGL((adapter_shrink_kernel<E, R, true, false>), grid, block, 0, s, a); \
    else hipLaunchKernelGGL((adapter_shrink_kernel<E, R, false, false>), grid, block, 0, s, a); \
    break;
  switch (p.rt) { POETX_RT(1) POETX_RT(2) POETX_RT(4) }
#undef POETX_RT
}

// A wave of the expand takes 64 columns, with rank 16 128; where the tiles times the width
// are at most this, 32: more workgroups, each sooner done.  Measured, 32 against 64 (128)
// columns: rank 16, 1024 x 2048 11.1 us against 11.9 us, 2048 x 2048 14.7, 15.7, fp32 backward
// of 333 x 600 20.6, 22.9; rank 32, 4099 x 2048 26.9, 28.3; rank 64, 4096 x 2048 24.1, 24.9; rank
// 128, 2048 x 2048 22.4, 24.8.  Above: rank 32, 8192 x 5632 64.1 us against 57.8 us, rank 64 85.3,
// 81.1, rank 128 121, 111.  Above rank 128 always 64 (rank 256, 2048 x 4096: 64.3 us with 32, 54.7 us with 64).
constexpr int64_t NARROW_WORK = 400 << 10;

template <typename E, int RT, bool NARROW>
void expand(const ExpandArgs& a, dim3 grid, bool vecy, bool vecw, hipStream_t s) {
  if (vecy && vecw) hipLaunchKernelGGL((adapter_expand_kernel<E, RT, NARROW, true, true>), grid, dim3(256), 0, s, a);
  else if (vecy) hipLaunchKernelGGL((adapter_expand_kernel<E, RT, NARROW, true, false>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((adapter_expand_kernel<E, RT, NARROW, false, false>), grid, dim3(256), 0, s, a);
}
template <typename E>
void launch_expand(ExpandArgs a, const AdPlan& p, bool vecw, hipStream_t s) {
  const size_t es = sizeof(E);
  const bool vecy = al16(a.Y) && a.ldy * es % 16 == 0 && a.width * es % 16 == 0;
  a.info = p.info;
  a.rpmax = p.rpmax;
  a.tiles = (int)p.tiles;
  const int rt = ceil_rt(p.rpmax / 16);
  const bool narrow = p.tiles * a.width <= NARROW_WORK;
  const int wide = 64 * expand_nc(rt, narrow);
  a.cols = a.Y ? (a.width + wide - 1) / wide : 0;
  const dim3 grid = tile_grid(a.cols + (a.rows[0] ? 2 : 0), p.tiles);
#define POETX_RT(R) \
  case R: \
    if (narrow && R < 16) expand<E, R, R < 16>(a, grid, vecy, vecw, s); \
    else expand<E, R, false>(a, grid, vecy, vecw, s); \
    break;
  switch (rt) { POETX_RT(1) POETX_RT(2) POETX_RT(4) POETX_RT(8) POETX_RT(16) }
#undef POETX_RT
}

// Whether the forward goes in one launch: each workgroup then reads its
// tile of x and all of A, so these have to be small, and the workgroups few.
// Measured with m, n in {2048, 5632, 4096, 11008, 520, 600}, ranks 8 to 32, 1 to 2048 tokens:
// where the rule holds one launch takes 8.5 to 12.3 us against 11 to 14.2 us,
// just outside it 12 to 15 us against 11 us.
bool small_forward(const poetx_adapters* set, const AdPlan& p, int64_t N, int32_t nseg) {
  if (p.rpmax > 32) return false;
  const int64_t tokens = (N + nseg - 1) / nseg < AD_T ? (N + nseg - 1) / nseg : AD_T;   // of a tile, on average
  const int64_t reads = (p.rpmax + tokens) * set->n * (set->dtype == POETX_F32 ? 4 : 2);
  const int64_t groups = p.tiles * ((set->m + SMALL_COLS - 1) / SMALL_COLS);
  return reads <= 200 * 1024 && (groups <= 304 || groups * reads <= 16 << 20);
}

template <typename E>
void launch_small(const poetx_adapters* set, const AdSegs& seg, const void* X, int64_t ldx, void* Y, int64_t ldy,
                  const AdPlan& p, hipStream_t s) {
  const size_t es = sizeof(E);
  SmallArgs a{X, Y, ldx, ldy, (int)set->n, (int)set->m, (int)p.tiles, seg, static_cast<const AdEntry*>(set->table)};
  const bool vec = al16(X) && ldx * es % 16 == 0 && set->n * es % 16 == 0 && al16(Y) && ldy * es % 16 == 0 &&
                   set->m * es % 16 == 0 && set->layout == (LAY_A16 | LAY_B16);
  const dim3 grid = tile_grid((set->m + SMALL_COLS - 1) / SMALL_COLS, p.tiles), block(64 * SMALL_WAVES);
  if (p.rpmax == 16) {
    if (vec) hipLaunchKernelGGL((adapter_small_kernel<E, 1, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((adapter_small_kernel<E, 1, false>), grid, block, 0, s, a);
  } else {
    if (vec) hipLaunchKernelGGL((adapter_small_kernel<E, 2, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((adapter_small_kernel<E, 2, false>), grid, block, 0, s, a);
  }
}

template <typename E>
int forward_impl(const poetx_adapters* set, const AdSegs& seg, const void* X, int64_t ldx, void* Y, int64_t ldy,
                 const AdPlan& p, hipStream_t s) {
  const size_t es = sizeof(E);
  const AdEntry* table = static_cast<const AdEntry*>(set->table);
  const double flops = 2.0 * seg.N * set->max_rank;
  if (small_forward(set, p, seg.N, seg.nseg)) {
    HostTimer tm(s, "adapter_small", flops * (set->m + set->n), (double)seg.N * (set->n + 2 * set->m) * es);
    launch_small<E>(set, seg, X, ldx, Y, ldy, p, s);
    return host_check_launch("adapters forward");
  }
  {
    HostTimer tm(s, "adapter_shrink", flops * set->n, (double)seg.N * set->n * es);
    ShrinkArgs a{};
    a.job[0] = ShrinkJob{X, p.F[0], ldx, (int)set->n, p.parts[0], 0};
    a.seg = seg;
    a.table = table;
    const bool vec = al16(X) && ldx * es % 16 == 0 && set->n * es % 16 == 0 && (set->layout & LAY_A16);
    launch_shrink<E>(a, p, 0, vec, streams(set, seg.N), s);
  }
  {
    HostTimer tm(s, "adapter_expand", flops * set->m, 2.0 * seg.N * set->m * es);
    ExpandArgs a{};
    a.Y = Y; a.ldy = ldy; a.width = (int)set->m; a.T = p.F[0]; a.parts = p.parts[0];
    launch_expand<E>(a, p, (set->layout & LAY_B16) != 0, s);
  }
  return host_check_launch("adapters forward");
}

template <typename E>
int backward_impl(const poetx_adapters* set, const AdSegs& seg, const void* X, int64_t ldx, const void* dY,
                  int64_t lddy, void* dX, int64_t lddx, const AdPlan& p, hipStream_t s) {
  const size_t es = sizeof(E);
  const int m = (int)set->m, n = (int)set->n;
  const AdEntry* table = static_cast<const AdEntry*>(set->table);
  const double flops = 2.0 * seg.N * set->max_rank;
  const bool xvec = al16(X) && ldx * es % 16 == 0 && n * es % 16 == 0;
  const bool yvec = al16(dY) && lddy * es % 16 == 0 && m * es % 16 == 0;
  const bool nt = streams(set, seg.N);
  const ListArgs lists{p.list, p.offs, (int)p.tiles, p.ordered && p.tiles > 0};
  if (p.tiles == 0) {
    hipLaunchKernelGGL(adapter_list_kernel, dim3((unsigned)set->count), dim3(256), 0, s, seg, lists);
  } else {
    {
      HostTimer tm(s, "adapter_shrink", flops * (m + n), (double)seg.N * (m + n) * es);
      ShrinkArgs a{};
      a.job[0] = ShrinkJob{X, p.F[0], ldx, n, p.parts[0], 0};
      a.job[1] = ShrinkJob{dY, p.F[1], lddy, m, p.parts[1], 1};
      a.seg = seg;
      a.table = table;
      a.lists = lists;
      // columns of A turned by a workgroup: a power of two whose ranks fit the LDS
      int tw = 64;
      while (tw > 8 && (size_t)tw * (set->max_rank + 3) * es > TURN_LDS) tw /= 2;
      a.turn = TurnArgs{dX ? p.At : nullptr, n, (n + tw - 1) / tw, tw};
      launch_shrink<E>(a, p, (int64_t)set->count * (1 + (dX ? a.turn.per : 0)), xvec && yvec && set->layout == (LAY_A16 | LAY_B16),
                       nt, s);
    }
    {
      HostTimer tm(s, "adapter_expand", flops * n, 2.0 * seg.N * n * es);
      ExpandArgs a{};
      a.Y = dX; a.ldy = lddx; a.width = n; a.T = p.F[1]; a.parts = p.parts[1];
      a.F[0] = p.F[0]; a.F[1] = p.F[1]; a.rows[0] = p.T; a.rows[1] = p.U;
      a.fparts[0] = p.parts[0]; a.fparts[1] = p.parts[1];
      launch_expand<E>(a, p, true, s);
    }
    {
      HostTimer tm(s, "adapter_outer", 2 * flops * (m + n), (double)seg.N * (m + n) * es);
      OuterArgs a{};
      a.job[0] = OuterJob{X, p.U, p.part[0], ldx, n};
      a.job[1] = OuterJob{dY, p.T, p.part[1], lddy, m};
      a.list = p.list; a.offs = p.offs; a.count = set->count; a.rpmax = p.rpmax; a.run = p.run; a.slabs0 = p.slabs[0];
      a.slabs = p.slabs[0] + p.slabs[1]; a.groups = p.rpmax / 16;
      a.N = seg.N;
      const dim3 grid((unsigned)((a.slabs + 7) / 8 * 8 * a.groups), (unsigned)p.runs);
      if (xvec && yvec && nt) hipLaunchKernelGGL((adapter_outer_kernel<E, true, true>), grid, dim3(256), 0, s, a);
      else if (xvec && yvec) hipLaunchKernelGGL((adapter_outer_kernel<E, true, false>), grid, dim3(256), 0, s, a);
      else hipLaunchKernelGGL((adapter_outer_kernel<E, false, false>), grid, dim3(256), 0, s, a);
    }
  }
  {
    HostTimer tm(s, "adapter_reduce", 0.0, 0.0);
    ReduceArgs a{};
    a.part[0] = p.part[0]; a.part[1] = p.part[1];
    a.offs = p.offs; a.table = table; a.width[0] = n; a.width[1] = m; a.rpmax = p.rpmax; a.run = p.run;
    a.accumulate = (set->flags & POETX_ACCUMULATE_GRAD) != 0;
    hipLaunchKernelGGL(adapter_reduce_kernel, dim3((unsigned)(((m > n ? m : n) + 63) / 64), (unsigned)set->count,
                                                   (unsigned)(2 * ((set->max_rank + 15) / 16))), dim3(256), 0, s, a);
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

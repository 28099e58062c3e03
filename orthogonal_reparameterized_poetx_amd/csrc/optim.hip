// Optimizer steps over many tensors with one launch: the global gradient norm
// with its clipping coefficient, and AdamW (Loshchilov & Hutter 2019) with
// 32-bit or 8-bit moments.  See include/poetx.h for formats and formulas.
//
// Both are streaming passes: per value the step reads p, g, m, v and writes
// p, m, v, 28 bytes with fp32 everywhere and 16 with 8-bit moments.  HBM bounds
// the norm and the step with fp32 moments (15 M values: vector units busy 19 % of
// the time); with 8-bit moments 105 vector instructions a value, most of them to
// decode and encode, keep the vector units busy all the time, and they bound it
// as well (fp32 tensors 6.0 TB/s; bf16 ones, 10 bytes a value, 4.0).  A table made once on the
// host maps workgroups to tensors: chunk c of the grid is a few state blocks of
// one tensor, and its record holds all that a workgroup needs of it, so that
// one scalar load comes before the data.
#include <cmath>
#include <cstring>

#include "../../include/poetx.h"
#include "global.h"
#include "grid.h"
#include "host.h"

namespace poetx {

constexpr int OPT_BLOCK = 256;     // values that share an exponent byte: one wave, four values a lane
constexpr int OPT_WAVES = 4;
constexpr int CHUNK_BLOCKS = OPT_WAVES;
constexpr int64_t OPT_FEW = 16 * 1024;   // blocks of a small set

struct OptChunk {
  void* p;           // at the chunk's first value
  const void* g;
  uint16_t* copy;
  int64_t block;     // its first state block
  float lr_mul, decay;
  int32_t left;      // values from here to the tensor's end, at most a chunk's
  int32_t flags;
};
enum { OPT_PBF = 1, OPT_GBF = 2, OPT_VEC = 4 };   // bf16 parameter, gradient; every pointer 16-byte aligned
struct OptHead {     // start of the table; the chunks follow
  uint32_t arrived;  // workgroups of a running norm that have stored their sum
  uint32_t pad[63];
};

// ---- the dither: fractional parts of pos alpha + step beta, alpha and beta
// the powers of the reciprocal plastic number (Roberts 2018), times 2^32.
// Over steps at one position, and over positions at one step, it fills [0, 1)
// evenly.  m takes bits 31..12, v bits 24..5 (the same sequence times 2^7, an
// irrational of its own), a bf16 parameter bits 31..16.
constexpr uint32_t kAlphaPos = 0xC13FA9A9u, kAlphaStep = 0x91E10DA5u;

template <bool SIGNED>
struct Code {
  static constexpr int LOW = SIGNED ? 15 : 31;        // exponent fields
  static constexpr int FIX = SIGNED ? 271 : 287;      // 127 + 127 + distance of the lowest step from E
};

// E of a block: the exponent of its largest magnitude after rounding up by
// the largest dither, so that no code overflows
__device__ __forceinline__ int block_exp(uint32_t maxbits) {
  if (maxbits >= 0x7f800000u) return 255;
  const int e = (int)((maxbits + 0xFFFFFu) >> 23);
  return e < 40 ? 40 : e > 254 ? 254 : e;
}

template <bool SIGNED>
__device__ __forceinline__ uint32_t encode8(float x, uint32_t u, int E) {
  const uint32_t bits = __float_as_uint(x) & 0x7fffffffu;
  // normal: add the dither below the third fraction bit and cut it off
  const int normal = (int)((bits + u) >> 20) - ((E - Code<SIGNED>::LOW) << 3);
  // below the lowest octave: steps of a fixed size
  const float unit = __uint_as_float((uint32_t)(Code<SIGNED>::FIX - E) << 23);
  const int tiny = (int)floorf(__fadd_rn(__fmul_rn(__uint_as_float(bits), unit), (float)u * 0x1p-20f));
  int c = (int)(bits >> 23) - E + Code<SIGNED>::LOW >= 1 ? normal : tiny;
  if (SIGNED) {
    c = c > 127 ? 127 : c;
    return (uint32_t)c | (x < 0.f ? 128u : 0u);
  }
  c = c > 255 ? 255 : c < 1 ? 1 : c;
  return bits ? (uint32_t)c : 0u;
}

template <bool SIGNED>
__device__ __forceinline__ float decode8(uint32_t c, int E) {
  const uint32_t e = (c >> 3) & Code<SIGNED>::LOW, f = c & 7u;
  const float tiny = (float)f * __uint_as_float((uint32_t)(E - Code<SIGNED>::LOW - 2) << 23);
  const float normal = __uint_as_float(((uint32_t)(E - Code<SIGNED>::LOW) + e) << 23 | f << 20);
  float v = e ? normal : tiny;
  if (SIGNED) v = __uint_as_float(__float_as_uint(v) | (c & 128u) << 24);
  return v;
}
// a stored exponent byte as it is read: at least 40; 255 makes the block NaN
__device__ __forceinline__ int exp_of(int byte) { return byte < 40 ? 40 : byte; }

// largest of x over the wave, in every lane
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#define POETX_DPP_MAX(ctrl, rows) \
  { const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, rows, 0xf, false); x = x > y ? x : y; }
  POETX_DPP_MAX(0x111, 0xf)   // row_shr 1, 2, 4, 8: lane 15 of each row of 16 holds the row's
  POETX_DPP_MAX(0x112, 0xf)
  POETX_DPP_MAX(0x114, 0xf)
  POETX_DPP_MAX(0x118, 0xf)
  POETX_DPP_MAX(0x142, 0xa)   // row 0 into 1, 2 into 3
  POETX_DPP_MAX(0x143, 0xc)   // rows 0, 1 into 2, 3
#undef POETX_DPP_MAX
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

struct F4 { float x[4]; };

// four values from `at` on; those at or past `left` read as zero.  Values and
// fp32 moments go past the caches (nontemporal), nothing of them is met again
// before the next step; 8-bit codes and their exponents go through
__device__ __forceinline__ F4 load4(const void* base, int64_t at, int left, bool bf, bool vec) {
  F4 r;
  if (vec && left >= 4) {
    if (bf) {
      const u32x2 w = gld_nt<u32x2>(static_cast<const uint16_t*>(base) + at);
      r.x[0] = __uint_as_float(w.x << 16); r.x[1] = __uint_as_float(w.x & 0xffff0000u);
      r.x[2] = __uint_as_float(w.y << 16); r.x[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      const f32x4 w = gld_nt<f32x4>(static_cast<const float*>(base) + at);
      r.x[0] = w[0]; r.x[1] = w[1]; r.x[2] = w[2]; r.x[3] = w[3];
    }
    return r;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    r.x[j] = j >= left ? 0.f : bf ? bits_to_f32(gld(static_cast<const uint16_t*>(base) + at + j))
                                  : gld(static_cast<const float*>(base) + at + j);
  return r;
}

__device__ __forceinline__ void store4_bf16(uint16_t* base, int64_t at, int left, bool vec, const uint16_t h[4]) {
  if (vec && left >= 4) {
    gst_nt(base + at, u32x2{pack2(h[0], h[1]), pack2(h[2], h[3])});
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < left) gst(base + at + j, h[j]);
}

struct StepArgs {
  const OptChunk* chunks;
  const float* coef;
  void *m, *v;
  uint8_t *me, *ve;
  const uint32_t* before;   // steps skipped before this one, see below; or NULL
  uint32_t* after;          // and after it
  int64_t step;
  float lr, b1, b2, ob1, ob2, eps, ibc1, ibc2;
};

// 1 / (1 - b^n), n >= 1
__device__ __forceinline__ float bias_of(float b, uint64_t n) {
  double p = 1.0, f = b;
  for (; n; n >>= 1, f *= f)
    if (n & 1) p *= f;
  return (float)(1.0 / (1.0 - p));
}

// A workgroup takes a chunk, each wave one block: small workgroups in the order
// of the memory.  With four blocks a wave, all loads ahead, 135.6 M values with
// 8-bit moments took 431 us, with two 418 us, with one 404 us; past the caches and
// with the hardware's reciprocal and root (one ulp each, on an update that is
// some 1e-3 of p) 353 us, 6.1 TB/s of the 16 bytes a value (345 to 370 us on other
// cards, calls back to back; one at a time under a profiler 380 us).
// A step whose coefficient is not finite writes nothing, and those after it
// take its number: step s reads the count of such steps from skipped[s % 2], and its
// first workgroup leaves the next step's in the other word, which no workgroup
// of this launch reads.  The host's bias corrections hold for a count of zero;
// with another they are formed here.
// The moments are formed with separate roundings (no contraction): the codes
// of the 8-bit state then follow from the formula alone.
// DEEP: for an eps that does not swallow the roots of subnormal values, which the
// hardware's root takes for zero.  They are below 2^-63: an eps from 2^-38 on is
// the same with and without them.  (Chosen in the kernel, it cost every call: 135.6 M
// values with 8-bit moments 383 us against 367 us.)
constexpr float DEEP_EPS = 0x1p-38f;

template <bool Q8, bool DEEP>
__global__ __launch_bounds__(256) void adamw_kernel(const StepArgs a) {
#pragma clang fp contract(off)
  const OptChunk ch = a.chunks[blockIdx.x];
  const float coef = a.coef ? *a.coef : 1.f;
  const bool finite = fabsf(coef) < INFINITY;
  const uint32_t skipped = a.before ? *a.before : 0u;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int at = wave * OPT_BLOCK + lane * 4;
  const bool in = wave * OPT_BLOCK < ch.left;   // (a wave without a block reads the chunk's first)
  const float lr = a.lr * ch.lr_mul;
  const bool pbf = ch.flags & OPT_PBF, gbf = ch.flags & OPT_GBF, vec = ch.flags & OPT_VEC;
  const int l = ch.left - at, left = l < 0 ? 0 : l > 4 ? 4 : l;   // values of the tensor from this lane's first on
  const int64_t sb = ch.block + (in ? wave : 0), s = sb * OPT_BLOCK + lane * 4;
  // every load before the first use of one
  F4 p = load4(ch.p, at, left, pbf, vec);
  const F4 g = load4(ch.g, at, left, gbf, vec);
  F4 m, v;
  uint32_t mc, vc;
  int em, ev;
  if (Q8) {
    em = a.me[sb];
    ev = a.ve[sb];
    mc = gld(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.m) + s));
    vc = gld(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.v) + s));
  } else {
    const f32x4 x = gld_nt<f32x4>(static_cast<const float*>(a.m) + s);
    const f32x4 y = gld_nt<f32x4>(static_cast<const float*>(a.v) + s);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m.x[j] = x[j];
      v.x[j] = y[j];
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.after) *a.after = skipped + (finite ? 0u : 1u);
  if (!in || !finite) return;
  float ibc1 = a.ibc1, ibc2 = a.ibc2;
  if (__builtin_expect(skipped != 0, 0)) {
    const uint64_t n = a.step > skipped ? (uint64_t)(a.step - skipped) : 1;   // (1: the counts are not of these steps)
    ibc1 = bias_of(a.b1, n);
    ibc2 = bias_of(a.b2, n);
  }
  if (Q8) {
    em = exp_of(em);
    ev = exp_of(ev);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m.x[j] = em == 255 ? NAN : decode8<true>(mc >> (8 * j) & 255u, em);
      v.x[j] = ev == 255 ? NAN : decode8<false>(vc >> (8 * j) & 255u, ev);
    }
  }
  const uint32_t h0 = (uint32_t)s * kAlphaPos + ((uint32_t)a.step - skipped) * kAlphaStep;
  uint16_t pb[4], cb[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float gj = g.x[j] * coef;
    float mj = m.x[j] * a.b1 + gj * a.ob1;
    float vj = v.x[j] * a.b2 + gj * gj * a.ob2;
    if (j >= left) mj = vj = 0.f;   // padding
    m.x[j] = mj;
    v.x[j] = vj;
    const float vh = vj * ibc2;
    float root = __builtin_amdgcn_sqrtf(vh);
    if (DEEP) root = vh < 0x1p-126f ? __builtin_amdgcn_sqrtf(vh * 0x1p64f) * 0x1p-32f : root;
    const float up = (mj * ibc1) * __builtin_amdgcn_rcpf(root + a.eps);
    const float q = p.x[j] - lr * (ch.decay * p.x[j] + up);
    p.x[j] = q;
    // the carry of the dither must not turn infinity or NaN into another value
    const uint32_t qb = __float_as_uint(q);
    const uint32_t d = (h0 + (uint32_t)j * kAlphaPos) >> 16;
    pb[j] = (uint16_t)((qb & 0x7f800000u) == 0x7f800000u ? f32_to_bits(q) : (qb + d) >> 16);
    cb[j] = f32_to_bits(q);
  }
  if (pbf) {
    store4_bf16(static_cast<uint16_t*>(ch.p), at, left, vec, pb);
  } else {
    float* dst = static_cast<float*>(ch.p) + at;
    if (vec && left == 4) {
      gst_nt(dst, f32x4{p.x[0], p.x[1], p.x[2], p.x[3]});
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) gst(dst + j, p.x[j]);
    }
    if (ch.copy) store4_bf16(ch.copy, at, left, vec, cb);
  }
  if (Q8) {
    uint32_t xm = 0, xv = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t bm = __float_as_uint(m.x[j]) & 0x7fffffffu, bv = __float_as_uint(v.x[j]) & 0x7fffffffu;
      xm = xm > bm ? xm : bm;
      xv = xv > bv ? xv : bv;
    }
    em = block_exp(wave_max(xm));
    ev = block_exp(wave_max(xv));
    uint32_t om = 0, ov = 0;
    if (em != 255) {
#pragma unroll
      for (int j = 0; j < 4; ++j) om |= encode8<true>(m.x[j], (h0 + (uint32_t)j * kAlphaPos) >> 12, em) << (8 * j);
    }
    if (ev != 255) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        ov |= encode8<false>(v.x[j], (h0 + (uint32_t)j * kAlphaPos) >> 5 & 0xFFFFFu, ev) << (8 * j);
    }
    gst(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.m) + s), om);
    gst(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.v) + s), ov);
    if (lane == 0) {
      a.me[sb] = (uint8_t)em;
      a.ve[sb] = (uint8_t)ev;
    }
  } else {
    gst_nt(static_cast<float*>(a.m) + s, f32x4{m.x[0], m.x[1], m.x[2], m.x[3]});
    gst_nt(static_cast<float*>(a.v) + s, f32x4{v.x[0], v.x[1], v.x[2], v.x[3]});
  }
}

// Squares are exact in fp64 and cannot overflow; their sums keep far more
// bits than the fp32 result, whatever the count.  The four waves of team t (of
// NORM_TEAMS a workgroup) sum every teams-th group of K chunks; the
// last workgroup to arrive adds the partial sums in index order, so the
// result does not depend on the order of arrival.  Arrivals wait for one
// another, some 20 ns each, so there is one workgroup for each compute unit:
// 120.6 M values in fp32 take 87 us (5.5 TB/s), with 512 workgroups 101 us, with
// 2048 of four waves 153 us.  fp64 sums cost nothing: with fp32 sums as long.
constexpr int NORM_TEAMS = 2, NORM_WAVES = NORM_TEAMS * OPT_WAVES;

template <int K>
__global__ __launch_bounds__(64 * NORM_WAVES) void grad_norm_kernel(OptHead* head, const OptChunk* chunks, int64_t nchunks,
                                                        float max_norm, double* part, float* out) {
  __shared__ double red[NORM_WAVES];
  __shared__ uint32_t last;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % OPT_WAVES;
  const int64_t teams = (int64_t)gridDim.x * NORM_TEAMS;
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  for (int64_t c = K * (int64_t)(blockIdx.x * NORM_TEAMS + __builtin_amdgcn_readfirstlane(threadIdx.x >> 8)); c < nchunks;
       c += K * teams) {
    F4 g[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t ck = c + k;
      const OptChunk* ch = chunks + (ck < nchunks ? ck : c);
      const int at = wave * OPT_BLOCK + lane * 4, l = (ck < nchunks ? ch->left : 0) - at;
      g[k] = load4(ch->g, at, l < 0 ? 0 : l > 4 ? 4 : l, ch->flags & OPT_GBF, ch->flags & OPT_VEC);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = fma((double)g[k].x[j], (double)g[k].x[j], acc[j]);
  }
  double sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
  auto block_sum = [&](double x) {
#pragma unroll
    for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
    if (lane == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.0;
#pragma unroll
    for (int q = 0; q < NORM_WAVES; ++q) x += red[q];
    __syncthreads();
    return x;
  };
  sum = block_sum(sum);
  if (threadIdx.x == 0) {
    __hip_atomic_store(&part[blockIdx.x], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(&head->arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  sum = 0.0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += 64 * NORM_WAVES)
    sum += __hip_atomic_load(&part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  sum = block_sum(sum);
  if (threadIdx.x == 0) {
    const double norm = sqrt(sum);
    out[0] = (float)norm;
    const double c = (double)max_norm / (norm + 1e-6);
    out[1] = !(norm < INFINITY) ? NAN : c < 1.0 ? (float)c : 1.f;
    __hip_atomic_store(&head->arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);   // for the next call
  }
}

// what 16 codes from `at` on stand for, in bf16
template <bool SIGNED>
__device__ __forceinline__ void moments16(const uint8_t* codes, const uint8_t* exps, uint16_t* out, int64_t at) {
  const int E = exp_of(exps[at / OPT_BLOCK]);
  const uint4 c = ldg16(codes + at);
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t h[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float x = decode8<SIGNED>(w[k / 2] >> (16 * (k & 1) + 8 * e) & 255u, E);
      h[e] = E == 255 ? 0x7fc0u : __float_as_uint(x) >> 16;   // at most four significant bits: exact
    }
    o[k] = h[0] | h[1] << 16;
  }
  stg16(out + at, make_uint4(o[0], o[1], o[2], o[3]));
  stg16(out + at + 8, make_uint4(o[4], o[5], o[6], o[7]));
}

// Both moments as bf16, 16 values a thread: 6 bytes a value, HBM (135.6 M values 158 us,
// 5.1 TB/s).
__global__ __launch_bounds__(256) void moments_kernel(const uint8_t* m, const uint8_t* v, const uint8_t* me,
                                                      const uint8_t* ve, uint16_t* mo, uint16_t* vo, int64_t blocks) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 16;
  if (at >= blocks * OPT_BLOCK) return;
  if (mo) moments16<true>(m, me, mo, at);
  if (vo) moments16<false>(v, ve, vo, at);
}

}  // namespace poetx

using namespace poetx;

namespace {

// workgroups of a norm: one for each compute unit; half of that for small sets
// (0.6 M values: 6.8 us, with 256 8.8 us)
constexpr int64_t kNormGroups = 256, kNormFew = 128;

int check_param(const poetx_param& p, int32_t i) {
  if (p.count < 0) return host_fail(POETX_ESHAPE, "tensor %d: count=%lld", (int)i, (long long)p.count);
  if ((p.param_dtype != POETX_F32 && p.param_dtype != POETX_BF16) ||
      (p.grad_dtype != POETX_F32 && p.grad_dtype != POETX_BF16))
    return host_fail(POETX_EDTYPE, "tensor %d: unsupported dtype", (int)i);
  if (p.copy_bf16 && p.param_dtype != POETX_F32)
    return host_fail(POETX_EDTYPE, "tensor %d: copy_bf16 goes with an fp32 tensor", (int)i);
  if (p.count == 0) return POETX_OK;
  if (!p.grad) return host_fail(POETX_EINVAL, "tensor %d: NULL gradient", (int)i);
  const uintptr_t pa = p.param_dtype == POETX_F32 ? 3 : 1, ga = p.grad_dtype == POETX_F32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(p.param) & pa) || (reinterpret_cast<uintptr_t>(p.grad) & ga) ||
      (reinterpret_cast<uintptr_t>(p.copy_bf16) & 1))
    return host_fail(POETX_EINVAL, "tensor %d: pointer not aligned to its type", (int)i);
  return POETX_OK;
}

// blocks, chunks and values of the tensors
int plan_params(const poetx_param* params, int32_t count, int64_t* blocks, int64_t* chunks, int64_t* values) {
  if (count < 0 || count > (1 << 20)) return host_fail(POETX_ESHAPE, "count=%d out of range [0, 1048576]", (int)count);
  if (count > 0 && !params) return host_fail(POETX_EINVAL, "params is NULL");
  *blocks = *chunks = *values = 0;
  for (int32_t i = 0; i < count; ++i) {
    const int rc = check_param(params[i], i);
    if (rc) return rc;
    if (params[i].count > (int64_t(1) << 37) - *values)
      return host_fail(POETX_ESHAPE, "more than 2^37 values in one set");
    const int64_t b = (params[i].count + OPT_BLOCK - 1) / OPT_BLOCK;
    *blocks += b;
    *chunks += (b + CHUNK_BLOCKS - 1) / CHUNK_BLOCKS;
    *values += params[i].count;
  }
  return POETX_OK;
}

size_t table_bytes(int64_t chunks) { return sizeof(OptHead) + (size_t)chunks * sizeof(OptChunk); }

int check_set(const poetx_param_set* set) {
  if (!set) return host_fail(POETX_EINVAL, "set is NULL");
  if (set->count < 0 || set->chunks < 0 || set->chunks > 0x7fffffffLL || set->blocks < 0 || set->norm_only > 1)
    return host_fail(POETX_EINVAL, "set was not made by poetx_param_table");
  if (set->chunks > 0 && (!set->table || (reinterpret_cast<uintptr_t>(set->table) & (kWsAlign - 1))))
    return host_fail(POETX_EINVAL, "set->table is NULL or not %zu-byte aligned", kWsAlign);
  return POETX_OK;
}

int check_state(const poetx_param_set* set, const poetx_adamw_state* st) {
  if (!st) return host_fail(POETX_EINVAL, "state is NULL");
  if (st->reserved) return host_fail(POETX_EINVAL, "state.reserved must be 0");
  if (st->kind != POETX_STATE_F32 && st->kind != POETX_STATE_8BIT)
    return host_fail(POETX_EINVAL, "state.kind=%d", (int)st->kind);
  if (set->blocks == 0) return POETX_OK;
  if (!st->m || !st->v || (st->kind == POETX_STATE_8BIT && (!st->m_exp || !st->v_exp)))
    return host_fail(POETX_EINVAL, "NULL state array");
  if ((reinterpret_cast<uintptr_t>(st->m) & 15) || (reinterpret_cast<uintptr_t>(st->v) & 15))
    return host_fail(POETX_EINVAL, "state arrays must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(st->skipped) & 3) return host_fail(POETX_EINVAL, "state.skipped not aligned to its type");
  return POETX_OK;
}

const OptChunk* chunks_of(const poetx_param_set* set) {
  return reinterpret_cast<const OptChunk*>(static_cast<const char*>(set->table) + sizeof(OptHead));
}

}  // namespace

extern "C" {

size_t poetx_param_table_bytes(const poetx_param* params, int32_t count) {
  int64_t blocks, chunks, values;
  if (plan_params(params, count, &blocks, &chunks, &values)) return 0;
  return table_bytes(chunks);
}

int poetx_param_table(const poetx_param* params, int32_t count, void* host_table, size_t bytes,
                      poetx_param_set* set) {
  int64_t blocks, chunks, values;
  const int rc = plan_params(params, count, &blocks, &chunks, &values);
  if (rc) return rc;
  if (!host_table || !set) return host_fail(POETX_EINVAL, "NULL argument");
  const size_t need = table_bytes(chunks);
  if (bytes < need) return host_fail(POETX_EWORKSPACE, "table has %zu bytes, needs %zu", bytes, need);
  memset(host_table, 0, sizeof(OptHead));
  OptChunk* c = reinterpret_cast<OptChunk*>(static_cast<char*>(host_table) + sizeof(OptHead));
  const int64_t span = (int64_t)CHUNK_BLOCKS * OPT_BLOCK;
  int64_t block = 0;
  uint32_t norm_only = 0;
  for (int32_t i = 0; i < count; ++i) {
    const poetx_param& p = params[i];
    const bool pbf = p.param_dtype == POETX_BF16, gbf = p.grad_dtype == POETX_BF16;
    const bool vec = !((reinterpret_cast<uintptr_t>(p.param) | reinterpret_cast<uintptr_t>(p.grad) |
                        reinterpret_cast<uintptr_t>(p.copy_bf16)) & 15);
    if (p.count > 0 && !p.param) norm_only = 1;
    for (int64_t at = 0; at < p.count; at += span) {
      const int64_t left = p.count - at < span ? p.count - at : span;
      *c++ = OptChunk{p.param ? static_cast<char*>(p.param) + at * (pbf ? 2 : 4) : nullptr,
                      static_cast<const char*>(p.grad) + at * (gbf ? 2 : 4),
                      p.copy_bf16 ? static_cast<uint16_t*>(p.copy_bf16) + at : nullptr, block + at / OPT_BLOCK, p.lr_mul,
                      p.weight_decay, (int32_t)left, (pbf ? OPT_PBF : 0) | (gbf ? OPT_GBF : 0) | (vec ? OPT_VEC : 0)};
    }
    block += (p.count + OPT_BLOCK - 1) / OPT_BLOCK;
  }
  *set = poetx_param_set{nullptr, blocks, chunks, values, count, norm_only};
  return POETX_OK;
}

size_t poetx_grad_norm_workspace_bytes(const poetx_param_set* set) {
  return kNormGroups * sizeof(double);
}

int poetx_grad_norm(const poetx_param_set* set, float max_norm, float* out, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_set(set);
  if (rc) return rc;
  if (!(max_norm > 0.f)) return host_fail(POETX_EINVAL, "max_norm must be positive");
  if (!out) return host_fail(POETX_EINVAL, "out is NULL");
  if (!set->table) return host_fail(POETX_EINVAL, "set->table is NULL");
  if ((rc = host_check_ws(ws, ws_bytes, poetx_grad_norm_workspace_bytes(set)))) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t most = (set->chunks + NORM_TEAMS - 1) / NORM_TEAMS, cap = set->blocks <= OPT_FEW ? kNormFew : kNormGroups,
                grid = most < 1 ? 1 : most < cap ? most : cap;
  {
    HostTimer tm(s, "grad_norm", 2.0 * set->values, 0.0);
    OptHead* head = static_cast<OptHead*>(const_cast<void*>(set->table));
    double* part = static_cast<double*>(ws);
    if (set->blocks <= OPT_FEW)
      hipLaunchKernelGGL(grad_norm_kernel<2>, dim3((unsigned)grid), dim3(64 * NORM_WAVES), 0, s, head, chunks_of(set),
                         set->chunks, max_norm, part, out);
    else
      hipLaunchKernelGGL(grad_norm_kernel<8>, dim3((unsigned)grid), dim3(64 * NORM_WAVES), 0, s, head, chunks_of(set),
                         set->chunks, max_norm, part, out);
  }
  return host_check_launch("gradient norm");
}

int poetx_adamw_step(const poetx_param_set* set, const poetx_adamw_state* state, const poetx_adamw_hyper* hyper,
                     int64_t step, const float* coef, void* stream) {
  int rc = check_set(set);
  if (rc) return rc;
  if ((rc = check_state(set, state))) return rc;
  if (set->norm_only) return host_fail(POETX_EINVAL, "a tensor of the set has no param");
  if (!hyper) return host_fail(POETX_EINVAL, "hyper is NULL");
  if (step < 1) return host_fail(POETX_EINVAL, "step must be >= 1");
  if (!(hyper->beta1 >= 0.f && hyper->beta1 < 1.f && hyper->beta2 >= 0.f && hyper->beta2 < 1.f))
    return host_fail(POETX_EINVAL, "betas must lie in [0, 1)");
  if (!(hyper->eps >= 0.f)) return host_fail(POETX_EINVAL, "eps must not be negative");
  if (set->chunks == 0) return POETX_OK;
  StepArgs a{};
  a.coef = coef;
  a.m = state->m; a.v = state->v;
  a.me = static_cast<uint8_t*>(state->m_exp); a.ve = static_cast<uint8_t*>(state->v_exp);
  a.lr = hyper->lr; a.b1 = hyper->beta1; a.b2 = hyper->beta2; a.eps = hyper->eps;
  a.ob1 = 1.f - hyper->beta1; a.ob2 = 1.f - hyper->beta2;
  a.ibc1 = (float)(1.0 / (1.0 - std::pow((double)hyper->beta1, (double)step)));
  a.ibc2 = (float)(1.0 / (1.0 - std::pow((double)hyper->beta2, (double)step)));
  if (state->skipped) {
    a.before = state->skipped + (step & 1);
    a.after = state->skipped + (~step & 1);
  }
  a.step = step;
  hipStream_t s = static_cast<hipStream_t>(stream);
  {
    const bool q8 = state->kind == POETX_STATE_8BIT, deep = hyper->eps < DEEP_EPS;
    HostTimer tm(s, "adamw", 0.0, (q8 ? 16.0 : 28.0) * set->values);
    launches(set->chunks, [&](int64_t first, uint32_t number) {
      a.chunks = chunks_of(set) + first;
      if (first > 0) a.after = nullptr;   // the first launch has left it
      if (q8 && deep) hipLaunchKernelGGL((adamw_kernel<true, true>), dim3(number), dim3(256), 0, s, a);
      else if (q8) hipLaunchKernelGGL((adamw_kernel<true, false>), dim3(number), dim3(256), 0, s, a);
      else if (deep) hipLaunchKernelGGL((adamw_kernel<false, true>), dim3(number), dim3(256), 0, s, a);
      else hipLaunchKernelGGL((adamw_kernel<false, false>), dim3(number), dim3(256), 0, s, a);
    });
  }
  return host_check_launch("adamw");
}

int poetx_adamw_moments(const poetx_param_set* set, const poetx_adamw_state* state, void* m_out, void* v_out,
                        void* stream) {
  int rc = check_set(set);
  if (rc) return rc;
  if ((rc = check_state(set, state))) return rc;
  if (state->kind != POETX_STATE_8BIT) return host_fail(POETX_EINVAL, "poetx_adamw_moments takes an 8-bit state");
  if ((reinterpret_cast<uintptr_t>(m_out) | reinterpret_cast<uintptr_t>(v_out)) & 15)
    return host_fail(POETX_EINVAL, "outputs must be 16-byte aligned");
  if (set->blocks == 0 || (!m_out && !v_out)) return POETX_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  {
    HostTimer tm(s, "adamw_moments", 0.0, 6.0 * OPT_BLOCK * set->blocks);
    launches((set->blocks + 15) / 16, [&](int64_t first, uint32_t number) {
      const int64_t at = first * 16, values = at * OPT_BLOCK;
      hipLaunchKernelGGL(moments_kernel, dim3(number), dim3(256), 0, s, static_cast<const uint8_t*>(state->m) + values,
                         static_cast<const uint8_t*>(state->v) + values, static_cast<const uint8_t*>(state->m_exp) + at,
                         static_cast<const uint8_t*>(state->v_exp) + at,
                         m_out ? static_cast<uint16_t*>(m_out) + values : nullptr,
                         v_out ? static_cast<uint16_t*>(v_out) + values : nullptr, set->blocks - at);
    });
  }
  return host_check_launch("adamw moments");
}

}  // extern "C"

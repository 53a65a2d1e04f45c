// Tokens in 8-bit integers with one scale each (include/gq.h, "Tokens in
// 8-bit integers"), plainly or behind the residual's addition and the
// root-mean-square norm, and the layout of packed codes as signed bytes.
//
// One pass over a row gives all statistics: with g = h * weight, y = g * f
// and f = 1 / sqrt(mean h^2 + eps), the factor f is positive, so max |y| =
// f max |g| and y / (max |y| / 127) = g / (max |g| / 127): the codes need
// max |g| only, and f goes into the scale.
#include <cfloat>

#include "gq_device.cuh"
#include "gq_internal.h"

namespace gq {
namespace {

struct QuantArgs {
  const void *x, *r;      // r: residual or NULL
  const void *w;          // fp32 or x-typed factors, or NULL
  void *h;                // x + r rounded, or NULL
  int8_t *codes;
  float *scales;
  int32_t *sums;          // or NULL
  int64_t n_tok, ldx;
  int d_in;
  float eps;
  int split, per;         // CTAs per row (a cluster) and elements per CTA
  int team, rows;         // threads per row and rows per CTA
};

// A unit is 16 bytes of a row, E = 8 (16-bit) or 4 (fp32) elements: what one
// load of a lane brings, so that a warp's loads are contiguous in every type.
// As fp32 its elements lie in pairs (f32x2), on which the additions, products
// and quotients run two at a time.
template <typename T>
constexpr int kE = 16 / static_cast<int>(sizeof(T));

// A unit's elements as pairs, by type (the last argument only names it).
__device__ __forceinline__ void widen(const uint4 &u, uint64_t (&v)[2], float) {
  v[0] = pair(u.x, u.y);
  v[1] = pair(u.z, u.w);
}
__device__ __forceinline__ uint64_t widen2(uint32_t u, __nv_bfloat16) {
  return pair(u << 16, u & 0xffff0000u);
}
__device__ __forceinline__ uint64_t widen2(uint32_t u, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
  return f32x2_pack(f.x, f.y);
}
template <typename T>
__device__ __forceinline__ void widen(const uint4 &u, uint64_t (&v)[4], T t) {
  v[0] = widen2(u.x, t);
  v[1] = widen2(u.y, t);
  v[2] = widen2(u.z, t);
  v[3] = widen2(u.w, t);
}
// The E factors of a unit as pairs.
template <typename T>
struct Factors {
  static constexpr int P = kE<T> / 2, Q = P / 2;     // pairs, and 16-byte pieces of them
  uint64_t f[P];
  template <typename WT>
  __device__ __forceinline__ void load(const WT *w) {
    const uint4 a = *reinterpret_cast<const uint4 *>(w);
    if constexpr (sizeof(WT) == sizeof(T)) {
      widen(a, f, T());
    } else {
      const uint4 b = *(reinterpret_cast<const uint4 *>(w) + 1);
      set(0, a);
      set(1, b);
    }
  }
  __device__ __forceinline__ void set(int p, const uint4 &a) {
    f[2 * p] = pair(a.x, a.y);
    f[2 * p + 1] = pair(a.z, a.w);
  }
  __device__ __forceinline__ uint4 piece(int p) const {
    uint4 a;
    f32x2_unpack(f[2 * p], a.x, a.y);
    f32x2_unpack(f[2 * p + 1], a.z, a.w);
    return a;
  }
  // v = v * factors
  __device__ __forceinline__ void times(uint64_t (&v)[P]) const {
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = mul2(v[i], f[i]);
  }
};
// Pairs rounded to T.
__device__ __forceinline__ uint4 narrow(const uint64_t (&v)[2], float) {
  uint4 u;
  f32x2_unpack(v[0], u.x, u.y);
  f32x2_unpack(v[1], u.z, u.w);
  return u;
}
__device__ __forceinline__ uint32_t narrow2(uint64_t v, __half) {
  uint32_t a, b;
  f32x2_unpack(v, a, b);
  const __half2 h = __floats2half2_rn(__uint_as_float(a), __uint_as_float(b));
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t narrow2(uint64_t v, __nv_bfloat16) {
  uint32_t a, b;
  f32x2_unpack(v, a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <typename T>
__device__ __forceinline__ uint4 narrow(const uint64_t (&v)[4], T t) {
  return make_uint4(narrow2(v[0], t), narrow2(v[1], t), narrow2(v[2], t), narrow2(v[3], t));
}

// 16 bytes that are read once (volatile, so that no load leaves its place
// behind chain_wait, as one that the compiler takes for a function of its
// address might).
__device__ __forceinline__ uint4 load16_once(const void *p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// The larger of a and |b|, |c|; NaN when one is NaN.
__device__ __forceinline__ float max_abs_nan(float a, uint64_t bc) {
  uint32_t b, c;
  f32x2_unpack(bc, b, c);
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;"
      : "=f"(r) : "f"(a), "f"(fabsf(__uint_as_float(b))), "f"(fabsf(__uint_as_float(c))));
  return r;
}
// Running largest magnitude of raw units (NaN when an element is NaN), two
// 16-bit ones at a time.
template <typename T>
struct RawTop;
template <>
struct RawTop<float> {
  float m = 0.0f;
  __device__ __forceinline__ void take(const uint4 &a) {
    m = max_abs_nan(max_abs_nan(m, pair(a.x, a.y)), pair(a.z, a.w));
  }
  __device__ __forceinline__ float value() const { return m; }
};
template <typename P>
struct RawTop16 {
  uint32_t m = 0u;
  __device__ __forceinline__ void take(const uint4 &a) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
    P t = *reinterpret_cast<const P *>(&m);
#pragma unroll
    for (int i = 0; i < 4; ++i) t = __hmax2_nan(t, __habs2(*reinterpret_cast<const P *>(&u[i])));
    m = *reinterpret_cast<const uint32_t *>(&t);
  }
  __device__ __forceinline__ float value() const {
    const P t = *reinterpret_cast<const P *>(&m);
    return static_cast<float>(__hmax_nan(t.x, t.y));
  }
};
template <>
struct RawTop<__half> : RawTop16<__half2> {};
template <>
struct RawTop<__nv_bfloat16> : RawTop16<__nv_bfloat162> {};

// Reductions over the threads of a row: over a warp, over the
// row's warps through shared memory (a slot per warp of the block), over the
// CTAs of a row's cluster through `mine` of each.  Every thread of the block
// takes part and all threads of a row get the result.  Each reduction has
// slots of its own, and the CTAs of a cluster meet once more before they
// leave (they arrive when they have read the others' slots and wait only
// before the next reduction, `again`, or the end), so no slot changes or goes
// while another thread reads it.
struct MaxSsq {          // max |g| as the bits of a float (NaN above infinity), and sum h^2
  uint32_t top;
  float ssq;
  __device__ __forceinline__ static MaxSsq zero() { return {0u, 0.0f}; }
  __device__ __forceinline__ MaxSsq warp() const {
    MaxSsq v{__reduce_max_sync(0xffffffffu, top), ssq};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v.ssq += __shfl_xor_sync(0xffffffffu, v.ssq, o);
    return v;
  }
};
struct MaxOnly {
  uint32_t top, unused;
  __device__ __forceinline__ static MaxOnly zero() { return {0u, 0u}; }
  __device__ __forceinline__ MaxOnly warp() const { return {__reduce_max_sync(0xffffffffu, top), 0u}; }
};
struct IntSum {
  int sum, unused;
  __device__ __forceinline__ static IntSum zero() { return {0, 0}; }
  __device__ __forceinline__ IntSum warp() const { return {__reduce_add_sync(0xffffffffu, sum), 0}; }
};
template <typename V>
__device__ __forceinline__ V row_reduce(V v, const QuantArgs &a, uint64_t *slots, uint64_t *mine,
                                        bool again) {
  static_assert(sizeof(V) == 8, "a slot holds 8 bytes");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tw = a.team >> 5;
  v = v.warp();
  if (tw > 1) {
    if (lane == 0) reinterpret_cast<V *>(slots)[warp] = v;
    __syncthreads();
    v = lane < tw ? reinterpret_cast<V *>(slots)[warp / tw * tw + lane] : V::zero();
    v = v.warp();
  }
  if (a.split > 1) {
    if (threadIdx.x == 0) *reinterpret_cast<V *>(mine) = v;
    if (again) cluster_wait();
    cluster_sync();
    v = V::zero();
    if (lane < a.split) {
      uint64_t u;
      asm volatile("ld.shared::cluster.u64 %0, [%1];"
                   : "=l"(u) : "r"(mapa_shared(smem_u32(mine), lane)) : "memory");
      v = *reinterpret_cast<const V *>(&u);
    }
    v = v.warp();
    cluster_arrive();  // waited for by the next reduction, or before the end
  }
  return v;
}

// Byte codes of four values from the sums t = q + 1.5 * 2^23 (their low
// bytes).
__device__ __forceinline__ uint32_t low_bytes(uint64_t a, uint64_t b) {
  uint32_t t[4];
  f32x2_unpack(a, t[0], t[1]);
  f32x2_unpack(b, t[2], t[3]);
  return __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
}
// 1 / sqrt(mean h^2 + eps) of one row.
__device__ __forceinline__ float inv_rms(float ssq, int d, float eps) {
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ssq, static_cast<float>(d)), eps)));
}
// sum h^2 in fp64 by one warp, for a row whose squares overflow fp32 or
// vanish in it (the row lies in memory: the caller has met the others at a
// barrier behind their stores of h).
template <typename T>
__device__ __noinline__ double ssq64(const T *h, int d_in) {
  double d = 0.0;
  __syncwarp();
  for (int c = threadIdx.x & 31; c < d_in; c += 32) {
    const double v = static_cast<double>(static_cast<float>(h[c]));
    d += v * v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  return d;
}

// What a row's values are before they are quantised.
enum Mode { kPlain, kCol, kNorm };

// The grid of a row from the bits of its largest magnitude.  A row whose
// values are so small that the quotient's steps could leave the normal range
// is divided 2^64 times larger, step and values alike (both exactly).
struct RowGrid {
  float s;             // the step
  float sq, rs;        // the step that the quotients use, and RN(1 / sq)
  bool bad, tiny;      // a value was not finite; sq = 2^64 s
};
__device__ __forceinline__ RowGrid row_grid(uint32_t bits) {
  RowGrid g;
  const float top = __uint_as_float(bits);
  g.bad = bits >= 0x7f800000u;
  g.tiny = top < 0x1p-90f;
  // (correctly rounded either way: the quotient from RN(1 / 127))
  g.s = g.tiny ? __fdiv_rn(top, 127.0f) : div_by_recip(top, 127.0f, 1.0f / 127.0f);
  if (g.s == 0.0f || g.bad) g.s = 1.0f;
  g.sq = g.tiny ? g.s * 0x1p64f : g.s;
  g.rs = __frcp_rn(g.sq);
  return g;
}
// Values of a tiny row, 2^64 times larger and at most 127 steps (a step that
// is subnormal may have been rounded down by more than rint would forgive).
__device__ __forceinline__ uint64_t tiny2(uint64_t g, float sq) {
  uint32_t a, b;
  f32x2_unpack(g, a, b);
  const float m = 127.0f * sq;
  return f32x2_pack(fminf(fmaxf(__uint_as_float(a) * 0x1p64f, -m), m),
                    fminf(fmaxf(__uint_as_float(b) * 0x1p64f, -m), m));
}
// The scale of a row, by the row's first warp (all its lanes).
template <typename T, bool NORM>
__device__ __forceinline__ float row_scale(const QuantArgs &a, const RowGrid &g, float ssq,
                                           const T *h) {
  if (g.bad) return __uint_as_float(0x7fc00000u);
  if (!NORM) return g.s;
  float f;
  if (ssq >= 1e-30f && ssq <= FLT_MAX)
    f = inv_rms(ssq, a.d_in, a.eps);
  else
    f = static_cast<float>(1.0 / sqrt(ssq64(h, a.d_in) / a.d_in + a.eps));
  return __fmul_rn(g.s, f);
}

// Statistics of a thread: max |g|, and sum h^2 in two halves.
template <Mode MODE, typename T>
struct Stats {
  RawTop<T> raw;
  float top = 0.0f;
  uint64_t ssq2 = 0ull;
  // h as it is stored in T -> the pairs of g (unset for kPlain)
  __device__ __forceinline__ void take(const uint4 &h, const Factors<T> &w, uint64_t (&g)[kE<T> / 2]) {
    if constexpr (MODE == kPlain) {
      raw.take(h);
    } else {
      widen(h, g, T());
      if (MODE == kNorm) {
#pragma unroll
        for (int i = 0; i < kE<T> / 2; ++i) ssq2 = fma2(g[i], g[i], ssq2);
      }
      w.times(g);
#pragma unroll
      for (int i = 0; i < kE<T> / 2; ++i) top = max_abs_nan(top, g[i]);
    }
  }
  __device__ __forceinline__ uint32_t bits() const {
    return __float_as_uint(MODE == kPlain ? raw.value() : top);
  }
  __device__ __forceinline__ float ssq() const {
    uint32_t a, b;
    f32x2_unpack(ssq2, a, b);
    return __uint_as_float(a) + __uint_as_float(b);
  }
};
// x + r rounded to T.
template <typename T>
__device__ __forceinline__ uint4 add_residual(const uint4 &x, const uint4 &r) {
  uint64_t a[kE<T> / 2], b[kE<T> / 2];
  widen(x, a, T());
  widen(r, b, T());
#pragma unroll
  for (int i = 0; i < kE<T> / 2; ++i) a[i] = add2(a[i], b[i]);
  return narrow(a, T());
}
// Writes the codes of the pairs of a unit; returns their sum.  rint(RN(g /
// s)) by the correctly rounded quotient from RN(1 / s) and the addition of
// 1.5 * 2^23, whose sum's low byte is the code (|g / s| <= 127 up to the
// step's rounding, which rint removes).
template <int P>
__device__ __forceinline__ int put(uint64_t (&g)[P], const RowGrid &gr, int8_t *out) {
  if (gr.tiny) {
#pragma unroll
    for (int i = 0; i < P; ++i) g[i] = tiny2(g[i], gr.sq);
  }
  const uint64_t rs2 = f32x2_pack(gr.rs, gr.rs), ns2 = f32x2_pack(-gr.sq, -gr.sq);
  const uint64_t c2 = f32x2_pack(12582912.0f, 12582912.0f);
#pragma unroll
  for (int i = 0; i < P; ++i) g[i] = quotient_plus_f32x2(g[i], rs2, ns2, c2);
  uint32_t q[P / 2];
  int sum = 0;
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    q[i] = gr.bad ? 0u : low_bytes(g[2 * i], g[2 * i + 1]);
    sum = __dp4a(static_cast<int>(q[i]), 0x01010101, sum);
  }
  if constexpr (P == 4)
    *reinterpret_cast<uint2 *>(out) = make_uint2(q[0], q[1]);
  else
    *reinterpret_cast<uint32_t *>(out) = q[0];
  return sum;
}

// ---------------------------------------------------------------- a block per row
// `team` threads take a row (or a slice of at most 8192 elements of one: the
// CTAs of a cluster share a longer row), N elements each, all loads first.
// N = 8 for a few tokens: the time is one load's latency, the reductions and
// the launch (one token of 4096: 1.7 us in a graph, 2.4 with residual and
// norm).  N = 32 while the rows fit the SMs at once, and for rows that the
// persistent kernel cannot hold (16 elements per thread were 4 to 13% faster
// around 4M elements and slower on both sides of that: not kept).  Measured
// (bf16, graph replays): 150 x 768, N = 8, plain 1.6 us, norm 2.0; N = 32: 512
// x 4096 plain 3.3 us, norm 5.1, 100 x 28672 norm with residual 8.4 us.
constexpr int kSlice = 8192;

template <typename T, typename WT, Mode MODE, int N>
__global__ void __launch_bounds__(N == 8 ? 1024 : 256, N == 8 ? 1 : 3) quant_block_kernel(const QuantArgs a) {
  constexpr bool NORM = MODE == kNorm;
  constexpr int E = kE<T>, U = N / E;
  __shared__ uint64_t slots[2][32], mine[2];
  chain_wait();
  chain_next();
  const int part = threadIdx.x / a.team, tid = threadIdx.x - part * a.team;
  const int rank = a.split > 1 ? static_cast<int>(blockIdx.x) % a.split : 0;
  const int64_t row = static_cast<int64_t>(blockIdx.x / a.split) * a.rows + part;
  const bool live = row < a.n_tok, res = NORM && a.r;
  const int c0 = rank * a.per + tid * E, cs = a.team * E;
  const int c1 = live ? min(rank * a.per + a.per, a.d_in) : 0;
  const T *x = static_cast<const T *>(a.x) + row * a.ldx;
  const T *r = static_cast<const T *>(a.r) + row * a.d_in;
  T *h = static_cast<T *>(a.h) + row * a.d_in;
  uint4 xr[U], rr[U];
#pragma unroll
  for (int v = 0; v < U; ++v) {
    const int c = c0 + v * cs;
    if (c < c1) {
      xr[v] = load16_once(x + c);
      if (res) rr[v] = load16_once(r + c);
    }
  }
  uint64_t g[U][E / 2];
  Stats<MODE, T> st;
#pragma unroll
  for (int v = 0; v < U; ++v) {
    const int c = c0 + v * cs;
    if (c < c1) {
      if (res) {
        xr[v] = add_residual<T>(xr[v], rr[v]);
        *reinterpret_cast<uint4 *>(h + c) = xr[v];
      }
      Factors<T> w;
      if (MODE != kPlain) w.load(static_cast<const WT *>(a.w) + c);
      st.take(xr[v], w, g[v]);
    }
  }
  uint32_t bits = st.bits();
  float ssq = 0.0f;
  if constexpr (NORM) {
    const MaxSsq m = row_reduce(MaxSsq{bits, st.ssq()}, a, slots[0], &mine[0], false);
    bits = m.top;
    ssq = m.ssq;
  } else {
    bits = row_reduce(MaxOnly{bits, 0u}, a, slots[0], &mine[0], false).top;
  }
  const RowGrid gr = row_grid(bits);
  int sum = 0;
#pragma unroll
  for (int v = 0; v < U; ++v) {
    const int c = c0 + v * cs;
    if (c < c1) {
      if (MODE == kPlain) widen(xr[v], g[v], T());
      sum += put(g[v], gr, a.codes + row * a.d_in + c);
    }
  }
  if (a.sums) sum = row_reduce(IntSum{sum, 0}, a, slots[1], &mine[1], true).sum;
  if (rank == 0 && live && tid < 32) {
    const float s = row_scale<T, NORM>(a, gr, ssq, res ? h : x);
    if (tid == 0) {
      a.scales[row] = s;
      if (a.sums) a.sums[row] = sum;
    }
  }
  if (a.split > 1) cluster_wait();
}

// ---------------------------------------------------------------- many rows
// Persistent blocks, 32 elements per thread: `team` threads take a row at a
// time, always the same columns, whose factors stay on the SM as fp32: in
// shared memory (the copies of a thread's own columns, 16 bytes a lane: no
// bank conflicts, no misses behind the stream of rows: 43 to 57% of the copy
// bandwidth when they came through L1), or, for fp32 rows of up to 20480
// elements, in registers (WREG: such rows need few instructions per byte, so
// fewer threads are enough; 134M elements with column factors 104 against
// 140 us).  Each thread copies its own units of the rows ahead into a ring of
// its own there (cp.async, AHEAD rows), so loads go on while a row is reduced
// and written, no registers wait for them and no thread waits for another's
// copies; a row is read once and stays in registers between the statistics
// and the codes, both of which take g from it (g itself would be twice the
// registers, and spill: 54% of the copy bandwidth instead of 77% when it was
// tried).  One barrier per row: the codes' sums of a row are added up behind
// the next row's.  x (and r) are read, codes (and h) written: plain rows and
// fp32 rows are bound by HBM (16384 x 28672 bf16 205 us = 105% of the copy
// bandwidth, 16384 x 8192 fp32 with factors 104 us = 99%), 16-bit rows with
// factors also by the instructions issued, 14 an element with column factors,
// 21 with the norm and 27 with its residual against 12 plain (16384 x 28672
// 264 us = 82%, 32768 x 8192 norm with residual 312 us = 92%, without 216 us
// = 57%).
constexpr int kRegThreads = 640;
constexpr size_t kRingMost = 225 * 1024;
__device__ __forceinline__ void cp_async16(uint32_t dst, const char *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t p, const uint4 &v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w) : "memory");
}

// FULL: every thread has all its units (d_in = 32 team), so that no unit is a
// branch of its own.  For 16-bit rows with column factors, which are bound by
// the instructions issued: 16384 x 28672 278 -> 264 us (plain rows, bound by
// HBM, 220 -> 250: not there).
template <typename T, typename WT, Mode MODE, int AHEAD, bool WREG, bool FULL>
__global__ void __launch_bounds__(WREG ? kRegThreads : 1024, 1) quant_rows_kernel(const QuantArgs a) {
  constexpr bool NORM = MODE == kNorm;
  constexpr int E = kE<T>, U = 32 / E;
  extern __shared__ uint4 ring[];
  __shared__ uint64_t slots[2][32];
  __shared__ int sums[2][32];
  chain_wait();
  chain_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = threadIdx.x / a.team, tid = threadIdx.x - part * a.team;
  const int tw = a.team >> 5, w0 = warp / tw * tw;
  const bool res = NORM && a.r;
  // operand o of unit v of ring row k: 16 bytes per thread at (k nin + o) U + v
  const uint32_t piece = blockDim.x * 16, rowb = piece * U * (res ? 2 : 1);
  const uint32_t sbase = smem_u32(ring) + threadIdx.x * 16;
  const int c0 = tid * E, cs = a.team * E;
  // this thread's units of a row
  const int nv = FULL ? U : c0 < a.d_in ? (a.d_in - c0 + cs - 1) / cs : 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * a.rows;
  int64_t row = static_cast<int64_t>(blockIdx.x) * a.rows + part;
  const char *xn = reinterpret_cast<const char *>(static_cast<const T *>(a.x) + row * a.ldx + c0);
  const char *rn = reinterpret_cast<const char *>(static_cast<const T *>(a.r) + row * a.d_in + c0);
  const int64_t xstep = step * a.ldx * sizeof(T), rstep = step * a.d_in * sizeof(T);
  const int unitb = cs * static_cast<int>(sizeof(T));
  int64_t ahead = row;                         // the row that xn and rn point into
  auto issue = [&](uint32_t at) {              // copies that row to ring row `at`
    if (ahead < a.n_tok) {
#pragma unroll
      for (int v = 0; v < U; ++v)
        if (FULL || v < nv) {
          cp_async16(at + v * piece, xn + v * unitb);
          if (res) cp_async16(at + (U + v) * piece, rn + v * unitb);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += step;
    xn += xstep;
    rn += rstep;
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) issue(sbase + k * rowb);
  // the factors of unit v as fp32: Q pieces behind the ring, at v Q + p, or
  // in registers
  constexpr int Q = Factors<T>::Q;
  const uint32_t wbase = sbase + AHEAD * rowb;
  Factors<T> wreg[WREG ? U : 1];
  if (MODE != kPlain) {
#pragma unroll
    for (int v = 0; v < U; ++v)
      if (v < nv) {
        Factors<T> f;
        f.load(static_cast<const WT *>(a.w) + c0 + v * cs);
        if constexpr (WREG) {
          wreg[v] = f;
        } else {
#pragma unroll
          for (int p = 0; p < Q; ++p) sts16(wbase + (v * Q + p) * piece, f.piece(p));
        }
      }
  }
  auto factors = [&](int v) {
    Factors<T> f{};
    if constexpr (WREG) {
      f = wreg[v];
    } else if (MODE != kPlain) {
#pragma unroll
      for (int p = 0; p < Q; ++p) f.set(p, lds16(wbase + (v * Q + p) * piece));
    }
    return f;
  };
  int64_t at = row * a.d_in + c0;              // of H and the codes
  uint32_t slot = sbase;
  int par = 0;                                 // parity of the round
  int64_t last = -1;
  // (all teams of a block make the same number of rounds)
  for (; row - part < a.n_tok; row += step, par ^= 1) {
    const bool live = row < a.n_tok;
    const int n = live ? nv : 0;
    uint4 x[U];
    Stats<MODE, T> st;
    asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
    if constexpr (NORM) {
#pragma unroll
      for (int v = 0; v < U; ++v)
        if (v < n) {
          x[v] = lds16(slot + v * piece);
          if (res) {
            x[v] = add_residual<T>(x[v], lds16(slot + (U + v) * piece));
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.h) + at + v * cs) = x[v];
          }
        }
#pragma unroll
      for (int v = 0; v < U; ++v)
        if (v < n) {
          uint64_t g[E / 2];
          st.take(x[v], factors(v), g);
        }
    } else if (live) {
#pragma unroll
      for (int v = 0; v < U; ++v)
        if (FULL || v < n) x[v] = lds16(slot + v * piece);
#pragma unroll
      for (int v = 0; v < U; ++v)
        if (FULL || v < n) {
          uint64_t g[E / 2];
          st.take(x[v], factors(v), g);
        }
    }
    issue(slot);                               // the row of this slot is in registers
    slot = AHEAD == 2 && slot == sbase ? sbase + rowb : sbase;
    uint32_t bits = st.bits();
    float ssq = 0.0f;
    if constexpr (NORM) {
      MaxSsq m = MaxSsq{bits, st.ssq()}.warp();
      if (lane == 0) reinterpret_cast<MaxSsq *>(slots[par])[warp] = m;
      __syncthreads();
      m = (lane < tw ? reinterpret_cast<MaxSsq *>(slots[par])[w0 + lane] : MaxSsq::zero()).warp();
      bits = m.top;
      ssq = m.ssq;
    } else {
      bits = __reduce_max_sync(0xffffffffu, bits);
      if (lane == 0) slots[par][warp] = bits;
      __syncthreads();
      bits = lane < tw ? static_cast<uint32_t>(slots[par][w0 + lane]) : 0u;
      bits = __reduce_max_sync(0xffffffffu, bits);
    }
    if (a.sums && warp == w0 && last >= 0) {  // the previous row's, whole since the barrier
      const int t = __reduce_add_sync(0xffffffffu, lane < tw ? sums[par ^ 1][w0 + lane] : 0);
      if (lane == 0) a.sums[last] = t;
    }
    const RowGrid gr = row_grid(bits);
    int sum = 0;
    if (live) {
      int8_t *out = a.codes + at;
#pragma unroll
      for (int v = 0; v < U; ++v)
        if (FULL || v < n) {
          uint64_t g[E / 2];
          widen(x[v], g, T());
          if (MODE != kPlain) factors(v).times(g);
          sum += put(g, gr, out + v * cs);
        }
    }
    if (a.sums) {
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (lane == 0) sums[par][warp] = sum;
    }
    if (warp == w0 && live) {
      const float s = row_scale<T, NORM>(a, gr, ssq, res ? static_cast<const T *>(a.h) + row * a.d_in
                                                         : static_cast<const T *>(a.x) + row * a.ldx);
      if (lane == 0) a.scales[row] = s;
    }
    last = live ? row : -1;
    at += step * a.d_in;
  }
  if (a.sums) {
    __syncthreads();
    if (warp == w0 && last >= 0) {
      const int t = __reduce_add_sync(0xffffffffu, lane < tw ? sums[par ^ 1][w0 + lane] : 0);
      if (lane == 0) a.sums[last] = t;
    }
  }
}

// Rows that the ring holds: two where those of all an SM's threads, with the
// factors, leave room.
template <typename T, Mode MODE>
constexpr int kAhead = sizeof(T) == 2 && MODE == kPlain ? 2 : 1;

template <typename T, typename WT, Mode MODE, bool WREG, bool FULL>
cudaError_t launch_many(const QuantArgs &a, size_t smem, cudaStream_t st) {
  static SmemOptIn opt;
  const auto kernel = quant_rows_kernel<T, WT, MODE, kAhead<T, MODE>, WREG, FULL>;
  opt.allow(kernel, kRingMost);
  const int threads = a.rows * a.team;
  int per_sm = (WREG ? kRegThreads : 1024) / threads;
  if (per_sm > static_cast<int>(kRingMost / (smem + 2048))) per_sm = static_cast<int>(kRingMost / (smem + 2048));
  if (per_sm < 1) per_sm = 1;
  const int64_t blocks = (a.n_tok + a.rows - 1) / a.rows, most = static_cast<int64_t>(num_sms()) * per_sm;
  return launch_chained(kernel, static_cast<unsigned>(blocks < most ? blocks : most), threads, smem, st, 1, a);
}

template <typename T, typename WT, Mode MODE, int N>
cudaError_t launch_block(QuantArgs a, cudaStream_t st) {
  a.team = ((a.per + N - 1) / N + 31) / 32 * 32;
  a.rows = N == 8 || a.split > 1 || a.team > 128 ? 1 : 256 / a.team;
  return launch_chained(quant_block_kernel<T, WT, MODE, N>,
                        static_cast<unsigned>((a.n_tok + a.rows - 1) / a.rows * a.split), a.rows * a.team, 0,
                        st, a.split, a);
}

template <typename T, typename WT, Mode MODE>
gq_status launch_rows(QuantArgs a, cudaStream_t st) {
  a.split = (a.d_in + kSlice - 1) / kSlice;
  a.per = ((a.d_in + a.split - 1) / a.split + 7) / 8 * 8;
  QuantArgs m = a;
  m.team = ((a.d_in + 31) / 32 + 31) / 32 * 32;
  m.rows = m.team >= 128 ? 1 : 128 / m.team;
  constexpr bool kCanReg = sizeof(T) == 4 && MODE != kPlain;
  constexpr bool kFull = sizeof(T) == 2 && MODE == kCol;
  const bool wreg = kCanReg && m.team <= kRegThreads;
  const size_t smem = static_cast<size_t>(m.rows * m.team) *
                      (32 * sizeof(T) * kAhead<T, MODE> * (a.r ? 2 : 1) + (MODE == kPlain || wreg ? 0 : 128));
  const int slot = timer_begin(GQ_KERNEL_QUANT_INT8, st);
  cudaError_t e;
  // Measured (graph replays, inputs from HBM): 8 elements per thread while a
  // row has an SM of its own or all rows together take few of its threads
  // (600 x 768 fp32 2.3 us, 32 per thread 3.0); 32 per thread in one wave
  // of blocks (512 x 4096 bf16 3.3 us, 8 per thread 4.3, persistent 3.6);
  // persistent beyond (4000 x 2048 fp32 9.7 us, a block per row 11.8).
  // Between 4M and 12M elements the persistent blocks make one round, so that
  // they copy their factors once for a row or two: norm of 2047 x 2048 fp16
  // 7.9 us, by a block per row 8.2 (N = 8) and 9.0 (32).
  const int64_t elems = a.n_tok * a.d_in, sms = num_sms();
  if (a.n_tok * a.split <= sms || elems <= sms * 512 * 8)
    e = launch_block<T, WT, MODE, 8>(a, st);
  else if (elems <= sms * 768 * 32 || m.team > 1024 || smem > kRingMost)
    e = launch_block<T, WT, MODE, 32>(a, st);
  else if (wreg)
    e = launch_many<T, WT, MODE, kCanReg, false>(m, smem, st);
  else if (kFull && a.d_in == 32 * m.team)
    e = launch_many<T, WT, MODE, false, kFull>(m, smem, st);
  else
    e = launch_many<T, WT, MODE, false, false>(m, smem, st);
  count_launch();
  timer_end(slot, st,
            static_cast<double>(a.n_tok) *
                    (static_cast<double>(a.d_in) * (sizeof(T) * (a.r ? 3 : 1) + 1) + 4 +
                     (a.sums ? 4 : 0)) +
                (a.w ? static_cast<double>(a.d_in) * sizeof(WT) : 0.0));
  return launched(e, "quant kernel");
}

// 16 codes per thread from the packed bit stream (once per layer).
__global__ void __launch_bounds__(256)
    unpack8_kernel(const uint32_t *q, const uint16_t *zeros, int64_t d_out, int64_t d_in, int bits,
                   int8_t *codes, int32_t *zpoint) {
  const int64_t per_row = d_in / 16, n = d_out * per_row;
  const int offset = 1 << (bits - 1);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; t < n;
       t += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = t / per_row, k0 = (t - row * per_row) * 16;
    const uint32_t *src = q + row * (d_in * bits / 32);
    __align__(16) int8_t c[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t bit = bits * (k0 + i), w = bit >> 5;
      const int off = static_cast<int>(bit & 31);
      uint32_t v = src[w] >> off;
      if (off + bits > 32) v |= src[w + 1] << (32 - off);
      c[i] = static_cast<int8_t>(static_cast<int>(v & ((1u << bits) - 1u)) - offset);
    }
    *reinterpret_cast<uint4 *>(codes + row * d_in + k0) = *reinterpret_cast<const uint4 *>(c);
    if (zpoint && k0 == 0)
      zpoint[row] = static_cast<int>(__half2float(__ushort_as_half(zeros[row]))) - offset;
  }
}

}  // namespace

gq_status launch_quant_int8(const void *X, const void *R, gq_dtype dt, int64_t n_tok, int64_t d_in,
                            int64_t ldx, const void *w, gq_dtype w_dtype, int norm, float eps,
                            void *H, int8_t *codes, float *scales, int32_t *sums,
                            cudaStream_t st) {
  if (n_tok == 0) return GQ_OK;
  const QuantArgs a{X, R, w, H, codes, scales, sums, n_tok, ldx, static_cast<int>(d_in), eps,
                    1, 0, 0, 0};
  if (norm) {
    switch (dt) {
      case GQ_F32: return launch_rows<float, float, kNorm>(a, st);
      case GQ_F16:
        return w_dtype == GQ_F32 ? launch_rows<__half, float, kNorm>(a, st)
                                 : launch_rows<__half, __half, kNorm>(a, st);
      default:
        return w_dtype == GQ_F32 ? launch_rows<__nv_bfloat16, float, kNorm>(a, st)
                                 : launch_rows<__nv_bfloat16, __nv_bfloat16, kNorm>(a, st);
    }
  }
  switch (dt) {
    case GQ_F32:
      return w ? launch_rows<float, float, kCol>(a, st) : launch_rows<float, float, kPlain>(a, st);
    case GQ_F16:
      return w ? launch_rows<__half, float, kCol>(a, st) : launch_rows<__half, float, kPlain>(a, st);
    default:
      return w ? launch_rows<__nv_bfloat16, float, kCol>(a, st)
               : launch_rows<__nv_bfloat16, float, kPlain>(a, st);
  }
}

gq_status launch_unpack_int8(const uint32_t *qpacked, const uint16_t *zeros, int64_t d_out,
                             int64_t d_in, int bits, int8_t *codes, int32_t *zpoint,
                             cudaStream_t st) {
  const int64_t blocks = (d_out * (d_in / 16) + 255) / 256;
  const int64_t most = 16 * static_cast<int64_t>(num_sms());
  unpack8_kernel<<<static_cast<unsigned>(blocks < most ? blocks : most), 256, 0, st>>>(
      qpacked, zeros, d_out, d_in, bits, codes, zpoint);
  count_launch();
  return check_launch("unpack8_kernel");
}

}  // namespace gq

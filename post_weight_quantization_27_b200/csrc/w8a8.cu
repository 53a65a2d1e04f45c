// Product of int8 tokens with a layer held in int8, scales per token and per
// output channel (include/gq.h, "Product of int8 tokens"):
//   Y = act(x_scale w_scale (sum_k x c - zpoint sum_k x) + bias) * M + R.
// The integers are exact in 32 bits: with at most 65536 columns, |sum x c|
// and |zpoint sum x| are at most 128 * 128 * 65536 = 2^30, and their
// difference sum x (c - zpoint) at most 128 * 255 * 65536 < 2^31.  One
// rounding takes it to fp32, where the epilogue works, and one more to the
// output's type.
#include <cfloat>
#include <type_traits>

#include "gq_device.cuh"
#include "gq_internal.h"

namespace gq {
namespace {

struct W8Args {
  const int8_t *w, *x;
  const uint16_t *ws;
  const int32_t *wz;      // or NULL (symmetric)
  const float *xs;
  const int32_t *xsum;
  const float *bias;      // or NULL
  const void *m, *r;      // or NULL
  void *y;
  int64_t d_out, n_tok;
  int d_in;
  int act;
  int *status;
  int n_tt, n_jt, nkb;    // tiles of tokens, tiles of outputs, K steps
  int pj;                 // outputs of a pair's tile
};

// acc - z xsum in two's complement.
__device__ __forceinline__ int sub_wrap(int acc, int z, int xsum) {
  return static_cast<int>(static_cast<uint32_t>(acc) -
                          static_cast<uint32_t>(z) * static_cast<uint32_t>(xsum));
}

// SiLU and GELU (tanh form, 0.5 v (1 + tanh u), u = sqrt(2 / pi) (v +
// 0.044715 v^3)) are v / (1 + 2^t) with t = -v log2 e and t = -2 u log2 e = v
// (c0 + c1 v^2), two at a time.  The approximate 2^t and reciprocal (a few
// ulps, and t's rounding) matter where 2^t is near 1; where it is large the
// value itself vanishes.  NaN stays NaN, in ReLU too.
__device__ __forceinline__ void over_1_plus_exp2(uint64_t v, uint64_t t, float &lo, float &hi) {
  uint32_t t0, t1;
  float e0, e1;
  f32x2_unpack(t, t0, t1);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(__uint_as_float(t0)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(__uint_as_float(t1)));
  f32x2_unpack(add2(f32x2_pack(e0, e1), f32x2_pack(1.0f, 1.0f)), t0, t1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(__uint_as_float(t0)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(__uint_as_float(t1)));
  f32x2_unpack(mul2(v, f32x2_pack(e0, e1)), t0, t1);
  lo = __uint_as_float(t0);
  hi = __uint_as_float(t1);
}
template <int N>
__device__ __forceinline__ void act_all(float (&v)[N], int act) {
  static_assert(N % 2 == 0, "pairs");
  if (act == GQ_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];
  } else if (act == GQ_ACT_SILU) {
    const uint64_t c = f32x2_pack(-1.4426950408889634f, -1.4426950408889634f);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint64_t p = f32x2_pack(v[i], v[i + 1]);
      over_1_plus_exp2(p, mul2(p, c), v[i], v[i + 1]);
    }
  } else if (act == GQ_ACT_GELU) {
    const uint64_t c0 = f32x2_pack(-2.302208198f, -2.302208198f);    // -2 log2(e) sqrt(2 / pi)
    const uint64_t c1 = f32x2_pack(-0.1029432396f, -0.1029432396f);  // .. 0.044715
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint64_t p = f32x2_pack(v[i], v[i + 1]);
      over_1_plus_exp2(p, mul2(p, fma2(mul2(p, p), c1, c0)), v[i], v[i + 1]);
    }
  }
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float &o) { o = v; }
__device__ __forceinline__ void from_f(float v, __half &o) { o = __float2half_rn(v); }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16 &o) { o = __float2bfloat16_rn(v); }

// The device status word, cleared by the launch's first block as it starts:
// a wait gives up 2 s after that at the earliest.
__device__ __forceinline__ void reset_status(int *status) { *reinterpret_cast<volatile int *>(status) = 0; }

// Output j of token t from its integer sum and the output's own scale,
// zero-point and bias, the token's scale and code sum, and M and R there.
// The product is taken as (v w_scale) x_scale: |v| < 2^31 times an fp16
// scale neither overflows nor loses a normal result.
struct OutCol {
  uint16_t ws;
  float bias;
  int wz;
  __device__ __forceinline__ float scale() const { return __half2float(__ushort_as_half(ws)); }
};
__device__ __forceinline__ OutCol out_col(const W8Args &a, int64_t j, bool live) {
  OutCol o;
  o.ws = live ? a.ws[j] : 0;
  o.wz = live && a.wz ? a.wz[j] : 0;
  o.bias = live && a.bias ? a.bias[j] : 0.0f;
  return o;
}
__device__ __forceinline__ float finish(const W8Args &a, const OutCol &o, int acc, float xs,
                                        int xsum, float m, float r) {
  if (a.wz) acc = sub_wrap(acc, o.wz, xsum);
  float v[2] = {static_cast<float>(acc) * o.scale(), 0.0f};
  v[0] = a.bias ? fmaf(v[0], xs, o.bias) : v[0] * xs;
  act_all(v, a.act);
  if (a.m) v[0] *= m;
  if (a.r) v[0] += r;
  return v[0];
}

// ---------------------------------------------------------------- 32 outputs of a token
__device__ __forceinline__ uint64_t int2float2(float a, float b) {  // of integers held as bits
  return f32x2_pack(static_cast<float>(__float_as_int(a)), static_cast<float>(__float_as_int(b)));
}
// v = the raw integer sums (as bits) -> x_scale w_scale (acc - z xsum) +
// bias, from the columns' operands in shared memory.  (Each option loops
// over all columns by itself: a branch per column would keep the compiler
// from interleaving them.)
__device__ __forceinline__ void scale32(const W8Args &a, const float *s, const int *z,
                                        const float *b, float xs, int xsum, float (&v)[32]) {
  if (a.wz) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const int4 z4 = *reinterpret_cast<const int4 *>(z + i);
      v[i] = __int_as_float(sub_wrap(__float_as_int(v[i]), z4.x, xsum));
      v[i + 1] = __int_as_float(sub_wrap(__float_as_int(v[i + 1]), z4.y, xsum));
      v[i + 2] = __int_as_float(sub_wrap(__float_as_int(v[i + 2]), z4.z, xsum));
      v[i + 3] = __int_as_float(sub_wrap(__float_as_int(v[i + 3]), z4.w, xsum));
    }
  }
  const uint64_t xs2 = f32x2_pack(xs, xs);
  uint64_t p[16];
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const ulonglong2 s4 = *reinterpret_cast<const ulonglong2 *>(s + 2 * i);
    p[i] = mul2(int2float2(v[2 * i], v[2 * i + 1]), s4.x);
    p[i + 1] = mul2(int2float2(v[2 * i + 2], v[2 * i + 3]), s4.y);
  }
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const ulonglong2 b4 = *reinterpret_cast<const ulonglong2 *>(b + 2 * i);
      p[i] = fma2(p[i], xs2, b4.x);
      p[i + 1] = fma2(p[i + 1], xs2, b4.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = mul2(p[i], xs2);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    uint32_t lo, hi;
    f32x2_unpack(p[i], lo, hi);
    v[2 * i] = __uint_as_float(lo);
    v[2 * i + 1] = __uint_as_float(hi);
  }
}
__device__ __forceinline__ void prefetch_l2(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ void prefetch_l2(const void *p, int bytes) {  // multiples of 16
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// M or R over a box of 32 tokens x BC = 64 / sizeof(T) outputs: four lanes
// take a row's 64 bytes (a lane per row would touch 32 lines an instruction:
// 2560 x 2048 x 8192 with a residual 51 against 40 us), and the rows change
// hands in the warp's staging buffer, laid out as the boxes that leave by it.
__device__ __forceinline__ int box_at(int r, int c) {   // 16-byte chunk c of row r
  return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}
template <typename T, bool WHOLE>
struct Box {
  static constexpr int E = 16 / static_cast<int>(sizeof(T));
  uint4 u[4];
  __device__ __forceinline__ void load(const W8Args &a, const void *base, int64_t row0, int64_t j0,
                                       int lane) {
    const int64_t j = j0 + (lane & 3) * E;
    const T *p = static_cast<const T *>(base) + (row0 + (lane >> 2)) * a.d_out + j;
#pragma unroll
    for (int i = 0; i < 4; ++i, p += 8 * a.d_out) {
      if (row0 + (lane >> 2) + 8 * i >= a.n_tok) break;
      if constexpr (WHOLE) {
        if (j < a.d_out) u[i] = *reinterpret_cast<const uint4 *>(p);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (j + e < a.d_out) reinterpret_cast<T *>(&u[i])[e] = p[e];
      }
    }
  }
  // This lane's row of the box, in place of what it loaded.
  __device__ __forceinline__ void to_row(uint8_t *stg, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4 *>(stg + box_at((lane >> 2) + 8 * i, lane & 3)) = u[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const uint4 *>(stg + box_at(lane, i));
    __syncwarp();
  }
  template <int H>
  __device__ __forceinline__ void times(float (&v)[32]) const {
#pragma unroll
    for (int i = 0; i < 4 * E; ++i) v[H * 4 * E + i] *= to_f(reinterpret_cast<const T *>(u)[i]);
  }
  template <int H>
  __device__ __forceinline__ void plus(float (&v)[32]) const {
#pragma unroll
    for (int i = 0; i < 4 * E; ++i) v[H * 4 * E + i] += to_f(reinterpret_cast<const T *>(u)[i]);
  }
};
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// The values v[H BC ..] of a token, BC = 64 / sizeof(T) of them, rounded to T
// into this lane's row of a box of 32 rows of 64 bytes (16-byte chunk c of
// row r at c ^ (r / 2 % 4): the tensor map's 64-byte swizzle, and no bank
// conflicts).
template <int H>
__device__ __forceinline__ void stage_row(uint8_t *stg, int r, const float (&v)[32], float) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<float4 *>(stg + box_at(r, c)) =
        make_float4(v[16 * H + 4 * c], v[16 * H + 4 * c + 1], v[16 * H + 4 * c + 2], v[16 * H + 4 * c + 3]);
}
template <int H, typename T>
__device__ __forceinline__ void stage_row(uint8_t *stg, int r, const float (&v)[32], T t) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4 u;
    u.x = pack2(v[8 * c], v[8 * c + 1], t);
    u.y = pack2(v[8 * c + 2], v[8 * c + 3], t);
    u.z = pack2(v[8 * c + 4], v[8 * c + 5], t);
    u.w = pack2(v[8 * c + 6], v[8 * c + 7], t);
    *reinterpret_cast<uint4 *>(stg + box_at(r, c)) = u;
  }
}
// 64 fp32 outputs of R tokens from shared memory (before M and R) to Y, where
// rows of Y, M and R are no multiple of 16 bytes long: M, R and Y at the same
// addresses, row after row.  A row's pieces follow one another, so that the
// sectors that two of them share are written whole: the stores of 2048 rows of
// 50257 alone take 99 us so and 230 in boxes of 16 outputs (65 where sectors
// are whole).
constexpr int kRowPitch = 68;                  // floats (no bank conflicts)
template <int R>
__device__ __forceinline__ void put_rows(const W8Args &a, const float *stg, int64_t at, int rows,
                                         int n, int lane) {
  float *y = static_cast<float *>(a.y) + at + lane;
  const float *mp = static_cast<const float *>(a.m) + at + lane;
  const float *rp = static_cast<const float *>(a.r) + at + lane;
  const int live[2] = {lane < n ? rows : 0, lane + 32 < n ? rows : 0};
#pragma unroll
  for (int r0 = 0; r0 < R; r0 += 4) {
    float v[4][2], u[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) v[i][h] = stg[(r0 + i) * kRowPitch + h * 32 + lane];
    if (a.m) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (r0 + i < live[h]) u[i][h] = mp[(r0 + i) * a.d_out + h * 32];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) v[i][h] *= u[i][h];
    }
    if (a.r) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (r0 + i < live[h]) u[i][h] = rp[(r0 + i) * a.d_out + h * 32];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) v[i][h] += u[i][h];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (r0 + i < live[h]) y[(r0 + i) * a.d_out + h * 32] = v[i][h];
  }
}
// A staged box of 16-bit outputs to such rows: a row per store, 32 lanes.
// (Rows of 64 in 4-byte stores, a lane's pair by its row's parity, took 253 us
// instead of 160 for 2048 rows of 50257 behind 768 inputs: more instructions.)
template <typename T>
__device__ __forceinline__ void store_box(const W8Args &a, const uint8_t *stg, int lane,
                                          int64_t row0, int64_t j0) {
  T *y = static_cast<T *>(a.y) + row0 * a.d_out + j0 + lane;
  const int rows = a.n_tok - row0 < 32 ? static_cast<int>(a.n_tok - row0) : 32;
  if (j0 + lane >= a.d_out) return;
  for (int r = 0; r < rows; ++r)
    y[r * a.d_out] = *reinterpret_cast<const T *>(stg + box_at(r, lane / 8) + (lane % 8) * 2);
}

// ---------------------------------------------------------------- many tokens
// Tiles of 256 tokens x PJ = 256 (or 224: a.pj) or 128 outputs on CTA pairs
// (tcgen05 cta_group::2, kind::i8), persistent, K in steps of 128 bytes:
//   warp 0      TMA: CTA r of the pair stages the tile's token rows 128 r ..
//               and output rows PJ / 2 r .., both CTAs' loads completing on
//               CTA 0's full[s]
//   warp 1      CTA 0: four MMAs of M = 256, N = PJ, K = 32 a stage into one
//               of two PJ-column TMEM accumulators; each CTA receives its 128
//               tokens' rows
//   the others  epilogue, a warp per 32 tokens x 64 outputs, a thread per
//               token: the outputs' scales, zero-points and bias pass through
//               shared memory of the warp's own, loaded a tile ahead; results
//               pass a 64-byte-swizzled buffer of the warp's own and leave
//               by TMA store; where Y's rows are no multiple of 16 bytes
//               (!TMA), by ordinary ones.  No warp waits for another one's tile
//               (operands shared by a barrier of all: 2560 x 2048 x 8192 with
//               GELU 42.7 us, so 40.5; 36.9 with all later steps).
// The issuing warps' lanes walk their loops together, so that a step's values
// stay in uniform registers (a loop of one lane: 0.35 us a step, so 0.25: they
// share their schedulers with the epilogue).  Bound by the tensor cores where K
// is long (8192 x 8192 x 28672: 1140 us = 3370 TOP/s in bursts), by the
// epilogue, about 4 us a tile of 256 x 256, where it is short, up to 2048 or so.
// Shared memory goes to operand stages first: 4 of them with two staged boxes
// per warp take 44 us instead of 35 at 2560 x 2048 x 8192, so deep is the
// loads' latency.
constexpr int PT = 256, PK = 128;
constexpr int P_STAGING = 2048;                        // per epilogue warp: 32 rows x 64 bytes

struct Cols {              // operands of an epilogue warp's outputs, in shared memory
  float s[64];
  int z[64];
  float b[64];
};
template <int PJ, bool TMA>
struct PairShape {
  static constexpr int kStages = PJ == 256 ? 5 : 7;
  static constexpr int kBoxes = PJ == 256 ? 1 : 2;       // staged boxes per epilogue warp
  static constexpr int kX = 128 * PK, kW = PJ / 2 * PK;  // one CTA's operands of a stage
  static constexpr int kStage = kX + kW;
  static constexpr int kWarps = PJ / 16;                 // of the epilogue
  static constexpr int kCols = 64;                       // outputs of each of its warps
  static constexpr int kThreads = 64 + 32 * kWarps;
  static constexpr int kRows = 16;                       // .. or rows of put_rows (PJ = 128)
  static constexpr int kStaging = PJ == 256 ? P_STAGING : 4608;
  static_assert(kBoxes * P_STAGING <= kStaging && (PJ == 256 || kRows * kRowPitch * 4 <= kStaging) &&
                    kStaging % 512 == 0, "what is staged fits, boxes on the swizzle's period");
  static constexpr size_t kSmem = 1024 + kStages * kStage + kWarps * (kStaging + sizeof(Cols)) + 256;
};
struct TileOps {           // what one thread brings for a tile: two outputs' operands, its token's
  int tt, jt;              // the tile
  uint16_t ws[2];
  int wz[2];
  float bias[2], xs;
  int xsum;
};

// Tile t -> (token tile, output tile) in groups of 8 token tiles, so that the
// tiles in flight (74 pairs: 8 x 9) share slabs of both operands in L2.
__device__ __forceinline__ void pair_tile(int t, int n_tt, int n_jt, int &tt, int &jt) {
  constexpr int G = 8;
  const int g = t / (G * n_jt), r = t - g * G * n_jt;
  const int rows = min(G, n_tt - g * G);
  tt = g * G + r % rows;
  jt = r / rows;
}

// TMA: rows of Y, M and R are a multiple of 16 bytes long (kernels of their
// own: 2048 x 768 x 50256 103 us with one kernel for both, so 93).
template <typename T, int PJ, bool TMA>
__global__ void __launch_bounds__(PairShape<PJ, TMA>::kThreads, 1)
    w8a8_pair_kernel(const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmY, W8Args a) {
  using S = PairShape<PJ, TMA>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *staging = smem + S::kStages * S::kStage;
  Cols *cols = reinterpret_cast<Cols *>(staging + S::kWarps * S::kStaging);
  uint64_t *full = reinterpret_cast<uint64_t *>(cols + S::kWarps);  // CTA 0: both CTAs' loads landed
  uint64_t *empty = full + S::kStages;                  // per CTA: MMAs done with the stage
  uint64_t *acc_full = empty + S::kStages;              // per CTA
  uint64_t *acc_empty = acc_full + 2;                       // CTA 0: both CTAs' epilogue warps
  uint64_t *drain = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x >> 1), n_pairs = static_cast<int>(gridDim.x >> 1);
  const int n_tiles = a.n_tt * a.n_jt, pj = PJ == 256 ? a.pj : PJ;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * S::kWarps);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    int tt, jt;
    pair_tile(pair, a.n_tt, a.n_jt, tt, jt);
    for (int kb = 0; kb < S::kStages && kb < a.nkb; ++kb)
      tma_prefetch_2d(&tmW, kb * PK, jt * pj + static_cast<int>(rank) * (pj / 2));
  }
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) reset_status(a.status);
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * PJ);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers initialised and TMEM allocated
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  chain_next();
  const int half0 = static_cast<int>(rank) * 128;  // this CTA's token rows in a tile

  if (warp == 0) {
    // (The two issuing warps share their schedulers with the epilogue's: all
    // their lanes walk the loop, so that its values stay in uniform registers
    // and a step is few instructions; one lane issues.)
    const bool leader = elect_one();
    bool ok = true;
    uint32_t s = 0, ph = 1, done = 0;
    const uint32_t bytes = 2 * (S::kX + pj / 2 * PK);
    const uint32_t base = smem_u32(smem), full0 = mapa_shared(smem_u32(full), 0);
    for (int t = pair; t < n_tiles && ok; t += n_pairs) {
      int tt, jt;
      pair_tile(t, a.n_tt, a.n_jt, tt, jt);
      const int yx = tt * PT + half0, yw = jt * pj + static_cast<int>(rank) * (pj / 2);
      for (int kb = 0; kb < a.nkb; ++kb) {
        if (!mbar_wait_warp(&empty[s], ph)) { ok = false; break; }
        if (leader) {
          const uint32_t st = base + s * S::kStage;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          tma_load_2d_pair(st, &tmX, full0 + 8 * s, kb * PK, yx);
          tma_load_2d_pair(st + S::kX, &tmW, full0 + 8 * s, kb * PK, yw);
        }
        done |= 1u << s;
        if (++s == S::kStages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (rank == 0) {  // the last loads of both CTAs have landed: stage q's was in this or the last lap
      for (uint32_t q = 0; q < S::kStages; ++q)
        if ((done >> q & 1) && !mbar_wait_warp(&full[q], q < s ? ph ^ 1 : ph)) ok = false;
    }
    if (!ok && leader) set_status(a.status, kDevTimeout);
  } else if (warp == 1) {
    if (rank == 0) {
      const bool leader = elect_one();
      bool ok = true;
      uint32_t s = 0, ph = 0, ch = 0;
      const uint32_t idesc = idesc_s8_s32(PT, pj);
      const uint64_t dx0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t dw0 = smem_desc_sw128(smem_u32(smem) + S::kX, 16, 1024);
      for (int t = pair; t < n_tiles && ok; t += n_pairs, ++ch) {
        const uint32_t buf = ch & 1, use = ch >> 1;
        if (!mbar_wait_cluster_warp(&acc_empty[buf], (use & 1) ^ 1)) { ok = false; break; }
        tc_fence_after();
        const uint32_t acc = tmem + buf * PJ;
        for (int kb = 0; kb < a.nkb; ++kb) {
          if (!mbar_wait_cluster_warp(&full[s], ph)) { ok = false; break; }
          tc_fence_after();
          if (leader) {
            const uint64_t dx = dx0 + s * (S::kStage >> 4), dw = dw0 + s * (S::kStage >> 4);
            mma_s8_pair(acc, dx, dw, idesc, kb != 0);
#pragma unroll
            for (int kk = 1; kk < PK / 32; ++kk) mma_s8_pair(acc, dx + 2 * kk, dw + 2 * kk, idesc, 1u);
            mma_commit_pair(&empty[s], 3);
          }
          if (++s == S::kStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        if (leader) mma_commit_pair(&acc_full[buf], 3);
      }
      if (leader) mma_commit_pair(drain, 1);
      if (!mbar_wait_warp(drain, 0)) ok = false;
      if (!ok && leader) set_status(a.status, kDevTimeout);
    }
  } else {
    constexpr int BC = 64 / sizeof(T);            // outputs per staged box
    const int ew = warp - 2, quarter = warp & 3, col0 = (ew >> 2) * S::kCols;
    const int blocks = min(S::kCols, pj - col0) / 32;  // of 32 outputs that this warp has in a tile
    uint8_t *stg = staging + ew * S::kStaging;
    uint32_t stg_at = 0;
    Cols &cl = cols[ew];
    auto load_ops = [&](int t) {
      TileOps o{};
      if (t >= n_tiles) return o;
      pair_tile(t, a.n_tt, a.n_jt, o.tt, o.jt);
      const int64_t j0 = static_cast<int64_t>(o.jt) * pj + col0 + lane;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (j0 + 32 * i < a.d_out) {
          o.ws[i] = a.ws[j0 + 32 * i];
          if (a.wz) o.wz[i] = a.wz[j0 + 32 * i];
          if (a.bias) o.bias[i] = a.bias[j0 + 32 * i];
        }
      const int64_t row = static_cast<int64_t>(o.tt) * PT + half0 + quarter * 32 + lane;
      if (row < a.n_tok) {
        o.xs = a.xs[row];
        if (a.wz) o.xsum = a.xsum[row];
      }
      return o;
    };
    TileOps next = load_ops(pair);
    uint32_t ch = 0;
    bool ok = true;
    for (int t = pair; t < n_tiles; t += n_pairs, ++ch) {
      const uint32_t buf = ch & 1, use = ch >> 1;
      const TileOps ops = next;
      const int tt = ops.tt, jt = ops.jt;
      __syncwarp();        // all lanes have read the last tile's operands
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        cl.s[lane + 32 * i] = __half2float(__ushort_as_half(ops.ws[i]));
        if (a.wz) cl.z[lane + 32 * i] = ops.wz[i];
        if (a.bias) cl.b[lane + 32 * i] = ops.bias[i];
      }
      __syncwarp();
      next = load_ops(t + n_pairs);
      const int64_t row0 = static_cast<int64_t>(tt) * PT + half0 + quarter * 32;
      // M and R: the next tile's go to L2 now; this tile's, 16-bit, come
      // before the sums are needed, fp32, twice the registers, when they are
      constexpr bool kEarly = sizeof(T) == 2;
      Box<T, TMA> m, r;
      auto load_mr = [&](int64_t j) {
        if (a.m) m.load(a, a.m, row0, j, lane);
        if (a.r) r.load(a, a.r, row0, j, lane);
      };
      if (a.m || a.r) {
        if (kEarly) load_mr(static_cast<int64_t>(jt) * pj + col0);
        if (t + n_pairs < n_tiles) {
          const int64_t next_row = static_cast<int64_t>(next.tt) * PT + half0 + quarter * 32 + lane;
          const int64_t jw = static_cast<int64_t>(next.jt) * pj + col0;
          for (int64_t j = jw; next_row < a.n_tok && j < jw + blocks * 32 && j < a.d_out; j += 128 / sizeof(T)) {
            if (a.m) prefetch_l2(static_cast<const T *>(a.m) + next_row * a.d_out + j);
            if (a.r) prefetch_l2(static_cast<const T *>(a.r) + next_row * a.d_out + j);
          }
        }
      }
      ok = mbar_wait_warp(&acc_full[buf], use & 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * PJ + col0;
      if constexpr (!TMA && sizeof(T) == 4) {
        float v[2][32];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          tmem_ld32(taddr + q * 32, v[q]);
          if (q == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(&acc_empty[buf], 0);
          }
          scale32(a, cl.s + q * 32, cl.z + q * 32, cl.b + q * 32, ops.xs, ops.xsum, v[q]);
          act_all(v[q], a.act);
        }
        constexpr int R = S::kRows;                                // rows that the buffer holds
        float *rows = reinterpret_cast<float *>(stg);
        const int64_t j0 = static_cast<int64_t>(jt) * pj + col0, left = a.n_tok - row0;
        const int n = a.d_out - j0 < 64 ? static_cast<int>(a.d_out - j0) : 64;
#pragma unroll 1
        for (int p = 0; p < 32; p += R) {
          if (lane / R == p / R) {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float *u = &v[c / 8][c % 8 * 4];
              *reinterpret_cast<float4 *>(rows + lane % R * kRowPitch + 4 * c) = make_float4(u[0], u[1], u[2], u[3]);
            }
          }
          __syncwarp();
          if (n > 0 && left > p)
            put_rows<R>(a, rows, (row0 + p) * a.d_out + j0, left - p < R ? static_cast<int>(left - p) : R, n, lane);
          __syncwarp();
        }
        continue;
      }
      // (rolled: the options' code per 32 columns is large, and the warps
      // would wait for instructions)
#pragma unroll 1
      for (int q = 0; q < blocks; ++q) {
        const int64_t j0 = static_cast<int64_t>(jt) * pj + col0 + q * 32;
        float v[32];
        tmem_ld32(taddr + q * 32, v);
        if (q == blocks - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(&acc_empty[buf], 0);
        }
        scale32(a, cl.s + q * 32, cl.z + q * 32, cl.b + q * 32, ops.xs, ops.xsum, v);
        act_all(v, a.act);
        auto put_box = [&](auto half) {
          constexpr int H = decltype(half)::value;
          const int64_t jb = j0 + H * BC;
          uint8_t *const box = stg + stg_at;
          if (S::kBoxes == 2) stg_at ^= P_STAGING;
          if constexpr (TMA) {                                     // the buffer's last box has left it
            if (lane == 0) {
              if (S::kBoxes == 2) bulk_wait_group_read1();
              else bulk_wait_group_read0();
            }
            __syncwarp();
          }
          if (a.m) {
            if (!kEarly) m.load(a, a.m, row0, jb, lane);
            m.to_row(box, lane);
            m.template times<H>(v);
          }
          if (a.r) {
            if (!kEarly) r.load(a, a.r, row0, jb, lane);
            r.to_row(box, lane);
            r.template plus<H>(v);
          }
          if (kEarly && q + 1 < blocks) load_mr(j0 + 32);
          stage_row<H>(box, lane, v, T());
          if constexpr (TMA) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (jb < a.d_out && row0 < a.n_tok)
                tma_store_2d(&tmY, box, static_cast<int32_t>(jb), static_cast<int32_t>(row0));
              bulk_commit_group();       // (an empty group too: the waits count them)
            }
          } else {
            __syncwarp();
            store_box<T>(a, box, lane, row0, jb);
            __syncwarp();
          }
        };
        put_box(std::integral_constant<int, 0>());
        if constexpr (BC == 16) put_box(std::integral_constant<int, 1>());
      }
    }
    if (lane == 0) bulk_wait_group0();
    if (!ok && lane == 0) set_status(a.status, kDevTimeout);
  }

  // every MMA of the pair has completed (CTA 0 waited for them) and both
  // CTAs are done with their TMEM and shared memory before either frees it
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * PJ);
  }
}

// ---------------------------------------------------------------- few tiles
// 128 outputs x up to 128 tokens per cluster of `split` CTAs, each summing
// its own range of K on the tensor cores (M = the outputs, N = the tokens
// rounded up to 16, so a short batch wastes no operand rows); two or more
// CTAs fit an SM, so one's epilogue runs beside another's loads.  With
// split > 1 every CTA lays its integer sums out in its (then idle) ring,
// and CTA r of the cluster adds the token columns r, r + split, .. of all
// of them over distributed shared memory: integers, so the order of the
// additions does not matter, no workspace and no second launch.
// A lane owns an output, so a warp's accesses to Y, M and R are contiguous
// whatever d_out is.  Bound by the weights' way from HBM and by what comes
// before and after it: 33 x 8192 x 8192 affine with residual 19.5 us (10.5 at
// the copy rate; 16384 inputs take 11.6 us more, 5.8 TB/s), 16 x 4096 x 11008
// 12.2, 33 x 4096 x 4096 9.2 (2.6 at the copy rate).  So about 7 us are this
// kernel's own (the dp4a kernel pays 2 around the same weights): TMEM, barriers
// and the first round of the ring, then the sums' exchange, which few_us puts
// at 1.5 us and 0.06 a token of the tile: each CTA reads them by 4-byte loads
// from the others between two cluster barriers.
constexpr int F_J = 128, F_T = 128, F_MAX_STAGES = 12, F_THREADS = 128;

struct FewPlan {
  int bn;            // tokens per tile, a multiple of 16
  int stages, split;
  int tmem_cols;
  int steps, held;   // K steps and CTAs on the fullest SM
};

__device__ __forceinline__ int ld_cluster_s32(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// The token columns c0, c0 + step, .. (NC of them, those below n) of output
// j, in stages over all of them: a warp is alone on its scheduler here, and
// one column after another would wait for each instruction in turn (128
// columns: 17.5 -> 10 us at 768 -> 2304).
template <typename T, int NC>
__device__ __forceinline__ void few_columns(const W8Args &a, const OutCol &o, bool live, int64_t t0,
                                            int c0, int step, int n, int64_t j, const float *xs,
                                            const int *xsum, int (&acc)[NC]) {
  const int64_t at = (t0 + c0) * a.d_out + j, pitch = a.d_out * step;
  T mv[NC], rv[NC];
  if (a.m) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (live && c0 + i * step < n) mv[i] = static_cast<const T *>(a.m)[at + i * pitch];
  }
  if (a.r) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (live && c0 + i * step < n) rv[i] = static_cast<const T *>(a.r)[at + i * pitch];
  }
  if (a.wz) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (c0 + i * step < n) acc[i] = sub_wrap(acc[i], o.wz, xsum[c0 + i * step]);
  }
  float v[NC];
  const float ws = o.scale();
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const float sx = c0 + i * step < n ? xs[c0 + i * step] : 0.0f;
    v[i] = static_cast<float>(acc[i]) * ws;
    v[i] = a.bias ? fmaf(v[i], sx, o.bias) : v[i] * sx;
  }
  act_all(v, a.act);
  if (a.m) {
#pragma unroll
    for (int i = 0; i < NC; ++i) v[i] *= to_f(mv[i]);
  }
  if (a.r) {
#pragma unroll
    for (int i = 0; i < NC; ++i) v[i] += to_f(rv[i]);
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (c0 + i * step < n) from_f(v[i], static_cast<T *>(a.y)[at + i * pitch]);
}

template <typename T>
__global__ void __launch_bounds__(F_THREADS)
    w8a8_few_kernel(const __grid_constant__ CUtensorMap tmX,
                    const __grid_constant__ CUtensorMap tmW, W8Args a, FewPlan p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[F_MAX_STAGES], empty[F_MAX_STAGES], acc_full;
  __shared__ uint32_t tmem_slot;
  __shared__ float xs[F_T];
  __shared__ int xsum[F_T];
  uint8_t *ring = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int rank = static_cast<int>(blockIdx.x) % p.split;
  const int tile = static_cast<int>(blockIdx.x) / p.split;
  const int tt = tile % a.n_tt, jt = tile / a.n_tt;
  const int stage_bytes = (F_J + p.bn) * PK;
  const int kb0 = static_cast<int>(static_cast<int64_t>(a.nkb) * rank / p.split);
  const int nkb = static_cast<int>(static_cast<int64_t>(a.nkb) * (rank + 1) / p.split) - kb0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    for (int it = 0; it < p.stages && it < nkb; ++it)
      tma_prefetch_2d(&tmW, (kb0 + it) * PK, jt * F_J);
  }
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) reset_status(a.status);
  if (warp == 1) {
    tmem_alloc(&tmem_slot, static_cast<uint32_t>(p.tmem_cols));
    tmem_relinquish();
  }
  // the epilogue's operands of this output, on their way while the tiles are
  const int64_t j = static_cast<int64_t>(jt) * F_J + threadIdx.x;
  const int64_t t0 = static_cast<int64_t>(tt) * p.bn;
  const int n = a.n_tok - t0 < p.bn ? static_cast<int>(a.n_tok - t0) : p.bn;
  const bool live = j < a.d_out;
  const OutCol o = out_col(a, j, live);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  chain_next();

  bool ok = true;
  if (warp == 0) {
    const bool leader = elect_one();
    const uint32_t base = smem_u32(ring);
    int s = 0;
    uint32_t ph = 1;
    int it = 0;
    for (; it < nkb; ++it) {
      if (!mbar_wait_warp(&empty[s], ph)) { ok = false; break; }
      if (leader) {
        const uint32_t st = base + s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        tma_load_2d(st, &tmW, &full[s], (kb0 + it) * PK, jt * F_J);
        tma_load_2d(st + F_J * PK, &tmX, &full[s], (kb0 + it) * PK, tt * p.bn);
      }
      if (++s == p.stages) {
        s = 0;
        ph ^= 1;
      }
    }
    for (int j = it - 1; j >= 0 && j >= it - p.stages; --j)  // the last loads have landed
      if (!mbar_wait_warp(&full[j % p.stages], (j / p.stages) & 1)) ok = false;
  } else if (warp == 1) {
    const bool leader = elect_one();
    const uint32_t idesc = idesc_s8_s32(F_J, p.bn), dstage = static_cast<uint32_t>(stage_bytes) >> 4;
    const uint64_t dw0 = smem_desc_sw128(smem_u32(ring), 16, 1024);
    int s = 0;
    uint32_t ph = 0;
    for (int it = 0; it < nkb; ++it) {
      if (!mbar_wait_warp(&full[s], ph)) { ok = false; break; }
      tc_fence_after();
      if (leader) {
        const uint64_t dw = dw0 + s * dstage, dx = dw + (F_J * PK >> 4);
        mma_s8(tmem, dw, dx, idesc, it != 0);
#pragma unroll
        for (int kk = 1; kk < PK / 32; ++kk) mma_s8(tmem, dw + 2 * kk, dx + 2 * kk, idesc, 1u);
        mma_commit(&empty[s]);
      }
      if (++s == p.stages) {
        s = 0;
        ph ^= 1;
      }
    }
    if (leader) mma_commit(&acc_full);
  } else if (warp >= 2) {
    for (int c = threadIdx.x - 64; c < n; c += 64) {
      xs[c] = a.xs[t0 + c];
      if (a.wz) xsum[c] = a.xsum[t0 + c];
      if (c % p.split == rank) {       // M and R of the columns that this CTA finishes: to L2
        const int64_t j0 = static_cast<int64_t>(jt) * F_J;
        for (int64_t q = j0; q < j0 + F_J && q < a.d_out; q += 128 / sizeof(T)) {
          if (a.m) prefetch_l2(static_cast<const T *>(a.m) + (t0 + c) * a.d_out + q);
          if (a.r) prefetch_l2(static_cast<const T *>(a.r) + (t0 + c) * a.d_out + q);
        }
      }
    }
  }
  __syncthreads();
  if (!__all_sync(0xffffffffu, mbar_wait(&acc_full, 0))) ok = false;
  tc_fence_after();

  const uint32_t taddr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  if (p.split == 1) {
    for (int c0 = 0; c0 < n; c0 += 32) {
      float v[32];
      tmem_ld32(taddr + c0, v);
      int acc[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[i] = __float_as_int(v[i]);
      few_columns<T, 32>(a, o, live, t0, c0, 1, n, j, xs, xsum, acc);
    }
    tc_fence_before();
    __syncthreads();
  } else {
    // every load of this CTA has landed and every MMA has read the ring
    int *sums = reinterpret_cast<int *>(ring);
    for (int c0 = 0; c0 < n; c0 += 32) {
      float v[32];
      tmem_ld32(taddr + c0, v);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c0 + i < n) sums[(c0 + i) * F_J + threadIdx.x] = __float_as_int(v[i]);
    }
    tc_fence_before();
    cluster_sync();
    for (int c0 = rank; c0 < n; c0 += 16 * p.split) {
      int acc[16] = {};
#pragma unroll 2
      for (int r = 0; r < p.split; ++r) {
        const uint32_t base = mapa_shared(smem_u32(sums + threadIdx.x), r);
        int part[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          part[i] = c0 + i * p.split < n ? ld_cluster_s32(base + (c0 + i * p.split) * (F_J * 4)) : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] += part[i];
      }
      few_columns<T, 16>(a, o, live, t0, c0, p.split, n, j, xs, xsum, acc);
    }
    cluster_sync();  // no CTA leaves while another reads its sums
  }
  if (!ok) set_status(a.status, kDevTimeout);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, static_cast<uint32_t>(p.tmem_cols));
  }
}

// ---------------------------------------------------------------- one to eight tokens
// A warp reads V_R = 4 or 8 output rows 512 bytes at a time (16 per lane, two
// to four steps in flight) straight from global memory and multiplies them
// with NT tokens by dp4a; `ks` warps of a block share a row group along K and
// add up through shared memory.  No barriers, no TMEM and no tensor maps to set up: the
// weights' bytes and one memory round trip are all there is.  HBM-bound: one
// token 4096 -> 11008 9.5 us of 6.9 at the copy rate, 8192 -> 28672 36.5 of
// 35.9, 768 -> 2304 2.1 us.  The
// first steps' weights start towards L2 before the stream's earlier work is
// done (whose results they may be: nothing is read yet): behind a token's norm
// 11.5 us instead of 12.3, 768 -> 2304 3.9 instead of 4.1.
constexpr int V_WARPS = 4;

__device__ __forceinline__ int4 ld_stream(const int8_t *p) {  // (not .nc: see chain_wait)
  int4 v;
  asm volatile("ld.global.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

template <typename T, int NT, int V_R>
__global__ void __launch_bounds__(V_WARPS * 32) w8a8_vec_kernel(W8Args a, int ks) {
  __shared__ int part[V_WARPS][V_R * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = V_WARPS / ks, kp = warp % ks, grp = warp / ks;
  const int64_t j0 = (static_cast<int64_t>(blockIdx.x) * groups + grp) * V_R;
  constexpr int ST = NT == 1 ? 16 / V_R : 2;   // steps in flight
  if (kp == 0 && lane < V_R && j0 + lane < a.d_out)
    prefetch_l2(a.w + (j0 + lane) * a.d_in, a.d_in < ST * ks * 512 ? a.d_in : ST * ks * 512);
  chain_wait();
  chain_next();
  if (blockIdx.x == 0 && threadIdx.x == 0) reset_status(a.status);
  int acc[V_R][NT] = {};
  const int8_t *w[V_R];
#pragma unroll
  for (int r = 0; r < V_R; ++r)  // rows past the end read the last one again
    w[r] = a.w + (j0 + r < a.d_out ? j0 + r : a.d_out - 1) * a.d_in;
  const int stride = ks * 512;
  for (int k = kp * 512 + lane * 16; k < a.d_in; k += ST * stride) {
    int4 wv[ST][V_R], xv[ST][NT];
#pragma unroll
    for (int u = 0; u < ST; ++u) {
      const int ku = k + u * stride;
      if (ku < a.d_in) {
#pragma unroll
        for (int r = 0; r < V_R; ++r) wv[u][r] = ld_stream(w[r] + ku);
      } else {
#pragma unroll
        for (int r = 0; r < V_R; ++r) wv[u][r] = make_int4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int u = 0; u < ST; ++u) {
      const int ku = k + u * stride;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        xv[u][t] = ku < a.d_in
                       ? *reinterpret_cast<const int4 *>(a.x + static_cast<int64_t>(t) * a.d_in + ku)
                       : make_int4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < ST; ++u)
#pragma unroll
      for (int r = 0; r < V_R; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          acc[r][t] = __dp4a(wv[u][r].x, xv[u][t].x, acc[r][t]);
          acc[r][t] = __dp4a(wv[u][r].y, xv[u][t].y, acc[r][t]);
          acc[r][t] = __dp4a(wv[u][r].z, xv[u][t].z, acc[r][t]);
          acc[r][t] = __dp4a(wv[u][r].w, xv[u][t].w, acc[r][t]);
        }
  }
#pragma unroll
  for (int r = 0; r < V_R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int v = __reduce_add_sync(0xffffffffu, acc[r][t]);
      if (lane == 0) part[warp][r * NT + t] = v;
    }
  __syncthreads();
  // thread (group, token, row): one output
  const int i = threadIdx.x;
  if (i < groups * V_R * NT) {
    const int r = i % V_R, g = i / V_R % groups, t = i / (V_R * groups);
    const int64_t j = (static_cast<int64_t>(blockIdx.x) * groups + g) * V_R + r;
    if (j < a.d_out) {
      int sum = 0;
      for (int q = 0; q < ks; ++q) sum += part[g * ks + q][r * NT + t];
      const int64_t at = t * a.d_out + j;
      from_f(finish(a, out_col(a, j, true), sum, a.xs[t], a.wz ? a.xsum[t] : 0,
                    a.m ? to_f(static_cast<const T *>(a.m)[at]) : 0.0f,
                    a.r ? to_f(static_cast<const T *>(a.r)[at]) : 0.0f),
             static_cast<T *>(a.y)[at]);
    }
  }
}

template <typename T>
constexpr CUtensorMapDataType tmap_type() {
  return sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

template <typename T, int PJ, bool TMA>
gq_status launch_pair_as(W8Args a, int pj, cudaStream_t st) {
  using S = PairShape<PJ, TMA>;
  static SmemOptIn opt;
  CUtensorMap tX, tW, tY{};
  gq_status s = make_tmap_2d(&tX, a.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.d_in, a.n_tok, a.d_in, PK, 128);
  if (s == GQ_OK)
    s = make_tmap_2d(&tW, a.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.d_in, a.d_out, a.d_in, PK, pj / 2);
  if (s == GQ_OK && TMA)
    s = make_tmap_2d(&tY, a.y, tmap_type<T>(), sizeof(T), a.d_out, a.n_tok, a.d_out, 64 / sizeof(T),
                     32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (s != GQ_OK) return s;
  a.n_tt = static_cast<int>((a.n_tok + PT - 1) / PT);
  a.n_jt = static_cast<int>((a.d_out + pj - 1) / pj);
  a.pj = pj;
  a.nkb = (a.d_in + PK - 1) / PK;
  const int tiles = a.n_tt * a.n_jt, pairs = num_sms() / 2;
  opt.allow(w8a8_pair_kernel<T, PJ, TMA>, S::kSmem);
  const int slot = timer_begin(GQ_KERNEL_W8A8, st);
  const cudaError_t e = launch_chained(w8a8_pair_kernel<T, PJ, TMA>, 2 * (tiles < pairs ? tiles : pairs),
                                       S::kThreads, S::kSmem, st, 2, tX, tW, tY, a);
  count_launch();
  timer_end(slot, st, 2.0 * static_cast<double>(a.n_tok) * a.d_out * a.d_in);
  return launched(e, "w8a8_pair_kernel");
}

// Whether rows of Y (and of M and R) are a multiple of 16 bytes long.
template <typename T>
bool whole_rows(const W8Args &a) {
  return a.d_out * sizeof(T) % 16 == 0;
}
template <typename T, int PJ>
gq_status launch_pair(const W8Args &a, int pj, cudaStream_t st) {
  if constexpr (sizeof(T) == 4 && PJ == 256)          // (ragged fp32 rows: 128 or few tiles)
    return launch_pair_as<T, PJ, true>(a, pj, st);
  else
    return whole_rows<T>(a) ? launch_pair_as<T, PJ, true>(a, pj, st) : launch_pair_as<T, PJ, false>(a, pj, st);
}

// CTAs per tile: the split whose fullest SM has the fewest K steps, the
// smallest such; each CTA keeps at least four steps.  The SM's shared memory
// is divided among the CTAs that it then holds (at most three).  A CTA of a
// split tile holds 72 KB or more: it never shares an SM with a CTA of a
// kernel that takes all of TMEM (their shared memory is above 190 KB), and
// at most three of them, 384 columns, share one, so no cluster waits for
// TMEM columns while it holds some that another cluster waits for.
FewPlan few_plan(int64_t n_tok, int64_t d_out, int nkb, int &n_tt, int &n_jt) {
  FewPlan p;
  n_tt = static_cast<int>((n_tok + F_T - 1) / F_T);
  const int64_t per = (n_tok + n_tt - 1) / n_tt;
  p.bn = static_cast<int>((per + 15) / 16 * 16);
  n_jt = static_cast<int>((d_out + F_J - 1) / F_J);
  const int64_t tiles = static_cast<int64_t>(n_tt) * n_jt;
  const int sms = num_sms();
  int64_t best = INT64_MAX, per_sm = 1;
  p.split = 1;
  for (int c = 1; c <= 8 && (c == 1 || nkb >= 4 * c); ++c) {
    const int64_t held = (tiles * c + sms - 1) / sms;
    if (c > 1 && held > 2) break;
    // (larger clusters do not fill the last SMs: 384 x 4096 x 4096 in threes,
    // 288 CTAs in 296 places, 30 us, unsplit 15)
    if (c > 2 && 10 * tiles * c > 9 * held * sms) continue;
    const int64_t cost = held * ((nkb + c - 1) / c);
    if (cost < best) {
      best = cost;
      p.split = c;
      per_sm = held;
    }
  }
  p.steps = static_cast<int>(best < INT32_MAX ? best : INT32_MAX);
  p.held = static_cast<int>(per_sm < INT32_MAX ? per_sm : INT32_MAX);
  const int stage = (F_J + p.bn) * PK;
  const int kb = per_sm == 1 ? 216 : per_sm == 2 ? 108 : 72;
  p.stages = kb * 1024 / stage;
  if (p.stages > F_MAX_STAGES) p.stages = F_MAX_STAGES;
  const int most = (nkb + p.split - 1) / p.split;
  // a split tile's sums lie in the ring, which is at least 72 KB then
  static_assert(F_T * F_J * 4 <= 72 * 1024, "the sums of a tile fit the ring");
  const int need = p.split > 1 ? (72 * 1024 + stage - 1) / stage : 1;
  if (p.stages > most) p.stages = most;
  if (p.stages < need) p.stages = need;
  p.tmem_cols = 32;
  while (p.tmem_cols < p.bn) p.tmem_cols *= 2;
  return p;
}

template <typename T>
gq_status launch_few(const W8Args &a, const FewPlan &p, cudaStream_t st) {
  static SmemOptIn opt;
  CUtensorMap tX, tW;
  gq_status s = make_tmap_2d(&tX, a.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.d_in, a.n_tok, a.d_in, PK, p.bn);
  if (s == GQ_OK)
    s = make_tmap_2d(&tW, a.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.d_in, a.d_out, a.d_in, PK, F_J);
  if (s != GQ_OK) return s;
  const size_t smem = 1024 + static_cast<size_t>(p.stages) * (F_J + p.bn) * PK;
  opt.allow(w8a8_few_kernel<T>, 1024 + 216 * 1024);
  const int slot = timer_begin(GQ_KERNEL_W8A8, st);
  const cudaError_t e = launch_chained(w8a8_few_kernel<T>, static_cast<unsigned>(a.n_tt) * a.n_jt * p.split,
                                       F_THREADS, smem, st, p.split, tX, tW, a, p);
  count_launch();
  timer_end(slot, st, 2.0 * static_cast<double>(a.n_tok) * a.d_out * a.d_in);
  return launched(e, "w8a8_few_kernel");
}

template <typename T, int NT, int V_R = 4>
gq_status launch_vec_n(const W8Args &a, cudaStream_t st) {
  // warps along K: while the row groups alone do not fill the SMs
  int ks = 1;
  const int64_t rows = (a.d_out + V_R - 1) / V_R;
  while (ks < V_WARPS && rows * ks < 8 * static_cast<int64_t>(num_sms()) && a.d_in > 512 * ks) ks *= 2;
  const int64_t groups = V_WARPS / ks;
  const int slot = timer_begin(GQ_KERNEL_W8A8, st);
  const cudaError_t e = launch_chained(w8a8_vec_kernel<T, NT, V_R>, static_cast<unsigned>((rows + groups - 1) / groups),
                                       V_WARPS * 32, 0, st, 1, a, ks);
  count_launch();
  timer_end(slot, st, 2.0 * static_cast<double>(a.n_tok) * a.d_out * a.d_in);
  return launched(e, "w8a8_vec_kernel");
}

template <typename T>
gq_status launch_vec(const W8Args &a, cudaStream_t st) {
  switch (a.n_tok) {
    case 1:  // (short rows: 768 -> 50257 9.6 us by eights, 13.7 by fours)
      return a.d_in <= 1024 && a.d_out >= int64_t(64) * num_sms() ? launch_vec_n<T, 1, 8>(a, st)
                                                                  : launch_vec_n<T, 1>(a, st);
    case 2: return launch_vec_n<T, 2>(a, st);
    case 3: return launch_vec_n<T, 3>(a, st);
    case 4: return launch_vec_n<T, 4>(a, st);
    case 5: return launch_vec_n<T, 5>(a, st);
    case 6: return launch_vec_n<T, 6>(a, st);
    case 7: return launch_vec_n<T, 7>(a, st);
    default: return launch_vec_n<T, 8>(a, st);
  }
}

// Expected microseconds of a pair kernel: launch and first loads, the first
// tile's MMAs, a round of tiles per 74 pairs, each bound by its MMAs or by its
// epilogue, and the last epilogue.  Steps of 0.35 (256 outputs) and 0.23 us
// (128): a narrow MMA reads its A tile more often per flop.  `pj`: the tile's
// outputs; 224 instead of 256 where the last round is so poorly filled that as
// many rounds of smaller tiles do (2560 x 2048 x 8192: 320 or 370 tiles, five
// rounds either way, 35.2 or 33.6 us; each epilogue warp keeps 32 outputs or
// more, so no less).
template <typename T, int PJ>
float pair_us(const W8Args &a, int nkb, int &pj) {
  const int64_t n_tt = (a.n_tok + PT - 1) / PT, pairs = num_sms() / 2;
  const bool whole = whole_rows<T>(a), wide = PJ == 256;
  if (!whole && wide && sizeof(T) == 4) return FLT_MAX;
  const float epi_full = sizeof(T) == 4 ? (whole ? (wide ? 4.7f : 3.2f) : 4.0f)
                                        : (whole ? (wide ? 3.8f : 2.5f) : (wide ? 5.5f : 3.8f));
  float best = FLT_MAX;
  for (int c = PJ; c >= (wide ? 224 : PJ); c -= 32) {
    const int64_t tiles = n_tt * ((a.d_out + c - 1) / c);
    const float rounds = static_cast<float>((tiles + pairs - 1) / pairs);
    const float epi = epi_full * static_cast<float>(c) / PJ;
    const float mma = static_cast<float>(nkb) * (0.11f + 0.24f / 256.0f * static_cast<float>(c));
    const float us = 3.5f + mma + (rounds - 1.0f) * (mma > epi ? mma : epi) + epi;
    if (us < best) {
      best = us;
      pj = c;
    }
  }
  return best;
}
// Of the kernel for few tiles: launch and first loads, the weights from HBM or
// the fullest SM's steps, and the epilogues (of tiles that share an SM they
// overlap in part; a split tile's sums are exchanged first).
float few_us(const W8Args &a, const FewPlan &p) {
  const float bn = static_cast<float>(p.bn);
  const float hbm = static_cast<float>(a.d_out) * static_cast<float>(a.d_in) / 6.5e6f;
  const float steps = static_cast<float>(p.steps) * (F_J + bn) * PK / 140e3f;
  return 3.5f + (hbm > steps ? hbm : steps) +
         (p.split > 1 ? 1.5f + 0.06f * bn : 0.035f * bn * (1.0f + 0.45f * static_cast<float>(p.held - 1)));
}

// The kernel is chosen by these estimates; dp4a for one token, and for up to
// eight while the layer is small and its products few.  Measured (us, graph
// replays, weights from HBM, bf16 out; fp32 in the last two lines; the chosen
// one is marked):
//   n    d_in   d_out    dp4a   few    256    128
//   1    4096   11008     9.9*  11.8   24.3   25.8
//   1    28672  8192     36.6*  41.2   82.7   86.0
//   2    8192   8192     18.0   16.7*  30.6   31.1
//   4    4096   4096      6.4*   8.6   14.6   12.6
//   8    4096   4096      9.3*   8.6   14.8   12.9
//   8    2048   8192      9.6*   8.0   11.6   10.7
//   8    8192   2048      9.2*  15.6   22.4   16.2
//   4    12288  2048      8.2*  18.2   30.5   22.8
//   7    5120   5120     14.3*  10.7   17.5   19.5
//   2    768    50257    11.2*   9.7   20.3   26.6
//   5    768    50257    17.8*   9.8   20.3   26.0
//   4    4096   11008    11.3*  12.0   21.9   23.4
//   8    4096   11008    17.1   12.1*  21.0   21.9
//   33   8192   28672       -   44.6*  52.3   58.8
//   64   8192   8192        -   18.9*  26.6   20.2
//   256  8192   8192        -   25.1   27.6   21.7*
//   384  4096   11008       -   22.6*  26.2   24.8
//   512  8192   8192        -   34.7   28.1*  31.4
//   512  4096   11008       -   30.4   26.9*  25.5
//   2048 4096   11008       -  102.5   61.7*  67.8
//   251  768    50257       -   28.9*     -   30.0
//   2048 2048   8191        -   51.3      -   38.8*
// The bounds of dp4a are coarse: from two tokens on its time follows the
// outputs as much as the layer's bytes, and the few-tile kernel's whether its
// clusters run at once (16 to 18 tiles in eights or sevens seem not to), so
// the slower one is taken for some layers, short rows with many outputs above
// all (7 tokens 512 -> 32768: 13.2 us of 6.0).
template <typename T>
gq_status launch_typed(W8Args a, cudaStream_t st) {
  const int64_t layer = a.d_in * a.d_out;
  if (a.n_tok == 1 || (a.n_tok <= 8 && layer < (int64_t(3) << 24) && a.n_tok * layer < (int64_t(3) << 26)))
    return launch_vec<T>(a, st);
  W8Args f = a;
  f.nkb = (a.d_in + PK - 1) / PK;
  const FewPlan p = few_plan(a.n_tok, a.d_out, f.nkb, f.n_tt, f.n_jt);
  const float few = few_us(a, p);
  int pj = 256, pj128 = 128;
  const float wide = pair_us<T, 256>(a, f.nkb, pj), narrow = pair_us<T, 128>(a, f.nkb, pj128);
  if (few <= wide && few <= narrow) return launch_few<T>(f, p, st);
  return wide <= narrow ? launch_pair<T, 256>(a, pj, st) : launch_pair<T, 128>(a, pj128, st);
}

}  // namespace

gq_status launch_w8a8(const int8_t *w_codes, const uint16_t *w_scales, const int32_t *w_zpoint,
                      int64_t d_out, int64_t d_in, const int8_t *x_codes, const float *x_scales,
                      const int32_t *x_sums, int64_t n_tok, const float *bias, int act,
                      const void *M, const void *R, void *Y, gq_dtype y_dtype, int *status,
                      cudaStream_t st) {
  if (n_tok == 0) {
    cudaMemsetAsync(status, 0, sizeof(int), st);
    return check_launch("memset");
  }
  const W8Args a{w_codes, x_codes, w_scales, w_zpoint, x_scales, x_sums, bias, M, R, Y,
                 d_out,   n_tok,   static_cast<int>(d_in), act, status, 0, 0, 0, 0};
  switch (y_dtype) {
    case GQ_F32: return launch_typed<float>(a, st);
    case GQ_F16: return launch_typed<__half>(a, st);
    default: return launch_typed<__nv_bfloat16>(a, st);
  }
}

}  // namespace gq

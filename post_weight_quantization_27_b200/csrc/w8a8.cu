// Product of int8 tokens with a layer held in int8, scales per token and per
// output channel (include/gq.h, "Product of int8 tokens"):
//   Y = act(x_scale w_scale (sum_k x c - zpoint sum_k x) + bias) * M + R.
// The integers are exact in 32 bits: with at most 65536 columns, |sum x c|
// and |zpoint sum x| are at most 128 * 128 * 65536 = 2^30, and their
// difference sum x (c - zpoint) at most 128 * 255 * 65536 < 2^31.  One
// rounding takes it to fp32, where the epilogue works, and one more to the
// output's type.
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
  int y_vec;              // rows of Y, M and R are a multiple of 16 bytes long
  int y_tma;              // .. and Y leaves by TMA
};

// acc - z xsum in two's complement.
__device__ __forceinline__ int sub_wrap(int acc, int z, int xsum) {
  return static_cast<int>(static_cast<uint32_t>(acc) -
                          static_cast<uint32_t>(z) * static_cast<uint32_t>(xsum));
}

__device__ __forceinline__ float act8(float v, int act) {
  if (act == GQ_ACT_RELU) return v < 0.0f ? 0.0f : v;   // keeps NaN
  // v / (1 + e^-w), w = v (SiLU) or 2 u (GELU's tanh form, 0.5 v (1 + tanh
  // u)).  The intrinsics' few ulps (e^-w: 2 + 1.17 |w|) matter where e^-w is
  // near 1; where it is large the value itself vanishes.
  if (act == GQ_ACT_SILU) return __fdividef(v, 1.0f + __expf(-v));
  if (act == GQ_ACT_GELU) {
    const float u = 0.7978845608028654f * fmaf(0.044715f * v, v * v, v);
    return __fdividef(v, 1.0f + __expf(-2.0f * u));
  }
  return v;
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
// zero-point and bias.  The product is taken as (v w_scale) x_scale: |v| <
// 2^31 times an fp16 scale neither overflows nor loses a normal result.
template <typename T>
__device__ __forceinline__ void finish(const W8Args &a, int64_t t, int64_t j, int acc, float ws,
                                       int wz, float bias) {
  if (a.wz) acc = sub_wrap(acc, wz, a.xsum[t]);
  float v = static_cast<float>(acc) * ws * a.xs[t];
  if (a.bias) v += bias;
  v = act8(v, a.act);
  const int64_t i = t * a.d_out + j;
  if (a.m) v *= to_f(static_cast<const T *>(a.m)[i]);
  if (a.r) v += to_f(static_cast<const T *>(a.r)[i]);
  from_f(v, static_cast<T *>(a.y)[i]);
}

// ---------------------------------------------------------------- 32 outputs of a token
// v = the raw integer sums (as bits) -> x_scale w_scale (acc - z xsum) + bias.
__device__ __forceinline__ void scale32(const W8Args &a, const float *s, const int *z,
                                        const float *b, float xs, int xsum, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 s4 = *reinterpret_cast<const float4 *>(s + i);
    const float sv[4] = {s4.x, s4.y, s4.z, s4.w};
    int zv[4] = {0, 0, 0, 0};
    float bv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (a.wz) {
      const int4 z4 = *reinterpret_cast<const int4 *>(z + i);
      zv[0] = z4.x; zv[1] = z4.y; zv[2] = z4.z; zv[3] = z4.w;
    }
    if (a.bias) {
      const float4 b4 = *reinterpret_cast<const float4 *>(b + i);
      bv[0] = b4.x; bv[1] = b4.y; bv[2] = b4.z; bv[3] = b4.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int acc = __float_as_int(v[i + e]);
      if (a.wz) acc = sub_wrap(acc, zv[e], xsum);
      v[i + e] = static_cast<float>(acc) * sv[e] * xs;
      if (a.bias) v[i + e] += bv[e];
    }
  }
}
__device__ __forceinline__ void act32(float (&v)[32], int act) {
  if (act == GQ_ACT_NONE) return;
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = act8(v[i], act);
}
// v = v * M + R for outputs j .. j + 31 of a token; the rows are read 16
// bytes at a time where they are a multiple of 16 bytes long.
template <typename T>
__device__ __forceinline__ void load32(const W8Args &a, const T *p, int64_t j, float (&f)[32]) {
  constexpr int E = 16 / sizeof(T);
  if (a.y_vec) {
#pragma unroll
    for (int i = 0; i < 32; i += E) {
      uint4 u = make_uint4(0u, 0u, 0u, 0u);
      if (j + i < a.d_out) u = *reinterpret_cast<const uint4 *>(p + i);
      const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
      for (int k = 0; k < E; ++k) f[i + k] = to_f(e[k]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = j + i < a.d_out ? to_f(p[i]) : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void mul_add32(const W8Args &a, int64_t row, int64_t j, float (&v)[32]) {
  const int64_t at = row * a.d_out + j;
  if (a.m) {
    float f[32];
    load32<T>(a, static_cast<const T *>(a.m) + at, j, f);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= f[i];
  }
  if (a.r) {
    float f[32];
    load32<T>(a, static_cast<const T *>(a.r) + at, j, f);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += f[i];
  }
}
// 32 values rounded to T into this lane's row of a 32-row box of 128-byte
// rows (16-byte chunk c of row r at c ^ (r % 8)).
__device__ __forceinline__ void stage32(uint8_t *row, int r, int, const float (&v)[32], float) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4 *>(row + ((c ^ (r & 7)) << 4)) =
        make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <typename T>
__device__ __forceinline__ void stage32(uint8_t *row, int r, int sub, const float (&v)[32], T t) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4 u;
    u.x = pack2(v[8 * c], v[8 * c + 1], t);
    u.y = pack2(v[8 * c + 2], v[8 * c + 3], t);
    u.z = pack2(v[8 * c + 4], v[8 * c + 5], t);
    u.w = pack2(v[8 * c + 6], v[8 * c + 7], t);
    *reinterpret_cast<uint4 *>(row + (((4 * sub + c) ^ (r & 7)) << 4)) = u;
  }
}
// A staged box to Y with ordinary stores, a row at a time.
template <typename T>
__device__ __forceinline__ void store_box(const W8Args &a, const uint8_t *stg, int lane,
                                          int64_t row0, int64_t j0) {
  constexpr int CC = 128 / sizeof(T), E = 16 / sizeof(T);
  T *y = static_cast<T *>(a.y) + row0 * a.d_out + j0;
  const int rows = a.n_tok - row0 < 32 ? static_cast<int>(a.n_tok - row0) : 32;
  for (int r = 0; r < rows; ++r) {
#pragma unroll
    for (int c = lane; c < CC; c += 32)
      if (j0 + c < a.d_out)
        y[r * a.d_out + c] = *reinterpret_cast<const T *>(stg + r * 128 + (((c / E) ^ (r & 7)) << 4) +
                                                          (c % E) * sizeof(T));
  }
}

// ---------------------------------------------------------------- many tokens
// 256 (tokens) x 256 (outputs) tiles on CTA pairs (tcgen05 cta_group::2,
// kind::i8), persistent, K in steps of 128 bytes:
//   warp 0      TMA: CTA r of the pair stages the tile's token rows 128 r ..
//               and output rows 128 r .., both CTAs' loads completing on CTA
//               0's full[s] (64 KB a stage)
//   warp 1      CTA 0: four MMAs of M = N = 256, K = 32 a stage into one of
//               two 256-column TMEM accumulators; each CTA receives its 128
//               tokens' rows
//   warps 2-9   epilogue: a thread owns a token, a warp 32 tokens x 128
//               outputs; the columns' scales, zero-points and bias come once
//               per tile through shared memory; results pass a 128-byte-
//               swizzled buffer of the warp's own and leave by TMA store
//               (by coalesced stores where Y's rows are no multiple of 16
//               bytes).
constexpr int PT = 256, PJ = 256, PK = 128, P_STAGES = 5;
constexpr int P_TILE_BYTES = 128 * PK;                 // one operand of one CTA: 16 KB
constexpr int P_STAGE_BYTES = 2 * P_TILE_BYTES;
constexpr int P_STAGING = 4096;                        // per epilogue warp: 32 rows x 128 bytes
constexpr int P_THREADS = 320;
constexpr size_t P_SMEM = 1024 + P_STAGES * P_STAGE_BYTES + 8 * P_STAGING + 2 * PJ * 12 + 256;

struct Cols {              // per-output operands of a tile, in shared memory
  float s[PJ];
  int z[PJ];
  float b[PJ];
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

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P_THREADS, 1)
    w8a8_pair_kernel(const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmY, W8Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *staging = smem + P_STAGES * P_STAGE_BYTES;
  Cols *cols = reinterpret_cast<Cols *>(staging + 8 * P_STAGING);
  uint64_t *full = reinterpret_cast<uint64_t *>(cols + 2);  // CTA 0: both CTAs' loads landed
  uint64_t *empty = full + P_STAGES;                        // per CTA: MMAs done with the stage
  uint64_t *acc_full = empty + P_STAGES;                    // per CTA
  uint64_t *acc_empty = acc_full + 2;                       // CTA 0: 16 epilogue warps
  uint64_t *drain = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x >> 1), n_pairs = static_cast<int>(gridDim.x >> 1);
  const int n_tiles = a.n_tt * a.n_jt;
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) reset_status(a.status);
    for (int s = 0; s < P_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 16);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers initialised and TMEM allocated
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int half0 = static_cast<int>(rank) * 128;  // this CTA's token and output rows in a tile

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      uint32_t it = 0;
      for (int t = pair; t < n_tiles && ok; t += n_pairs) {
        int tt, jt;
        pair_tile(t, a.n_tt, a.n_jt, tt, jt);
        for (int kb = 0; kb < a.nkb; ++kb, ++it) {
          const uint32_t s = it % P_STAGES, r = it / P_STAGES;
          if (!mbar_wait(&empty[s], (r & 1) ^ 1)) { ok = false; break; }
          uint8_t *st = smem + s * P_STAGE_BYTES;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * P_STAGE_BYTES);
          tma_load_2d_pair(st, &tmX, &full[s], kb * PK, tt * PT + half0);
          tma_load_2d_pair(st + P_TILE_BYTES, &tmW, &full[s], kb * PK, jt * PJ + half0);
        }
      }
      if (rank == 0) {  // the last loads of both CTAs have landed
        const uint32_t n_wait = it < P_STAGES ? it : P_STAGES;
        for (uint32_t k = 0; k < n_wait; ++k) {
          const uint32_t j = it - 1 - k;
          if (!mbar_wait(&full[j % P_STAGES], (j / P_STAGES) & 1)) ok = false;
        }
      }
      if (!ok) set_status(a.status, kDevTimeout);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      bool ok = true;
      uint32_t it = 0, ch = 0;
      constexpr uint32_t idesc = idesc_s8_s32(PT, PJ);
      for (int t = pair; t < n_tiles && ok; t += n_pairs, ++ch) {
        const uint32_t buf = ch & 1, use = ch >> 1;
        if (!mbar_wait_cluster(&acc_empty[buf], (use & 1) ^ 1)) { ok = false; break; }
        tc_fence_after();
        for (int kb = 0; kb < a.nkb; ++kb, ++it) {
          const uint32_t s = it % P_STAGES, r = it / P_STAGES;
          if (!mbar_wait_cluster(&full[s], r & 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sx = smem_u32(smem + s * P_STAGE_BYTES), sw = sx + P_TILE_BYTES;
#pragma unroll
          for (int kk = 0; kk < PK / 32; ++kk)
            mma_s8_pair(tmem + buf * PJ, smem_desc_sw128(sx + kk * 32, 16, 1024),
                        smem_desc_sw128(sw + kk * 32, 16, 1024), idesc, (kb | kk) != 0);
          mma_commit_pair(&empty[s], 3);
        }
        if (!ok) break;
        mma_commit_pair(&acc_full[buf], 3);
      }
      mma_commit_pair(drain, 1);
      if (!mbar_wait(drain, 0)) ok = false;
      if (!ok) set_status(a.status, kDevTimeout);
    }
  } else {
    constexpr int CC = 128 / sizeof(T);           // outputs per staged box
    const int ew = warp - 2, quarter = warp & 3, half = ew >> 2;
    uint8_t *stg = staging + ew * P_STAGING;
    uint8_t *stg_row = stg + lane * 128;
    uint32_t ch = 0;
    bool ok = true;
    for (int t = pair; t < n_tiles; t += n_pairs, ++ch) {
      int tt, jt;
      pair_tile(t, a.n_tt, a.n_jt, tt, jt);
      const uint32_t buf = ch & 1, use = ch >> 1;
      Cols &cl = cols[buf];
      {
        // the other buffer may still be read: this one was last read before
        // every warp passed the previous tile's barrier
        const int c = threadIdx.x - 64;
        const int64_t j = static_cast<int64_t>(jt) * PJ + c;
        const bool in = j < a.d_out;
        cl.s[c] = in ? __half2float(__ushort_as_half(a.ws[j])) : 0.0f;
        cl.z[c] = in && a.wz ? a.wz[j] : 0;
        cl.b[c] = in && a.bias ? a.bias[j] : 0.0f;
      }
      const int64_t row0 = static_cast<int64_t>(tt) * PT + half0 + quarter * 32;
      const int64_t row = row0 + lane;
      const bool live = row < a.n_tok;
      const float xs = live ? a.xs[row] : 0.0f;
      const int xsum = live && a.wz ? a.xsum[row] : 0;
      named_bar_sync(1, 256);
      // (a warp whose wait gave up keeps meeting the others at the barrier)
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], use & 1));
      if (!ok) continue;
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * PJ + half * 128;
#pragma unroll 1
      for (int b = 0; b < 128 / CC; ++b) {
        const int c0 = half * 128 + b * CC;                       // column in the tile
        const int64_t j0 = static_cast<int64_t>(jt) * PJ + c0;
        if (a.y_tma) {
          if (lane == 0) bulk_wait_group_read0();
          __syncwarp();
        }
#pragma unroll
        for (int sub = 0; sub < CC / 32; ++sub) {
          float v[32];
          tmem_ld32(taddr + b * CC + sub * 32, v);
          scale32(a, cl.s + c0 + sub * 32, cl.z + c0 + sub * 32, cl.b + c0 + sub * 32, xs, xsum, v);
          act32(v, a.act);
          if (live) mul_add32<T>(a, row, j0 + sub * 32, v);
          stage32(stg_row, lane, sub, v, T());
        }
        if (b == 128 / CC - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(&acc_empty[buf], 0);
        }
        if (a.y_tma) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && j0 < a.d_out && row0 < a.n_tok) {
            tma_store_2d(&tmY, stg, static_cast<int32_t>(j0), static_cast<int32_t>(row0));
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          store_box<T>(a, stg, lane, row0, j0);
          __syncwarp();
        }
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
    tmem_dealloc_pair(tmem, 512);
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
// whatever d_out is.
constexpr int F_J = 128, F_T = 128, F_MAX_STAGES = 8, F_THREADS = 128;

struct FewPlan {
  int bn;            // tokens per tile, a multiple of 16
  int stages, split;
  int tmem_cols;
};

__device__ __forceinline__ int ld_cluster_s32(uint32_t saddr, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(saddr, rank)) : "memory");
  return v;
}

template <typename T>
__global__ void __launch_bounds__(F_THREADS)
    w8a8_few_kernel(const __grid_constant__ CUtensorMap tmX,
                    const __grid_constant__ CUtensorMap tmW, W8Args a, FewPlan p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[F_MAX_STAGES], empty[F_MAX_STAGES], acc_full;
  __shared__ uint32_t tmem_slot;
  uint8_t *ring = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % p.split;
  const int tile = static_cast<int>(blockIdx.x) / p.split;
  const int tt = tile % a.n_tt, jt = tile / a.n_tt;
  const int stage_bytes = (F_J + p.bn) * PK;
  const int kb0 = static_cast<int>(static_cast<int64_t>(a.nkb) * rank / p.split);
  const int nkb = static_cast<int>(static_cast<int64_t>(a.nkb) * (rank + 1) / p.split) - kb0;
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) reset_status(a.status);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, static_cast<uint32_t>(p.tmem_cols));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  bool ok = true;
  if (warp == 0 && lane == 0) {
    int it = 0;
    for (; it < nkb; ++it) {
      const int s = it % p.stages, r = it / p.stages;
      if (!mbar_wait(&empty[s], (r & 1) ^ 1)) { ok = false; break; }
      uint8_t *st = ring + s * stage_bytes;
      mbar_arrive_expect_tx(&full[s], stage_bytes);
      tma_load_2d(st, &tmW, &full[s], (kb0 + it) * PK, jt * F_J);
      tma_load_2d(st + F_J * PK, &tmX, &full[s], (kb0 + it) * PK, tt * p.bn);
    }
    for (int j = it - 1; j >= 0 && j >= it - p.stages; --j)  // the last loads have landed
      if (!mbar_wait(&full[j % p.stages], (j / p.stages) & 1)) ok = false;
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_s8_s32(F_J, p.bn);
    for (int it = 0; it < nkb; ++it) {
      const int s = it % p.stages, r = it / p.stages;
      if (!mbar_wait(&full[s], r & 1)) { ok = false; break; }
      tc_fence_after();
      const uint32_t sw = smem_u32(ring + s * stage_bytes), sx = sw + F_J * PK;
#pragma unroll
      for (int kk = 0; kk < PK / 32; ++kk)
        mma_s8(tmem, smem_desc_sw128(sw + kk * 32, 16, 1024), smem_desc_sw128(sx + kk * 32, 16, 1024),
               idesc, (it | kk) != 0);
      mma_commit(&empty[s]);
    }
    mma_commit(&acc_full);
  }
  __syncwarp();
  if (!__all_sync(0xffffffffu, mbar_wait(&acc_full, 0))) ok = false;
  tc_fence_after();

  const int64_t j = static_cast<int64_t>(jt) * F_J + threadIdx.x;
  const int64_t t0 = static_cast<int64_t>(tt) * p.bn;
  const int n = a.n_tok - t0 < p.bn ? static_cast<int>(a.n_tok - t0) : p.bn;
  const uint32_t taddr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  const bool live = j < a.d_out;
  const float ws = live ? __half2float(__ushort_as_half(a.ws[j])) : 0.0f;
  const int wz = live && a.wz ? a.wz[j] : 0;
  const float bias = live && a.bias ? a.bias[j] : 0.0f;
  if (p.split == 1) {
    for (int c0 = 0; c0 < n; c0 += 32) {
      float v[32];
      tmem_ld32(taddr + c0, v);
      if (live) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c0 + i < n) finish<T>(a, t0 + c0 + i, j, __float_as_int(v[i]), ws, wz, bias);
      }
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
    if (live) {
      for (int c = rank; c < n; c += p.split) {
        const uint32_t at = smem_u32(sums + c * F_J + threadIdx.x);
        int part[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) part[r] = r < p.split ? ld_cluster_s32(at, r) : 0;
        int acc = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r) acc += part[r];
        finish<T>(a, t0 + c, j, acc, ws, wz, bias);
      }
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

// Opts a kernel in to its shared memory, once per device.
template <typename K>
void allow_smem(K kernel, size_t bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes)) == cudaSuccess)
    done.fetch_or(bit, std::memory_order_relaxed);
}

template <typename T>
constexpr CUtensorMapDataType tmap_type() {
  return sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

template <typename T>
gq_status launch_pair(W8Args a, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  CUtensorMap tX, tW, tY{};
  gq_status s = make_tmap_2d(&tX, a.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.d_in, a.n_tok, a.d_in, PK, 128);
  if (s == GQ_OK)
    s = make_tmap_2d(&tW, a.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.d_in, a.d_out, a.d_in, PK, 128);
  if (s == GQ_OK && a.y_vec)
    s = make_tmap_2d(&tY, a.y, tmap_type<T>(), sizeof(T), a.d_out, a.n_tok, a.d_out, 128 / sizeof(T), 32);
  if (s != GQ_OK) return s;
  a.y_tma = a.y_vec;
  a.n_tt = static_cast<int>((a.n_tok + PT - 1) / PT);
  a.n_jt = static_cast<int>((a.d_out + PJ - 1) / PJ);
  a.nkb = (a.d_in + PK - 1) / PK;
  const int tiles = a.n_tt * a.n_jt, pairs = num_sms() / 2;
  allow_smem(w8a8_pair_kernel<T>, P_SMEM, done);
  const int slot = timer_begin(GQ_KERNEL_W8A8, st);
  w8a8_pair_kernel<T><<<2 * (tiles < pairs ? tiles : pairs), P_THREADS, P_SMEM, st>>>(tX, tW, tY, a);
  count_launch();
  timer_end(slot, st, 2.0 * static_cast<double>(a.n_tok) * a.d_out * a.d_in);
  return check_launch("w8a8_pair_kernel");
}

// Clusters of CTAs per tile: enough of them for two CTAs per SM, each with
// at least four K steps.  A CTA of a split tile so holds four stages or its
// share of 108 KB, 72 KB and more: it never shares an SM with a CTA of a
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
  p.split = 1;
  while (p.split < 8 && tiles * p.split * 2 <= 2 * num_sms() + num_sms() / 2 && nkb >= 8 * p.split) p.split *= 2;
  const int stage = (F_J + p.bn) * PK;
  p.stages = (108 * 1024) / stage;
  if (p.stages > F_MAX_STAGES) p.stages = F_MAX_STAGES;
  const int most = (nkb + p.split - 1) / p.split;
  const int need = p.split > 1 ? (p.bn * F_J * 4 + stage - 1) / stage : 1;
  if (p.stages > most) p.stages = most > need ? most : need;
  p.tmem_cols = 32;
  while (p.tmem_cols < p.bn) p.tmem_cols *= 2;
  return p;
}

template <typename T>
gq_status launch_few(W8Args a, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  a.nkb = (a.d_in + PK - 1) / PK;
  const FewPlan p = few_plan(a.n_tok, a.d_out, a.nkb, a.n_tt, a.n_jt);
  CUtensorMap tX, tW;
  gq_status s = make_tmap_2d(&tX, a.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.d_in, a.n_tok, a.d_in, PK, p.bn);
  if (s == GQ_OK)
    s = make_tmap_2d(&tW, a.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.d_in, a.d_out, a.d_in, PK, F_J);
  if (s != GQ_OK) return s;
  const size_t smem = 1024 + static_cast<size_t>(p.stages) * (F_J + p.bn) * PK;
  allow_smem(w8a8_few_kernel<T>, 1024 + 108 * 1024, done);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_tt) * a.n_jt * p.split);
  cfg.blockDim = dim3(F_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  const int slot = timer_begin(GQ_KERNEL_W8A8, st);
  cudaLaunchKernelEx(&cfg, w8a8_few_kernel<T>, tX, tW, a, p);
  count_launch();
  timer_end(slot, st, 2.0 * static_cast<double>(a.n_tok) * a.d_out * a.d_in);
  return check_launch("w8a8_few_kernel");
}

template <typename T>
gq_status launch_typed(W8Args a, cudaStream_t st) {
  a.y_vec = a.d_out * sizeof(T) % 16 == 0;
  if (a.n_tok > 256) return launch_pair<T>(a, st);
  return launch_few<T>(a, st);
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
                 d_out,   n_tok,   static_cast<int>(d_in), act, status, 0, 0, 0, 0, 0};
  switch (y_dtype) {
    case GQ_F32: return launch_typed<float>(a, st);
    case GQ_F16: return launch_typed<__half>(a, st);
    default: return launch_typed<__nv_bfloat16>(a, st);
  }
}

}  // namespace gq

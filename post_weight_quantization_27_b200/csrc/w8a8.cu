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

// One output element.  The product is taken as (v w_scale) x_scale: |v| <
// 2^31 times an fp16 scale neither overflows nor loses a normal result.
template <typename T>
__device__ __forceinline__ void finish(const W8Args &a, int64_t t, int64_t j, int acc) {
  if (a.wz) acc = sub_wrap(acc, a.wz[j], a.xsum[t]);
  float v = static_cast<float>(acc) * __half2float(__ushort_as_half(a.ws[j])) * a.xs[t];
  if (a.bias) v += a.bias[j];
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

// 64 x 64 outputs per block of 256 threads, 4 x 4 per thread, K in steps of
// 64 bytes through shared memory.
template <typename T>
__global__ void __launch_bounds__(256) w8a8_tile_kernel(W8Args a) {
  __shared__ int sx[64][17], sw[64][17];
  const int64_t j0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int lr = threadIdx.x >> 2, lc = threadIdx.x & 3;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.y) * 64; t0 < a.n_tok;
       t0 += static_cast<int64_t>(gridDim.y) * 64) {
    int acc[4][4] = {};
    for (int k0 = 0; k0 < a.d_in; k0 += 64) {
      int4 vx = make_int4(0, 0, 0, 0), vw = vx;
      const int k = k0 + lc * 16;
      if (k < a.d_in && t0 + lr < a.n_tok)
        vx = *reinterpret_cast<const int4 *>(a.x + (t0 + lr) * a.d_in + k);
      if (k < a.d_in && j0 + lr < a.d_out)
        vw = *reinterpret_cast<const int4 *>(a.w + (j0 + lr) * a.d_in + k);
      __syncthreads();
      sx[lr][lc * 4] = vx.x; sx[lr][lc * 4 + 1] = vx.y;
      sx[lr][lc * 4 + 2] = vx.z; sx[lr][lc * 4 + 3] = vx.w;
      sw[lr][lc * 4] = vw.x; sw[lr][lc * 4 + 1] = vw.y;
      sw[lr][lc * 4 + 2] = vw.z; sw[lr][lc * 4 + 3] = vw.w;
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < 16; ++kk) {
        int xv[4], wv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xv[i] = sx[ty + 16 * i][kk];
          wv[i] = sw[tx + 16 * i][kk];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xv[i], wv[j], acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = t0 + ty + 16 * i, jj = j0 + tx + 16 * j;
        if (t < a.n_tok && jj < a.d_out) finish<T>(a, t, jj, acc[i][j]);
      }
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

template <typename T>
gq_status launch_typed(W8Args a, cudaStream_t st) {
  a.y_vec = a.d_out * sizeof(T) % 16 == 0;
  if (a.n_tok > 128) return launch_pair<T>(a, st);
  const int64_t rows = (a.n_tok + 63) / 64;
  const dim3 grid(static_cast<unsigned>((a.d_out + 63) / 64),
                  static_cast<unsigned>(rows < 65535 ? rows : 65535));
  const int slot = timer_begin(GQ_KERNEL_W8A8, st);
  w8a8_tile_kernel<T><<<grid, 256, 0, st>>>(a);
  count_launch();
  timer_end(slot, st, 2.0 * static_cast<double>(a.n_tok) * a.d_out * a.d_in);
  return check_launch("w8a8_tile_kernel");
}

}  // namespace

gq_status launch_w8a8(const int8_t *w_codes, const uint16_t *w_scales, const int32_t *w_zpoint,
                      int64_t d_out, int64_t d_in, const int8_t *x_codes, const float *x_scales,
                      const int32_t *x_sums, int64_t n_tok, const float *bias, int act,
                      const void *M, const void *R, void *Y, gq_dtype y_dtype, int *status,
                      cudaStream_t st) {
  if (cudaMemsetAsync(status, 0, sizeof(int), st) != cudaSuccess) return check_launch("memset");
  if (n_tok == 0) return GQ_OK;
  const W8Args a{w_codes, x_codes, w_scales, w_zpoint, x_scales, x_sums, bias, M, R, Y,
                 d_out,   n_tok,   static_cast<int>(d_in), act, status, 0, 0, 0, 0, 0};
  switch (y_dtype) {
    case GQ_F32: return launch_typed<float>(a, st);
    case GQ_F16: return launch_typed<__half>(a, st);
    default: return launch_typed<__nv_bfloat16>(a, st);
  }
}

}  // namespace gq

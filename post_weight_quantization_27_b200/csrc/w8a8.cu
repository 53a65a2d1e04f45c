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
};

__device__ __forceinline__ float act8(float v, int act) {
  if (act == GQ_ACT_RELU) return v < 0.0f ? 0.0f : v;   // keeps NaN
  if (act == GQ_ACT_SILU) return v / (1.0f + expf(-v));
  if (act == GQ_ACT_GELU) {
    const float u = 0.7978845608028654f * fmaf(0.044715f * v, v * v, v);
    return v / (1.0f + expf(-2.0f * u));
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
  if (a.wz) acc = static_cast<int>(static_cast<uint32_t>(acc) - static_cast<uint32_t>(a.wz[j]) * static_cast<uint32_t>(a.xsum[t]));
  float v = static_cast<float>(acc) * __half2float(__ushort_as_half(a.ws[j])) * a.xs[t];
  if (a.bias) v += a.bias[j];
  v = act8(v, a.act);
  const int64_t i = t * a.d_out + j;
  if (a.m) v *= to_f(static_cast<const T *>(a.m)[i]);
  if (a.r) v += to_f(static_cast<const T *>(a.r)[i]);
  from_f(v, static_cast<T *>(a.y)[i]);
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

template <typename T>
gq_status launch_typed(const W8Args &a, cudaStream_t st) {
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
                 d_out,   n_tok,   static_cast<int>(d_in), act, status};
  switch (y_dtype) {
    case GQ_F32: return launch_typed<float>(a, st);
    case GQ_F16: return launch_typed<__half>(a, st);
    default: return launch_typed<__nv_bfloat16>(a, st);
  }
}

}  // namespace gq

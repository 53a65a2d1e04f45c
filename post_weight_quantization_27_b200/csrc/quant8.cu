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
  int norm;
  float eps;
};

// 8 consecutive elements as fp32.
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __half *p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4 *>(p);
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4 *>(p);
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
// 8 values rounded to T (and the rounded values back in v).
__device__ __forceinline__ void store8(float *p, float (&v)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__half *p, float (&v)[8]) {
  __align__(16) __half t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = __float2half_rn(v[i]);
    v[i] = __half2float(t[i]);
  }
  *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(t);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, float (&v)[8]) {
  __align__(16) __nv_bfloat16 t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = __float2bfloat16_rn(v[i]);
    v[i] = __bfloat162float(t[i]);
  }
  *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(t);
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *red) {
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) v = max(v, red[i]);
  return v;
}
template <typename S>
__device__ __forceinline__ S block_sum(S v, S *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) v += red[i];
  return v;
}

// 1 / sqrt(mean h^2 + eps) of one row.
__device__ __forceinline__ float inv_rms(float ssq, int d, float eps) {
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(ssq, static_cast<float>(d)), eps)));
}

// One block per row, two passes over it.
template <typename T, typename WT>
__global__ void __launch_bounds__(256) quant_rows_kernel(QuantArgs a) {
  __shared__ uint32_t red_u[8];
  __shared__ float red_f[8];
  __shared__ double red_d[8];
  __shared__ int red_i[8];
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T *>(a.x) + row * a.ldx;
  const T *r = a.r ? static_cast<const T *>(a.r) + row * a.d_in : nullptr;
  T *h = a.h ? static_cast<T *>(a.h) + row * a.d_in : nullptr;
  const WT *w = static_cast<const WT *>(a.w);
  uint32_t top = 0;
  float ssq = 0.0f;
  for (int c = threadIdx.x * 8; c < a.d_in; c += 2048) {
    float v[8], f[8];
    load8(x + c, v);
    if (r) {
      load8(r + c, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __fadd_rn(v[i], f[i]);
      store8(h + c, v);
    }
    if (w) load8(w + c, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ssq = fmaf(v[i], v[i], ssq);
      const float g = w ? __fmul_rn(v[i], f[i]) : v[i];
      top = max(top, __float_as_uint(g) & 0x7fffffffu);
    }
  }
  top = block_max(top, red_u);
  const bool bad = top >= 0x7f800000u;
  const float amax = __uint_as_float(top);
  float s = __fdiv_rn(amax, 127.0f);
  if (s == 0.0f) s = 1.0f;
  if (a.norm) ssq = block_sum(ssq, red_f);
  const T *src = h ? h : x;
  double ssq64 = 0.0;
  const bool lost = a.norm && !(ssq >= 1e-30f && ssq <= FLT_MAX);
  int sum = 0;
  for (int c = threadIdx.x * 8; c < a.d_in; c += 2048) {
    float v[8], f[8];
    load8(src + c, v);
    if (lost) {
#pragma unroll
      for (int i = 0; i < 8; ++i) ssq64 += static_cast<double>(v[i]) * v[i];
    }
    if (w) load8(w + c, f);
    __align__(8) int8_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float g = w ? __fmul_rn(v[i], f[i]) : v[i];
      const int k = bad ? 0 : static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(g, s)), -127.0f), 127.0f));
      q[i] = static_cast<int8_t>(k);
      sum += k;
    }
    *reinterpret_cast<uint2 *>(a.codes + row * a.d_in + c) = *reinterpret_cast<const uint2 *>(q);
  }
  if (a.sums) sum = block_sum(sum, red_i);
  if (lost) ssq64 = block_sum(ssq64, red_d);
  if (threadIdx.x == 0) {
    if (a.norm)
      s = __fmul_rn(s, lost ? static_cast<float>(1.0 / sqrt(ssq64 / a.d_in + a.eps))
                            : inv_rms(ssq, a.d_in, a.eps));
    a.scales[row] = bad ? __uint_as_float(0x7fc00000u) : s;
    if (a.sums) a.sums[row] = sum;
  }
}

template <typename T, typename WT>
gq_status launch_rows(const QuantArgs &a, cudaStream_t st) {
  const int slot = timer_begin(GQ_KERNEL_QUANT_INT8, st);
  quant_rows_kernel<T, WT><<<static_cast<unsigned>(a.n_tok), 256, 0, st>>>(a);
  count_launch();
  timer_end(slot, st,
            static_cast<double>(a.n_tok) *
                    (static_cast<double>(a.d_in) * (sizeof(T) * (a.r ? 3 : 1) + 1) + 4 +
                     (a.sums ? 4 : 0)) +
                (a.w ? static_cast<double>(a.d_in) * sizeof(WT) : 0.0));
  return check_launch("quant_rows_kernel");
}

// 16 codes per thread from the packed bit stream.
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
  const QuantArgs a{X,    R,    w,     H,   codes, scales, sums, n_tok, ldx, static_cast<int>(d_in),
                    norm, eps};
  switch (dt) {
    case GQ_F32: return launch_rows<float, float>(a, st);
    case GQ_F16:
      return w_dtype == GQ_F32 ? launch_rows<__half, float>(a, st)
                               : launch_rows<__half, __half>(a, st);
    default:
      return w_dtype == GQ_F32 ? launch_rows<__nv_bfloat16, float>(a, st)
                               : launch_rows<__nv_bfloat16, __nv_bfloat16>(a, st);
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

// q8_common.cuh -- the 8-bit codes of the quantised slot cache, shared by the
// kernels that write it (q8_cache.cu) and the decode step (q8_decode.cu).
//
// A block of `block` consecutive slots of one head has one fp32 scale a for K and
// one for V; the value of a code c is c a.  With top the largest code value:
//     a = max(max|x| / top, 2^-126),   c = rne(x * (1 / a)),
// each step one fp32 operation rounded to nearest (the floor keeps 1 / a finite
// for blocks of zeros and subnormals).  |x - c a| is then at most half a code step
// (int8: a / 2; e4m3: 2^-4 |x|, or half its smallest step 2^-10 a) up to fp32 rounding.
#pragma once

#include <cuda_fp8.h>

#include <cfloat>

#include "kvc_internal.cuh"

namespace kvc {

template <int FMT> struct Q8;

template <> struct Q8<KV_Q8_S8> {
  static constexpr float kTop = 127.f;
  __device__ __forceinline__ static uint32_t pack4(float a, float b, float c, float d) {
    const int i0 = max(-127, min(127, __float2int_rn(a))), i1 = max(-127, min(127, __float2int_rn(b)));
    const int i2 = max(-127, min(127, __float2int_rn(c))), i3 = max(-127, min(127, __float2int_rn(d)));
    return (uint32_t)(i0 & 255) | ((uint32_t)(i1 & 255) << 8) | ((uint32_t)(i2 & 255) << 16) |
           ((uint32_t)i3 << 24);
  }
  __device__ __forceinline__ static void unpack4(uint32_t w, float *out) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = (float)(int8_t)(w >> (8 * i));
  }
};

template <> struct Q8<KV_Q8_E4M3> {
  static constexpr float kTop = 448.f;
  __device__ __forceinline__ static uint32_t pack4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
  __device__ __forceinline__ static void unpack4(uint32_t w, float *out) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
    out[0] = a.x;
    out[1] = a.y;
    out[2] = b.x;
    out[3] = b.y;
  }
};

// The scale of a block whose largest magnitude is `big`.
template <int FMT>
__device__ __forceinline__ float q8_scale(float big) {
  return fmaxf(__fdiv_rn(big, Q8<FMT>::kTop), FLT_MIN);
}

// 16 values as one vector of codes; inv = 1 / scale.
template <int FMT>
__device__ __forceinline__ uint4 q8_pack16(const float (&x)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = Q8<FMT>::pack4(__fmul_rn(x[4 * i], inv), __fmul_rn(x[4 * i + 1], inv),
                          __fmul_rn(x[4 * i + 2], inv), __fmul_rn(x[4 * i + 3], inv));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 consecutive elements of a row in the cache's dtype (16-byte aligned).
template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&x)[16]) {
  constexpr int N = Vec16<T>::N;
#pragma unroll
  for (int i = 0; i < 16 / N; ++i)
    Vec16<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(p) + i), x + i * N);
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&v);
  }
  reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void store16(float *p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4 *>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ float max_abs16(const float (&x)[16]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
  return m;
}

// Largest v of the block (blockDim.x a multiple of 32, at most 1024); sm: 32 floats.
__device__ __forceinline__ float block_max(float v, float *sm) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  float m = lane < nw ? sm[lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return m;
}

}  // namespace kvc

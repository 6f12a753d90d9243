// q8_common.cuh -- the 8-bit codes of the quantised slot cache, shared by the
// kernels that write it (q8_cache.cu) and the decode step (q8_decode.cu).
//
// A block of `block` consecutive slots of one head has one fp32 scale a for K and
// one for V; the value of a code c is c a.  With top the largest code value:
//     a = max(max|x| / top, 2^-126),   c = rne(x * (1 / a)),
// each step one fp32 operation rounded to nearest (the floor keeps 1 / a finite
// for blocks of zeros and subnormals).  |x - c a| is then at most half a code step
// (int8: a / 2; e4m3: 2^-4 |x|, or half its smallest step 2^-10 a) up to fp32 rounding.
// A block with a NaN or an infinity has the scale NaN, so that all its values are NaN and stay
// it when its rows move: magnitudes are searched with maxima that keep a NaN, where fmaxf would
// drop it, and across threads as bits, which order a NaN above every number.
#pragma once

#include <cuda_fp8.h>

#include <cfloat>

#include "kvc_internal.cuh"

namespace kvc {

template <int FMT> struct Q8;

// int8 codes without the conversion instructions, which run at an eighth of the rate of
// an addition: adding 1.5 2^23 to |y| <= 2^22 leaves rne(y) in the low bits of the sum
// (its last place is 1), and an integer c + 128 placed there is read back by subtraction.
// A code depends on the rounding of the product and on that of the sum: both are scalar
// intrinsics, which are never fused (the packed f32x2 multiply and add are, even as
// mul.rn and add.rn).
template <> struct Q8<KV_Q8_S8> {
  static constexpr float kTop = 127.f;
  __device__ __forceinline__ static uint32_t low(float y) { return __float_as_uint(__fadd_rn(y, 12582912.f)); }
  // |y| <= 127 (1 + 2^-22): no code passes 127 (with a NaN scale a code is any byte)
  __device__ __forceinline__ static uint32_t pack4(float2 a, float2 b) {
    return __byte_perm(__byte_perm(low(a.x), low(a.y), 0x0040), __byte_perm(low(b.x), low(b.y), 0x0040), 0x5410);
  }
  __device__ __forceinline__ static void unpack4(uint32_t w, float2 &a, float2 &b) {
    const uint32_t u = w ^ 0x80808080u;  // c + 128
    const float2 k = make_float2(-8388736.f, -8388736.f);
    a = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)),
                               __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441))), k);
    b = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)),
                               __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443))), k);
  }
  // Largest |c| of 16 codes: a 16-bit lane orders by its upper byte, so the lanes' maxima
  // hold the largest upper bytes, and those of the swapped bytes the largest lower ones.
  __device__ __forceinline__ static float big16(const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = __vabsdiffu4(w[i] ^ 0x80808080u, 0x80808080u);
    uint32_t hi = __vimax3_u16x2(m[0], m[1], __vimax3_u16x2(m[2], m[3], 0u));
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = __byte_perm(m[i], 0u, 0x2301);
    hi = __vimax3_u16x2(hi, __vimax3_u16x2(m[0], m[1], m[2]), m[3]);
    return (float)(max(hi & 0xFFFFu, hi >> 16) >> 8);
  }
};

template <> struct Q8<KV_Q8_E4M3> {
  static constexpr float kTop = 448.f;
  __device__ __forceinline__ static uint32_t pack4(float2 a, float2 b) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
  __device__ __forceinline__ static void unpack4(uint32_t w, float2 &a, float2 &b) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    a = __half22float2(__half2(lo));
    b = __half22float2(__half2(hi));
  }
  // largest |c| of 16 codes: without the sign their bits order like their values
  __device__ __forceinline__ static float big16(const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vimax3_u16x2(m, w[i] & 0x007F007Fu, (w[i] >> 8) & 0x007F007Fu);
    float2 a, b;
    unpack4(max(m & 0xFFFFu, m >> 16), a, b);
    return a.x;
  }
};

// The larger one; NaN (0x7FFFFFFF) when either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// The scale of a block whose largest magnitude has the bits `big`; NaN when that is not finite.
template <int FMT>
__device__ __forceinline__ float q8_scale(uint32_t big) {
  return big < 0x7F800000u ? fmaxf(__fdiv_rn(__uint_as_float(big), Q8<FMT>::kTop), FLT_MIN)
                           : __uint_as_float(0x7FFFFFFFu);
}

// 16 values as one vector of codes; inv = 1 / scale.
template <int FMT>
__device__ __forceinline__ uint4 q8_pack16(const float2 (&x)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = x[2 * i], b = x[2 * i + 1];
    w[i] = Q8<FMT>::pack4(make_float2(__fmul_rn(a.x, inv), __fmul_rn(a.y, inv)),
                          make_float2(__fmul_rn(b.x, inv), __fmul_rn(b.y, inv)));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int FMT>
__device__ __forceinline__ uint4 q8_pack16(const float (&x)[16], float inv) {
  float2 y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = make_float2(x[2 * i], x[2 * i + 1]);
  return q8_pack16<FMT>(y, inv);
}

// 16 codes of scale a as codes of the scale whose reciprocal is inv.
template <int FMT>
__device__ __forceinline__ uint4 q8_requantise16(const uint4 &v, float a, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const float2 a2 = make_float2(a, a);
  float2 x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    Q8<FMT>::unpack4(w[i], x[2 * i], x[2 * i + 1]);
    x[2 * i] = __fmul2_rn(x[2 * i], a2);
    x[2 * i + 1] = __fmul2_rn(x[2 * i + 1], a2);
  }
  return q8_pack16<FMT>(x, inv);
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
  for (int i = 0; i < 16; ++i) m = max_nan(m, fabsf(x[i]));
  return m;
}

// Bits of the largest magnitude v of the block (blockDim.x a multiple of 32, at most 1024); sm: 32 words.
__device__ __forceinline__ uint32_t block_max(float v, uint32_t *sm) {
  const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v));
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = w;
  __syncthreads();
  const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  return __reduce_max_sync(0xFFFFFFFFu, lane < nw ? sm[lane] : 0u);
}

}  // namespace kvc

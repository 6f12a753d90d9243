// mma_common.cuh -- warp-level products (mma.sync) with fp32 results: bf16 operands, and fp32
// operands split into two tf32 parts.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace kvc {

__device__ __forceinline__ uint32_t tf32_hi(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
struct Split {
  uint32_t hi, lo;
  __device__ __forceinline__ void set(float x) {
    hi = tf32_hi(x);
    lo = __float_as_uint(x - __uint_as_float(hi));
  }
};
__device__ __forceinline__ void mma1688(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c + small += a b to fp32 accuracy.  The unit cuts its sums off rather than rounding them: the
// two small products have a sum of their own, so that only the large one's steps are cut at
// the sum's own size.
__device__ __forceinline__ void mma_split(float (&c)[4], float (&small)[4], const Split (&a)[4], const Split &b0,
                                          const Split &b1) {
  mma1688(small, a[0].lo, a[1].lo, a[2].lo, a[3].lo, b0.hi, b1.hi);
  mma1688(c, a[0].hi, a[1].hi, a[2].hi, a[3].hi, b0.hi, b1.hi);
  mma1688(small, a[0].hi, a[1].hi, a[2].hi, a[3].hi, b0.lo, b1.lo);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements, two of a row in each lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

}  // namespace kvc

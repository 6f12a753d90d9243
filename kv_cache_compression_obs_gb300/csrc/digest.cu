// digest.cu -- least and largest key per block of cache slots and channel.
//
// Minima and maxima are exact in the cache's type.  A NaN in a block's keys stays in its digest.
// A warp reads a block's rows, 16 bytes a lane and several rows at a time; where there are too
// few blocks to fill the GPU four warps share one.  Bound by memory (one read of K): 64 heads of 31000 to
// 32768 slots 79 us, the copy rate; the newest block of 64 heads 2.8 us.
#include "kvc_internal.cuh"
#include "pdl.cuh"

namespace kvc {
namespace {

constexpr int NW = 4, NT = 32 * NW;

struct DigestArgs {
  const void *K;
  const int32_t *len;
  void *digest;
  int *status;
  int cap, nb;    // slots and blocks of a unit
  int b_log2;
  int n_new;      // newest slots
  int per;        // blocks looked at per unit
  long items;     // units x per
  int share;      // 1: the CTA's warps share a block
};

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, __nv_bfloat16) {
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __nv_bfloat16) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, float) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
  return __float_as_uint(r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, float) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
  return __float_as_uint(r);
}

template <typename T, int D>
__global__ void __launch_bounds__(NT) digest_kernel(const __grid_constant__ DigestArgs A) {
  constexpr int LPR = D * (int)sizeof(T) / 16, RPI = 32 / LPR;  // lanes per row, rows at a time
  constexpr int U = 8;
  __shared__ uint4 part[2][NW][LPR];
  pdl_wait();
  pdl_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int el = lane % LPR, rl = lane / LPR;
  const int block = 1 << A.b_log2;
  const long step = (long)gridDim.x * (A.share ? 1 : NW);
  for (long item = A.share ? (long)blockIdx.x : (long)blockIdx.x * NW + warp; item < A.items; item += step) {
    const long u = item / A.per;
    const int n = A.len ? A.len[u] : A.cap;
    int j = (int)(item - u * A.per);
    if (n < 0 || n > A.cap) {
      if (j == 0 && lane == 0 && A.status) atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
      continue;
    }
    j += max(0, n - A.n_new) >> A.b_log2;
    const int rows = min(block, n - j * block);
    if (rows <= 0) continue;
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(A.K) + (u * (long)A.cap + (long)j * block) * D) + el;
    // rows behind the last stand for it
    const int first = (A.share ? warp * RPI : 0) + rl, by = A.share ? NW * RPI : RPI;
    uint4 lo = __ldcs(src + (long)min(first, rows - 1) * LPR), hi = lo;
    for (int r = first + by; r - rl < rows; r += U * by) {
      uint4 x[U];
#pragma unroll
      for (int i = 0; i < U; ++i) x[i] = __ldcs(src + (long)min(r + i * by, rows - 1) * LPR);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        lo.x = min2(lo.x, x[i].x, T());
        lo.y = min2(lo.y, x[i].y, T());
        lo.z = min2(lo.z, x[i].z, T());
        lo.w = min2(lo.w, x[i].w, T());
        hi.x = max2(hi.x, x[i].x, T());
        hi.y = max2(hi.y, x[i].y, T());
        hi.z = max2(hi.z, x[i].z, T());
        hi.w = max2(hi.w, x[i].w, T());
      }
    }
    auto merge = [&](const uint4 &a, const uint4 &b) {
      lo = make_uint4(min2(lo.x, a.x, T()), min2(lo.y, a.y, T()), min2(lo.z, a.z, T()), min2(lo.w, a.w, T()));
      hi = make_uint4(max2(hi.x, b.x, T()), max2(hi.y, b.y, T()), max2(hi.z, b.z, T()), max2(hi.w, b.w, T()));
    };
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
      uint4 a, b;
      a.x = __shfl_xor_sync(0xFFFFFFFFu, lo.x, o);
      a.y = __shfl_xor_sync(0xFFFFFFFFu, lo.y, o);
      a.z = __shfl_xor_sync(0xFFFFFFFFu, lo.z, o);
      a.w = __shfl_xor_sync(0xFFFFFFFFu, lo.w, o);
      b.x = __shfl_xor_sync(0xFFFFFFFFu, hi.x, o);
      b.y = __shfl_xor_sync(0xFFFFFFFFu, hi.y, o);
      b.z = __shfl_xor_sync(0xFFFFFFFFu, hi.z, o);
      b.w = __shfl_xor_sync(0xFFFFFFFFu, hi.w, o);
      merge(a, b);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(A.digest) + (u * A.nb + j) * 2L * D) + el;
    if (A.share) {  // one item per CTA and turn: the whole CTA is here
      if (warp > 0 && rl == 0) {
        part[0][warp][el] = lo;
        part[1][warp][el] = hi;
      }
      __syncthreads();
      if (warp == 0 && rl == 0) {
#pragma unroll
        for (int w = 1; w < NW; ++w) merge(part[0][w][el], part[1][w][el]);
        dst[0] = lo;
        dst[LPR] = hi;
      }
      __syncthreads();
    } else if (rl == 0) {
      dst[0] = lo;
      dst[LPR] = hi;
    }
  }
}

template <typename T, int D>
int run(const DigestArgs &A, cudaStream_t st) {
  const long ctas = A.share ? A.items : (A.items + NW - 1) / NW, most = 0x7FFFFFFFL;
  const cudaError_t e = launch_pdl(digest_kernel<T, D>, (unsigned)(ctas < most ? ctas : most), NT, 0, st, A);
  if (e != cudaSuccess) return cuda_failure(e, "block digests");
  return launch_status();
}

}  // namespace

int launch_block_digest(const void *K, const int32_t *len, long units, int cap, int d, int block, int n_new, int dtype,
                        void *digest, int *status, cudaStream_t st) {
  DigestArgs A{};
  A.K = K;
  A.len = len;
  A.digest = digest;
  A.status = status;
  A.cap = cap;
  A.nb = (int)(((long)cap + block - 1) / block);
  A.b_log2 = block == 128 ? 7 : block == 64 ? 6 : block == 32 ? 5 : 4;
  A.n_new = n_new;
  // n_new slots touch at most this many blocks, wherever they begin
  const long touched = ((long)n_new + block - 2) / block + 1;
  A.per = (int)(n_new >= cap || touched > A.nb ? A.nb : touched);
  A.items = units * A.per;
  A.share = A.items < 4L * kNumSmsHint;
  if (dtype == KV_BF16) return d == 128 ? run<__nv_bfloat16, 128>(A, st) : run<__nv_bfloat16, 64>(A, st);
  return d == 128 ? run<float, 128>(A, st) : run<float, 64>(A, st);
}

}  // namespace kvc

// blocks.cu -- attention of a few new tokens over the blocks of a long cache that their digests
// choose, for each token and KV head on its own.
//
// With the least and largest key of a block per channel, low and top, and the group's queries,
//     u_j = max_g sum_c max(q_gc, 0) top_jc + min(q_gc, 0) low_jc
// is at least every logit (before the scale) of block j.  The first `sink` and last `recent`
// of the blocks that a token sees and the best others by (u descending, j ascending) are
// attended, all of their visible slots with a plain softmax.
//
// The choice is the one that u in 64 bits makes.  The bounds are computed by warp-level
// products with fp32 sums, which are off by at most e = 2^-16 max|digest| max_g |q_g|_1 (16 steps
// of a sum that may be cut off, 2^-22 each; the products are exact, or 2^-21 from split fp32
// operands).  With a the m-th largest of them, a block above a + 2e is among the true best m, one
// below a - 2e is not; when those between (mostly one block, the m-th itself) are more than
// the places left, they alone are computed again in 64 bits.
//
// One launch, a cluster of CTAs for each (row, KV head, token): the CTAs share out the digests,
// exchange the bounds through distributed shared memory, find the same m-th
// largest each for itself (by halving the range of their bits), share out the chosen blocks'
// slots and join their softmax shares as they exchanged the bounds.
#include <cooperative_groups.h>

#include "pdl.cuh"
#include "rows_stream.cuh"

namespace kvc {
namespace {

constexpr int NW = 4, NT = 32 * NW;
constexpr int kMaxBlocks = 12288;  // 14 bytes of shared memory each

struct BlkArgs {
  const void *q, *K, *V;
  const int32_t *len;
  const void *digest;
  void *o;
  float *lse;
  int32_t *sel;
  int *status;
  long long sq[3], so[3];  // batch, head, token
  int Hq, Hkv, G, nq, cap, nb;
  int b_log2, n_sel, sink, recent;
  int area;   // bytes of the part of shared memory that the choice, the warps' rings and their shares take in turn
  float c_log2;
};

__device__ __forceinline__ uint32_t order(float x) {  // orders like x; a NaN like +inf
  const uint32_t u = x != x ? 0x7F800000u : __float_as_uint(x);
  return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unorder(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// max(q, 0) and min(q, 0) of a vector, NaN kept; the largest magnitude in a vector.
__device__ __forceinline__ uint32_t part2(uint32_t q, bool pos, __nv_bfloat16) {
  const __nv_bfloat162 x = *reinterpret_cast<__nv_bfloat162 *>(&q), z = __float2bfloat162_rn(0.f);
  const __nv_bfloat162 r = pos ? __hmax2_nan(x, z) : __hmin2_nan(x, z);
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t part2(uint32_t q, bool pos, float) {
  const float x = __uint_as_float(q);
  return x != x || (x > 0.f) == pos ? q : 0u;
}
template <typename T>
__device__ __forceinline__ uint4 part(const uint4 &q, bool pos) {
  return make_uint4(part2(q.x, pos, T()), part2(q.y, pos, T()), part2(q.z, pos, T()), part2(q.w, pos, T()));
}
__device__ __forceinline__ void grow(uint32_t &big, const uint4 &x, __nv_bfloat16) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7FFF7FFFu;
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162 *>(&big), *reinterpret_cast<const __nv_bfloat162 *>(&a));
    big = *reinterpret_cast<const uint32_t *>(&r);
  }
}
__device__ __forceinline__ void grow(uint32_t &big, const uint4 &x, float) {
  const float a = fmaxf(fabsf(__uint_as_float(x.x)), fabsf(__uint_as_float(x.y)));
  const float b = fmaxf(fabsf(__uint_as_float(x.z)), fabsf(__uint_as_float(x.w)));
  big = __float_as_uint(fmaxf(__uint_as_float(big), fmaxf(a, b)));
}
__device__ __forceinline__ float magnitude(uint32_t big, __nv_bfloat16) {
  return fmaxf(__uint_as_float(big << 16), __uint_as_float(big & 0xFFFF0000u));
}
__device__ __forceinline__ float magnitude(uint32_t big, float) { return __uint_as_float(big); }

// Sum over the CTA; `slot` alternates between calls so that one barrier is enough.
__device__ __forceinline__ int cta_sum(int x, int (*red)[NW], int slot) {
  x = __reduce_add_sync(0xFFFFFFFFu, x);
  if ((threadIdx.x & 31) == 0) red[slot][threadIdx.x >> 5] = x;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) s += red[slot][w];
  return s;
}

// u of block j in 64 bits: one warp, lanes over the channels; every lane gets it.
template <typename T, int D>
__device__ double bound64(const BlkArgs &A, const T *q, const T *digest, int j) {
  const int lane = threadIdx.x & 31;
  const T *low = digest + (long)j * 2 * D, *top = low + D;
  double best = -INFINITY;
  for (int g = 0; g < A.G; ++g) {
    double s = 0.;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int c = lane + 32 * i;
      const double x = (double)to_f32(q[g * A.sq[1] + c]);
      s += (x != x || x > 0. ? x : 0.) * (double)to_f32(top[c]) + (x != x || x < 0. ? x : 0.) * (double)to_f32(low[c]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (s != s) s = INFINITY;
    best = s > best ? s : best;
  }
  return best;
}

// Shared memory of the choice.
struct Choice {
  uint32_t *key;   // [blocks] bounds' bits, then 1 (chosen) or 0
  double *exact;   // [blocks] of the undecided blocks
  uint16_t *list;  // [blocks] undecided blocks; then the chosen ones, ascending
};

// Marks the best `m` of the n candidates (block lo + i) in c.key; err: how far a bound may be off.
template <typename T, int D>
__device__ void choose(const BlkArgs &A, const Choice &c, const T *q, const T *digest, int lo, int n, int m, float err,
                       int (*red)[NW], uint32_t (*redu)[NW], int &undecided) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t least = 0xFFFFFFFFu, most = 0u;
  for (int i = threadIdx.x; i < n; i += NT) {
    least = min(least, c.key[i]);
    most = max(most, c.key[i]);
  }
  least = __reduce_min_sync(0xFFFFFFFFu, least);
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane == 0) {
    redu[0][warp] = least;
    redu[1][warp] = most;
  }
  if (threadIdx.x == 0) undecided = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    least = min(least, redu[0][w]);
    most = max(most, redu[1][w]);
  }
  // at least m keys are >= L, fewer than m are >= H
  uint32_t L = least, H = most + 1;
  int slot = 0;
  bool split = false;
  while (H - L > 1) {
    const uint32_t mid = L + (H - L) / 2;
    int x = 0;
    for (int i = threadIdx.x; i < n; i += NT) x += c.key[i] >= mid;
    x = cta_sum(x, red, slot);
    slot ^= 1;
    if (x >= m) L = mid; else H = mid;
    if (x == m) {
      split = true;
      break;
    }
  }
  if (split) {  // the m-th largest is the least key from here on
    uint32_t k = 0xFFFFFFFFu;
    for (int i = threadIdx.x; i < n; i += NT)
      if (c.key[i] >= L) k = min(k, c.key[i]);
    k = __reduce_min_sync(0xFFFFFFFFu, k);
    __syncthreads();  // redu was read above
    if (lane == 0) redu[0][warp] = k;
    __syncthreads();
    L = redu[0][0];
#pragma unroll
    for (int w = 1; w < NW; ++w) L = min(L, redu[0][w]);
  }
  const float a = unorder(L), above = a + 2.f * err, below = a - 2.f * err;
  int sure = 0, maybe = 0;
  for (int i = threadIdx.x; i < n; i += NT) {
    const float x = unorder(c.key[i]);
    if (x > above) ++sure;
    else if (!(x < below)) ++maybe;
  }
  const int both = cta_sum(sure + (maybe << 16), red, slot);
  slot ^= 1;
  sure = both & 0xFFFF;
  maybe = both >> 16;
  const bool again = maybe > m - sure;
  for (int i = threadIdx.x; i < n; i += NT) {
    const float x = unorder(c.key[i]);
    const bool in = x > above, open = !in && !(x < below);
    if (again && open) c.list[atomicAdd(&undecided, 1)] = (uint16_t)i;
    c.key[i] = in || (open && !again);
  }
  __syncthreads();
  if (!again) return;
  for (int i = warp; i < maybe; i += NW) {
    const double x = bound64<T, D>(A, q, digest, lo + c.list[i]);
    if (lane == 0) c.exact[i] = x;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < maybe; i += NT) {
    const double x = c.exact[i];
    const int j = c.list[i];
    int better = 0;
    for (int k = 0; k < maybe; ++k) better += c.exact[k] > x || (c.exact[k] == x && c.list[k] < j);
    if (better < m - sure) c.key[j] = 1;
  }
  __syncthreads();
}

template <typename T, int D>
__global__ void __launch_bounds__(NT, sizeof(T) == 2 || D == 64 ? 2 : 1) blocks_kernel(const __grid_constant__ BlkArgs A) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ float wm[NW * 8], wz[NW * 8];
  __shared__ float2 mz[8], all[16][8];
  __shared__ float sM[8], sI[8];
  __shared__ float err_part[NW], err_cta;
  __shared__ int red[2][NW], undecided;
  __shared__ uint32_t redu[2][NW];
  constexpr int NCH = RowStream<T, D>::NCH;
  const int G = A.G;
  float *sh = reinterpret_cast<float *>(dyn);              // [G][D] this CTA's share
  unsigned char *area = dyn + G * D * 4;
  float *so = reinterpret_cast<float *>(area);             // [NW][G][D]
  float *mine = reinterpret_cast<float *>(area + A.area);  // this CTA's bounds
  pdl_wait();
  pdl_launch();
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  const int CL = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long u = blockIdx.x / CL, bh = u / A.nq;
  const int t = (int)(u - bh * A.nq), b = (int)(bh / A.Hkv), h = (int)(bh - (long)b * A.Hkv);
  const int n = A.len[bh];
  int32_t *sel = A.sel ? A.sel + u * A.n_sel : nullptr;
  if (n < 0 || n > A.cap) {  // every CTA of the cluster alike
    if (rank == 0 && threadIdx.x == 0 && A.status) atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
    return;
  }
  T *o = static_cast<T *>(A.o) + b * A.so[0] + (long)h * G * A.so[1] + t * A.so[2];
  float *lse = A.lse ? A.lse + ((long)b * A.Hq + (long)h * G) * A.nq + t : nullptr;
  const int seen = n - A.nq + t + 1;
  if (seen <= 0) {
    if (rank == 0) {
      for (int i = threadIdx.x; i < G * D; i += NT) o[i / D * A.so[1] + i % D] = T(0.f);
      for (int i = threadIdx.x; i < A.n_sel && sel; i += NT) sel[i] = -1;
      if (threadIdx.x < G && lse) lse[(long)threadIdx.x * A.nq] = -INFINITY;
    }
    return;
  }
  const int block = 1 << A.b_log2;
  const int nbk = (seen + block - 1) >> A.b_log2;
  const T *q = static_cast<const T *>(A.q) + b * A.sq[0] + (long)h * G * A.sq[1] + t * A.sq[2];
  RowStream<T, D> R;
  R.init(area + warp * R.RING);
  R.load_q(q + min(R.g, G - 1) * A.sq[1]);

  // ---- which blocks ----
  const int ns = min(nbk, A.n_sel);
  const int m = A.n_sel - A.sink - A.recent;  // places that bounds decide, where nbk > n_sel
  const int lo = A.sink, nm = nbk - A.sink - A.recent;
  const bool choice = nbk > A.n_sel;
  const int cap_c = choice && m > 0 ? nm : 0;
  Choice c;
  c.exact = reinterpret_cast<double *>(area);
  c.key = reinterpret_cast<uint32_t *>(c.exact + A.nb);
  c.list = reinterpret_cast<uint16_t *>(mine + (A.nb + CL - 1) / CL + 16);
  if (cap_c > 0) {
    const T *digest = static_cast<const T *>(A.digest) + bh * A.nb * 2L * D;
    const int per = (((nm + CL - 1) / CL) + 15) & ~15;
    const int i0 = min(nm, rank * per), i1 = min(nm, i0 + per);
    uint32_t big = 0u;
    float norm = 0.f;
#pragma unroll
    for (int x = 0; x < NCH; ++x) {
      const uint32_t w[4] = {R.q[x].x, R.q[x].y, R.q[x].z, R.q[x].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        norm += sizeof(T) == 4 ? fabsf(__uint_as_float(w[i]))
                               : fabsf(__uint_as_float(w[i] << 16)) + fabsf(__uint_as_float(w[i] & 0xFFFF0000u));
    }
    norm += __shfl_xor_sync(0xFFFFFFFFu, norm, 1);
    norm += __shfl_xor_sync(0xFFFFFFFFu, norm, 2);
    norm = rows_max(norm);
    for (int i = i0 + warp * 16; i < i1; i += NW * 16) {
      uint4 x[2][2][NCH];  // low, top of blocks i + g and i + g + 8
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const char *p = reinterpret_cast<const char *>(digest + (long)(lo + min(i + R.g + 8 * k, i1 - 1)) * 2 * D) + R.t * 16;
#pragma unroll
        for (int y = 0; y < NCH; ++y) {
          x[0][k][y] = __ldcs(reinterpret_cast<const uint4 *>(p + y * 64));
          x[1][k][y] = __ldcs(reinterpret_cast<const uint4 *>(p + D * sizeof(T) + y * 64));
        }
      }
      float s[4] = {0.f, 0.f, 0.f, 0.f}, small[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int y = 0; y < NCH; ++y) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          grow(big, x[0][k][y], T());
          grow(big, x[1][k][y], T());
        }
        dot16(s, small, x[0][0][y], x[0][1][y], part<T>(R.q[y], false), T());
        dot16(s, small, x[1][0][y], x[1][1][y], part<T>(R.q[y], true), T());
      }
      if (sizeof(T) == 4)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] += small[k];
      // the largest of the group's: columns behind G repeat its last query
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float v = max_nan(s[2 * k], s[2 * k + 1]);
        v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
        v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
        if (R.t == 0 && i + R.g + 8 * k < i1) mine[i - i0 + R.g + 8 * k] = v;
      }
    }
    float e = magnitude(big, T());
#pragma unroll
    for (int x = 16; x; x >>= 1) e = fmaxf(e, __shfl_xor_sync(0xFFFFFFFFu, e, x));
    if (lane == 0) err_part[warp] = e;
    __syncthreads();
    if (threadIdx.x == 0) err_cta = fmaxf(fmaxf(err_part[0], err_part[1]), fmaxf(err_part[2], err_part[3]));
    cl.sync();
    float err = 0.f;
    bool wild = false;
    for (int r = 0; r < CL; ++r) err = fmaxf(err, *cl.map_shared_rank(&err_cta, r));
    err *= norm * 0x1p-16f;
    for (int i = threadIdx.x; i < nm; i += NT) {
      const int r = i / per;
      const float v = cl.map_shared_rank(mine, r)[i - r * per];
      wild |= !(fabsf(v) < INFINITY);
      c.key[i] = order(v);
    }
    // a bound that is no number, or too large for fp32: 64 bits decide for all of them
    if (__syncthreads_or(wild || !(err < INFINITY))) err = INFINITY;
    choose<T, D>(A, c, q, digest, lo, nm, m, err, red, redu, undecided);
  }
  {
    // the chosen ones in order
    const int chunk = (nbk + NT - 1) / NT, j0 = min(nbk, (int)threadIdx.x * chunk), j1 = min(nbk, j0 + chunk);
    auto chosen = [&](int j) { return !choice || j < lo || j >= nbk - A.recent || (m > 0 && c.key[j - lo]); };
    int cnt = 0;
    for (int j = j0; j < j1; ++j) cnt += chosen(j);
    int incl = cnt;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, incl, x);
      if (lane >= x) incl += y;
    }
    __syncthreads();
    if (lane == 31) red[0][warp] = incl;
    __syncthreads();
    int at = incl - cnt;
    for (int w = 0; w < warp; ++w) at += red[0][w];
    for (int j = j0; j < j1; ++j)
      if (chosen(j)) c.list[at++] = (uint16_t)j;
    __syncthreads();
  }
  if (rank == 0 && sel)
    for (int i = threadIdx.x; i < A.n_sel; i += NT) sel[i] = i < ns ? (int)c.list[i] : -1;

  // ---- attention over them ----
  {
    const int tl = A.b_log2 - 4, in_last = (seen - ((nbk - 1) << A.b_log2) + 15) >> 4;
    const int tiles = ((ns - 1) << tl) + in_last, per = (tiles + CL - 1) / CL;
    const int x0 = min(tiles, rank * per), x1 = min(tiles, x0 + per);
    const T *K = static_cast<const T *>(A.K) + bh * A.cap * (long)D, *V = static_cast<const T *>(A.V) + bh * A.cap * (long)D;
    const int lim[2] = {seen, seen};
    R.run((x1 - x0 - warp + NW - 1) / NW,
          [&](int y) {
            const int x = x0 + y * NW + warp;
            return ((int)c.list[x >> tl] << A.b_log2) + ((x & ((1 << tl) - 1)) << 4);
          },
          K, D, V, D, seen - 1, A.c_log2, lim, seen);
    __syncthreads();
    R.leave(G, wm + warp * 8, wz + warp * 8, so + warp * G * D);
    __syncthreads();
    join_warps<D, NW>(G, wm, wz, so, sh, mz);
  }
  cl.sync();
  for (int i = threadIdx.x; i < CL * G; i += NT) all[i / G][i % G] = cl.map_shared_rank(mz, i / G)[i % G];
  __syncthreads();
  if ((int)threadIdx.x < G) {
    float M = -INFINITY, Z = 0.f;
    for (int s = 0; s < CL; ++s)
      if (all[s][threadIdx.x].y != 0.f) M = fmaxf(M, all[s][threadIdx.x].x);
    for (int s = 0; s < CL; ++s)
      if (all[s][threadIdx.x].y != 0.f) Z += all[s][threadIdx.x].y * tc::ex2(M == -INFINITY ? 0.f : all[s][threadIdx.x].x - M);
    sM[threadIdx.x] = M;
    sI[threadIdx.x] = 1.f / Z;
    if (rank == 0 && lse) lse[(long)threadIdx.x * A.nq] = (M + log2f(Z)) * 0.6931471805599453f;
  }
  __syncthreads();
  for (int i = rank * NT + threadIdx.x; i < G * D; i += CL * NT) {
    const int r = i / D;
    float v = 0.f;
    for (int s = 0; s < CL; ++s)
      if (all[s][r].y != 0.f) v += tc::ex2(sM[r] == -INFINITY ? 0.f : all[s][r].x - sM[r]) * cl.map_shared_rank(sh, s)[i];
    o[r * A.so[1] + i % D] = T(v * sI[r]);
  }
  cl.sync();  // nobody leaves while its shares are read
}

template <typename T, int D>
int run(BlkArgs A, long units, cudaStream_t st) {
  // CTAs per unit: as many as run at once, two an SM (fp32, d = 128: one)
  const long room = (sizeof(T) == 2 || D == 64 ? 2L : 1L) * kNumSmsHint;
  int CL = 16;
  while (CL > 1 && units * CL > room) CL /= 2;
  const size_t warps = NW * RowStream<T, D>::RING, choice = (size_t)A.nb * 12;
  A.area = (int)(((warps > choice ? warps : choice) + 15) & ~(size_t)15);
  const size_t bytes = (size_t)A.G * D * 4 + A.area + ((size_t)(A.nb + CL - 1) / CL + 16) * 4 + (size_t)A.nb * 2 + 16;
  if (units * CL > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  if (ensure_smem((const void *)blocks_kernel<T, D>, bytes)) return KV_ERR_CUDA;
  if (CL > 8) {
    const cudaError_t e = cudaFuncSetAttribute(blocks_kernel<T, D>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return cuda_failure(e, "block-sparse attention: clusters of 16");
  }
  const cudaError_t e = launch_pdl_cluster(blocks_kernel<T, D>, (unsigned)(units * CL), NT, bytes, st, CL, A);
  if (e != cudaSuccess) return cuda_failure(e, "block-sparse attention");
  return launch_status();
}

}  // namespace

bool attn_blocks_fits(int nb) { return nb <= kMaxBlocks; }

int launch_attn_blocks(const void *q, const void *K, const void *V, const int32_t *len, const void *digest, int B, int Hq,
                       int Hkv, int nq, int cap, int d, int block, int n_sel, int sink, int recent, const long long *sq,
                       const long long *so, float scale, int dtype, void *o, float *lse, int32_t *sel, int *status,
                       cudaStream_t st) {
  BlkArgs A{};
  A.q = q;
  A.K = K;
  A.V = V;
  A.len = len;
  A.digest = digest;
  A.o = o;
  A.lse = lse;
  A.sel = sel;
  A.status = status;
  for (int i = 0; i < 3; ++i) {
    A.sq[i] = sq[i];
    A.so[i] = so[i];
  }
  A.Hq = Hq;
  A.Hkv = Hkv;
  A.G = Hq / Hkv;
  A.nq = nq;
  A.cap = cap;
  A.nb = (int)(((long)cap + block - 1) / block);
  A.b_log2 = block == 128 ? 7 : block == 64 ? 6 : block == 32 ? 5 : 4;
  A.n_sel = n_sel;
  A.sink = sink;
  A.recent = recent;
  A.c_log2 = scale * 1.4426950408889634f;
  const long units = (long)B * Hkv * nq;
  if (dtype == KV_BF16)
    return d == 128 ? run<__nv_bfloat16, 128>(A, units, st) : run<__nv_bfloat16, 64>(A, units, st);
  return d == 128 ? run<float, 128>(A, units, st) : run<float, 64>(A, units, st);
}

}  // namespace kvc

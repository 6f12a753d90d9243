// attn_prompt.cu -- causal attention of a prompt, grouped heads, packed sequences
// (KV-cache survey blog §1.1: softmax(Q K^T / sqrt(d)) V): fp32, and bf16 calls that the
// tcgen05 kernel (attn_prompt_tc.cu) does not take.
//
//     m' = max(m, max_j l_j), z' = z 2^(m - m') + sum_j 2^(l_j - m'), O likewise,
// over key tiles of BN, l in log2 units, so that 2^l is one instruction.
//
// The products keep fp32 accuracy on the tensor cores: every operand x is hi + lo, hi = x
// rounded to tf32 (11 significant bits) and lo the exact rest, and a product is
// hi hi + hi lo + lo hi in mma.m16n8k8 with fp32 sums; lo lo, below 2^-22 of the product,
// and lo's own bits past its 11 are dropped.  On the CUDA cores the same tiles were bound by
// shared memory: a 16-byte load takes four cycles whatever it shares, and a thread's few
// results do not pay for its operands (4 heads of 512 tokens
// 26.7 us; here 11.6 us, and 55 TFLOP/s over 4096 tokens of 32/8 heads).  With one running sum
// for everything, which the unit cuts off at every step, 4000 tokens were off by 4e-6 of the
// output's norm and ran at 59; with sums of their own for the small products and for each tile
// they are off by 4.6e-7, where fp32 matrix products are off by 5.6e-7.
//
// A warp holds 16 query rows.  Which element of d (or which key) stands at which k is free as
// long as both operands agree: a lane takes 16 consecutive bytes of a K row for two k steps,
// the weights of keys 2t and 2t + 1, which it holds after the first product, are columns t
// and t + 4 of the second's operand, and 16 consecutive bytes of V rows 2t and 2t + 1 serve
// four of its n tiles.  Row strides of D + 16 and D + 4 words make both reads free of bank
// conflicts.  K and V tiles come by asynchronous copies (bf16: converted on the way).
//   SPLIT 0: four warps, 64 rows, share the tiles, double buffered.
//   SPLIT 1: all warps have the same 16 rows and every NW-th tile each, in buffers of their
//            own, and are joined at the end: where 64-row tiles would leave SMs idle.
#include <cmath>

#include "attn_common.cuh"
#include "tc_common.cuh"

namespace kvc {
namespace {

constexpr int BN = 32;

template <int D, int SPLIT>
struct Geo {
  static constexpr int NW = SPLIT ? (D == 64 ? 8 : 4) : 4;  // warps
  static constexpr int BM = SPLIT ? 16 : 64;
  static constexpr int LK = D + 16, LV = D + 4;    // padded rows, in floats
  static constexpr int TILE = BN * (LK + LV);      // a K and a V tile
  static constexpr int BUFS = SPLIT ? NW : 2;
  static constexpr int SMEM = (BM * LK + BUFS * TILE) * 4;
};

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

template <typename T, int D, int SPLIT>
__global__ void __launch_bounds__(32 * Geo<D, SPLIT>::NW) attn_kernel(const T *__restrict__ Q, const T *__restrict__ K,
                                                                      const T *__restrict__ V, T *__restrict__ O,
                                                                      const __grid_constant__ AttnArgs A) {
  using Gm = Geo<D, SPLIT>;
  constexpr int NW = Gm::NW, NT = 32 * NW, BM = Gm::BM, LK = Gm::LK, LV = Gm::LV, EV = Vec16<T>::N;
  constexpr int NO = D / 8;  // n tiles of O
  extern __shared__ __align__(16) float sh[];
  float *sQ = sh, *sX = sh + BM * LK;
  __shared__ AttnTile st;
  const AttnShape &S = A.S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int h = blockIdx.x % S.Hq;
  if (threadIdx.x < 32) {
    const AttnTile t = attn_locate(S, blockIdx.x / S.Hq, BM, blockIdx.x == 0, A.status);
    if (threadIdx.x == 0) st = t;
  }
  __syncthreads();
  const AttnTile t = st;
  if (t.nq <= 0) return;
  const int hk = h / (S.Hq / S.Hkv);
  const T *q = Q + t.b * S.q[0] + h * S.q[1] + (long long)(t.q0 + t.r0) * S.q[2];
  const T *k = K + t.b * S.k[0] + hk * S.k[1] + (long long)t.k0 * S.k[2];
  const T *v = V + t.b * S.v[0] + hk * S.v[1] + (long long)t.k0 * S.v[2];
  const int rows = min(BM, t.nq - t.r0);
  const int off = t.nk - t.nq + t.r0;      // row i of the tile sees keys <= off + i
  const int kend = min(t.nk, off + rows);  // keys that some row sees
  const int ntile = kend > 0 ? (kend + BN - 1) / BN : 0;

  // Rows [0, n) of a tile with ld floats each; rows behind `have` become 0.  first / step: this
  // thread's part of the copying threads.
  auto copy_rows = [&](float *dst, int ld, const T *p, long long stride, int n, int have, int first, int step) {
    for (int e = first; e < n * (D / EV); e += step) {
      const int r = e / (D / EV), c = (e % (D / EV)) * EV;
      if constexpr (sizeof(T) == 4) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst + r * ld + c)),
                     "l"(p + (r < have ? r * stride : 0) + c), "r"(r < have ? 16 : 0)
                     : "memory");
      } else {
        float x[EV];
#pragma unroll
        for (int i = 0; i < EV; ++i) x[i] = 0.f;
        if (r < have) Vec16<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(p + r * stride + c)), x);
#pragma unroll
        for (int i = 0; i < EV; i += 4)
          *reinterpret_cast<float4 *>(dst + r * ld + c + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      }
    }
  };
  auto fetch = [&](int j, float *buf, int first, int step) {  // tile j's K and V, one copy group
    if (j < ntile) {
      copy_rows(buf, LK, k + (long long)j * BN * S.k[2], S.k[2], BN, kend - j * BN, first, step);
      copy_rows(buf + BN * LK, LV, v + (long long)j * BN * S.v[2], S.v[2], BN, kend - j * BN, first, step);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  copy_rows(sQ, LK, q, S.q[2], BM, rows, threadIdx.x, NT);  // joins the first tile's group
  if (SPLIT) fetch(warp, sX + warp * Gm::TILE, lane, 32);
  else fetch(0, sX, threadIdx.x, NT);

  const int r0 = SPLIT ? 0 : warp * 16;                    // this warp's rows of the tile
  const float *mq = sQ + r0 * LK;
  // last keys that rows g and g + 8 of the warp see
  const int lim0 = min(kend - 1, off + r0 + g), lim1 = min(kend - 1, off + r0 + g + 8);
  const int wend = SPLIT ? kend : min(t.nk, off + min(rows, r0 + 16));  // keys that some row of the warp sees
  float m0 = -INFINITY, m1 = -INFINITY, z0 = 0.f, z1 = 0.f, o[NO][4];
#pragma unroll
  for (int i = 0; i < NO; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) o[i][x] = 0.f;
  if (SPLIT) {  // Q is everyone's
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
  }
  int turn = 0;
  for (int j = SPLIT ? warp : 0; j < ntile; j += SPLIT ? NW : 1, turn ^= 1) {
    const float *sK;
    if (SPLIT) {
      if (j != warp) fetch(j, sX + warp * Gm::TILE, lane, 32);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
      sK = sX + warp * Gm::TILE;
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();  // everyone's pieces have landed, and the other buffer has been read
      fetch(j + 1, sX + (turn ^ 1) * Gm::TILE, threadIdx.x, NT);
      sK = sX + turn * Gm::TILE;
    }
    const float *sV = sK + BN * LK;
    const int j0 = j * BN;
    if (j0 < wend) {
      float s[BN / 8][4], sl[BN / 8][4];
#pragma unroll
      for (int n = 0; n < BN / 8; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[n][x] = sl[n][x] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {  // two k steps
        const float4 qa = *reinterpret_cast<const float4 *>(mq + g * LK + c * 16 + t4 * 4);
        const float4 qb = *reinterpret_cast<const float4 *>(mq + (g + 8) * LK + c * 16 + t4 * 4);
        Split a[2][4];
        a[0][0].set(qa.x);
        a[0][1].set(qb.x);
        a[0][2].set(qa.y);
        a[0][3].set(qb.y);
        a[1][0].set(qa.z);
        a[1][1].set(qb.z);
        a[1][2].set(qa.w);
        a[1][3].set(qb.w);
#pragma unroll
        for (int n = 0; n < BN / 8; ++n) {
          const float4 kb = *reinterpret_cast<const float4 *>(sK + (n * 8 + g) * LK + c * 16 + t4 * 4);
          Split b[4];
          b[0].set(kb.x);
          b[1].set(kb.y);
          b[2].set(kb.z);
          b[3].set(kb.w);
          mma_split(s[n], sl[n], a[0], b[0], b[1]);
          mma_split(s[n], sl[n], a[1], b[2], b[3]);
        }
      }
      // logits of keys j0 + 8 n + 2 t4 (+ 1)
      float x0 = m0, x1 = m1;
      const bool part = j0 + BN - 1 > min(lim0, off + r0);
#pragma unroll
      for (int n = 0; n < BN / 8; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int key = j0 + n * 8 + 2 * t4 + x;
          s[n][x] = part && key > lim0 ? -INFINITY : (s[n][x] + sl[n][x]) * A.c_log2;
          s[n][2 + x] = part && key > lim1 ? -INFINITY : (s[n][2 + x] + sl[n][2 + x]) * A.c_log2;
          x0 = fmaxf(x0, s[n][x]);
          x1 = fmaxf(x1, s[n][2 + x]);
        }
#pragma unroll
      for (int w = 1; w < 4; w <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, w));
        x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, w));
      }
      if (__any_sync(0xFFFFFFFFu, x0 > m0 || x1 > m1)) {
        const float f0 = x0 > m0 ? tc::ex2(m0 - x0) : 1.f, f1 = x1 > m1 ? tc::ex2(m1 - x1) : 1.f;
        m0 = x0;
        m1 = x1;
        z0 *= f0;
        z1 *= f1;
#pragma unroll
        for (int i = 0; i < NO; ++i) {
          o[i][0] *= f0;
          o[i][1] *= f0;
          o[i][2] *= f1;
          o[i][3] *= f1;
        }
      }
      const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;  // no key seen yet
      Split a[BN / 8][4];  // rows g, g + 8 against keys 2 t4, 2 t4 + 1: columns t4 and t4 + 4
#pragma unroll
      for (int n = 0; n < BN / 8; ++n) {
        const float p0 = tc::ex2(s[n][0] - b0), p1 = tc::ex2(s[n][1] - b0);
        const float p2 = tc::ex2(s[n][2] - b1), p3 = tc::ex2(s[n][3] - b1);
        z0 += p0 + p1;
        z1 += p2 + p3;
        a[n][0].set(p0);
        a[n][1].set(p2);
        a[n][2].set(p1);
        a[n][3].set(p3);
      }
      // a tile's sums start at 0 and join O by an addition that rounds: O's error does not
      // grow with every step that the unit cuts off
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float y[4][4], yl[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) y[i][x] = yl[i][x] = 0.f;
#pragma unroll
        for (int n = 0; n < BN / 8; ++n) {
          const float4 va = *reinterpret_cast<const float4 *>(sV + (n * 8 + 2 * t4) * LV + c * 32 + g * 4);
          const float4 vb = *reinterpret_cast<const float4 *>(sV + (n * 8 + 2 * t4 + 1) * LV + c * 32 + g * 4);
          const float xa[4] = {va.x, va.y, va.z, va.w}, xb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            Split ba, bb;
            ba.set(xa[i]);
            bb.set(xb[i]);
            mma_split(y[i], yl[i], a[n], ba, bb);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[c * 4 + i][x] += y[i][x] + yl[i][x];
      }
    }
    if (SPLIT) __syncwarp();  // the buffer has been read
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int w = 1; w < 4; w <<= 1) {
    z0 += __shfl_xor_sync(0xFFFFFFFFu, z0, w);
    z1 += __shfl_xor_sync(0xFFFFFFFFu, z1, w);
  }
  // O's tile 4 c + i holds columns 32 c + 8 t4 + i and + 4: four tiles give the lane columns
  // 32 c + 8 t4 .. + 7
  auto store = [&](int r, int col, float4 w) {
    T *dst = O + t.b * S.o[0] + h * S.o[1] + (long long)(t.q0 + t.r0 + r) * S.o[2] + col;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4 *>(dst) = w;
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(w.x, w.y), b = __floats2bfloat162_rn(w.z, w.w);
      *reinterpret_cast<uint2 *>(dst) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
  };
  auto store_lse = [&](int r, float m, float z) {
    if (A.lse)
      A.lse[((long long)t.b * S.Hq + h) * S.Tq + t.q0 + t.r0 + r] =
          z != 0.f ? (m + log2f(z)) * 0.6931471805599453f : -INFINITY;
  };
  if constexpr (!SPLIT) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = r0 + g + 8 * half;
      if (r >= rows) continue;
      const float z = half ? z1 : z0, inv = z != 0.f ? 1.f / z : 0.f;  // no key seen: 0 (a NaN is passed on)
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          store(r, c * 32 + 8 * t4 + 4 * x,
                make_float4(o[4 * c][2 * half + x] * inv, o[4 * c + 1][2 * half + x] * inv, o[4 * c + 2][2 * half + x] * inv,
                            o[4 * c + 3][2 * half + x] * inv));
      if (t4 == 0) store_lse(r, half ? m1 : m0, z);
    }
  } else {
    __shared__ float sm[NW][16], sz[NW][16];
    __syncthreads();
    float *mine = sX + warp * Gm::TILE;  // [16][D]
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          *reinterpret_cast<float4 *>(mine + (g + 8 * half) * D + c * 32 + 8 * t4 + 4 * x) =
              make_float4(o[4 * c][2 * half + x], o[4 * c + 1][2 * half + x], o[4 * c + 2][2 * half + x],
                          o[4 * c + 3][2 * half + x]);
      if (t4 == 0) {
        sm[warp][g + 8 * half] = half ? m1 : m0;
        sz[warp][g + 8 * half] = half ? z1 : z0;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < rows * (D / 4); e += NT) {
      const int r = e / (D / 4), col = (e % (D / 4)) * 4;
      float M = -INFINITY, Z = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, sm[w][r]);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = sz[w][r] != 0.f ? tc::ex2(sm[w][r] - M) : 0.f;  // a warp without a visible key
        const float4 x = *reinterpret_cast<const float4 *>(sX + w * Gm::TILE + r * D + col);
        Z += f * sz[w][r];
        y = make_float4(y.x + f * x.x, y.y + f * x.y, y.z + f * x.z, y.w + f * x.w);
      }
      const float inv = Z != 0.f ? 1.f / Z : 0.f;
      store(r, col, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
      if (col == 0) store_lse(r, M, Z);
    }
  }
}

template <typename T, int D, int SPLIT>
int run(const void *Q, const void *K, const void *V, void *O, const AttnArgs &A, cudaStream_t st) {
  using Gm = Geo<D, SPLIT>;
  const long ctas = attn_tiles(A.S, Gm::BM) * A.S.Hq;
  if (ctas > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  if (ensure_smem((const void *)attn_kernel<T, D, SPLIT>, Gm::SMEM)) return KV_ERR_CUDA;
  attn_kernel<T, D, SPLIT><<<(unsigned)ctas, 32 * Gm::NW, Gm::SMEM, st>>>(
      static_cast<const T *>(Q), static_cast<const T *>(K), static_cast<const T *>(V), static_cast<T *>(O), A);
  return launch_status();
}

// 64-row tiles read K and V a quarter as often; the split form only where they would leave
// SMs without work.
template <typename T, int D>
int run_rows(const void *Q, const void *K, const void *V, void *O, const AttnArgs &A, cudaStream_t st) {
  if (attn_tiles(A.S, 64) * A.S.Hq < kNumSmsHint) return run<T, D, 1>(Q, K, V, O, A, st);
  return run<T, D, 0>(Q, K, V, O, A, st);
}

}  // namespace

// For bf16, whose rows may be split over their keys; fp32 needs none.
size_t attn_prompt_workspace_bytes(int B, int Hq, int Hkv, int Tq, int Tk, int d, int n_seq) {
  AttnShape S{};
  S.B = B;
  S.Hq = Hq;
  S.Hkv = Hkv;
  S.Tq = Tq;
  S.Tk = Tk;
  S.d = d;
  S.n_seq = n_seq;
  return attn_tc_workspace_bytes(S);
}

int launch_attn_prompt(const void *Q, const void *K, const void *V, const AttnShape &S, float scale, int dtype,
                       void *O, float *lse, void *ws, int *status, cudaStream_t st) {
  AttnArgs A{S, scale * 1.4426950408889634f, lse, status};
  if (attn_tc_eligible(S, scale, dtype)) return launch_attn_prompt_tc(Q, K, V, A, O, ws, st);
  if (dtype == KV_BF16)
    return S.d == 128 ? run_rows<__nv_bfloat16, 128>(Q, K, V, O, A, st) : run_rows<__nv_bfloat16, 64>(Q, K, V, O, A, st);
  return S.d == 128 ? run_rows<float, 128>(Q, K, V, O, A, st) : run_rows<float, 64>(Q, K, V, O, A, st);
}

}  // namespace kvc

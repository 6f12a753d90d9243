// attn_prompt.cu -- causal attention of a prompt, grouped heads, packed sequences
// (KV-cache survey blog §1.1: softmax(Q K^T / sqrt(d)) V): the CUDA-core kernel.
//
// One CTA per (query tile of BM rows, query head) walks the sequence's keys in tiles
// of 64 with a running row maximum m and sum z:
//     m' = max(m, max_j l_j), z' = z 2^(m - m') + sum_j 2^(l_j - m'), O likewise,
// l in log2 units, so that 2^l is one instruction.  256 threads as 16 x 16: thread
// (ty, tx) holds rows ty RT .. ty RT + RT - 1 against keys tx + 16 i, and of O the
// columns 4 tx .. 4 tx + 3 (+ 64).  All arithmetic is fp32.
// fp32 tiles come by asynchronous copies, K and V double buffered, so that a short prompt
// (one CTA an SM, nothing else to run meanwhile) does not wait for memory in every tile:
// 4 heads of 512 tokens 13 us against 36 us with one buffer that K and V take turns in,
// which bf16 (converted on the way; the tensor cores take all but odd scales) keeps.
#include <cmath>

#include "attn_common.cuh"
#include "tc_common.cuh"

namespace kvc {
namespace {

constexpr int NT = 256;
constexpr int BN = 64;

template <typename T, int D, int RT>
struct Geo {
  static constexpr int BM = 16 * RT;
  static constexpr int LD = D + 4;   // padded row of the Q and K/V buffers
  static constexpr int LP = BN + 4;  // padded row of P
  static constexpr bool ASYNC = sizeof(T) == 4;
  static constexpr int SMEM = (BM * LD + (ASYNC ? 4 : 1) * BN * LD + BM * LP) * 4;
};

template <typename T, int D, int RT>
__global__ void __launch_bounds__(NT) attn_kernel(const T *__restrict__ Q, const T *__restrict__ K,
                                                  const T *__restrict__ V, T *__restrict__ O,
                                                  const __grid_constant__ AttnArgs A) {
  using Gm = Geo<T, D, RT>;
  constexpr int BM = Gm::BM, LD = Gm::LD, LP = Gm::LP, NV = D / 64, EV = Vec16<T>::N;
  extern __shared__ __align__(16) float sh[];
  float *sQ = sh, *sP = sQ + BM * LD, *sX = sP + BM * LP;  // sX: K, or K K V V in turns of two
  __shared__ AttnTile st;
  const AttnShape &S = A.S;
  const int h = blockIdx.x % S.Hq;
  const int index = blockIdx.x / S.Hq;
  if (threadIdx.x < 32) {
    const AttnTile t = attn_locate(S, index, BM, blockIdx.x == 0, A.status);
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
  const int off = t.nk - t.nq + t.r0;                 // row i of the tile sees keys <= off + i
  const int kend = min(t.nk, off + rows);             // keys that some row sees
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;

  for (int e = threadIdx.x; e < BM * (D / EV); e += NT) {
    const int r = e / (D / EV), c = (e % (D / EV)) * EV;
    float x[EV];
    if (r < rows) {
      Vec16<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(q + r * S.q[2] + c)), x);
    } else {
#pragma unroll
      for (int i = 0; i < EV; ++i) x[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < EV; ++i) sQ[r * LD + c + i] = x[i] * A.c_log2;
  }
  auto load_tile = [&](const T *p, long long stride, int j0) {  // rows behind the last key become 0
    for (int e = threadIdx.x; e < BN * (D / EV); e += NT) {
      const int r = e / (D / EV), c = (e % (D / EV)) * EV;
      float x[EV];
      if (j0 + r < kend) {
        Vec16<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(p + (j0 + r) * stride + c)), x);
      } else {
#pragma unroll
        for (int i = 0; i < EV; ++i) x[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < EV; i += 4)
        *reinterpret_cast<float4 *>(sX + r * LD + c + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    }
  };
  auto copy_tile = [&](float *dst, const T *p, long long stride, int j0) {  // the same, asynchronously
    if (j0 < kend)
      for (int e = threadIdx.x; e < BN * (D / 4); e += NT) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;
        const bool have = j0 + r < kend;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst + r * LD + c)),
                     "l"(p + (have ? (j0 + r) * stride : 0) + c), "r"(have ? 16 : 0)
                     : "memory");
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float m[RT], z[RT], o[RT][NV][4];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    m[i] = -INFINITY;
    z[i] = 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[i][c][x] = 0.f;
  }
  if constexpr (Gm::ASYNC) {
    copy_tile(sX, k, S.k[2], 0);
    copy_tile(sX + 2 * BN * LD, v, S.v[2], 0);
  }
  int buf = 0;
  for (int j0 = 0; j0 < kend; j0 += BN, buf ^= 1) {
    const float *sK = sX, *sV = sX;
    if constexpr (Gm::ASYNC) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");  // K
      __syncthreads();  // everyone's pieces, and the other buffers have been read
      copy_tile(sX + (buf ^ 1) * BN * LD, k, S.k[2], j0 + BN);
      copy_tile(sX + (2 + (buf ^ 1)) * BN * LD, v, S.v[2], j0 + BN);
      sK = sX + buf * BN * LD;
      sV = sX + (2 + buf) * BN * LD;
    } else {
      load_tile(k, S.k[2], j0);
      __syncthreads();
    }
    float s[RT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[i][x] = 0.f;
#pragma unroll 8
    for (int c = 0; c < D; c += 4) {
      float4 a[RT], b[4];
#pragma unroll
      for (int i = 0; i < RT; ++i) a[i] = *reinterpret_cast<const float4 *>(sQ + (ty * RT + i) * LD + c);
#pragma unroll
      for (int x = 0; x < 4; ++x) b[x] = *reinterpret_cast<const float4 *>(sK + (tx + 16 * x) * LD + c);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          s[i][x] += a[i].x * b[x].x + a[i].y * b[x].y + a[i].z * b[x].z + a[i].w * b[x].w;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int lim = min(kend - 1, off + ty * RT + i) - j0;  // last key of the tile that the row sees
      float mx = m[i];
#pragma unroll
      for (int x = 0; x < 4; ++x) mx = tx + 16 * x <= lim ? fmaxf(mx, s[i][x]) : mx;
#pragma unroll
      for (int w = 8; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, w));
      const float f = mx == m[i] ? 1.f : tc::ex2(m[i] - mx);
      m[i] = mx;
      float sum = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float p = tx + 16 * x <= lim ? tc::ex2(s[i][x] - mx) : 0.f;
        sP[(ty * RT + i) * LP + tx + 16 * x] = p;
        sum += p;
      }
      z[i] = z[i] * f + sum;
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[i][c][x] *= f;
    }
    if constexpr (Gm::ASYNC) {
      asm volatile("cp.async.wait_group 2;" ::: "memory");  // V
      __syncthreads();
    } else {
      __syncthreads();
      load_tile(v, S.v[2], j0);
      __syncthreads();
    }
#pragma unroll 4
    for (int j = 0; j < BN; j += 4) {
      float4 p[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) p[i] = *reinterpret_cast<const float4 *>(sP + (ty * RT + i) * LP + j);
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        float4 x[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) x[y] = *reinterpret_cast<const float4 *>(sV + (j + y) * LD + 4 * tx + 64 * c);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          o[i][c][0] += p[i].x * x[0].x + p[i].y * x[1].x + p[i].z * x[2].x + p[i].w * x[3].x;
          o[i][c][1] += p[i].x * x[0].y + p[i].y * x[1].y + p[i].z * x[2].y + p[i].w * x[3].y;
          o[i][c][2] += p[i].x * x[0].z + p[i].y * x[1].z + p[i].z * x[2].z + p[i].w * x[3].z;
          o[i][c][3] += p[i].x * x[0].w + p[i].y * x[1].w + p[i].z * x[2].w + p[i].w * x[3].w;
        }
      }
    }
    if constexpr (!Gm::ASYNC) __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    float sum = z[i];
#pragma unroll
    for (int w = 8; w; w >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, w);
    const int r = ty * RT + i;
    if (r >= rows) continue;
    const float inv = sum > 0.f ? 1.f / sum : 0.f;  // no key seen: 0
    T *dst = O + t.b * S.o[0] + h * S.o[1] + (long long)(t.q0 + t.r0 + r) * S.o[2];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const float4 w = make_float4(o[i][c][0] * inv, o[i][c][1] * inv, o[i][c][2] * inv, o[i][c][3] * inv);
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(dst + 4 * tx + 64 * c) = w;
      } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(w.x, w.y), b = __floats2bfloat162_rn(w.z, w.w);
        *reinterpret_cast<uint2 *>(dst + 4 * tx + 64 * c) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
      }
    }
    if (A.lse && tx == 0)
      A.lse[((long long)t.b * S.Hq + h) * S.Tq + t.q0 + t.r0 + r] =
          sum > 0.f ? (m[i] + log2f(sum)) * 0.6931471805599453f : -INFINITY;
  }
}

template <typename T, int D, int RT>
int run(const void *Q, const void *K, const void *V, void *O, const AttnArgs &A, cudaStream_t st) {
  using Gm = Geo<T, D, RT>;
  const long ctas = attn_tiles(A.S, Gm::BM) * A.S.Hq;
  if (ctas > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  if (ensure_smem((const void *)attn_kernel<T, D, RT>, Gm::SMEM)) return KV_ERR_CUDA;
  attn_kernel<T, D, RT><<<(unsigned)ctas, NT, Gm::SMEM, st>>>(static_cast<const T *>(Q), static_cast<const T *>(K),
                                                            static_cast<const T *>(V), static_cast<T *>(O), A);
  return launch_status();
}

// Tiles of 64 rows reuse K and V four times as often as tiles of 16, which give four
// times the CTAs: the small ones when the large ones would leave SMs without work.
template <typename T, int D>
int run_rows(const void *Q, const void *K, const void *V, void *O, const AttnArgs &A, cudaStream_t st) {
  if (attn_tiles(A.S, 64) * A.S.Hq < kNumSmsHint) return run<T, D, 1>(Q, K, V, O, A, st);
  return run<T, D, 4>(Q, K, V, O, A, st);
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

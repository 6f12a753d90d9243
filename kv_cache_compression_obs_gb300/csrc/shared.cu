// shared.cu -- attention of a batch of rows over one common prefix and each row's own slots.
//
//     o = sum over the prefix and the row's visible slots of softmax(scale <q, k>) v.
// The prefix's keys are the same for all rows, so the rows of all batch entries and of a KV
// head's group form the one operand of its products (shared_tc.cu; fp32: below), in shares of
// its keys that leave their sums, references and normalisers in the workspace.
// The second launch has a cluster of CTAs for each 8 query rows of a (batch row, KV head): they share out
// its own slots, which need nothing of the first launch, then join everything:
//     M = max m_s, z = sum z_s 2^(m_s - M), o = sum o_s 2^(m_s - M) / z.
#include <cooperative_groups.h>

#include "pdl.cuh"
#include "rows_stream.cuh"
#include "shared_common.cuh"

namespace kvc {
namespace {

constexpr int NW = 4, NT = 32 * NW;
constexpr int kMaxSplits = 64;

__device__ __forceinline__ long q_offset(const long long (&s)[3], int b, int h, int G, int nq, int row) {
  const int g = row / nq, t = row - g * nq;
  return (long)b * s[0] + ((long)h * G + g) * s[1] + t * s[2];
}

// ---- fp32 prefix: 8 rows and a share of the keys per CTA ----
template <typename T, int D>
__global__ void __launch_bounds__(NT, sizeof(T) == 2 ? 4 : 2) prefix_rows_kernel(const __grid_constant__ SharedArgs A, int groups, int per) {
  extern __shared__ __align__(16) float so[];  // [NW][8][D]
  __shared__ float wm[NW * 8], wz[NW * 8];
  pdl_wait();
  pdl_launch();
  const int warp = threadIdx.x >> 5;
  const int grp = blockIdx.x % groups, rest = blockIdx.x / groups, h = rest % A.Hkv, s = rest / A.Hkv;
  const int r0 = grp * 8, R = min(8, A.rows - r0), gn = A.G * A.nq;
  const int k0 = s * per, k1 = min(A.P, k0 + per);
  RowStream<T, D> S;
  S.init();
  {
    const int row = r0 + min(S.g, R - 1), b = row / gn;
    S.load_q(static_cast<const T *>(A.q) + q_offset(A.sq, b, h, A.G, A.nq, row - b * gn));
  }
  const T *K = static_cast<const T *>(A.Kp) + h * A.skp[0], *V = static_cast<const T *>(A.Vp) + h * A.svp[0];
  const int lim[2] = {k1, k1};
  int j = k0 + warp * 16;
  if (j < k1) {
    S.load_k(K, A.skp[1], j, k1 - 1);
    S.load_v(V, A.svp[1], j, k1 - 1);
  }
  for (; j < k1; j += NW * 16) {
    const int nj = j + NW * 16;
    float l[4];
    S.logits(A.c_log2, l);
    if (nj < k1) S.load_k(K, A.skp[1], nj, k1 - 1);
    if (j + 16 > k1) S.hide(l, S.g, j, lim);
    S.add(l);
    if (nj < k1) S.load_v(V, A.svp[1], nj, k1 - 1);
  }
  S.leave(R, wm + warp * 8, wz + warp * 8, so + warp * R * D);
  __syncthreads();
  const long at = ((long)s * A.Hkv + h) * A.rows + r0;
  join_warps<D, NW>(R, wm, wz, so, A.part + at * D, A.stat + at);
}

// ---- own slots, and everything joined ----
template <typename T, int D>
__global__ void __launch_bounds__(NT, sizeof(T) == 2 ? 4 : 2) shared_join_kernel(const __grid_constant__ SharedArgs A, int groups) {
  extern __shared__ __align__(16) float dyn[];
  __shared__ float wm[NW * 8], wz[NW * 8];
  __shared__ float2 mz[8], all[8][8];
  __shared__ float2 st[kMaxSplits][8];
  __shared__ float sM[8], sI[8];
  float *sh = dyn, *so = dyn + 8 * D;  // [8][D], [NW][8][D]
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  const int CL = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int warp = threadIdx.x >> 5;
  const long u = blockIdx.x / CL, bh = u / groups;
  const int grp = (int)(u - bh * groups), b = (int)(bh / A.Hkv), h = (int)(bh - (long)b * A.Hkv);
  const int gn = A.G * A.nq, r0 = grp * 8, R = min(8, gn - r0);
  // Without a prefix launch in front nothing has waited for the kernels before this one.
  if (A.splits == 0) pdl_wait();
  const int n = A.cap ? __ldcg(A.len + bh) : 0;
  const bool bad = n < 0 || n > A.cap;
  if (!bad && n > 0) {
    RowStream<T, D> S;
    S.init();
    S.load_q(static_cast<const T *>(A.q) + q_offset(A.sq, b, h, A.G, A.nq, r0 + min(S.g, R - 1)));
    const T *K = static_cast<const T *>(A.K) + bh * A.cap * (long)D, *V = static_cast<const T *>(A.V) + bh * A.cap * (long)D;
    int lim[2];  // slots that rows 2t, 2t + 1 see
#pragma unroll
    for (int x = 0; x < 2; ++x) lim[x] = n - A.nq + (r0 + min(2 * S.t + x, R - 1)) % A.nq + 1;
    const int tiles = (n + 15) >> 4, per = (tiles + CL - 1) / CL, x1 = min(tiles, (rank + 1) * per);
    int x = rank * per + warp;
    if (x < x1) {
      S.load_k(K, D, x * 16, n - 1);
      S.load_v(V, D, x * 16, n - 1);
    }
    for (; x < x1; x += NW) {
      const int nx = x + NW;
      float l[4];
      S.logits(A.c_log2, l);
      if (nx < x1) S.load_k(K, D, nx * 16, n - 1);
      if (x * 16 + 16 > n - A.nq) S.hide(l, S.g, x * 16, lim);
      S.add(l);
      if (nx < x1) S.load_v(V, D, nx * 16, n - 1);
    }
    S.leave(R, wm + warp * 8, wz + warp * 8, so + warp * R * D);
    __syncthreads();
    join_warps<D, NW>(R, wm, wz, so, sh, mz);
  } else if ((int)threadIdx.x < 8) {
    mz[threadIdx.x] = make_float2(-INFINITY, 0.f);
  }
  if (A.splits) pdl_wait();  // the prefix's shares are there
  pdl_launch();
  if (bad) {  // every CTA of the cluster alike
    if (rank == 0 && grp == 0 && threadIdx.x == 0 && A.status) atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
    return;
  }
  const long row0 = (long)b * gn + r0;
  for (int i = threadIdx.x; i < A.splits * 8; i += NT) {
    const int s = i >> 3, r = min(i & 7, R - 1);
    st[s][i & 7] = A.stat[((long)s * A.Hkv + h) * A.rows + row0 + r];
  }
  cl.sync();
  for (int i = threadIdx.x; i < CL * 8; i += NT) all[i >> 3][i & 7] = cl.map_shared_rank(mz, i >> 3)[min(i & 7, R - 1)];
  __syncthreads();
  if ((int)threadIdx.x < R) {
    const int r = threadIdx.x;
    float M = -INFINITY, Z = 0.f;
    for (int s = 0; s < CL; ++s)
      if (all[s][r].y != 0.f) M = fmaxf(M, all[s][r].x);
    for (int s = 0; s < A.splits; ++s)
      if (st[s][r].y != 0.f) M = fmaxf(M, st[s][r].x);
    // factors take the references' places
    for (int s = 0; s < CL; ++s) {
      const float f = all[s][r].y != 0.f ? tc::ex2(M == -INFINITY ? 0.f : all[s][r].x - M) : 0.f;
      Z += f * all[s][r].y;
      all[s][r].x = f;
    }
    for (int s = 0; s < A.splits; ++s) {
      const float f = st[s][r].y != 0.f ? tc::ex2(M == -INFINITY ? 0.f : st[s][r].x - M) : 0.f;
      Z += f * st[s][r].y;
      st[s][r].x = f;
    }
    sI[r] = Z != 0.f ? 1.f / Z : 0.f;  // 0: no key seen; a NaN is passed on
    if (rank == 0 && A.lse) {
      const int g = (r0 + r) / A.nq, t = r0 + r - g * A.nq;
      A.lse[((long)b * A.Hq + (long)h * A.G + g) * A.nq + t] = Z != 0.f ? (M + log2f(Z)) * 0.6931471805599453f : -INFINITY;
    }
  }
  __syncthreads();
  const float *part = A.part + ((long)h * A.rows + row0) * D;
  const long share = (long)A.Hkv * A.rows * D;
  for (int i = (rank * NT + threadIdx.x) * 4; i < R * D; i += CL * NT * 4) {
    const int r = i / D;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4 &x, const float2 &w) {
      v.x += w.x * x.x;
      v.y += w.x * x.y;
      v.z += w.x * x.z;
      v.w += w.x * x.w;
    };
#pragma unroll 4
    for (int s = 0; s < A.splits; ++s)
      if (st[s][r].y != 0.f) add(__ldcs(reinterpret_cast<const float4 *>(part + s * share + i)), st[s][r]);
    for (int s = 0; s < CL; ++s)
      if (all[s][r].y != 0.f) add(*reinterpret_cast<const float4 *>(cl.map_shared_rank(sh, s) + i), all[s][r]);
    T *o = static_cast<T *>(A.o) + q_offset(A.so, b, h, A.G, A.nq, r0 + r) + i % D;
    const float f = sI[r];
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * f, v.y * f), c = __floats2bfloat162_rn(v.z * f, v.w * f);
      *reinterpret_cast<uint2 *>(o) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&c));
    } else {
      *reinterpret_cast<float4 *>(o) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    }
  }
  cl.sync();  // nobody leaves while its shares are read
}

// fp32: two CTAs an SM, a few rounds of them; at least 64 keys each.
SharedPlan rows_plan(long rows, int Hkv, int P) {
  const long items = (rows + 7) / 8 * Hkv, want = 4L * kNumSmsHint;
  long s = items > 0 ? (want + items - 1) / items : 1;
  if (s > P / 64) s = P / 64;
  s = s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s;
  const int per = (int)((((P + s - 1) / s) + 63) / 64 * 64);
  return SharedPlan{(P + per - 1) / per, per};
}

SharedPlan make_plan(long rows, int Hkv, int P, int dtype) {
  if (P == 0 || rows == 0) return SharedPlan{0, 0};
  return dtype == KV_BF16 ? shared_tc_plan(rows, Hkv, P) : rows_plan(rows, Hkv, P);
}

template <typename T, int D>
int run(const SharedArgs &A, const SharedPlan &plan, cudaStream_t st) {
  const size_t so = (size_t)NW * 8 * D * 4, smem = so + 8 * D * 4;
  if (A.splits > 0) {
    if (sizeof(T) == 2) {
      const int rc = launch_shared_prefix_tc(A, D, st);
      if (rc != KV_OK) return rc;
    } else {
      const int groups = (A.rows + 7) / 8;
      const long ctas = (long)groups * A.Hkv * A.splits;
      if (ctas > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
      const cudaError_t e = launch_pdl(prefix_rows_kernel<float, D>, (unsigned)ctas, NT, so, st, A, groups, plan.per);
      if (e != cudaSuccess) return cuda_failure(e, "shared prefix");
      count_launches(1);
    }
  }
  const int gn = A.G * A.nq, groups = (gn + 7) / 8;
  const long units = (long)A.B * A.Hkv * groups, room = (sizeof(T) == 2 ? 4L : 2L) * kNumSmsHint;
  int CL = 8;
  while (CL > 1 && (units * CL > room || CL * 64 > A.cap)) CL /= 2;
  if (units * CL > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  if (ensure_smem((const void *)shared_join_kernel<T, D>, smem)) return KV_ERR_CUDA;
  const cudaError_t e = launch_pdl_cluster(shared_join_kernel<T, D>, (unsigned)(units * CL), NT, smem, st, CL, A, groups);
  if (e != cudaSuccess) return cuda_failure(e, "shared prefix: own slots");
  return launch_status();
}

}  // namespace

size_t attn_shared_workspace_bytes(int B, int Hq, int Hkv, int nq, int P, int d, int dtype) {
  const long rows = (long)B * (Hq / Hkv) * nq;
  const SharedPlan plan = make_plan(rows, Hkv, P, dtype);
  return (size_t)plan.splits * Hkv * rows * ((size_t)d * sizeof(float) + sizeof(float2)) + (plan.splits ? 32 : 0);
}

int launch_attn_shared(const void *q, const void *Kp, const void *Vp, const void *K, const void *V, const int32_t *len, int B,
                       int Hq, int Hkv, int nq, int P, int cap, int d, const long long *strides, float scale, int dtype, void *o,
                       float *lse, void *ws, int *status, cudaStream_t st) {
  SharedArgs A{};
  A.q = q;
  A.Kp = Kp;
  A.Vp = Vp;
  A.K = K;
  A.V = V;
  A.len = len;
  A.o = o;
  A.lse = lse;
  A.status = status;
  for (int i = 0; i < 3; ++i) {
    A.sq[i] = strides[i];
    A.so[i] = strides[7 + i];
  }
  for (int i = 0; i < 2; ++i) {
    A.skp[i] = strides[3 + i];
    A.svp[i] = strides[5 + i];
  }
  A.B = B;
  A.Hq = Hq;
  A.Hkv = Hkv;
  A.G = Hq / Hkv;
  A.nq = nq;
  A.P = P;
  A.cap = cap;
  A.rows = B * A.G * nq;
  const SharedPlan plan = make_plan(A.rows, Hkv, P, dtype);
  A.splits = plan.splits;
  A.c_log2 = scale * 1.4426950408889634f;
  A.part = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(ws) + 31) & ~uintptr_t(31));
  A.stat = reinterpret_cast<float2 *>(A.part + (size_t)A.splits * Hkv * A.rows * d);
  if (dtype == KV_BF16) return d == 128 ? run<__nv_bfloat16, 128>(A, plan, st) : run<__nv_bfloat16, 64>(A, plan, st);
  return d == 128 ? run<float, 128>(A, plan, st) : run<float, 64>(A, plan, st);
}

}  // namespace kvc

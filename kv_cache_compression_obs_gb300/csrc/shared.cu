// shared.cu -- attention of a batch of rows over one common prefix and each row's own slots.
//
//     o = sum over the prefix and the row's visible slots of softmax(scale <q, k>) v.
// The prefix's keys are the same for all rows, so the rows of all batch entries and of a KV
// head's group form the one operand of its products (shared_tc.cu; fp32: below), in shares of
// its keys that leave their sums, references and normalisers in the workspace.
// A second launch streams the rows' own slots, which needs nothing of the first, in equal stretches; a
// third joins everything:  M = max m_s, z = sum z_s 2^(m_s - M), o = sum o_s 2^(m_s - M) / z.
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

// Dynamic shared memory of a streaming CTA: the warps' rings, which their shares take over at the end.
template <typename T, int D>
constexpr int kRings = NW * RowStream<T, D>::RING;
static_assert(kRings<__nv_bfloat16, 64> >= NW * 8 * 64 * 4, "shares");
// CTAs an SM holds.
template <typename T, int D>
constexpr int kPerSm = sizeof(T) == 4 && D == 128 ? 1 : 2;

// ---- fp32 prefix: 8 rows and a share of the keys per CTA ----
template <typename T, int D>
__global__ void __launch_bounds__(NT, kPerSm<T, D>) prefix_rows_kernel(const __grid_constant__ SharedArgs A, int groups, int per) {
  extern __shared__ __align__(16) unsigned char rings[];
  __shared__ float wm[NW * 8], wz[NW * 8];
  pdl_wait();
  pdl_launch();
  const int warp = threadIdx.x >> 5;
  const int grp = blockIdx.x % groups, rest = blockIdx.x / groups, h = rest % A.Hkv, s = rest / A.Hkv;
  const int r0 = grp * 8, R = min(8, A.rows - r0), gn = A.G * A.nq;
  const int k0 = s * per, k1 = min(A.P, k0 + per);
  RowStream<T, D> S;
  S.init(rings + warp * S.RING);
  {
    const int row = r0 + min(S.g, R - 1), b = row / gn;
    S.load_q(static_cast<const T *>(A.q) + q_offset(A.sq, b, h, A.G, A.nq, row - b * gn));
  }
  const int lim[2] = {k1, k1}, tiles = (k1 - k0 + 15) >> 4;
  S.run((tiles - warp + NW - 1) / NW, [&](int y) { return k0 + (y * NW + warp) * 16; }, static_cast<const T *>(A.Kp) + h * A.skp[0],
        A.skp[1], static_cast<const T *>(A.Vp) + h * A.svp[0], A.svp[1], k1 - 1, A.c_log2, lim, k1);
  __syncthreads();
  float *so = reinterpret_cast<float *>(rings);
  S.leave(R, wm + warp * 8, wz + warp * 8, so + warp * R * D);
  __syncthreads();
  const long at = ((long)s * A.Hkv + h) * A.rows + r0;
  join_warps<D, NW>(R, wm, wz, so, A.part + at * D, A.stat + at);
}

// ---- own slots ----
// The units (batch row, KV head, 8 of its query rows) one behind the other are a line of tiles of 16
// slots, and every CTA takes an equal stretch of it: lengths differ, and a CTA per unit would wait for
// the longest.  A stretch inside one unit is a piece; piece number = CTA + unit, which no two share.
struct OwnArgs {
  float *part;   // [pieces][8][D]
  float2 *stat;  // [pieces][8]
  int2 *info;    // [units] first piece, pieces
  int groups;    // of 8 query rows
  int units;
};
constexpr int kMinTiles = 8;  // of a stretch

template <typename T, int D>
__global__ void __launch_bounds__(NT, kPerSm<T, D>) own_slots_kernel(const __grid_constant__ SharedArgs A,
                                                                    const __grid_constant__ OwnArgs W) {
  extern __shared__ __align__(16) unsigned char rings[];
  float *so = reinterpret_cast<float *>(rings);  // [NW][8][D]
  __shared__ float wm[NW * 8], wz[NW * 8];
  __shared__ int wsum[NW], at_tile, at_unit;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Without a prefix launch in front nothing has waited for the kernels before this one.
  if (A.splits == 0) pdl_wait();
  pdl_launch();
  const int heads = A.B * A.Hkv;
  auto length = [&](int bh) {
    const int n = __ldcg(A.len + bh);
    return n < 0 || n > A.cap ? 0 : n;
  };
  // tiles of this thread's stretch of heads, then of those in front
  const int each = (heads + NT - 1) / NT, h0 = min(heads, (int)threadIdx.x * each), h1 = min(heads, h0 + each);
  int mine = 0;
  for (int bh = h0; bh < h1; ++bh) mine += (length(bh) + 15) >> 4;
  mine *= W.groups;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int total = 0, before = incl - mine;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  const int per = max(kMinTiles, (int)(((unsigned)total + gridDim.x - 1) / gridDim.x));
  const int lo = (int)min((long)total, (long)per * blockIdx.x), hi = min(total - lo, per) + lo;
  if (lo < total && before <= lo && lo < before + mine) {  // the thread whose heads hold tile lo
    int x = before;
    int u = h0 * W.groups;
    for (int bh = h0; bh < h1; ++bh) {
      const int t = (length(bh) + 15) >> 4;
      if (x + t * W.groups <= lo) {
        x += t * W.groups;
        u += W.groups;
        continue;
      }
      const int g = (lo - x) / t;
      x += g * t;
      u += g;
      break;
    }
    at_unit = u;
    at_tile = x;
  }
  __syncthreads();
  if (lo < hi) {
    int u = at_unit;
    int start = at_tile;  // unit u's first tile
    for (int x = lo; x < hi;) {
      const int bh = u / W.groups, grp = u - bh * W.groups, n = length(bh), t = (n + 15) >> 4;
      if (t == 0) {
        ++u;
        continue;
      }
      const int b = bh / A.Hkv, h = bh - b * A.Hkv, gn = A.G * A.nq, r0 = grp * 8, R = min(8, gn - r0);
      const int x0 = x - start, x1 = min(t, hi - start);
      RowStream<T, D> S;
      S.init(rings + warp * S.RING);
      S.load_q(static_cast<const T *>(A.q) + q_offset(A.sq, b, h, A.G, A.nq, r0 + min(S.g, R - 1)));
      int lim[2];  // slots that rows 2t, 2t + 1 see
#pragma unroll
      for (int i = 0; i < 2; ++i) lim[i] = n - A.nq + (r0 + min(2 * S.t + i, R - 1)) % A.nq + 1;
      S.run((x1 - x0 - warp + NW - 1) / NW, [&](int y) { return (x0 + y * NW + warp) * 16; },
            static_cast<const T *>(A.K) + (long)bh * A.cap * D, D, static_cast<const T *>(A.V) + (long)bh * A.cap * D, D, n - 1,
            A.c_log2, lim, n - A.nq + 1);
      __syncthreads();
      S.leave(R, wm + warp * 8, wz + warp * 8, so + warp * R * D);
      __syncthreads();
      const long piece = (long)blockIdx.x + u;
      join_warps<D, NW>(R, wm, wz, so, W.part + piece * 8 * D, W.stat + piece * 8);
      if (x0 == 0 && threadIdx.x == 0) {
        const int first = start / per, last = (start + t - 1) / per;
        W.info[u] = make_int2(first + u, last - first + 1);
      }
      __syncthreads();  // the shares are read before the next piece's
      x = start + x1;
      start += t;
      ++u;
    }
  }
  if (A.splits) pdl_wait();  // this kernel does not end before the prefix's
}

// ---- everything joined: one warp a query row ----
template <typename T, int D>
__global__ void __launch_bounds__(NT) shared_join_kernel(const __grid_constant__ SharedArgs A, const __grid_constant__ OwnArgs W) {
  constexpr int E = D / 32;  // elements of a lane
  pdl_wait();
  pdl_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gn = A.G * A.nq;
  const long at = (long)blockIdx.x * NW + warp;
  if (at >= (long)A.B * A.Hkv * gn) return;
  const long bh = at / gn;
  const int row = (int)(at - bh * gn), b = (int)(bh / A.Hkv), h = (int)(bh - (long)b * A.Hkv);
  const int n = A.cap ? A.len[bh] : 0;
  if (n < 0 || n > A.cap) {
    if (row == 0 && lane == 0 && A.status) atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
    return;
  }
  const int2 own = n > 0 ? W.info[bh * W.groups + row / 8] : make_int2(0, 0);
  const int shares = A.splits + own.y;
  // share s: the prefix's first, then the pieces
  auto stat = [&](int s) {
    return s < A.splits ? A.stat[((long)s * A.Hkv + h) * A.rows + (long)b * gn + row]
                        : W.stat[((long)own.x + s - A.splits) * 8 + row % 8];
  };
  float M = -INFINITY;
  for (int s = lane; s < shares; s += 32) {
    const float2 x = stat(s);
    if (x.y != 0.f) M = fmaxf(M, x.x);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float Z = 0.f, v[E];
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = 0.f;
  for (int s0 = 0; s0 < shares; s0 += 32) {
    float f = 0.f;  // share s0 + lane's factor; 0: it saw nothing and left no sums
    if (s0 + lane < shares) {
      const float2 x = stat(s0 + lane);
      if (x.y != 0.f) f = tc::ex2(M == -INFINITY ? 0.f : x.x - M);
      Z += f * x.y;
    }
    const unsigned live = __ballot_sync(0xFFFFFFFFu, f != 0.f);
#pragma unroll
    for (int half = 0; half < 32; half += 16) {
      if (s0 + half >= shares) break;
      float x[16][E];  // all on their way together
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int s = s0 + half + i;
        const float *p = s < A.splits ? A.part + (((long)s * A.Hkv + h) * A.rows + (long)b * gn + row) * D
                                      : W.part + (((long)own.x + s - A.splits) * 8 + row % 8) * D;
#pragma unroll
        for (int y = 0; y < E; ++y) x[i][y] = 0.f;
        if (live >> (half + i) & 1) {
          if constexpr (E == 4) {
            const float4 y = __ldcs(reinterpret_cast<const float4 *>(p) + lane);
            x[i][0] = y.x;
            x[i][1] = y.y;
            x[i][2] = y.z;
            x[i][3] = y.w;
          } else {
            const float2 y = __ldcs(reinterpret_cast<const float2 *>(p) + lane);
            x[i][0] = y.x;
            x[i][1] = y.y;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float w = __shfl_sync(0xFFFFFFFFu, f, half + i);
#pragma unroll
        for (int y = 0; y < E; ++y) v[y] += w * x[i][y];
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) Z += __shfl_xor_sync(0xFFFFFFFFu, Z, o);
  const float inv = Z != 0.f ? 1.f / Z : 0.f;  // 0: no key seen; a NaN is passed on
  const int g = row / A.nq, t = row - g * A.nq;
  T *o = static_cast<T *>(A.o) + (long)b * A.so[0] + ((long)h * A.G + g) * A.so[1] + t * A.so[2] + lane * E;
  if constexpr (sizeof(T) == 4) {
    if constexpr (E == 4) *reinterpret_cast<float4 *>(o) = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    else *reinterpret_cast<float2 *>(o) = make_float2(v[0] * inv, v[1] * inv);
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 2) *reinterpret_cast<__nv_bfloat162 *>(o + i) = __floats2bfloat162_rn(v[i] * inv, v[i + 1] * inv);
  }
  if (lane == 0 && A.lse)
    A.lse[((long)b * A.Hq + (long)h * A.G + g) * A.nq + t] = Z != 0.f ? (M + log2f(Z)) * 0.6931471805599453f : -INFINITY;
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

// CTAs of the own slots' kernel: those that run at once.
int own_ctas(int elem_bytes, int d) { return (elem_bytes == 4 && d == 128 ? 1 : 2) * kNumSmsHint; }

template <typename T, int D>
int run(const SharedArgs &A, const OwnArgs &W, const SharedPlan &plan, cudaStream_t st) {
  const size_t smem = kRings<T, D>;
  if (A.splits > 0) {
    if (sizeof(T) == 2) {
      const int rc = launch_shared_prefix_tc(A, D, st);
      if (rc != KV_OK) return rc;
    } else {
      const int groups = (A.rows + 7) / 8;
      const long ctas = (long)groups * A.Hkv * A.splits;
      if (ctas > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
      if (ensure_smem((const void *)prefix_rows_kernel<float, D>, kRings<float, D>)) return KV_ERR_CUDA;
      const cudaError_t e = launch_pdl(prefix_rows_kernel<float, D>, (unsigned)ctas, NT, kRings<float, D>, st, A, groups, plan.per);
      if (e != cudaSuccess) return cuda_failure(e, "shared prefix");
      count_launches(1);
    }
  }
  if (A.cap > 0) {
    if (ensure_smem((const void *)own_slots_kernel<T, D>, smem)) return KV_ERR_CUDA;
    const cudaError_t e = launch_pdl(own_slots_kernel<T, D>, (unsigned)own_ctas(sizeof(T), D), NT, smem, st, A, W);
    if (e != cudaSuccess) return cuda_failure(e, "shared prefix: own slots");
    count_launches(1);
  }
  const long ctas = ((long)A.rows * A.Hkv + NW - 1) / NW;
  if (ctas > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  const cudaError_t e = launch_pdl(shared_join_kernel<T, D>, (unsigned)ctas, NT, 0, st, A, W);
  if (e != cudaSuccess) return cuda_failure(e, "shared prefix: joining the shares");
  return launch_status();
}

// Where the shares stand in the workspace.
struct Layout {
  size_t prefix, prefix_stat, own, own_stat, info, bytes;
  Layout(const SharedPlan &plan, int Hkv, long rows, long units, int d, int dtype) {
    const size_t n = (size_t)plan.splits * Hkv * rows, pieces = (size_t)own_ctas(dtype == KV_BF16 ? 2 : 4, d) + units;
    prefix = 0;
    own = prefix + n * d * sizeof(float);
    prefix_stat = own + pieces * 8 * d * sizeof(float);
    own_stat = prefix_stat + n * sizeof(float2);
    info = own_stat + pieces * 8 * sizeof(float2);
    bytes = info + units * sizeof(int2) + 32;
  }
};

}  // namespace

size_t attn_shared_workspace_bytes(int B, int Hq, int Hkv, int nq, int P, int d, int dtype) {
  const long gn = (long)(Hq / Hkv) * nq, rows = B * gn, units = (long)B * Hkv * ((gn + 7) / 8);
  return Layout(make_plan(rows, Hkv, P, dtype), Hkv, rows, units, d, dtype).bytes;
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
  OwnArgs W{};
  W.groups = (A.G * nq + 7) / 8;
  W.units = B * Hkv * W.groups;
  char *p = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(ws) + 31) & ~uintptr_t(31));
  const Layout l(plan, Hkv, A.rows, W.units, d, dtype);
  A.part = reinterpret_cast<float *>(p + l.prefix);
  A.stat = reinterpret_cast<float2 *>(p + l.prefix_stat);
  W.part = reinterpret_cast<float *>(p + l.own);
  W.stat = reinterpret_cast<float2 *>(p + l.own_stat);
  W.info = reinterpret_cast<int2 *>(p + l.info);
  if (dtype == KV_BF16) return d == 128 ? run<__nv_bfloat16, 128>(A, W, plan, st) : run<__nv_bfloat16, 64>(A, W, plan, st);
  return d == 128 ? run<float, 128>(A, W, plan, st) : run<float, 64>(A, W, plan, st);
}

}  // namespace kvc

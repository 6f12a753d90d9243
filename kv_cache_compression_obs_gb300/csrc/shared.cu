// shared.cu -- attention of a batch of rows over one common prefix and each row's own slots.
//
//     o = sum over the prefix and the row's visible slots of softmax(scale <q, k>) v.
// The prefix's keys are the same for all rows, so the rows of all batch entries and of a KV
// head's group form the one operand of its products (shared_tc.cu; fp32: below), in shares of
// its keys that leave their sums, references and normalisers in the workspace.
// A second launch streams the rows' own slots, which needs nothing of the first, in equal stretches; a
// third joins everything:  M = max m_s, z = sum z_s 2^(m_s - M), o = sum o_s 2^(m_s - M) / z.
//
// Bound by memory: 64 rows of 32/8 heads behind 32768 keys with 200 to 2047 slots of their own 93 us (430 MB:
// 63 us): prefix 31, own slots 47 at 6.3 TB/s, joining 8, starts and ends between.  24 rows of
// 3 tokens and 32 heads behind 8191 keys 70 us (49).  4 rows behind 4096 keys 14 us, three kernels'
// latencies.  With the own slots by a cluster of CTAs per unit, which also joined, 188, 113 and 21 us.
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

// Two CTAs an SM (fp32, d = 128: one) of four warps with what shared memory holds of tiles.
template <typename T, int D>
using Rows = RowStream<T, D, (D == 64 && sizeof(T) == 2 ? 6 : 3)>;
// Dynamic shared memory of a streaming CTA: the warps' rings, which their shares take over at the end.
template <typename T, int D>
constexpr int kRings = NW * Rows<T, D>::RING;
static_assert(kRings<__nv_bfloat16, 64> >= NW * 8 * 64 * 4, "shares");
// CTAs an SM holds.
template <typename T, int D>
constexpr int kPerSm = sizeof(T) == 4 && D == 128 ? 1 : 2;

// A warp's share of the prefix (tiles first, first + NW, ..., `count` of them) made anew.
template <typename T, int D>
__device__ __noinline__ void prefix_again(const SharedArgs &A, int h, int r0, int first, int count, int last, int R, float2 *mz,
                                          float *so) {
  rows_again<T, D>(AgainArgs<T>{static_cast<const T *>(A.q) + h * A.G * A.sq[1], A.sq[0], A.sq[1], A.sq[2], A.G * A.nq, A.nq, r0,
                                static_cast<const T *>(A.Kp) + h * A.skp[0], static_cast<const T *>(A.Vp) + h * A.svp[0], A.skp[1],
                                A.svp[1], nullptr, 0, first, NW, count, last, 0, A.c_log2},
                   R, mz, so);
}

// ---- fp32 prefix: 8 rows and a share of the keys per CTA ----
template <typename T, int D>
__global__ void __launch_bounds__(NT, kPerSm<T, D>) prefix_rows_kernel(const __grid_constant__ SharedArgs A, int groups, int per) {
  extern __shared__ __align__(16) unsigned char rings[];
  __shared__ float2 wmz[NW * 8];
  pdl_wait();
  pdl_launch();  // in this order: the next launch takes it that what precedes the call is complete (pdl.cuh)
  const int warp = threadIdx.x >> 5;
  const int grp = blockIdx.x % groups, rest = blockIdx.x / groups, h = rest % A.Hkv, s = rest / A.Hkv;
  const int r0 = grp * 8, R = min(8, A.rows - r0), gn = A.G * A.nq;
  const int k0 = s * per, k1 = min(A.P, k0 + per);
  Rows<T, D> S;
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
  if (S.leave(R, wmz + warp * 8, so + warp * R * D))
    prefix_again<T, D>(A, h, r0, k0 / 16 + warp, (tiles - warp + NW - 1) / NW, k1, R, wmz + warp * 8, so + warp * R * D);
  __syncthreads();
  const long at = ((long)s * A.Hkv + h) * A.rows + r0;
  join_warps<D, NW>(R, wmz, so, A.part + at * D, A.stat + at);
}

// ---- own slots ----
// The units (batch row, KV head, 8 of its query rows) one behind the other are a line of tiles of 16
// slots, and every warp takes an equal stretch of it: lengths differ, and what is done unit by unit
// waits for the longest.  A stretch inside one unit is a piece; piece number = warp + unit, which no
// two share.  The warp's ring runs on across the units, and no barrier follows the first one.
struct OwnArgs {
  float *part;   // [pieces][8][D]
  float2 *stat;  // [pieces][8]
  int2 *info;    // [units] first piece, pieces
  int groups;    // of 8 query rows
};
// CTAs of the own slots' kernel: those that run at once, and as many again with short stretches.
__host__ __device__ constexpr int own_ctas(int elem_bytes, int d) { return 2 * (elem_bytes == 4 && d == 128 ? 1 : 2) * kNumSmsHint; }
constexpr int kMinTiles = 4;      // of a stretch
constexpr int kLongShare = 90;    // per cent of the tiles
constexpr int kKeptHeads = 2048;  // lengths that are kept in shared memory

// Where the warps' stretches begin.  The first half of the warps, all of which run at once, have the larger
// part of the tiles; the others, which follow as CTAs end, have short stretches that even out
// what some SMs are slower than others.
struct Stretches {
  int total, half, big, small;
  __device__ __forceinline__ Stretches(int tiles, int warps) : total(tiles), half(warps / 2) {
    big = max(kMinTiles, (int)((long)tiles * kLongShare / 100 / half));
    const int rest = tiles - min((long)tiles, (long)big * half);
    small = max(kMinTiles, (rest + half - 1) / half);
  }
  __device__ __forceinline__ int first(int w) const {
    return (int)min((long)total, w <= half ? (long)big * w : (long)big * half + (long)small * (w - half));
  }
  __device__ __forceinline__ int of(int tile) const {
    return tile / big < half ? tile / big : half + (tile - big * half) / small;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(NT, kPerSm<T, D>) own_slots_kernel(const __grid_constant__ SharedArgs A,
                                                                    const __grid_constant__ OwnArgs W) {
  extern __shared__ __align__(16) unsigned char rings[];
  __shared__ int wsum[NW], upto[NT], kept[kKeptHeads];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Without a prefix launch in front nothing has waited for the kernels before this one.
  if (A.splits == 0) pdl_wait();
  pdl_launch();
  const int heads = A.B * A.Hkv;
  auto fetch = [&](int bh) {
    const int n = __ldcg(A.len + bh);
    return n < 0 || n > A.cap ? 0 : n;
  };
  auto length = [&](int bh) { return bh < kKeptHeads ? kept[bh] : fetch(bh); };
#pragma unroll 4
  for (int bh = threadIdx.x; bh < min(heads, kKeptHeads); bh += NT) kept[bh] = fetch(bh);
  __syncthreads();
  const int each = (heads + NT - 1) / NT, mine0 = threadIdx.x * each;
  int mine = 0;
  for (int bh = mine0; bh < min(heads, mine0 + each); ++bh) mine += (length(bh) + 15) >> 4;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) incl += wsum[w];
    total += wsum[w];
  }
  upto[threadIdx.x] = incl * W.groups;  // tiles up to this thread's last head
  __syncthreads();
  const Stretches P(total * W.groups, (int)gridDim.x * NW);
  const int me = blockIdx.x * NW + warp, lo = P.first(me), hi = P.first(me + 1);
  if (lo < hi) {
    // the head that tile lo is in
    int src = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) src += __popc(__ballot_sync(0xFFFFFFFFu, upto[i * 32 + lane] <= lo));
    int bh = src * each, before = src > 0 ? upto[src - 1] : 0;
    for (;; ++bh) {
      const int t = ((length(bh) + 15) >> 4) * W.groups;
      if (before + t > lo) break;
      before += t;
    }
    struct Cursor {
      int bh, grp, n, tiles, x;  // head, group, its slots and tiles, the tile at hand
    };
    Cursor at;
    at.bh = bh;
    at.n = length(bh);
    at.tiles = (at.n + 15) >> 4;
    at.grp = (lo - before) / at.tiles;
    at.x = lo - before - at.grp * at.tiles;
    auto advance = [&](Cursor &c) {
      if (++c.x < c.tiles) return;
      c.x = 0;
      if (++c.grp < W.groups) return;
      c.grp = 0;
      do {
        c.n = length(++c.bh);
      } while (c.n == 0);  // only called where a tile follows
      c.tiles = (c.n + 15) >> 4;
    };
    const int gn = A.G * A.nq;
    Rows<T, D> S;
    S.init(rings + warp * S.RING);
    Cursor ahead = at;
    auto fill = [&](int stage) {
      S.fill(stage, static_cast<const T *>(A.K) + (long)ahead.bh * A.cap * D, D,
             static_cast<const T *>(A.V) + (long)ahead.bh * A.cap * D, D, ahead.x * 16, ahead.n - 1);
    };
    const int count = hi - lo;
#pragma unroll
    for (int s = 0; s < S.STAGES - 1; ++s) {
      if (s < count) {
        if (s > 0) advance(ahead);
        fill(s);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    int stage = 0, lim[2];
    bool first = true;  // of a piece
    for (int y = 0; y < count; ++y) {
      const int R = min(8, gn - at.grp * 8);
      if (first) {
        const int b = at.bh / A.Hkv, h = at.bh - b * A.Hkv, r0 = at.grp * 8;
        S.load_q(static_cast<const T *>(A.q) + q_offset(A.sq, b, h, A.G, A.nq, r0 + min(S.g, R - 1)));
        // slots that rows 2t, 2t + 1 see
#pragma unroll
        for (int i = 0; i < 2; ++i) lim[i] = at.n - A.nq + (r0 + min(2 * S.t + i, R - 1)) % A.nq + 1;
        first = false;
        if (at.x == 0 && lane == 0) {
          const int u = at.bh * W.groups + at.grp, from = P.of(lo + y), to = P.of(lo + y + at.tiles - 1);
          W.info[u] = make_int2(from + u, to - from + 1);
        }
      }
      if (y + S.STAGES - 1 < count) {
        advance(ahead);
        fill(stage == 0 ? S.STAGES - 1 : stage - 1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group %0;" ::"n"(S.STAGES - 1) : "memory");
      __syncwarp();
      float l[4], small[4];
      S.logits(stage, l, small);
      if (at.x * 16 + 16 > at.n - A.nq + 1) S.hide(l, S.g, at.x * 16, lim);
      S.add(stage, l, small, A.c_log2);
      __syncwarp();  // the stage may be filled again
      if (++stage == S.STAGES) stage = 0;
      if (at.x + 1 == at.tiles || y + 1 == count) {
        const long piece = (long)me + at.bh * W.groups + at.grp;
        S.leave(R, W.stat + piece * 8, W.part + piece * 8 * D);  // what it could not hold is seen at the join
        S.fresh();
        first = true;
      }
      if (y + 1 < count) advance(at);
    }
  }
  if (A.splits) pdl_wait();  // this kernel does not end before the prefix's
}

// Piece s of a unit (of head bh, from tile `at` of its head's line on, `tiles` long): its first tile and how many.  Found
// anew from the lengths, by a warp, where a piece has to be attended again.
__device__ int2 piece_tiles(const int32_t *len, int cap, int heads, int groups, int warps, int bh, int at, int tiles, int s) {
  int before = 0, all = 0;
  for (int i = threadIdx.x & 31; i < heads; i += 32) {
    const int n = len[i], t = n < 0 || n > cap ? 0 : ((n + 15) >> 4) * groups;
    all += t;
    if (i < bh) before += t;
  }
  for (int o = 16; o; o >>= 1) {
    all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
    before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
  }
  at += before;
  const Stretches P(all, warps);
  const int w = P.of(at) + s, first = max(at, P.first(w)), last = min(at + tiles, P.first(w + 1));
  return make_int2(first - at, last - first);
}

// Attends again those of a row's pieces that are not finite, by a warp; whether there was one.
template <typename T, int D>
__device__ __noinline__ bool own_row_again(const SharedArgs &A, const OwnArgs &W, int bh, int row, int2 own, int n) {
  const int b = bh / A.Hkv, h = bh - b * A.Hkv, tiles = (n + 15) >> 4;
  bool some = false;
#pragma unroll 1
  for (int s = 0; s < own.y; ++s) {
    const long at = (long)(own.x + s) * 8 + row % 8;
    bool bad = W.stat[at].y != W.stat[at].y;
    for (int i = threadIdx.x & 31; i < D; i += 32) bad |= !(fabsf(W.part[at * D + i]) < INFINITY);
    if (!__any_sync(0xFFFFFFFFu, bad)) continue;
    const int2 of = piece_tiles(A.len, A.cap, A.B * A.Hkv, W.groups, own_ctas(sizeof(T), D) * NW, bh, row / 8 * tiles, tiles, s);
    const AgainArgs<T> args{static_cast<const T *>(A.q) + q_offset(A.sq, b, h, A.G, A.nq, row), 0, 0, 0, 1, 1, 0,
                            static_cast<const T *>(A.K) + (long)bh * A.cap * D, static_cast<const T *>(A.V) + (long)bh * A.cap * D, D, D,
                            nullptr, 0, of.x, 1, of.y, n - A.nq + row % A.nq + 1, 0, A.c_log2};
    some_rows_again<T, D, 1>(args, 1, W.stat + at, W.part + at * D);
    some = true;
  }
  return some;
}

// ---- everything joined: one warp a query row ----
// Latency counts: the row's length is read before the wait, and the prefix's first sums are on
// their way beside the statistics that say what they weigh.  Every share has left its sums (zeros where it saw
// nothing), and all are taken, so that a NaN reaches the output however little its share weighs.
template <typename T, int D>
__global__ void __launch_bounds__(NT) shared_join_kernel(const __grid_constant__ SharedArgs A, const __grid_constant__ OwnArgs W) {
  constexpr int E = D / 32, N = 16;  // elements of a lane, sums in flight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gn = A.G * A.nq;
  const long at = (long)blockIdx.x * NW + warp;
  const bool mine = at < (long)A.B * A.Hkv * gn;
  const int bh = mine ? (int)(at / gn) : 0;
  const int row = mine ? (int)(at - (long)bh * gn) : 0, b = bh / A.Hkv, h = bh - b * A.Hkv;
  // The launch before waits for the one before it, so what precedes the call is complete (nothing is known
  // of it where that launch is the call's first and may still be waiting).
  const bool early = A.splits > 0 && A.cap > 0;
  int n = 0;
  if (early) n = __ldcg(A.len + bh);
  pdl_wait();
  pdl_launch();
  if (!mine) return;
  if (!early && A.cap > 0) n = A.len[bh];
  if (n < 0 || n > A.cap) {
    if (row == 0 && lane == 0 && A.status) atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
    return;
  }
  float x[N][E];
  auto load = [&](int i, const float *p, bool there) {
#pragma unroll
    for (int y = 0; y < E; ++y) x[i][y] = 0.f;
    if (there) {
      if constexpr (E == 4) {
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(p) + lane);
        x[i][0] = v.x;
        x[i][1] = v.y;
        x[i][2] = v.z;
        x[i][3] = v.w;
      } else {
        const float2 v = __ldcs(reinterpret_cast<const float2 *>(p) + lane);
        x[i][0] = v.x;
        x[i][1] = v.y;
      }
    }
  };
  const long share = (long)A.Hkv * A.rows, first = (long)h * A.rows + (long)b * gn + row;
  const int2 own = n > 0 ? W.info[bh * W.groups + row / 8] : make_int2(0, 0);
  float2 st0 = make_float2(-INFINITY, 0.f), st1 = st0;  // prefix shares `lane` and 32 + lane (at most 64)
  if (lane < A.splits) st0 = A.stat[lane * share + first];
  if (32 + lane < A.splits) st1 = A.stat[(32 + lane) * share + first];
  const float2 *ws = W.stat + (long)own.x * 8 + row % 8;
  const float *wp = W.part + ((long)own.x * 8 + row % 8) * D;
  float M, Z, v[E];
#pragma unroll 1
  for (bool again = false;; again = true) {
#pragma unroll
    for (int i = 0; i < N; ++i) load(i, A.part + (i * share + first) * D, i < A.splits);
    M = -INFINITY;
    for (int s = lane; s < own.y; s += 32) {
      const float2 y = ws[s * 8];
      if (y.y != 0.f) M = fmaxf(M, y.x);
    }
    if (st0.y != 0.f) M = fmaxf(M, st0.x);
    if (st1.y != 0.f) M = fmaxf(M, st1.x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    auto factor = [&](const float2 &y) { return y.y != 0.f ? tc::ex2(M == -INFINITY ? 0.f : y.x - M) : 0.f; };
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = 0.f;
    // the N sums in registers, weighed by lanes from .. from + N - 1's f
    auto take = [&](float f, int from) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float w = __shfl_sync(0xFFFFFFFFu, f, from + i);
#pragma unroll
        for (int y = 0; y < E; ++y) v[y] += w * x[i][y];
      }
    };
    const float f0 = factor(st0), f1 = factor(st1);
    Z = f0 * st0.y + f1 * st1.y;
    if (A.splits > 0) take(f0, 0);
    for (int s0 = N; s0 < A.splits; s0 += N) {
#pragma unroll
      for (int i = 0; i < N; ++i) load(i, A.part + ((s0 + i) * share + first) * D, s0 + i < A.splits);
      take(s0 < 32 ? f0 : f1, s0 % 32);
    }
    for (int s0 = 0; s0 < own.y; s0 += N) {
#pragma unroll
      for (int i = 0; i < N; ++i) load(i, wp + (long)(s0 + i) * 8 * D, s0 + i < own.y);
      float f = 0.f;
      if (lane < N && s0 + lane < own.y) {
        const float2 y = ws[(s0 + lane) * 8];
        f = factor(y);
        Z += f * y.y;
      }
      take(f, 0);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) Z += __shfl_xor_sync(0xFFFFFFFFu, Z, o);
    // A row that is not finite: those of its own slots' pieces that are not are attended again (bf16: a sum of weights
    // that is no number is so by the formula).
    float zero = 0.f;  // stays so where all are finite
#pragma unroll
    for (int i = 0; i < E; ++i) zero = __fmaf_rn(v[i], 0.f, zero);
    if (again || !__any_sync(0xFFFFFFFFu, zero != 0.f || Z != Z) || (sizeof(T) == 2 && Z != Z)) break;
    if (!own_row_again<T, D>(A, W, bh, row, own, n)) break;
    __syncwarp();
  }
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
    const size_t n = (size_t)plan.splits * Hkv * rows, pieces = (size_t)own_ctas(dtype == KV_BF16 ? 2 : 4, d) * NW + units;
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
  char *p = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(ws) + 31) & ~uintptr_t(31));
  const Layout l(plan, Hkv, A.rows, (long)B * Hkv * W.groups, d, dtype);
  A.part = reinterpret_cast<float *>(p + l.prefix);
  A.stat = reinterpret_cast<float2 *>(p + l.prefix_stat);
  W.part = reinterpret_cast<float *>(p + l.own);
  W.stat = reinterpret_cast<float2 *>(p + l.own_stat);
  W.info = reinterpret_cast<int2 *>(p + l.info);
  if (dtype == KV_BF16) return d == 128 ? run<__nv_bfloat16, 128>(A, W, plan, st) : run<__nv_bfloat16, 64>(A, W, plan, st);
  return d == 128 ? run<float, 128>(A, W, plan, st) : run<float, 64>(A, W, plan, st);
}

}  // namespace kvc

// rows_stream.cuh -- softmax attention of up to 8 query rows over a stream of cache slots, one
// warp's share: what block-sparse attention and the shared prefix's own slots have in common.
//
// The warp takes 16 slots at a time as the long side of warp-level products: logits
// L^T = K Q^T (16 slots x 8 rows), outputs O^T += V^T P^T (d x 8 rows).  Which element of d stands at
// which k is free as long as both operands agree, so a lane takes 16 consecutive bytes of a
// row and K and V are used as they lie in memory; only P is transposed
// (in registers).  A lane holds the rows 2t and 2t + 1 of the 8, t = lane % 4.
//   bf16: K and q are exact; P enters as hi + lo, so that the weights keep 16 bits.
//   fp32: every operand as two tf32 parts (mma_common.cuh), sums joined outside the unit, which cuts off: logits by
//   a tree over the steps, O's tile by tile (logits of one sum in the unit: O twice as far off, where logits are large 4.5 times
//   as far as by plain fp32 operations; the tree takes no longer).
// The reference m of a row moves only when a logit passes it by kLazyRows (log2 units), so O
// is rarely rescaled.
//
// K and V rows come by asynchronous 16-byte copies into a ring of tiles that belongs to the warp
// alone, so that no barrier holds warps up and what is in flight takes no registers (with the
// next tile in registers and four CTAs an SM, 512 ragged units of 1124 slots ran at 4.6 TB/s, half of
// the stalls waiting for the one tile ahead).  16-byte pieces of a row are permuted so that the
// eight lanes of a shared-memory phase read different banks: K lanes read pieces 4c + t of rows g
// and g + 1, V lanes pieces 8c + g of four rows.  Rows that do not exist are filled with 0.
// The copies go past the first-level cache: a kernel that has not yet waited for the one in front
// of it (but knows that those before that one are complete) may read what they wrote.
#pragma once

#include "kvc_internal.cuh"
#include "mma_common.cuh"
#include "tc_common.cuh"

namespace kvc {

constexpr float kLazyRows = 6.f;

// c (+)= 16 rows x 8 columns over the 32 (bf16) or 16 (fp32) elements that four lanes' vectors hold.
__device__ __forceinline__ void dot16(float (&c)[4], float (&)[4], const uint4 &x0, const uint4 &x1, const uint4 &q,
                                      __nv_bfloat16) {
  mma_bf16(c, x0.x, x1.x, x0.y, x1.y, q.x, q.y);
  mma_bf16(c, x0.z, x1.z, x0.w, x1.w, q.z, q.w);
}
__device__ __forceinline__ void dot16(float (&c)[4], float (&small)[4], const uint4 &x0, const uint4 &x1, const uint4 &q,
                                      float) {
  Split a[4], b0, b1;
  a[0].set(__uint_as_float(x0.x));
  a[1].set(__uint_as_float(x1.x));
  a[2].set(__uint_as_float(x0.y));
  a[3].set(__uint_as_float(x1.y));
  b0.set(__uint_as_float(q.x));
  b1.set(__uint_as_float(q.y));
  mma_split(c, small, a, b0, b1);
  a[0].set(__uint_as_float(x0.z));
  a[1].set(__uint_as_float(x1.z));
  a[2].set(__uint_as_float(x0.w));
  a[3].set(__uint_as_float(x1.w));
  b0.set(__uint_as_float(q.z));
  b1.set(__uint_as_float(q.w));
  mma_split(c, small, a, b0, b1);
}

__device__ __forceinline__ void add4(const float (&a)[4], const float (&b)[4], float (&c)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const float2 x = __fadd2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
    c[i] = x.x;
    c[i + 1] = x.y;
  }
}
// The same for fp32 with the large products' sums from 0 for each of the two steps, joined by an addition that rounds where
// the unit would cut off.
__device__ __forceinline__ void dot16_from_0(float (&c)[4], float (&small)[4], const uint4 &x0, const uint4 &x1, const uint4 &q) {
  const uint32_t a[4] = {x0.x, x1.x, x0.y, x1.y}, b[4] = {x0.z, x1.z, x0.w, x1.w};
  float sum[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    Split x[4], y0, y1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i].set(__uint_as_float(h ? b[i] : a[i]));
      sum[h][i] = 0.f;
    }
    y0.set(__uint_as_float(h ? q.z : q.x));
    y1.set(__uint_as_float(h ? q.w : q.y));
    mma_split(sum[h], small, x, y0, y1);
  }
  add4(sum[0], sum[1], c);
}

// log2 units
__device__ __forceinline__ float rows_max(float x) {  // over the 16 slots: the lanes with the same t
  x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
}

template <typename T, int D, int NS>  // NS: tiles of a warp's ring
struct RowStream {
  static constexpr int NCH = D * (int)sizeof(T) / 64;  // 64-byte chunks of a row
  static constexpr int EV = 16 / (int)sizeof(T);       // elements of a 16-byte piece
  static constexpr int VV = D / 8 / EV;                // pieces of a lane's D / 8 elements of a V row
  static constexpr int MT = D / 16;
  static constexpr int ROW = D * (int)sizeof(T), TILE = 32 * ROW;  // bytes; 16 rows of K, then 16 of V
  static constexpr int STAGES = NS;
  static constexpr int RING = STAGES * TILE;  // bytes of a warp

  uint4 q[NCH];    // column g = lane / 4 of the 8: its row's chunks, bytes 16 t
  float o[MT][4];  // elements at(i) + {0, 0, 1, 1}, rows 2t + {0, 1, 0, 1}
  float m[2], z[2];
  int g, t;
  unsigned char *ring;

  __device__ __forceinline__ void init(unsigned char *warp_ring) {
    const int lane = threadIdx.x & 31;
    g = lane >> 2;
    t = lane & 3;
    ring = warp_ring;
    fresh();
  }
  __device__ __forceinline__ int at(int i) const { return 2 * i / EV * 8 * EV + EV * g + 2 * i % EV; }
  // `row`: the query row of column g
  __device__ __forceinline__ void load_q(const T *row) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) q[c] = __ldcg(reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(row) + c * 64 + t * 16));
  }
  __device__ __forceinline__ static int k_swizzle(int row) { return (row & 1) << 2; }
  // the slots of a lane: bf16 2t, 2t + 1, 2t + 8, 2t + 9 (the k indices of its operand); fp32 t, t + 4, t + 8, t + 12
  __device__ __forceinline__ static int v_slot(int t, int r) { return sizeof(T) == 2 ? 2 * t + (r & 1) + 8 * (r >> 1) : t + 4 * r; }
  __device__ __forceinline__ static int v_swizzle(int row) { return (sizeof(T) == 2 ? row >> 1 & 3 : row & 3) << 1; }
  // Slots j .. j + 15 into a stage; those behind `last` become 0.
  __device__ __forceinline__ void fill(int stage, const T *k, long ks, const T *v, long vs, int j, int last) {
    constexpr int CPR = ROW / 16;
    unsigned char *dst = ring + stage * TILE;
#pragma unroll
    for (int i = 0; i < 16 * CPR / 32; ++i) {
      const int e = i * 32 + (threadIdx.x & 31), row = e / CPR, c = e % CPR;
      const bool there = j + row <= last;
      const long at = there ? j + row : last;
      const uint32_t n = there ? 16 : 0;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst + row * ROW + ((c ^ k_swizzle(row)) << 4))),
                   "l"(reinterpret_cast<const char *>(k + at * ks) + c * 16), "r"(n)
                   : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       tc::smem_u32(dst + 16 * ROW + row * ROW + ((c ^ v_swizzle(row)) << 4))),
                   "l"(reinterpret_cast<const char *>(v + at * vs) + c * 16), "r"(n)
                   : "memory");
    }
  }
  __device__ __forceinline__ void fresh() {  // nothing attended yet
    m[0] = m[1] = -INFINITY;
    z[0] = z[1] = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
  }
  // Attends `count` tiles of 16 slots; slot(y): tile y's first.  Slots behind `last` are not there; row 2t + x sees
  // those below lim[x], and all of them below `whole`.
  template <typename F>
  __device__ __forceinline__ void run(int count, F slot, const T *k, long ks, const T *v, long vs, int last, float c_log2,
                                      const int (&lim)[2], int whole) {
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
      if (s < count) fill(s, k, ks, v, vs, slot(s), last);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    int stage = 0;
    for (int y = 0; y < count; ++y) {
      const int ahead = y + STAGES - 1;
      if (ahead < count) fill(stage == 0 ? STAGES - 1 : stage - 1, k, ks, v, vs, slot(ahead), last);
      asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
      __syncwarp();
      float l[4], small[4];
      logits(stage, l, small);
      const int j = slot(y);
      if (j + 16 > whole) hide(l, g, j, lim);
      add(stage, l, small, c_log2);
      __syncwarp();  // the stage may be filled again
      if (++stage == STAGES) stage = 0;
    }
  }
  // Logits of a stage's K tile before the scale, l + small (0 in bf16): l[0], l[1] slot g of rows 2t, 2t + 1; l[2], l[3] slot g + 8.
  __device__ __forceinline__ void logits(int stage, float (&l)[4], float (&small)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) l[i] = small[i] = 0.f;
    const unsigned char *p = ring + stage * TILE + g * ROW;
    const int sw = k_swizzle(g);  // of row g + 8 too
    auto piece = [&](int c, int r) { return *reinterpret_cast<const uint4 *>(p + r * ROW + (((4 * c + t) ^ sw) << 4)); };
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) dot16(l, small, piece(c, 0), piece(c, 8), q[c], T());
    } else {
      // a tree: what is added up step by step is off by 2^-24 of the whole sum each time
#pragma unroll
      for (int c = 0; c < NCH; c += 2) {
        float u[4], v[4];
        dot16_from_0(u, small, piece(c, 0), piece(c, 8), q[c]);
        dot16_from_0(v, small, piece(c + 1, 0), piece(c + 1, 8), q[c + 1]);
        add4(u, v, u);
        add4(l, u, l);
      }
    }
  }
  // Row 2t + x sees the slots below n[x]; j: the tile's first slot.
  __device__ __forceinline__ static void hide(float (&l)[4], int g, int j, const int (&n)[2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j + g + 8 * (i >> 1) >= n[i & 1]) l[i] = -INFINITY;
  }
  // The softmax's step and O += P V with a stage's V tile.
  // (The small products' sum joins the others where the reference has been subtracted: a large logit has fewer places.)
  __device__ __forceinline__ void add(int stage, const float (&l)[4], const float (&small)[4], float c_log2) {
    const float a = fmaxf(l[0], l[2]) * c_log2, b = fmaxf(l[1], l[3]) * c_log2;
    if (__any_sync(0xFFFFFFFFu, a > m[0] + kLazyRows || b > m[1] + kLazyRows)) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float mn = fmaxf(m[x], rows_max(x ? b : a));
        const float f = mn == -INFINITY ? 1.f : tc::ex2(m[x] - mn);
        m[x] = mn;
        z[x] *= f;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          o[i][x] *= f;
          o[i][2 + x] *= f;
        }
      }
    }
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float ref = m[i & 1];
      const float x = __fmaf_rn(l[i], c_log2, ref == -INFINITY ? 0.f : -ref);
      p[i] = tc::ex2(sizeof(T) == 4 ? __fmaf_rn(small[i], c_log2, x) : x);
    }
    z[0] += p[0] + p[2];
    z[1] += p[1] + p[3];
    uint4 vw[4][VV];  // pieces 8c + g of the lane's four slots
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = v_slot(t, r);
      const unsigned char *src = ring + stage * TILE + (16 + row) * ROW;
#pragma unroll
      for (int c = 0; c < VV; ++c) vw[r][c] = *reinterpret_cast<const uint4 *>(src + (((8 * c + g) ^ v_swizzle(row)) << 4));
    }
    product(vw, p, T());
  }
  __device__ __forceinline__ void product(const uint4 (&vw)[4][VV], const float (&p)[4], __nv_bfloat16) {
    uint32_t b[2][2];  // hi, lo
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __nv_bfloat162 hi = __floats2bfloat162_rn(p[2 * h], p[2 * h + 1]);
      const uint32_t w = *reinterpret_cast<const uint32_t *>(&hi);
      const __nv_bfloat162 lo =
          __floats2bfloat162_rn(p[2 * h] - __uint_as_float(w << 16), p[2 * h + 1] - __uint_as_float(w & 0xFFFF0000u));
      b[0][h] = transpose8x8(w);
      b[1][h] = transpose8x8(*reinterpret_cast<const uint32_t *>(&lo));
    }
#pragma unroll
    for (int c = 0; c < VV; ++c) {
      const uint32_t w0[4] = {vw[0][c].x, vw[0][c].y, vw[0][c].z, vw[0][c].w};
      const uint32_t w1[4] = {vw[1][c].x, vw[1][c].y, vw[1][c].z, vw[1][c].w};
      const uint32_t w2[4] = {vw[2][c].x, vw[2][c].y, vw[2][c].z, vw[2][c].w};
      const uint32_t w3[4] = {vw[3][c].x, vw[3][c].y, vw[3][c].z, vw[3][c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = __byte_perm(w0[i], w1[i], 0x5410), a1 = __byte_perm(w0[i], w1[i], 0x7632);
        const uint32_t a2 = __byte_perm(w2[i], w3[i], 0x5410), a3 = __byte_perm(w2[i], w3[i], 0x7632);
        mma_bf16(o[c * 4 + i], a0, a1, a2, a3, b[0][0], b[0][1]);
        mma_bf16(o[c * 4 + i], a0, a1, a2, a3, b[1][0], b[1][1]);
      }
    }
  }
  __device__ __forceinline__ void product(const uint4 (&vw)[4][VV], const float (&p)[4], float) {
    // operand of the two k steps: slots t, t + 4 and t + 8, t + 12 of row g; lane 4 s + r / 2 holds slot s of row r
    Split b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int src = (t + 4 * (k & 1)) * 4 + (g >> 1);
      const float even = __shfl_sync(0xFFFFFFFFu, p[2 * (k >> 1)], src), odd = __shfl_sync(0xFFFFFFFFu, p[2 * (k >> 1) + 1], src);
      b[k].set(g & 1 ? odd : even);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      float c[4] = {0.f, 0.f, 0.f, 0.f}, small[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        Split a[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {  // (element, slot): (0, t), (1, t), (0, t + 4), (1, t + 4)
          const uint4 &w = vw[2 * k + (x >> 1)][i >> 1];
          a[x].set(__uint_as_float(i & 1 ? (x & 1 ? w.w : w.z) : (x & 1 ? w.y : w.x)));
        }
        mma_split(c, small, a, b[2 * k], b[2 * k + 1]);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) o[i][x] += c[x] + small[x];
    }
  }
  // A warp's share of the rows below R alone: reference and sum of weights mz [R], output sums so [R][D].  True
  // where the products could not hold it (rows_again).
  __device__ __forceinline__ bool leave(int R, float2 *mz, float *so) {
    bool bad = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      z[x] += __shfl_xor_sync(0xFFFFFFFFu, z[x], 4);
      z[x] += __shfl_xor_sync(0xFFFFFFFFu, z[x], 8);
      z[x] += __shfl_xor_sync(0xFFFFFFFFu, z[x], 16);
      const int r = 2 * t + x;
      if (r < R) {
        if (g == 0) mz[r] = make_float2(m[x], z[x]);
        float2 zero = make_float2(0.f, 0.f);  // stays so where all are finite
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const float2 v = make_float2(o[i][x], o[i][2 + x]);
          *reinterpret_cast<float2 *>(so + r * D + at(i)) = v;
          zero = __ffma2_rn(v, make_float2(0.f, 0.f), zero);
        }
        // bf16: a logit that is no number is so by the formula, and the row with it
        bad |= zero.x + zero.y != 0.f && (sizeof(T) == 4 || z[x] == z[x]);
      }
    }
    return __any_sync(0xFFFFFFFFu, bad);
  }
};

// A share made anew where sums came out that are not finite.  The products cannot hold an infinity in V (its weight's
// lower part, or a hidden slot's weight of 0, makes it a NaN), nor in fp32 one in K or q or what is so large that its
// upper tf32 part is infinite.  Here each weight is one float, its products are sums of fp32, slots that a row does
// not see are left out, and weights are at most 1, so that what is finite in the end is so on the way.  32 slots at a time, a
// lane's logits for all rows, then their V rows one by one; it costs several times what
// the products do.
template <typename T>
struct AgainArgs {
  const T *q;          // row r is row r0 + r: batch entry / gn, head / nq, token % nq
  long sb, sg, st;
  int gn, nq, r0;
  const T *k, *v;
  long ks, vs;
  const uint16_t *list;  // tile x is that of block list[x >> tl] (NULL: slots 16 x and on)
  int tl;
  int x0, step, count;   // tiles x0, x0 + step, ...
  int lim, by_token;     // slots that row r sees: lim + by_token * its token
  float c_log2;
};
template <typename T, int D, int N>  // at most N rows
__device__ __noinline__ void some_rows_again(const AgainArgs<T> &A, int R, float2 *mz, float *so) {
  constexpr int EV = 16 / (int)sizeof(T), E = D / 32;
  const int lane = threadIdx.x & 31;
  __syncwarp();  // mz, so
  int lim[N], most = 0;
  const uint4 *q[N];
  float ref[N], z[N], acc[N][E];
  bool search = false;  // a reference is to be found anew
#pragma unroll
  for (int r = 0; r < N; ++r) {
    const int row = A.r0 + min(r, R - 1), b = row / A.gn, in = row - b * A.gn;
    q[r] = reinterpret_cast<const uint4 *>(A.q + b * A.sb + in / A.nq * A.sg + in % A.nq * A.st);
    lim[r] = r < R ? A.lim + A.by_token * (row % A.nq) : 0;
    most = max(most, lim[r]);
    const float2 s = mz[min(r, R - 1)];
    ref[r] = s.x == -INFINITY ? s.x : s.x + kLazyRows;
    search |= s.y != s.y;
    z[r] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[r][e] = 0.f;
  }
  // this lane's slot of the 32 from tile y on (-1: none), and its logits
  auto slot = [&](int y) {
    y += lane >> 4;
    if (y >= A.count) return -1;
    const int x = A.x0 + y * A.step;
    const int j = (A.list ? ((int)A.list[x >> A.tl] << (A.tl + 4)) + ((x & ((1 << A.tl) - 1)) << 4) : x << 4) + (lane & 15);
    return j < most ? j : -1;
  };
  auto logits = [&](int j, float (&l)[N]) {
    const uint4 *k = reinterpret_cast<const uint4 *>(A.k + max(j, 0) * A.ks);
#pragma unroll
    for (int r = 0; r < N; ++r) l[r] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D / EV; ++c) {
      float x[EV], y[EV];
      Vec16<T>::unpack(k[c], x);
#pragma unroll
      for (int r = 0; r < N; ++r) {
        Vec16<T>::unpack(q[r][c], y);
#pragma unroll
        for (int e = 0; e < EV; ++e) l[r] = __fmaf_rn(x[e], y[e], l[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < N; ++r) l[r] = j >= 0 && j < lim[r] ? l[r] : -INFINITY;
  };
  if (search) {
#pragma unroll
    for (int r = 0; r < N; ++r) ref[r] = -INFINITY;
#pragma unroll 1
    for (int y = 0; y < A.count; y += 2) {
      float l[N];
      logits(slot(y), l);
#pragma unroll
      for (int r = 0; r < N; ++r) ref[r] = fmaxf(ref[r], l[r] * A.c_log2);
    }
#pragma unroll
    for (int r = 0; r < N; ++r)
      for (int o = 16; o; o >>= 1) ref[r] = fmaxf(ref[r], __shfl_xor_sync(0xFFFFFFFFu, ref[r], o));
  }
#pragma unroll 1
  for (int y = 0; y < A.count; y += 2) {
    const int j = slot(y);
    float p[N];
    logits(j, p);
#pragma unroll
    for (int r = 0; r < N; ++r) {
      p[r] = tc::ex2(__fmaf_rn(p[r], A.c_log2, ref[r] == -INFINITY ? 0.f : -ref[r]));
      z[r] += p[r];
    }
#pragma unroll 8
    for (int s = 0; s < 32; ++s) {
      const int js = __shfl_sync(0xFFFFFFFFu, j, s);
      const T *v = A.v + max(js, 0) * A.vs + lane * E;
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = to_f32(v[e]);
#pragma unroll
      for (int r = 0; r < N; ++r) {
        const float w = __shfl_sync(0xFFFFFFFFu, p[r], s);
        const bool sees = js >= 0 && js < lim[r];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] = sees ? __fmaf_rn(w, x[e], acc[r][e]) : acc[r][e];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < N; ++r) {
    for (int o = 16; o; o >>= 1) z[r] += __shfl_xor_sync(0xFFFFFFFFu, z[r], o);
    // the reference and the sum of weights stay as they are where they can
    constexpr float up = 1 << (int)kLazyRows;
    bool over = search;
#pragma unroll
    for (int e = 0; e < E; ++e) over |= fabsf(acc[r][e]) < INFINITY && !(fabsf(acc[r][e] * up) < INFINITY);
    over = __any_sync(0xFFFFFFFFu, over);
    if (r < R) {
      if (lane == 0 && over) mz[r] = make_float2(ref[r], z[r]);
#pragma unroll
      for (int e = 0; e < E; ++e) so[r * D + lane * E + e] = over ? acc[r][e] : acc[r][e] * up;
    }
  }
}

template <typename T, int D>
__device__ __forceinline__ void rows_again(AgainArgs<T> A, int R, float2 *mz, float *so) {
  constexpr int N = 4;  // the calling kernel has to have the registers
#pragma unroll 1
  for (int r = 0; r < R; r += N, A.r0 += N) some_rows_again<T, D, N>(A, min(N, R - r), mz + r, so + r * D);
}

// The shares of NW warps (wmz [NW][8], so [NW][R][D]) as one: sh [R][D], mz [R].  A share without
// slots has z = 0, sums of 0 and weighs nothing; a NaN in z or in the sums is passed on.
template <int D, int NW>
__device__ __forceinline__ void join_warps(int R, const float2 *wmz, const float *so, float *sh, float2 *mz) {
  for (int i = threadIdx.x; i < R * D; i += 32 * NW) {
    const int r = i / D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w)
      if (wmz[w * 8 + r].y != 0.f) M = fmaxf(M, wmz[w * 8 + r].x);
    float v = 0.f, Z = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float2 s = wmz[w * 8 + r];
      const float f = s.y == 0.f ? 0.f : M == -INFINITY ? 1.f : tc::ex2(s.x - M);
      v += f * so[w * R * D + i];
      Z += f * s.y;
    }
    sh[i] = v;
    if (i % D == 0) mz[r] = make_float2(M, Z);
  }
}

}  // namespace kvc

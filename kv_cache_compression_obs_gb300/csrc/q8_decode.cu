// q8_decode.cu -- one decode step over the 8-bit slot cache (H2O page, 问题形式化:
// attention renormalised over the kept keys; 贪心驱逐算法: the softmax accumulates
// into a per-token score).
//
// A unit is (b, KV head); its rows are the n cached slots and the new token (row n).
// With codes c and block scales a (q8_common.cuh), for the G query heads of a unit:
//     l_gj = scale a_j <q_g, c_j>,  P_g = softmax_j(l_gj),  o_g = sum_j P_gj b_j v_j,
//     acc_j += sum_g P_gj  (the new token's starts with its own sum).
// Two launches:
//
//   stream   -- the codes of the full blocks in ns splits per unit, one CTA each,
//               and one more CTA per unit for the unfinished block's rows and the
//               new token.  A warp takes 16 slots at a time and feeds them to
//               mma.m16n8k16: codes are exact in fp16, so
//               an int8 becomes 1024 + 128 + c by a byte permutation and a packed
//               subtraction, an e4m3 by the hardware conversion.  Which element of
//               d stands at which k of the product is free as long as both operands
//               agree, so every lane takes 16 consecutive bytes of a row and nothing is
//               transposed: for K the k index runs over d, for V over the slots, two
//               neighbouring slots' bytes interleaved.  Rows go from memory to
//               registers (through shared memory by bulk copies measured 5% slower:
//               the warps then wait for one another), the next tile's as soon as the
//               registers are free.
//               fp32 accuracy: the queries and the weights P enter as hi + lo pairs of
//               fp16 (22 bits; each scaled by a power of two so that nothing that
//               matters is subnormal) in neighbouring columns of the 8-column operand:
//               columns 2i, 2i+1 are query i's hi and lo, and a lane's two
//               accumulators of a row add up to the result.  Four queries fill one
//               operand; five to eight take two.
//               Logits (log2 units) also go to the workspace.
//   finalize -- combines the splits into o, turns the stored logits into
//               probabilities and adds them to acc, and quantises the unfinished
//               block when the new token fills it.
// Bound by memory: 64 units of 131000 int8 slots 385 us, the stream launch at 0.97 of the copy
// rate; 256 units of 700 to 8191 e4m3 slots 62.7 us, where a CTA's start (length, queries,
// first rows) shows.  Short caches take one launch (below): 8 units of 1638 slots 10.8 us.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "pdl.cuh"
#include "q8_common.cuh"
#include "tc_common.cuh"

namespace kvc {
namespace {

constexpr int NW = 4;            // warps of a stream CTA
constexpr int NT = 32 * NW;
constexpr int NTF = 256;         // finalize threads
constexpr int SLOTS_F = 2048;    // slots per finalize CTA (1024 and 4096: 2% slower)
constexpr int kMaxSplits = 256;
constexpr float kLazy = 6.f;     // log2 units a logit may pass the running reference by
constexpr int kMinExp = -118;    // smallest exponent of a V scale that is told apart (2^(8 + 118) is finite)
constexpr int kPScale = 8;       // weights enter the product as P 2^kPScale (at most 2^(6 + 8 + 1))

struct DecArgs {
  const void *q, *k_new, *v_new;
  kv_q8_cache c;
  const int32_t *row_pos;
  int32_t new_pos;
  int32_t *len_out;
  int G, ns, b_log2;
  float c_log2;      // scale log2(e)
  float *o;
  float *lgw;        // [units][cap + 1][G] logits
  float2 *pmz;       // [units][ns + 1][G] max and normaliser
  float *po;         // [units][ns + 1][G][d]
  int32_t *nsave;    // [units] len at entry, -1 when out of range
  int *status;
};

// slots [k0, k1) of split s of a unit with nf slots in full blocks
__device__ __forceinline__ int split_len(int nf, int ns) { return ((nf + ns - 1) / ns + 63) & ~63; }

template <int FMT>
__device__ __forceinline__ uint32_t to_half2_lo(uint32_t w);  // codes 0, 1 of a word
template <int FMT>
__device__ __forceinline__ uint32_t to_half2_hi(uint32_t w);  // codes 2, 3

__device__ __forceinline__ uint32_t sub_bias(uint32_t h) {
  uint32_t r;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));  // (1024 + 128 + c) - 1152
  return r;
}
__device__ __forceinline__ uint32_t cvt_e4m3(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
  return r;
}
// int8 words arrive with every sign bit flipped (c + 128)
template <> __device__ __forceinline__ uint32_t to_half2_lo<KV_Q8_S8>(uint32_t w) {
  return sub_bias(__byte_perm(w, 0x64646464u, 0x4140));
}
template <> __device__ __forceinline__ uint32_t to_half2_hi<KV_Q8_S8>(uint32_t w) {
  return sub_bias(__byte_perm(w, 0x64646464u, 0x4342));
}
template <> __device__ __forceinline__ uint32_t to_half2_lo<KV_Q8_E4M3>(uint32_t w) { return cvt_e4m3(w); }
template <> __device__ __forceinline__ uint32_t to_half2_hi<KV_Q8_E4M3>(uint32_t w) { return cvt_e4m3(w >> 16); }
template <int FMT> __device__ __forceinline__ uint32_t fix(uint32_t w) {
  return FMT == KV_Q8_S8 ? w ^ 0x80808080u : w;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// The largest |x| of a query row -> the exponent e with max 2^e in [2^13, 2^14).
__device__ __forceinline__ int query_shift(float big) {
  if (!(big > 0.f)) return 0;
  int ex;
  frexpf(big, &ex);  // big = f 2^ex, 0.5 <= f < 1
  return max(-126, min(126, 14 - ex));
}

// ---- the unfinished block's rows and the new token ------------------------------------
// Rows 0 .. rows - 1 (the last one the new token) over the warps of one CTA: D / 16 lanes a
// row, 16 elements each, all rows of a warp in flight at once.  Leaves each warp's maximum,
// normaliser and output share where the stream's warps leave theirs, and the rows' logits in lg.
template <typename T, int D>
__device__ void tail_part(const DecArgs &A, long u, int n, float *lg, float *qs, float *wm, float *wz, float *so) {
  constexpr int LPR = D / 16, RPS = 32 / LPR, STEPS = 128 / (NW * RPS);
  const int G = A.G, block = A.c.block;
  const int nf = n / block * block, rows = n - nf + 1;  // at most block
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % LPR, rl = lane / LPR;
  const T *q = static_cast<const T *>(A.q) + u * (long)G * D;
  const T *kn = static_cast<const T *>(A.k_new) + u * (long)D, *vn = static_cast<const T *>(A.v_new) + u * (long)D;
  T *kt = static_cast<T *>(A.c.Kt) + u * (long)block * D, *vt = static_cast<T *>(A.c.Vt) + u * (long)block * D;
  for (int i = threadIdx.x; i < G * D; i += NT) qs[i] = to_f32(q[i]) * A.c_log2;
  for (int i = threadIdx.x; i < D; i += NT) {  // append: nobody reads this row as a cached one
    kt[(long)(rows - 1) * D + i] = kn[i];
    vt[(long)(rows - 1) * D + i] = vn[i];
  }
  if (threadIdx.x == 0) A.c.pos[u * (long)A.c.cap + n] = A.row_pos ? A.row_pos[u / A.c.Hkv] : A.new_pos;
  __syncthreads();
  for (int gb = 0; gb < G; gb += 4) {  // four query heads at a time
    float l[STEPS][4];
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int row = (s * NW + warp) * RPS + rl;
      if ((s * NW + warp) * RPS >= rows) break;
      float x[16];
      if (row < rows) {
        load16((row == rows - 1 ? kn : kt + (long)row * D) + sub * 16, x);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float t = 0.f;
        const float4 *q4 = reinterpret_cast<const float4 *>(qs + min(gb + g, G - 1) * D + sub * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 y = q4[i];
          t += x[4 * i] * y.x + x[4 * i + 1] * y.y + x[4 * i + 2] * y.z + x[4 * i + 3] * y.w;
        }
#pragma unroll
        for (int o = LPR / 2; o; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
        l[s][g] = row < rows ? t : -INFINITY;
        m[g] = fmaxf(m[g], l[s][g]);
        if (A.c.acc && sub == 0 && row < rows && gb + g < G)
          lg[row * G + gb + g] = t;
      }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) m[g] = fmaxf(m[g], __shfl_xor_sync(0xFFFFFFFFu, m[g], o));
    float o[4][16];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[g][i] = 0.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int row = (s * NW + warp) * RPS + rl;
      if ((s * NW + warp) * RPS >= rows) break;
      float x[16];
      if (row < rows) {
        load16((row == rows - 1 ? vn : vt + (long)row * D) + sub * 16, x);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float p = row < rows ? tc::ex2(l[s][g] - m[g]) : 0.f;
        z[g] += p;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[g][i] += p * x[i];
      }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
#pragma unroll
      for (int w = LPR; w < 32; w <<= 1) z[g] += __shfl_xor_sync(0xFFFFFFFFu, z[g], w);
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int w = LPR; w < 32; w <<= 1) o[g][i] += __shfl_xor_sync(0xFFFFFFFFu, o[g][i], w);
      if (gb + g < G && rl == 0) {
        float *dst = so + (warp * G + gb + g) * D + sub * 16;
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[i] = o[g][i];
        if (sub == 0) {
          wm[warp * 8 + gb + g] = m[g];
          wz[warp * 8 + gb + g] = z[g];
        }
      }
    }
  }
}

// The warps' shares (wm, wz, so) as one: po [G][D], pmz [G].
template <int D>
__device__ __forceinline__ void combine_warps(int G, const float *wm, const float *wz, const float *so, float *po,
                                              float2 *pmz) {
  __syncthreads();
  for (int i = threadIdx.x; i < G * D; i += NT) {
    const int qi = i / D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, wm[w * 8 + qi]);
    float v = 0.f, Z = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = tc::ex2(wm[w * 8 + qi] - M);  // a warp without a row: 2^-inf = 0, its o and z are 0
      v += f * so[w * G * D + i];
      Z += f * wz[w * 8 + qi];
    }
    po[i] = v;
    if (i % D == 0) pmz[qi] = make_float2(M, Z);
  }
}

// ---- stream -----------------------------------------------------------------------------
// Slots [k0, k1) (whole blocks) of unit u over the warps of one CTA; their logits to lg, each
// warp's maximum, normaliser and output share to wm, wz and so.
// NSET operands of four queries each; D head dim.
template <typename T, int FMT, int D, int NSET>
__device__ __forceinline__ void stream_range(const DecArgs &A, long u, int k0, int k1, float *lg, float *wm, float *wz,
                                             float *so) {
  constexpr int VB = D / 8;       // V bytes per lane and slot
  constexpr int MT = D / 16;      // 16-row tiles of V^T
  constexpr int NCH = D / 64;     // 64-byte chunks of a K row
  const int G = A.G, bl = A.b_log2;
  const uint8_t *kc = static_cast<const uint8_t *>(A.c.K) + u * (long)A.c.cap * D;
  const uint8_t *vc = static_cast<const uint8_t *>(A.c.V) + u * (long)A.c.cap * D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  // this lane's pieces of a tile: 16 bytes (or 2 x 16) of the K rows g and g + 8, VB bytes of
  // the V rows 2t, 2t + 1, 2t + 8 and 2t + 9
  uint4 kw[2][NCH];
  uint32_t vw[4][VB / 4];
  auto load_k = [&](int j) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < NCH; ++c)
        kw[h][c] = __ldcs(reinterpret_cast<const uint4 *>(kc + (long)(j + g + 8 * h) * D + c * 64 + t * 16));
  };
  auto load_v = [&](int j) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t *p = vc + (long)(j + 2 * t + (r & 1) + 8 * (r >> 1)) * D + g * VB;
      if constexpr (VB == 16) {
        const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p));
        vw[r][0] = w.x;
        vw[r][1] = w.y;
        vw[r][2] = w.z;
        vw[r][3] = w.w;
      } else {
        const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(p));
        vw[r][0] = w.x;
        vw[r][1] = w.y;
      }
    }
  };
  const int first = k0 + warp * 16;
  if (first < k1) {  // on their way before the queries are read
    load_k(first);
    load_v(first);
  }

  // queries: column 2i hi, 2i + 1 lo of query i of the set; this lane holds column g
  uint32_t qb[NSET][NCH * 4][2];
  float qf[NSET];  // query t's factor back to log2 units
#pragma unroll
  for (int st = 0; st < NSET; ++st) {
    const int qi = st * 4 + (g >> 1);
    const T *q = static_cast<const T *>(A.q) + (u * G + min(qi, G - 1)) * (long)D;
    float x[NCH][16];
    float big = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      load16(q + c * 64 + t * 16, x[c]);
      big = fmaxf(big, max_abs16(x[c]));
    }
    big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
    const int sh = query_shift(big);
    const float f = exp2i(sh);
    // query t's shift sits in the lanes with g = 2t
    qf[st] = A.c_log2 * exp2i(-__shfl_sync(0xFFFFFFFFu, sh, 8 * t));
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float a = x[c][4 * i + 2 * p] * f, b = x[c][4 * i + 2 * p + 1] * f;
          const uint32_t hi = pack_half2(a, b);
          const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
          const uint32_t lo = pack_half2(a - back.x, b - back.y);
          qb[st][c * 4 + i][p] = qi < G ? ((g & 1) ? lo : hi) : 0u;
        }
  }
  float o[NSET][MT][4], m[NSET], z[NSET];
#pragma unroll
  for (int st = 0; st < NSET; ++st) {
    m[st] = -INFINITY;
    z[st] = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[st][i][j] = 0.f;
  }
  int rv = kMinExp;  // o stands for o 2^(rv - kPScale)
  const float *ks = A.c.Ks + u * (long)(A.c.cap >> bl), *vs = A.c.Vs + u * (long)(A.c.cap >> bl);

  for (int j = first; j < k1; j += NW * 16) {
    const int next = j + NW * 16;
    const float ak = ks[j >> bl], av = vs[j >> bl];

    float sc[NSET][4];
#pragma unroll
    for (int st = 0; st < NSET; ++st)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[st][i] = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const uint32_t w0[4] = {kw[0][c].x, kw[0][c].y, kw[0][c].z, kw[0][c].w};
      const uint32_t w1[4] = {kw[1][c].x, kw[1][c].y, kw[1][c].z, kw[1][c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x0 = fix<FMT>(w0[i]), x1 = fix<FMT>(w1[i]);
        const uint32_t a0 = to_half2_lo<FMT>(x0), a1 = to_half2_lo<FMT>(x1);
        const uint32_t a2 = to_half2_hi<FMT>(x0), a3 = to_half2_hi<FMT>(x1);
#pragma unroll
        for (int st = 0; st < NSET; ++st)
          mma16816(sc[st], a0, a1, a2, a3, qb[st][c * 4 + i][0], qb[st][c * 4 + i][1]);
      }
    }
    if (next < k1) load_k(next);  // the registers are free; V's after the second product
    // logits of query t (+ 4 st) for slots j + g and j + g + 8
    float l0[NSET], l1[NSET];
    bool over = false;
#pragma unroll
    for (int st = 0; st < NSET; ++st) {
      const float f = qf[st] * ak;
      l0[st] = (sc[st][0] + sc[st][1]) * f;
      l1[st] = (sc[st][2] + sc[st][3]) * f;
      const int qi = st * 4 + t;
      if (A.c.acc && qi < G) {
        lg[(long)(j - k0 + g) * G + qi] = l0[st];
        lg[(long)(j - k0 + g + 8) * G + qi] = l1[st];
      }
      over |= fmaxf(l0[st], l1[st]) > m[st] + kLazy;
    }
    const int ev = max(kMinExp, min(126, ilogbf(av)));
    if (__any_sync(0xFFFFFFFFu, over) || ev > rv) {
      const int drv = ev > rv ? rv - ev : 0;
      rv = max(rv, ev);
      const float fv = drv < -126 ? 0.f : exp2i(drv);
#pragma unroll
      for (int st = 0; st < NSET; ++st) {
        float mx = fmaxf(l0[st], l1[st]);
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
        const float mn = fmaxf(m[st], mx);
        const float f = exp2f(m[st] - mn);  // 0 on the first tile (m = -inf)
        z[st] *= f;
        m[st] = mn;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) o[st][i][jj] *= f * fv;
      }
    }
    const float pf = av * exp2i(kPScale - rv);  // av 2^-rv below 2
    uint32_t b0[NSET], b1[NSET];
#pragma unroll
    for (int st = 0; st < NSET; ++st) {
      const float p0 = tc::ex2(l0[st] - m[st]), p1 = tc::ex2(l1[st] - m[st]);
      z[st] += p0 + p1;
      const float w0 = p0 * pf, w1 = p1 * pf;
      const float h0 = __half2float(__float2half_rn(w0)), h1 = __half2float(__float2half_rn(w1));
      b0[st] = transpose8x8(pack_half2(h0, w0 - h0));
      b1[st] = transpose8x8(pack_half2(h1, w1 - h1));
    }
#pragma unroll
    for (int w = 0; w < VB / 4; ++w) {
      const uint32_t w0 = fix<FMT>(vw[0][w]), w1 = fix<FMT>(vw[1][w]), w2 = fix<FMT>(vw[2][w]), w3 = fix<FMT>(vw[3][w]);
      const uint32_t e0 = __byte_perm(w0, w1, 0x5140), e1 = __byte_perm(w0, w1, 0x7362);
      const uint32_t f0 = __byte_perm(w2, w3, 0x5140), f1 = __byte_perm(w2, w3, 0x7362);
      const uint32_t a0 = to_half2_lo<FMT>(e0), a1 = to_half2_hi<FMT>(e0);
      const uint32_t a2 = to_half2_lo<FMT>(f0), a3 = to_half2_hi<FMT>(f0);
      const uint32_t c0 = to_half2_lo<FMT>(e1), c1 = to_half2_hi<FMT>(e1);
      const uint32_t c2 = to_half2_lo<FMT>(f1), c3 = to_half2_hi<FMT>(f1);
#pragma unroll
      for (int st = 0; st < NSET; ++st) {
        mma16816(o[st][2 * w], a0, a1, a2, a3, b0[st], b1[st]);
        mma16816(o[st][2 * w + 1], c0, c1, c2, c3, b0[st], b1[st]);
      }
    }
    if (next < k1) load_v(next);
  }

  const float back = exp2i(rv - kPScale);
#pragma unroll
  for (int st = 0; st < NSET; ++st) {
    float zz = z[st];
    zz += __shfl_xor_sync(0xFFFFFFFFu, zz, 4);
    zz += __shfl_xor_sync(0xFFFFFFFFu, zz, 8);
    zz += __shfl_xor_sync(0xFFFFFFFFu, zz, 16);
    if (g == 0) {
      wm[warp * 8 + st * 4 + t] = m[st];
      wz[warp * 8 + st * 4 + t] = zz;
    }
    const int qi = st * 4 + t;
    if (qi < G) {
      float *dst = so + (warp * G + qi) * D + g * VB;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        dst[2 * i] = (o[st][i][0] + o[st][i][1]) * back;
        dst[2 * i + 1] = (o[st][i][2] + o[st][i][3]) * back;
      }
    }
  }
}

template <typename T, int FMT, int D, int NSET>
__global__ void __launch_bounds__(NT, NSET == 1 || D == 64 ? 4 : 3) q8_stream_kernel(const __grid_constant__ DecArgs A) {
  __shared__ __align__(16) float qs[8 * 128];
  __shared__ float wm[NW * 8], wz[NW * 8];
  extern __shared__ float so[];   // [NW][G][D]
  pdl_wait();
  pdl_launch();
  const long u = blockIdx.x / (A.ns + 1);
  const int s = blockIdx.x % (A.ns + 1);
  const int n = A.c.len[u];
  if (n < 0 || n >= A.c.cap) {
    if (s == A.ns && threadIdx.x == 0) {
      A.nsave[u] = -1;
      if (A.status) atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
    }
    return;
  }
  const int nf = n >> A.b_log2 << A.b_log2;
  const long at = u * (A.ns + 1) + s;
  float *lg = A.lgw + u * (long)(A.c.cap + 1) * A.G;
  if (s == A.ns) {
    if (threadIdx.x == 0) A.nsave[u] = n;
    tail_part<T, D>(A, u, n, lg + (long)nf * A.G, qs, wm, wz, so);
  } else {
    const int per = split_len(nf, A.ns);
    const int k0 = s * per, k1 = min(nf, k0 + per);
    if (k0 >= k1) return;
    stream_range<T, FMT, D, NSET>(A, u, k0, k1, lg + (long)k0 * A.G, wm, wz, so);
  }
  combine_warps<D>(A.G, wm, wz, so, A.po + at * A.G * D, A.pmz + at * A.G);
}

// ---- quantising the block that the new token fills -------------------------------------------
template <typename T, int FMT>
__device__ __forceinline__ void quantise_tail(const DecArgs &A, long u, int n, int kv, uint32_t *red) {
  const int D = A.c.d, block = A.c.block, nf = n >> A.b_log2 << A.b_log2;
  const T *rows = static_cast<const T *>(kv ? A.c.Vt : A.c.Kt) + u * (long)block * D;
  // the new token's row as it came in: its copy in the cache may be this kernel's own
  const T *fresh = static_cast<const T *>(kv ? A.v_new : A.k_new) + u * (long)D;
  uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(kv ? A.c.V : A.c.K) + (u * (long)A.c.cap + nf) * D);
  const int pieces = block * D / 16, old = (block - 1) * D / 16;
  auto load = [&](int i, float (&x)[16]) { load16(i < old ? rows + (long)i * 16 : fresh + (i - old) * 16, x); };
  float big = 0.f;
  for (int i = threadIdx.x; i < pieces; i += blockDim.x) {
    float x[16];
    load(i, x);
    big = max_nan(big, max_abs16(x));
  }
  const float a = q8_scale<FMT>(block_max(big, red));
  const float inv = __fdiv_rn(1.f, a);
  for (int i = threadIdx.x; i < pieces; i += blockDim.x) {
    float x[16];
    load(i, x);
    to[i] = q8_pack16<FMT>(x, inv);
  }
  if (threadIdx.x == 0) (kv ? A.c.Vs : A.c.Ks)[(u * (long)A.c.cap + nf) >> A.b_log2] = a;
  __syncthreads();  // red is used again
}

// ---- short caches: one launch ------------------------------------------------------------------
// A cluster of CTAs per unit, each with a range of its slots, whose logits stay in shared memory;
// maxima, normalisers and output shares are exchanged through distributed shared memory, then
// every CTA adds its own slots' probabilities to acc.  The last CTA takes the unfinished block
// and the new token, and slots as well where the ranges are long.
template <typename T, int FMT, int D, int NSET>
__global__ void __launch_bounds__(NT, NSET == 1 || D == 64 ? 4 : 3)
    q8_cluster_kernel(const __grid_constant__ DecArgs A, int slots) {
  __shared__ __align__(16) float qs[8 * 128];
  __shared__ float wm[NW * 8], wz[NW * 8];
  __shared__ float2 mz[2][8];       // this CTA's shares: slots, unfinished block
  __shared__ float2 all[9][8];      // everybody's
  __shared__ float sM[8], sI[8];
  __shared__ uint32_t red[32];
  extern __shared__ __align__(16) float dyn[];
  const int G = A.G;
  float *so = dyn;                  // [NW][G][D]
  float *sh = so + NW * G * D;      // [2][G][D] shares
  float *lg = sh + 2 * G * D;       // [slots][G], then [128][G] of the unfinished block
  float *lgt = lg + (long)slots * G;
  pdl_wait();
  pdl_launch();
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  const int CL = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const long u = blockIdx.x / CL;
  const int n = A.c.len[u];
  if (n < 0 || n >= A.c.cap) {  // every CTA of the cluster alike
    if (rank == 0 && threadIdx.x == 0 && A.status) atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
    return;
  }
  const int nf = n >> A.b_log2 << A.b_log2;
  const bool tail = rank == CL - 1;
  const int mr = CL > 1 && nf <= (CL - 1) * 256 ? CL - 1 : CL;  // CTAs with slots
  const int per = split_len(nf, mr);
  const int k0 = min(nf, rank * per), k1 = rank < mr ? min(nf, k0 + per) : k0;
  if (k0 < k1) {
    stream_range<T, FMT, D, NSET>(A, u, k0, k1, lg, wm, wz, so);
    combine_warps<D>(G, wm, wz, so, sh, mz[0]);
  } else if ((int)threadIdx.x < 8) {
    mz[0][threadIdx.x] = make_float2(-INFINITY, 0.f);
  }
  if (tail) {
    __syncthreads();
    tail_part<T, D>(A, u, n, lgt, qs, wm, wz, so);
    combine_warps<D>(G, wm, wz, so, sh + G * D, mz[1]);
  }
  // the slots' accumulators are on their way while the others finish
  float *acc = A.c.acc ? A.c.acc + u * (long)A.c.cap : nullptr;
  constexpr int AP = 8;
  float old[AP];
  if (acc) {
#pragma unroll
    for (int k = 0; k < AP; ++k) {
      const int j = k0 + k * NT + (int)threadIdx.x;
      old[k] = j < k1 ? acc[j] : 0.f;
    }
  }
  cl.sync();
  const int shares = mr + 1;  // CTAs with slots, then the unfinished block
  for (int i = threadIdx.x; i < shares * G; i += NT) {
    const int s = i / G, q = i - s * G;
    all[s][q] = s < mr ? cl.map_shared_rank(&mz[0][0], s)[q] : cl.map_shared_rank(&mz[1][0], CL - 1)[q];
  }
  __syncthreads();
  if ((int)threadIdx.x < G) {
    float M = -INFINITY, Z = 0.f;
    for (int s = 0; s < shares; ++s) M = fmaxf(M, all[s][threadIdx.x].x);
    for (int s = 0; s < shares; ++s) Z += all[s][threadIdx.x].y * tc::ex2(all[s][threadIdx.x].x - M);
    sM[threadIdx.x] = M;
    sI[threadIdx.x] = 1.f / Z;
  }
  __syncthreads();
  for (int i = rank * NT + threadIdx.x; i < G * D; i += CL * NT) {
    const int q = i / D;
    float v = 0.f;
    for (int s = 0; s < shares; ++s) {
      if (all[s][q].y == 0.f) continue;  // a CTA without slots has no share (one with slots: at least 1)
      const float f = tc::ex2(all[s][q].x - sM[q]);
      v += f * (s < mr ? cl.map_shared_rank(sh, s)[i] : cl.map_shared_rank(sh, CL - 1)[G * D + i]);
    }
    A.o[u * (long)G * D + i] = v * sI[q];
  }
  if (acc) {
    auto mass = [&](const float *l) {
      float p = 0.f;
      for (int q = 0; q < G; ++q) p += tc::ex2(l[q] - sM[q]) * sI[q];
      return p;
    };
#pragma unroll
    for (int k = 0; k < AP; ++k) {
      const int j = k0 + k * NT + (int)threadIdx.x;
      if (j < k1) acc[j] = old[k] + mass(lg + (j - k0) * G);
    }
    for (int j = k0 + AP * NT + threadIdx.x; j < k1; j += NT) acc[j] += mass(lg + (j - k0) * G);
    if (tail)
      for (int j = nf + threadIdx.x; j <= n; j += NT) acc[j] = (j < n ? acc[j] : 0.f) + mass(lgt + (j - nf) * G);
  }
  if (rank == 0 && threadIdx.x == 0) A.len_out[u] = n + 1;  // every CTA has read len
  if (((n + 1) & (A.c.block - 1)) == 0)
    for (int kv = rank; kv < 2; kv += CL) quantise_tail<T, FMT>(A, u, n, kv, red);
  cl.sync();  // nobody leaves while its shares are read
}

// ---- finalize -----------------------------------------------------------------------------
// `chunks` CTAs per unit, each SLOTS_F slots of acc; the query heads' outputs and the block
// that the new token may have filled are shared out over the same CTAs.
// A slot's G logits (GV = 1, 2, 4 or 8 of them as one or two vectors; 0: any G, read late).
template <int GV>
struct SlotLogits {
  float l[GV ? GV : 1];
  __device__ __forceinline__ void load(const float *p) {
    if constexpr (GV == 1) {
      l[0] = __ldcs(p);
    } else if constexpr (GV == 2) {
      const float2 v = __ldcs(reinterpret_cast<const float2 *>(p));
      l[0] = v.x;
      l[1] = v.y;
    } else if constexpr (GV >= 4) {
#pragma unroll
      for (int i = 0; i < GV / 4; ++i) {
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(p) + i);
        l[4 * i] = v.x;
        l[4 * i + 1] = v.y;
        l[4 * i + 2] = v.z;
        l[4 * i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ float mass(const float *p, int G, const float *sM, const float *sI) const {
    float v = 0.f;
    if constexpr (GV == 0) {
      for (int q = 0; q < G; ++q) v += tc::ex2(__ldcs(p + q) - sM[q]) * sI[q];
    } else {
#pragma unroll
      for (int q = 0; q < GV; ++q) v += tc::ex2(l[q] - sM[q]) * sI[q];
    }
    return v;
  }
};

template <typename T, int FMT, int GV>
__global__ void __launch_bounds__(NTF) q8_finalize_kernel(const __grid_constant__ DecArgs A, int chunks) {
  __shared__ float sM[8], sI[8];           // the unit's maximum and 1 / normaliser
  __shared__ float sF[8][kMaxSplits + 1];  // the splits' factors
  __shared__ float4 sO[NTF / 32][32];
  __shared__ uint32_t red[32];
  pdl_wait();
  pdl_launch();
  const int G = A.G, D = A.c.d, block = A.c.block, cap = A.c.cap;
  const long u = blockIdx.x / chunks;
  const int e = blockIdx.x % chunks;
  // what does not depend on the unit's length is on its way before the length is known
  const int lo = e * SLOTS_F;
  constexpr int SPT = SLOTS_F / NTF;
  SlotLogits<GV> lg[SPT];
  float old[SPT];
  const float *lgu = A.lgw + u * (long)(cap + 1) * G;
  if (A.c.acc) {
#pragma unroll
    for (int k = 0; k < SPT; ++k) {
      const int j = lo + k * NTF + threadIdx.x;
      if (j < cap) {
        lg[k].load(lgu + (long)j * G);
        old[k] = A.c.acc[u * (long)cap + j];
      }
    }
  }
  const int n = A.nsave[u];
  if (n < 0) return;
  const int hi = min(lo + SLOTS_F, n + 1);
  const bool fills = (n + 1) % block == 0;
  const bool scores = A.c.acc && lo < hi;
  if (!scores && e >= G && !(fills && e < 2)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nf = n / block * block;
  const int per = split_len(nf, A.ns);
  const int used = per ? (nf + per - 1) / per : 0;  // splits that hold rows; the tail is split ns
  const float2 *mz = A.pmz + u * (A.ns + 1) * G;
  if (warp < G) {  // one warp per query head
    float M = -INFINITY;
    for (int s = lane; s <= used; s += 32) M = fmaxf(M, mz[(s < used ? s : A.ns) * G + warp].x);
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    float Z = 0.f;
    for (int s = lane; s <= used; s += 32) {
      const float2 v = mz[(s < used ? s : A.ns) * G + warp];
      const float f = tc::ex2(v.x - M);
      sF[warp][s] = f;
      Z += v.y * f;
    }
    for (int o = 16; o; o >>= 1) Z += __shfl_xor_sync(0xFFFFFFFFu, Z, o);
    if (lane == 0) {
      sM[warp] = M;
      sI[warp] = 1.f / Z;
    }
  }
  __syncthreads();
  if (scores) {
    float *acc = A.c.acc + u * (long)cap;
#pragma unroll
    for (int k = 0; k < SPT; ++k) {
      const int j = lo + k * NTF + threadIdx.x;
      if (j < hi) acc[j] = (j < n ? old[k] : 0.f) + lg[k].mass(lgu + (long)j * G, G, sM, sI);
    }
  }
  const int d4 = D / 4;
  for (int q = e; q < G; q += chunks) {
    const float4 *po = reinterpret_cast<const float4 *>(A.po + (u * (A.ns + 1) * G + q) * (long)D);
    const int el = lane % d4, sp = warp * (32 / d4) + lane / d4, step = (NTF / 32) * (32 / d4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = sp; s <= used; s += step) {
      const float4 x = po[(long)(s < used ? s : A.ns) * G * d4 + el];
      const float f = sF[q][s];
      v.x += f * x.x;
      v.y += f * x.y;
      v.z += f * x.z;
      v.w += f * x.w;
    }
    sO[warp][lane] = v;
    __syncthreads();
    if ((int)threadIdx.x < d4) {
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < NTF / 32; ++w)
        for (int y = threadIdx.x; y < 32; y += d4) {
          const float4 x = sO[w][y];
          t.x += x.x;
          t.y += x.y;
          t.z += x.z;
          t.w += x.w;
        }
      const float i = sI[q];
      float *o = A.o + (u * (long)G + q) * D + 4 * threadIdx.x;
      o[0] = t.x * i;
      o[1] = t.y * i;
      o[2] = t.z * i;
      o[3] = t.w * i;
    }
    __syncthreads();
  }
  if (e == 0 && threadIdx.x == 0) A.len_out[u] = n + 1;
  if (!fills) return;
  for (int kv = e; kv < 2; kv += chunks) quantise_tail<T, FMT>(A, u, n, kv, red);
}

size_t al(size_t x) { return (x + 255) & ~(size_t)255; }

// Splits per unit: CTAs of about equal length, several waves of four an SM, so that units of
// different lengths even out; at least one tile a warp, and no more splits than the finalize
// kernel holds factors for.
int splits(long units, int cap) {
  const long want = (16L * kNumSmsHint + units - 1) / (units > 0 ? units : 1);
  const long most = (cap + 16 * NW - 1) / (16 * NW);
  const long ns = want < most ? want : most;
  return (int)(ns < 1 ? 1 : ns > kMaxSplits ? kMaxSplits : ns);
}

// The one-launch kernel where its CTAs hold short ranges and nearly all run at once (four an SM;
// three for G > 4 and d = 128, the rest then follow: a cluster waits for its own CTAs alone): CTAs
// per unit (0: not), slots of a CTA.  One KV group of 8 with 1638 slots 11.0 us (two launches: 12.3),
// 64 units of up to 8192 slots 32.7 us (34.0); but 256 units of up to 8192 slots 84 us (66), where
// CTAs that wait for the rest of their cluster leave the memory idle.  As the doubling looks one CTA
// a unit ahead, 77 to 121 units and 153 to 202 are taken past the room and get two launches.
int cluster_plan(long units, int G, int cap, int *slots) {
  const long room = 4L * kNumSmsHint;
  int cl = 1;
  while (cl < 8 && (cl + 1) * units <= room) cl *= 2;
  if (cl > 8) cl = 8;
  *slots = ((cap + cl - 1) / cl + 127) & ~63;  // split_len over one CTA less, or over all
  if (cl > 1 && *slots < 256) *slots = 256;
  return *slots <= 1088 && (long)*slots * G * 4 <= 36 * 1024 && units * cl <= room ? cl : 0;
}

template <typename T, int FMT, int D, int NSET>
int run(const DecArgs &A, long units, cudaStream_t st) {
  int slots;
  if (const int cl = cluster_plan(units, A.G, A.c.cap, &slots)) {
    const size_t bytes = ((size_t)(NW + 2) * A.G * D + (size_t)(slots + 128) * A.G) * sizeof(float);
    if (ensure_smem((const void *)q8_cluster_kernel<T, FMT, D, NSET>, bytes)) return KV_ERR_CUDA;
    const cudaError_t e = launch_pdl_cluster(q8_cluster_kernel<T, FMT, D, NSET>, (unsigned)(units * cl), NT, bytes, st,
                                             cl, A, slots);
    if (e != cudaSuccess) return cuda_failure(e, "8-bit decode: cluster kernel");
    return launch_status();
  }
  const size_t smem = (size_t)NW * A.G * D * sizeof(float);
  if (ensure_smem((const void *)q8_stream_kernel<T, FMT, D, NSET>, smem)) return KV_ERR_CUDA;
  const long ctas = units * (A.ns + 1);
  const int chunks = A.c.acc ? (A.c.cap + SLOTS_F - 1) / SLOTS_F : A.G;
  if (ctas > 0x7FFFFFFFL || units * chunks > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  cudaError_t e = launch_pdl(q8_stream_kernel<T, FMT, D, NSET>, (unsigned)ctas, NT, smem, st, A);
  if (e != cudaSuccess) return cuda_failure(e, "8-bit decode: stream kernel");
  count_launches(1);
  auto *fin = A.G == 1   ? q8_finalize_kernel<T, FMT, 1>
              : A.G == 2 ? q8_finalize_kernel<T, FMT, 2>
              : A.G == 4 ? q8_finalize_kernel<T, FMT, 4>
              : A.G == 8 ? q8_finalize_kernel<T, FMT, 8>
                         : q8_finalize_kernel<T, FMT, 0>;
  e = launch_pdl(fin, (unsigned)(units * chunks), NTF, 0, st, A, chunks);
  if (e != cudaSuccess) return cuda_failure(e, "8-bit decode: finalize kernel");
  return launch_status();
}

template <typename T, int FMT>
int run_d(const DecArgs &A, long units, cudaStream_t st) {
  if (A.c.d == 128) return A.G > 4 ? run<T, FMT, 128, 2>(A, units, st) : run<T, FMT, 128, 1>(A, units, st);
  return A.G > 4 ? run<T, FMT, 64, 2>(A, units, st) : run<T, FMT, 64, 1>(A, units, st);
}

}  // namespace

size_t decode_q8_workspace_bytes(long units, int G, int cap, int d) {
  int slots;
  if (units == 0 || cluster_plan(units, G, cap, &slots)) return 0;
  const int ns = splits(units, cap);
  return al((size_t)units * (cap + 1) * G * 4) + al((size_t)units * (ns + 1) * G * 8) +
         al((size_t)units * (ns + 1) * G * d * 4) + al((size_t)units * 4);
}

int launch_decode_q8(const void *q, const void *k_new, const void *v_new, const kv_q8_cache &c, int Hq,
                     int32_t new_pos, const int32_t *row_pos, int32_t *len_out, float scale, float *o, void *ws,
                     int *status, cudaStream_t st) {
  const long units = (long)c.B * c.Hkv;
  DecArgs A{};
  A.q = q;
  A.k_new = k_new;
  A.v_new = v_new;
  A.c = c;
  A.row_pos = row_pos;
  A.new_pos = new_pos;
  A.len_out = len_out;
  A.G = Hq / c.Hkv;
  A.ns = splits(units, c.cap);
  A.b_log2 = c.block == 128 ? 7 : c.block == 64 ? 6 : 5;
  A.c_log2 = scale * 1.4426950408889634f;
  A.o = o;
  A.status = status;
  char *p = static_cast<char *>(ws);
  A.lgw = reinterpret_cast<float *>(p);
  p += al((size_t)units * (c.cap + 1) * A.G * 4);
  A.pmz = reinterpret_cast<float2 *>(p);
  p += al((size_t)units * (A.ns + 1) * A.G * 8);
  A.po = reinterpret_cast<float *>(p);
  p += al((size_t)units * (A.ns + 1) * A.G * c.d * 4);
  A.nsave = reinterpret_cast<int32_t *>(p);
  if (c.dtype == KV_BF16)
    return c.format == KV_Q8_S8 ? run_d<__nv_bfloat16, KV_Q8_S8>(A, units, st)
                                : run_d<__nv_bfloat16, KV_Q8_E4M3>(A, units, st);
  return c.format == KV_Q8_S8 ? run_d<float, KV_Q8_S8>(A, units, st) : run_d<float, KV_Q8_E4M3>(A, units, st);
}

}  // namespace kvc

// blocks.cu -- attention of a few new tokens over the blocks of a long cache that their digests
// choose, for each token and KV head on its own.
//
// With the least and largest key of a block per channel, low and top, and the group's queries,
//     u_j = max_g sum_c max(q_gc, 0) top_jc + min(q_gc, 0) low_jc
// is at least every logit (before the scale) of block j.  The first `sink` and last `recent`
// of the blocks that a token sees and the best others by (u descending, j ascending) are
// attended, all of their visible slots with a plain softmax.
//
// The choice is the one that u in 64 bits makes.  The bounds are computed by warp-level products,
// whose terms are exact (2^-21 from split fp32 operands) and whose fp32 sums the unit may cut off
// at each term: by 2^-23 of the sum so far, which never passes S = max_g sum_c |q_gc| max_j |digest_jc|.
// In four sums of 64 terms each they are off by at most e = 2^-16 S, a factor of two to spare.  With a
// the m-th largest of them, a block above a + 2e is among the true best m, one below a - 2e is not; when
// those between (mostly one block, the m-th itself) are more than the places left, they alone are
// computed again, in three parts of fp32 (error-free products and sums, then rounded to 64 bits; the
// 64-bit unit is 40 times slower), or in 64 bits where fp32 would over- or underflow.
// Equal keys leave every block open, so the cluster's CTAs share out what is more than a few, and ranks
// come from histograms of the bounds as whole numbers: 12000 equal blocks of 8 heads take 400 us, 66 when
// they differ (each CTA for itself, all against all: 111 ms).  A block whose digest is no number or
// infinite has the bound +inf and needs none of this.
//
// One launch, a cluster of CTAs for each (row, KV head, token): the CTAs share out the digests,
// exchange the bounds through distributed shared memory, find the same m-th
// largest each for itself (a histogram over the range of their bits, then the few in its bin),
// share out the chosen blocks' slots and join their softmax shares as they exchanged the bounds.  Digests and slots come
// through the same rings (rows_stream.cuh), whose memory the choice borrows between.
#include <cooperative_groups.h>

#include <cfloat>
#include <map>
#include <mutex>
#include <tuple>

#include "pdl.cuh"
#include "rows_stream.cuh"

namespace kvc {
namespace {

constexpr int NW = 4, NT = 32 * NW;
constexpr int kMaxBlocks = 12288;  // 14 bytes of shared memory each and 4 shared out over the cluster (18 with one CTA)
constexpr int kBins = 256, kFew = 64;
constexpr int kAlone = 32;  // near bounds that a CTA computes by itself, without waiting for the others of its cluster
template <typename T, int D>
using Rows = RowStream<T, D, (D == 64 && sizeof(T) == 2 ? 4 : 2)>;
// CTAs an SM holds.
template <typename T, int D>
constexpr int kPerSm = sizeof(T) == 4 ? (D == 64 ? 2 : 1) : 3;

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
__device__ __forceinline__ unsigned long long order(double x) {  // orders like x; -0 like 0
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.);
  return u ^ (u >> 63 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// max(q, 0) and min(q, 0) of a vector, NaN kept.
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
// The larger magnitudes, element by element (a NaN is not kept).
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b, __nv_bfloat16) {
  b &= 0x7FFF7FFFu;
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b, float) {
  return __float_as_uint(fmaxf(__uint_as_float(a), fabsf(__uint_as_float(b))));
}
// |a| |b| summed over a word's elements
__device__ __forceinline__ float products(uint32_t a, uint32_t b, __nv_bfloat16) {
  return fabsf(__uint_as_float(a << 16) * __uint_as_float(b << 16)) +
         fabsf(__uint_as_float(a & 0xFFFF0000u) * __uint_as_float(b & 0xFFFF0000u));
}
__device__ __forceinline__ float products(uint32_t a, uint32_t b, float) { return fabsf(__uint_as_float(a) * __uint_as_float(b)); }
// whether a pair of elements has a product other than 0
__device__ __forceinline__ bool meet(uint32_t a, uint32_t b, __nv_bfloat16) {
  return ((a & 0x7FFFu) != 0 && (b & 0x7FFFu) != 0) || ((a & 0x7FFF0000u) != 0 && (b & 0x7FFF0000u) != 0);
}
__device__ __forceinline__ bool meet(uint32_t a, uint32_t b, float) { return (a & 0x7FFFFFFFu) != 0 && (b & 0x7FFFFFFFu) != 0; }

// The passes below run once or twice per launch, so their instructions come from memory: short loops beat
// unrolled ones (keys held in registers and everything unrolled: 13.8 us for 12.2 then), and what few calls need stands in
// functions of its own (in line with the rest: 48.4 us for 44.5, fp32, 32 units of 32768 slots).

// u of block j in 64 bits (q [G][D] as floats): one warp, lanes over the channels; every lane gets it.
template <typename T, int D>
__device__ __noinline__ double bound64(int G, const float *q, const T *digest, int j) {
  const int lane = threadIdx.x & 31;
  const T *low = digest + (long)j * 2 * D, *top = low + D;
  double best = -INFINITY;
  for (int g = 0; g < G; ++g) {
    double s = 0.;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int c = lane + 32 * i;
      const double x = (double)q[g * D + c];
      s += (x != x || x > 0. ? x : 0.) * (double)to_f32(top[c]) + (x != x || x < 0. ? x : 0.) * (double)to_f32(low[c]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (s != s) s = INFINITY;
    best = s > best ? s : best;
  }
  return best;
}

// The same in three parts of fp32: hi + lo is the sum without the error of its own additions (the sum of two floats and
// what its rounding lost, by Knuth's six operations, twice), `rest` sums up what those lose, some 2^-70 of the terms' size.
__device__ __forceinline__ void two_sum(float a, float b, float &s, float &e) {
  s = __fadd_rn(a, b);
  const float x = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, x)), __fsub_rn(b, x));
}
// The bounds of the blocks list[e0 .. e1 - 1], ordered as whole numbers: `out` (0 before) gets the larger of it and them.
// An item is a block and a query, and has LPI lanes: one for each 16 bytes of a digest's row where there are few items and
// they wait for one another's steps, eight where there are many (the sums over lanes cost more than those of a lane).
template <typename T, int D, int LPI>
__device__ __noinline__ void bounds_in_parts(int G, const float *q, const T *digest, const uint16_t *list, int e0, int e1,
                                             unsigned long long *out) {
  constexpr int EV = Vec16<T>::N, IPW = 32 / LPI, NV = D / EV / LPI;  // items of a warp, 16-byte pieces of a lane
  const int lane = threadIdx.x & 31, l = lane % LPI, items = (e1 - e0) * G;
#pragma unroll 1
  for (int first = (threadIdx.x >> 5) * IPW; first < items; first += NW * IPW) {
    const int item = min(first + lane / LPI, items - 1), i = e0 + item / G, g = item % G;
    const uint4 *row = reinterpret_cast<const uint4 *>(digest + (long)list[i] * 2 * D) + l;
    float low[NV * EV], top[NV * EV], hi = 0.f, lo = 0.f, rest = 0.f, x1, x2, x3;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      Vec16<T>::unpack(row[v * LPI], low + v * EV);
      Vec16<T>::unpack(row[D / EV + v * LPI], top + v * EV);
    }
    int bad = 0;
#pragma unroll
    for (int e = 0; e < NV * EV; ++e) {
      const float x = q[g * D + (l + e / EV * LPI) * EV + e % EV], y = x >= 0.f ? top[e] : low[e];
      const float p = __fmul_rn(x, y), px = __fmaf_rn(x, y, -p);
      bad |= !(fabsf(low[e]) < INFINITY) || !(fabsf(top[e]) < INFINITY);
      two_sum(hi, p, hi, x1);
      two_sum(lo, x1, lo, x2);
      two_sum(lo, px, lo, x3);
      rest = __fadd_rn(rest, __fadd_rn(x2, x3));
    }
#pragma unroll 1
    for (int o = LPI / 2; o; o >>= 1) {
      const float a = __shfl_xor_sync(0xFFFFFFFFu, hi, o), b = __shfl_xor_sync(0xFFFFFFFFu, lo, o);
      const float c = __shfl_xor_sync(0xFFFFFFFFu, rest, o);
      const bool upper = lane & o;  // the same sum in both lanes
      bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, o);
      two_sum(upper ? a : hi, upper ? hi : a, hi, x1);
      two_sum(upper ? b : lo, upper ? lo : b, lo, x2);
      two_sum(lo, x1, lo, x3);
      rest = __fadd_rn(__fadd_rn(rest, c), __fadd_rn(x2, x3));
    }
    const double s = (double)hi + ((double)lo + (double)rest);
    if (l == 0) atomicMax(out + i, order(bad || s != s ? (double)INFINITY : s));
  }
}

// S of the whole cluster without the digests' infinities and without queries with a NaN, whose bounds are all +inf; [i0, i1)
// are this CTA's blocks, part [NW][8] and mine its memory.
template <typename T, int D>
__device__ __noinline__ float finite_size(int G, const float *q, const T *digest, int i0, int i1, float *part, float &mine) {
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  const int c = threadIdx.x % D, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float big = 0.f;
#pragma unroll 8
  for (int i = i0 + (int)threadIdx.x / D; i < i1; i += NT / D) {
    const float low = fabsf(to_f32(digest[(long)i * 2 * D + c])), top = fabsf(to_f32(digest[(long)i * 2 * D + D + c]));
    if (low < INFINITY) big = fmaxf(big, low);
    if (top < INFINITY) big = fmaxf(big, top);
  }
  for (int g = 0; g < G; ++g) {
    const float x = q[g * D + c];
    float e = fabsf(x) * big;
    for (int o = 16; o; o >>= 1) e += __shfl_xor_sync(0xFFFFFFFFu, e, o);
    const bool nan = __any_sync(0xFFFFFFFFu, x != x);
    if (lane == 0) part[warp * 8 + g] = nan ? -INFINITY : fminf(e, FLT_MAX);
  }
  cl.sync();  // all have read `mine`
  if (threadIdx.x == 0) {
    mine = 0x1p-100f;
    for (int g = 0; g < G; ++g) {
      const float x = (part[g] + part[8 + g]) + (part[16 + g] + part[24 + g]);
      mine = fmaxf(mine, x < 0.f ? 0x1p-60f : x < INFINITY ? x : INFINITY);
    }
  }
  cl.sync();
  float size = 0.f;
  for (int r = 0; r < (int)cl.num_blocks(); ++r) size = fmaxf(size, *cl.map_shared_rank(&mine, r));
  return size;
}

// Shared memory of the choice.
struct Choice {
  uint32_t *key;              // [blocks] bounds' bits
  unsigned long long *exact;  // [blocks] bounds in 64 bits of the undecided blocks, ordered as whole numbers
  uint16_t *list;             // [blocks] undecided blocks, ascending; then the chosen ones
  int *hist;                  // [kBins]
  uint32_t *few;              // [kFew]
  unsigned long long (*ends)[NW];
};
constexpr uint32_t kIn = 0xFFFFFFFFu;  // no bound's bits

// In which of the histogram's bins the m-th largest is, how many it holds, and how many are above it.  `count` becomes 0.
__device__ __forceinline__ int bin_of(const Choice &c, int m, int (*red)[NW], uint32_t (*redu)[NW], int &count, uint32_t &bin,
                                      int &held) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // keys in this thread's two bins and in all above
  const int b = kBins - 2 - 2 * (int)threadIdx.x, h1 = c.hist[b + 1], h0 = c.hist[b];
  int incl = h0 + h1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) red[0][warp] = incl;
  __syncthreads();
  for (int w = 0; w < warp; ++w) incl += red[0][w];
  const int above = incl - h0 - h1;
  if (above < m && m <= incl) {  // one thread
    const bool upper = m <= above + h1;
    redu[0][0] = b + upper;
    redu[0][1] = upper ? above : above + h1;
    redu[0][2] = upper ? h1 : h0;
    count = 0;
  }
  __syncthreads();
  bin = redu[0][0];
  held = (int)redu[0][2];
  return (int)redu[0][1];
}

// The m-th largest of the n keys, whose least and largest this thread's `least`, `most` are a part of.
__device__ uint32_t mth_largest(const Choice &c, int n, int m, uint32_t least, uint32_t most, int (*red)[NW],
                                uint32_t (*redu)[NW], int &count) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  least = __reduce_min_sync(0xFFFFFFFFu, least);
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane == 0) {
    redu[0][warp] = least;
    redu[1][warp] = most;
  }
  for (int i = threadIdx.x; i < kBins; i += NT) c.hist[i] = 0;
  __syncthreads();  // the keys too
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    least = min(least, redu[0][w]);
    most = max(most, redu[1][w]);
  }
  for (;;) {
    const uint32_t range = most - least;
    const int s = max(0, 24 - __clz(range));  // range >> s is below kBins
    for (int i = threadIdx.x; i < n; i += NT) {
      const uint32_t k = c.key[i] - least;
      if (k <= range) atomicAdd(c.hist + (k >> s), 1);
    }
    __syncthreads();
    uint32_t bin;
    int held;
    m -= bin_of(c, m, red, redu, count, bin, held);
    least += bin << s;
    most = min(most, least + (uint32_t)((1ull << s) - 1));
    if (most == least) return least;
    if (held <= kFew) {
      for (int i = threadIdx.x; i < n; i += NT) {
        const uint32_t k = c.key[i];
        if (k >= least && k <= most) c.few[atomicAdd(&count, 1)] = k;
      }
      __syncthreads();
      // every warp alike: the range of the bits halved
      const uint32_t k0 = lane < held ? c.few[lane] : 0u, k1 = lane + 32 < held ? c.few[lane + 32] : 0u;
      uint32_t L = least, H = most;  // at least m keys are >= L, fewer than m are > H
      while (L < H) {
        const uint32_t mid = L + (H - L) / 2 + 1;
        const int x = __popc(__ballot_sync(0xFFFFFFFFu, k0 >= mid)) + __popc(__ballot_sync(0xFFFFFFFFu, k1 >= mid));
        if (x >= m) L = mid; else H = mid - 1;
        if (x == m) return __reduce_min_sync(0xFFFFFFFFu, min(k0 >= mid ? k0 : kIn, k1 >= mid ? k1 : kIn));
      }
      return L;
    }
    for (int i = threadIdx.x; i < kBins; i += NT) c.hist[i] = 0;
    __syncthreads();
  }
}

// Marks the m largest of c.exact[0, n), of equal ones the first, in c.key.  A histogram over the range that is left cuts
// eight bits off it, so that any number of them, equal or not, takes a few passes.
__device__ __noinline__ void mark_best(const Choice &c, int n, int m, int (*red)[NW], uint32_t (*redu)[NW], int &count) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned long long least = ~0ull, most = 0ull;
  for (int i = threadIdx.x; i < n; i += NT) {
    least = min(least, c.exact[i]);
    most = max(most, c.exact[i]);
  }
#pragma unroll 1
  for (int o = 16; o; o >>= 1) {
    least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
    most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
  }
  if (lane == 0) {
    c.ends[0][warp] = least;
    c.ends[1][warp] = most;
  }
  __syncthreads();
  for (int w = 0; w < NW; ++w) {
    least = min(least, c.ends[0][w]);
    most = max(most, c.ends[1][w]);
  }
  while (least < most) {
    const unsigned long long range = most - least;
    const int s = max(0, 56 - __clzll(range));  // range >> s is below kBins
    for (int i = threadIdx.x; i < kBins; i += NT) c.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += NT) {
      const unsigned long long k = c.exact[i] - least;
      if (k <= range) atomicAdd(c.hist + (int)(k >> s), 1);
    }
    __syncthreads();
    uint32_t bin;
    int held;
    m -= bin_of(c, m, red, redu, count, bin, held);
    least += (unsigned long long)bin << s;
    most = min(most, least + ((1ull << s) - 1));
  }
  // all above `least`, and the first m of those that are equal to it
  const int stretch = (n + NT - 1) / NT * 32, i0 = min(n, warp * stretch), i1 = min(n, i0 + stretch);
  int equal = 0;
  for (int i = i0 + lane; i < i0 + stretch; i += 32) equal += __popc(__ballot_sync(0xFFFFFFFFu, i < i1 && c.exact[i] == least));
  __syncthreads();  // `red` has been read
  if (lane == 0) red[0][warp] = equal;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < warp; ++w) at += red[0][w];
  for (int i = i0 + lane; i < i0 + stretch; i += 32) {
    const unsigned long long k = i < i1 ? c.exact[i] : 0ull;
    const bool same = i < i1 && k == least;
    const unsigned who = __ballot_sync(0xFFFFFFFFu, same);
    if (i < i1 && (k > least || (same && at + __popc(who & ((1u << lane) - 1)) < m))) c.key[c.list[i]] = kIn;
    at += __popc(who);
  }
}

// The blocks between `below` and `above` of the n candidates (`all_open` of them) again, and the best `places` marked.  A
// function of its own: few clusters come here, and the others should not fetch its instructions.
template <typename T, int D>
__device__ __noinline__ void second_look(const Choice &c, int G, const float *q, const T *digest, int n, int places, int all_open,
                                         float err, bool wide, float above, float below, int (*red)[NW], uint32_t (*redu)[NW],
                                         int &count) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stretch = (n + NT - 1) / NT * 32, i0 = min(n, warp * stretch), i1 = min(n, i0 + stretch);
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  int to = 0;
  for (int w = 0; w < warp; ++w) to += red[1][w];
  for (int i = i0 + lane; i < i0 + stretch; i += 32) {
    const float u = i < i1 ? unorder(c.key[i]) : -INFINITY;
    const bool between = i < i1 && !(u > above) && !(u < below);
    const unsigned who = __ballot_sync(0xFFFFFFFFu, between);
    if (between) {
      const int x = to + __popc(who & ((1u << lane) - 1));
      c.list[x] = (uint16_t)i;
      c.exact[x] = 0ull;
    }
    to += __popc(who);
  }
  __syncthreads();
  // where there are many the cluster's CTAs, which all have the same list, have a share of them each
  const int CL = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const bool spread = CL > 1 && all_open > kAlone;
  const int each = spread ? (all_open + CL - 1) / CL : all_open, e0 = spread ? min(all_open, rank * each) : 0;
  const int e1 = min(all_open, e0 + each);
  if (err == 0.f || below == INFINITY) {  // every term is 0, or all of these are +inf: the bounds are exact
    for (int i = e0 + threadIdx.x; i < e1; i += NT) c.exact[i] = order((double)unorder(c.key[c.list[i]]));
  } else if (wide) {
    for (int i = e0 + warp; i < e1; i += NW) {
      const double x = bound64<T, D>(G, q, digest, c.list[i]);
      if (lane == 0) c.exact[i] = order(x);
    }
  } else {
    if (all_open > kAlone) bounds_in_parts<T, D, 8>(G, q, digest, c.list, e0, e1, c.exact);
    else bounds_in_parts<T, D, D / Vec16<T>::N>(G, q, digest, c.list, e0, e1, c.exact);
  }
  if (spread) {
    cl.sync();
    for (int i = threadIdx.x; i < all_open; i += NT) {
      const int r = i / each;
      if (r != rank) c.exact[i] = cl.map_shared_rank(c.exact, r)[i];
    }
    cl.sync();  // the rings take the place of what has been read
  } else {
    __syncthreads();
  }
  if (all_open > kFew) {
    mark_best(c, all_open, places, red, redu, count);
  } else if ((int)threadIdx.x < all_open) {
    const int i = threadIdx.x;
    const unsigned long long x = c.exact[i];
    int better = 0;
    for (int k = 0; k < all_open; ++k) better += c.exact[k] > x || (c.exact[k] == x && k < i);
    if (better < places) c.key[c.list[i]] = kIn;
  }
  __syncthreads();
}

// The best `m` of the n candidates (block lo + i; their bounds' bits in c.key) to c.list, ascending, as blocks.
// err: how far a bound may be off; wide: only 64 bits tell them apart.
template <typename T, int D>
__device__ void choose(int G, const Choice &c, const float *q, const T *digest, int lo, int n, int m, float err,
                       bool wide, uint32_t least, uint32_t most, int (*red)[NW], uint32_t (*redu)[NW], int &count) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float a = unorder(mth_largest(c, n, m, least, most, red, redu, count));
  const float above = a + 2.f * err, below = a - 2.f * err;
  // each warp has a stretch of the candidates, 32 at a time
  const int stretch = (n + NT - 1) / NT * 32, i0 = min(n, warp * stretch), i1 = min(n, i0 + stretch);
  int sure = 0, open = 0;
  for (int i = i0 + lane; i < i0 + stretch; i += 32) {
    const float x = i < i1 ? unorder(c.key[i]) : -INFINITY;
    sure += __popc(__ballot_sync(0xFFFFFFFFu, i < i1 && x > above));
    open += __popc(__ballot_sync(0xFFFFFFFFu, i < i1 && !(x > above) && !(x < below)));
  }
  if (lane == 0) {
    red[0][warp] = sure;
    red[1][warp] = open;
  }
  __syncthreads();
  int at = 0, all_sure = 0, all_open = 0, sure_before = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) at += red[0][w] + red[1][w], sure_before += red[0][w];
    all_sure += red[0][w];
    all_open += red[1][w];
  }
  const int places = m - all_sure;
  const bool again = all_open > places;
  if (again) {
    second_look<T, D>(c, G, q, digest + (long)lo * 2 * D, n, places, all_open, err, wide, above, below, red, redu, count);
    // how many of those each warp's stretch has now
    int in = 0;
    for (int i = i0 + lane; i < i0 + stretch; i += 32) in += __popc(__ballot_sync(0xFFFFFFFFu, i < i1 && c.key[i] == kIn));
    if (lane == 0) red[1][warp] = in;
    __syncthreads();
    at = sure_before;
    for (int w = 0; w < warp; ++w) at += red[1][w];
  }
  for (int i = i0 + lane; i < i0 + stretch; i += 32) {
    const uint32_t k = i < i1 ? c.key[i] : 0u;
    const float x = unorder(k);
    const bool in = i < i1 && (k == kIn || x > above || (!again && !(x < below)));
    const unsigned who = __ballot_sync(0xFFFFFFFFu, in);
    if (in) c.list[at + __popc(who & ((1u << lane) - 1))] = (uint16_t)(lo + i);
    at += __popc(who);
  }
}

// A warp's share of the chosen tiles (first, first + NW, ..., `count` of them) made anew.
template <typename T, int D>
__device__ __noinline__ void share_again(const BlkArgs &A, const T *q, long bh, const uint16_t *list, int first, int count, int seen,
                                         float2 *mz, float *so) {
  const T *K = static_cast<const T *>(A.K) + bh * A.cap * (long)D, *V = static_cast<const T *>(A.V) + bh * A.cap * (long)D;
  rows_again<T, D>(AgainArgs<T>{q, 0, A.sq[1], 0, 8, 1, 0, K, V, D, D, list, A.b_log2 - 4, first, NW, count, seen, 0, A.c_log2}, A.G, mz,
                   so);
}

template <typename T, int D>
__global__ void __launch_bounds__(NT, kPerSm<T, D>) blocks_kernel(const __grid_constant__ BlkArgs A) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ float2 wmz[NW * 8];
  __shared__ float2 mz[8], all[16][8];
  __shared__ float sI[8];
  __shared__ float err_part[NW], err_cta;
  __shared__ int red[2][NW], counter, hist[kBins];
  __shared__ uint32_t redu[2][NW], few[kFew];
  __shared__ unsigned long long ends[2][NW];
  constexpr int NCH = Rows<T, D>::NCH;
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
  Rows<T, D> R;
  R.init(area + warp * R.RING);
  R.load_q(q + min(R.g, G - 1) * A.sq[1]);

  // ---- which blocks ----
  const int ns = min(nbk, A.n_sel);
  const int m = A.n_sel - A.sink - A.recent;  // places that bounds decide, where nbk > n_sel
  const int lo = A.sink, nm = nbk - A.sink - A.recent;
  const bool choice = nbk > A.n_sel;
  const int cap_c = choice && m > 0 ? nm : 0;
  Choice c;
  c.hist = hist;
  c.few = few;
  c.exact = reinterpret_cast<unsigned long long *>(area);
  c.ends = ends;
  c.key = reinterpret_cast<uint32_t *>(c.exact + A.nb);
  c.list = reinterpret_cast<uint16_t *>(mine + ((A.nb / CL + 20) & ~3));
  if (cap_c > 0) {
    for (int i = threadIdx.x; i < G * D; i += NT) sh[i] = to_f32(q[i / D * A.sq[1] + i % D]);  // for the near bounds
    const T *digest = static_cast<const T *>(A.digest) + bh * A.nb * 2L * D;
    const int per = (((nm + CL - 1) / CL) + 15) & ~15;
    const int i0 = min(nm, rank * per), i1 = min(nm, i0 + per);
    uint32_t big[NCH * 4];  // largest magnitudes of this lane's channels
#pragma unroll
    for (int x = 0; x < NCH * 4; ++x) big[x] = 0u;
    // tiles of 16 blocks: low rows where K's stand, top rows where V's do
    const int count = (i1 - i0 + 15) / 16, tiles = (count - warp + NW - 1) / NW;
    const T *rows = digest + (long)lo * 2 * D;
    auto first = [&](int y) { return i0 + (y * NW + warp) * 16; };
#pragma unroll
    for (int y = 0; y < R.STAGES - 1; ++y) {
      if (y < tiles) R.fill(y, rows, 2 * D, rows + D, 2 * D, first(y), i1 - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    for (int y = 0, stage = 0; y < tiles; ++y) {
      const int ahead = y + R.STAGES - 1;
      if (ahead < tiles) R.fill(stage == 0 ? R.STAGES - 1 : stage - 1, rows, 2 * D, rows + D, 2 * D, first(ahead), i1 - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group %0;" ::"n"(R.STAGES - 1) : "memory");
      __syncwarp();
      float sum[4][4], small[4] = {0.f, 0.f, 0.f, 0.f}, s[4];
#pragma unroll
      for (int x = 0; x < 16; ++x) sum[x / 4][x % 4] = 0.f;
      const unsigned char *low = R.ring + stage * R.TILE + R.g * R.ROW, *top = low + 16 * R.ROW;
#pragma unroll
      for (int x = 0; x < NCH; ++x) {
        const int at = ((4 * x + R.t) ^ R.k_swizzle(R.g)) << 4, bt = ((4 * x + R.t) ^ R.v_swizzle(R.g)) << 4;
        const uint4 l0 = *reinterpret_cast<const uint4 *>(low + at), l1 = *reinterpret_cast<const uint4 *>(low + 8 * R.ROW + at);
        const uint4 t0 = *reinterpret_cast<const uint4 *>(top + bt);
        const uint4 t1 = *reinterpret_cast<const uint4 *>(top + 8 * R.ROW + (((4 * x + R.t) ^ R.v_swizzle(R.g + 8)) << 4));
        auto grow = [&](const uint4 &v) {
          big[4 * x] = larger(big[4 * x], v.x, T());
          big[4 * x + 1] = larger(big[4 * x + 1], v.y, T());
          big[4 * x + 2] = larger(big[4 * x + 2], v.z, T());
          big[4 * x + 3] = larger(big[4 * x + 3], v.w, T());
        };
        grow(l0);
        grow(l1);
        grow(t0);
        grow(t1);
        dot16(sum[x & 1], small, l0, l1, part<T>(R.q[x], false), T());
        dot16(sum[2 + (x & 1)], small, t0, t1, part<T>(R.q[x], true), T());
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] = (sum[0][k] + sum[1][k]) + (sum[2][k] + sum[3][k]) + (sizeof(T) == 4 ? small[k] : 0.f);
      // the largest of the group's: columns behind G repeat its last query
      const int i = first(y);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float v = max_nan(s[2 * k], s[2 * k + 1]);
        v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
        v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
        if (R.t == 0 && i + R.g + 8 * k < i1) mine[i - i0 + R.g + 8 * k] = v;
      }
      __syncwarp();  // the stage may be filled again
      if (++stage == R.STAGES) stage = 0;
    }
    // S over this warp's blocks: the channels' largest over the lanes with the same ones, times |q|, each lane
    // for the query of its column
    float e = 0.f;
    bool some = false;
#pragma unroll
    for (int x = 0; x < NCH * 4; ++x) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) big[x] = larger(big[x], __shfl_xor_sync(0xFFFFFFFFu, big[x], o), T());
      const uint4 &q4 = R.q[x / 4];
      const uint32_t qw = x % 4 == 0 ? q4.x : x % 4 == 1 ? q4.y : x % 4 == 2 ? q4.z : q4.w;
      e += products(big[x], qw, T());
      some |= meet(big[x], qw, T());
    }
    if (some && e < 0x1p-100f) e = 0x1p-100f;  // 0 only where every term is: not where they underflow
    e += __shfl_xor_sync(0xFFFFFFFFu, e, 1);
    e += __shfl_xor_sync(0xFFFFFFFFu, e, 2);
    if (!(e < INFINITY)) e = INFINITY;  // an infinity, or a NaN in q
    e = rows_max(e);
    if (lane == 0) err_part[warp] = e;
    __syncthreads();
    if (threadIdx.x == 0) err_cta = fmaxf(fmaxf(err_part[0], err_part[1]), fmaxf(err_part[2], err_part[3]));
    cl.sync();
    float size = 0.f;  // of the terms of a bound
    for (int r = 0; r < CL; ++r) size = fmaxf(size, *cl.map_shared_rank(&err_cta, r));
    if (size == INFINITY)  // a block with an infinite key has the bound +inf, and says nothing of the others' terms
      size = finite_size<T, D>(G, sh, rows, i0, i1, reinterpret_cast<float *>(wmz), err_cta);
    uint32_t least = 0xFFFFFFFFu, most = 0u;
    // a stretch of four (of a CTA's bounds, whose number is a multiple of 16) at a time
    for (int i = threadIdx.x * 4; i < nm; i += NT * 4) {
      const int r = i / per;
      const float4 v = *reinterpret_cast<const float4 *>(cl.map_shared_rank(mine, r) + (i - r * per));
      const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k < nm) {
          const uint32_t y = order(x[k]);
          c.key[i + k] = y;
          least = min(least, y);
          most = max(most, y);
        }
    }
    // terms that fp32 does not hold: 64 bits decide for all of them.  (Otherwise a bound that is no number or infinite comes
    // from such a digest, and is +inf: one of max(q, 0) and min(q, 0) is 0.)
    const bool wide = !(size < 0x1p120f) || (size > 0.f && size < 0x1p-60f);
    c.list += A.sink;  // behind the first blocks
    choose<T, D>(G, c, sh, digest, lo, nm, m, wide ? INFINITY : size * 0x1p-16f, wide, least, most, red, redu, counter);
    c.list -= A.sink;
  }
  for (int i = threadIdx.x; i < ns; i += NT)  // those that no bound decides
    if (!choice || i < A.sink) c.list[i] = (uint16_t)i;
    else if (i >= ns - A.recent) c.list[i] = (uint16_t)(nbk - ns + i);
  __syncthreads();
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
    if (R.leave(G, wmz + warp * 8, so + warp * G * D))
      share_again<T, D>(A, q, bh, c.list, x0 + warp, (x1 - x0 - warp + NW - 1) / NW, seen, wmz + warp * 8, so + warp * G * D);
    __syncthreads();
    join_warps<D, NW>(G, wmz, so, sh, mz);
  }
  cl.sync();
  for (int i = threadIdx.x; i < CL * G; i += NT) all[i / G][i % G] = cl.map_shared_rank(mz, i / G)[i % G];
  __syncthreads();
  if ((int)threadIdx.x < G) {
    const int r = threadIdx.x;
    float M = -INFINITY, Z = 0.f;
    for (int s = 0; s < CL; ++s)
      if (all[s][r].y != 0.f) M = fmaxf(M, all[s][r].x);
    for (int s = 0; s < CL; ++s) {
      const float f = all[s][r].y != 0.f ? tc::ex2(M == -INFINITY ? 0.f : all[s][r].x - M) : 0.f;
      Z += f * all[s][r].y;
      all[s][r].x = f;  // the share's factor
    }
    sI[r] = 1.f / Z;
    if (rank == 0 && lse) lse[(long)r * A.nq] = (M + log2f(Z)) * 0.6931471805599453f;
  }
  __syncthreads();
  for (int i = rank * NT + threadIdx.x; i < G * D; i += CL * NT) {
    const int r = i / D;
    float x[16], v = 0.f;
#pragma unroll
    for (int s = 0; s < 16; ++s) x[s] = s < CL ? cl.map_shared_rank(sh, s)[i] : 0.f;
#pragma unroll
    for (int s = 0; s < 16; ++s)
      if (s < CL) v += all[s][r].x * x[s];
    o[r * A.so[1] + i % D] = T(v * sI[r]);
  }
  cl.sync();  // nobody leaves while its shares are read
}

// How many clusters of `size` such CTAs the current device holds at once (remembered; 0: none).
long clusters_at_once(const void *kernel, int threads, size_t bytes, int size) {
  static std::mutex mu;
  static std::map<std::tuple<int, const void *, size_t, int>, int> known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple(dev, kernel, bytes, size);
  const auto it = known.find(key);
  if (it != known.end()) return it->second;
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)size);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = bytes;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)size;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (ensure_smem(kernel, bytes) ||
      (size > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (known.size() < 4096) known[key] = n;
  return n;
}

template <typename T, int D>
int run(BlkArgs A, long units, cudaStream_t st) {
  const size_t warps = NW * Rows<T, D>::RING, choice = (size_t)A.nb * 12;
  A.area = (int)(((warps > choice ? warps : choice) + 15) & ~(size_t)15);
  auto need = [&](int CL) {
    return (size_t)A.G * D * 4 + A.area + (((size_t)A.nb / CL + 20) & ~(size_t)3) * 4 + (size_t)A.nb * 2 + 16;
  };
  // CTAs per unit: the largest cluster of which every unit's is on the GPU at once.  Clusters do not
  // cross groups of SMs, so that is asked for and not computed (448 CTAs in clusters of 7 on room for
  // 456 ran in two rounds: 69 us, 59 in clusters of 4).
  const long share = (long)kPerSm<T, D> * kNumSmsHint / units;
  int CL = (int)(share > 16 ? 16 : share < 1 ? 1 : share);
  for (; CL > 1; --CL)
    if (clusters_at_once((const void *)blocks_kernel<T, D>, NT, need(CL), CL) >= units) break;
  const size_t bytes = need(CL);
  if (units * CL > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  if (ensure_smem((const void *)blocks_kernel<T, D>, bytes)) return KV_ERR_CUDA;
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

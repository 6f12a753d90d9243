// rope.cu -- RMS norm of query and key heads, rotary positions and the rows of the cache,
// in one pass over a projection.
//
// A row is one head of one token; its d elements are d / 16 lanes' 16 each, as 8 pairs
// (a, b) that turn together, so that a rotation needs no exchange.  Where in the row
// a lane's two runs of 8 elements lie depends on the pairing:
//   halves       8i and rot/2 + 8i below rot, neighbouring runs behind it;
//   neighbours   16i and 16i + 8;
// and when rot / 2 is no multiple of 8 (halves only) elements are read one by one.
// A warp takes groups of rows of one token, queries, then keys, then values; the lanes that hold
// the same pairs of the group's rows share out the cosines and sines, and a token's are made once.
// No barrier: small calls are bound by latency (one token of 32/8 heads 2.8 us, 64 tokens 3.3 us).
//
// Angles: a frequency in turns is held as a 64-bit fraction of a turn, so position x
// frequency modulo 1 is one wrapping integer product, exact at any position; the upper
// 32 bits go to sincospif.  The fraction comes from the double's own bits by one integer product
// with 2^66 / (2 pi): the 64-bit floating-point unit is slow here.  It is off by 2^-64 turns
// and 2^-63 of itself, the angle by |pos| times that, far below the 2^-32 turns that are cut off;
// fp32 products would lose it from positions of a few thousand on.
//
// Long calls move as much as a copy and as fast: 32768 tokens of 32/8 heads 124 us, 6.5 TB/s (0.96 of
// a copy's rate; without the arithmetic 122).  Rows loaded in batches of four groups with nothing in
// flight meanwhile 147 us (4.7 of 10 cycles of an instruction waiting for them), 8 elements a lane
// and twice the warps 157, heads fixed to a warp that goes through the tokens 171.
#include <cmath>

#include "kvc_internal.cuh"
#include "pdl.cuh"

namespace kvc {
namespace {

constexpr int NT = 128, NW = NT / 32;
constexpr int kPerSm = 4;       // CTAs of an SM
constexpr int kDeep = 6;        // groups that may be on their way behind the one at hand
enum { HALVES = 0, NEIGHBOURS = 1, HALVES_ODD = 2 };

struct RopeArgs {
  kv_qkv_heads h;
  int *status;
  int groups[3];  // row groups (what a warp holds at a time) of queries, keys, values
  int steps;      // groups per item
  int chunks;     // items per token
};

constexpr int RUN = 8, PAIRS = 8;  // elements of a lane's two runs, which make as many pairs

// 16 elements in two runs.
template <typename T> struct Raw {
  static constexpr int H = sizeof(T) / 2;  // 16-byte vectors of a run
  uint4 v[2 * H];
};

// The pairs' first and second elements, packed by twos.
struct Pairs {
  float2 a[PAIRS / 2], b[PAIRS / 2];
};
__device__ __forceinline__ void words(const uint4 &v, uint32_t *w) {
  w[0] = v.x;
  w[1] = v.y;
  w[2] = v.z;
  w[3] = v.w;
}
template <int MODE>
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16> &r, Pairs &p) {
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
  uint32_t w[8];
  words(r.v[0], w);
  words(r.v[1], w + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (MODE == NEIGHBOURS) {
      p.a[i] = make_float2(lo(w[2 * i]), lo(w[2 * i + 1]));
      p.b[i] = make_float2(hi(w[2 * i]), hi(w[2 * i + 1]));
    } else {
      p.a[i] = make_float2(lo(w[i]), hi(w[i]));
      p.b[i] = make_float2(lo(w[4 + i]), hi(w[4 + i]));
    }
  }
}
template <int MODE>
__device__ __forceinline__ void unpack(const Raw<float> &r, Pairs &p) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) words(r.v[i], w + 4 * i);
  auto f = [&](int i) { return __uint_as_float(w[i]); };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p.a[i] = MODE == NEIGHBOURS ? make_float2(f(4 * i), f(4 * i + 2)) : make_float2(f(2 * i), f(2 * i + 1));
    p.b[i] = MODE == NEIGHBOURS ? make_float2(f(4 * i + 1), f(4 * i + 3)) : make_float2(f(8 + 2 * i), f(9 + 2 * i));
  }
}
template <int MODE>
__device__ __forceinline__ void pack(const Pairs &p, Raw<__nv_bfloat16> &r) {
  uint32_t w[8];
  auto two = [](float x, float y) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[MODE == NEIGHBOURS ? 2 * i : i] = MODE == NEIGHBOURS ? two(p.a[i].x, p.b[i].x) : two(p.a[i].x, p.a[i].y);
    w[MODE == NEIGHBOURS ? 2 * i + 1 : 4 + i] = MODE == NEIGHBOURS ? two(p.a[i].y, p.b[i].y) : two(p.b[i].x, p.b[i].y);
  }
  r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
  r.v[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
template <int MODE>
__device__ __forceinline__ void pack(const Pairs &p, Raw<float> &r) {
  float w[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[MODE == NEIGHBOURS ? 4 * i : 2 * i] = p.a[i].x;
    w[MODE == NEIGHBOURS ? 4 * i + 2 : 2 * i + 1] = p.a[i].y;
    w[MODE == NEIGHBOURS ? 4 * i + 1 : 8 + 2 * i] = p.b[i].x;
    w[MODE == NEIGHBOURS ? 4 * i + 3 : 9 + 2 * i] = p.b[i].y;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.v[i] = make_uint4(__float_as_uint(w[4 * i]), __float_as_uint(w[4 * i + 1]), __float_as_uint(w[4 * i + 2]), __float_as_uint(w[4 * i + 3]));
}

// Elements of pair x of a row whose rot / 2 is no multiple of RUN.
__device__ __forceinline__ int2 odd_pair(int x, int rot) {
  return x < rot / 2 ? make_int2(x, x + rot / 2) : make_int2(2 * x, 2 * x + 1);
}

// This lane's elements of a row; one that is read once makes way for others in the caches.
template <typename T, int MODE, bool ONCE = true>
__device__ __forceinline__ void load_row(const T *p, int a, int b, int rot, Raw<T> &r) {
  if constexpr (MODE == HALVES_ODD) {
    T *e = reinterpret_cast<T *>(r.v);
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      const int2 at = odd_pair(a + j, rot);
      e[j] = p[at.x];
      e[RUN + j] = p[at.y];
    }
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T>::H; ++i) {
      const uint4 *x = reinterpret_cast<const uint4 *>(p + a) + i, *y = reinterpret_cast<const uint4 *>(p + b) + i;
      r.v[i] = ONCE ? __ldcs(x) : *x;
      r.v[Raw<T>::H + i] = ONCE ? __ldcs(y) : *y;
    }
  }
}
template <typename T, int MODE>
__device__ __forceinline__ void store_row(T *p, int a, int b, int rot, const Raw<T> &r) {
  if constexpr (MODE == HALVES_ODD) {
    const T *e = reinterpret_cast<const T *>(r.v);
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      const int2 at = odd_pair(a + j, rot);
      p[at.x] = e[j];
      p[at.y] = e[RUN + j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T>::H; ++i) {
      reinterpret_cast<uint4 *>(p + a)[i] = r.v[i];
      reinterpret_cast<uint4 *>(p + b)[i] = r.v[Raw<T>::H + i];
    }
  }
}

// x / (2 pi) modulo 1 in units of 2^-64, from the bits of the double x.
__device__ __forceinline__ unsigned long long turn_fraction(double x) {
  const unsigned long long bits = (unsigned long long)__double_as_longlong(x);
  const int e = (int)(bits >> 52 & 0x7FF) - 1023;
  // x = m 2^(e - 63); m 2^66 / (2 pi) = hi 2^64 + lo; the fraction is that 2^(e - 65)
  const unsigned long long m = (bits << 11) | 0x8000000000000000ull, c = 0xA2F9836E4E44152Aull;
  const unsigned long long hi = __umul64hi(m, c), lo = m * c;
  const int s = 65 - e;  // to the right
  unsigned long long r = 0;
  if (s >= 64) r = s < 128 ? hi >> (s - 64) : 0;
  else if (s > 0) r = hi << (64 - s) | lo >> s;
  return bits >> 63 ? 0ull - r : r;
}

// What a lane knows for good: its place in a row and the frequencies whose cosines it makes.
// PART: not all pairs of a row turn.
template <typename T, int D, int MODE, bool PART>
struct Lane {
  static constexpr int LPR = D / (2 * RUN), RPW = 32 / LPR;  // lanes per row, rows of a group
  static constexpr int NP = PAIRS / RPW;                     // pairs whose cosines a lane makes
  int li, lr, a, b;  // lane of a row, row of a group, the lane's runs
  int turning;       // how many of the lane's pairs turn: the first ones
  unsigned long long frac[NP];

  __device__ __forceinline__ Lane(int rot) {
    const int lane = threadIdx.x & 31;
    li = lane % LPR;
    lr = lane / LPR;
    turning = min(PAIRS, max(0, rot / 2 - PAIRS * li));
    if constexpr (MODE == HALVES) {
      const int turning = rot / (2 * RUN);
      a = li < turning ? RUN * li : 2 * RUN * li;
      b = li < turning ? RUN * li + rot / 2 : 2 * RUN * li + RUN;
    } else if constexpr (MODE == NEIGHBOURS) {
      a = 2 * RUN * li;
      b = a + RUN;
    } else {
      a = RUN * li;
      b = 0;
    }
  }
  __device__ __forceinline__ void frequencies(const kv_qkv_heads &h) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int x = PAIRS * li + lr * NP + i;
      frac[i] = x < h.rot / 2 ? turn_fraction(h.inv_freq[x]) : 0ull;
    }
  }
  // Cosines and sines of this lane's pairs at a position; those of pairs that do not turn are not used.
  __device__ __forceinline__ void angles(const kv_qkv_heads &h, int pos, float2 (&c)[PAIRS / 2], float2 (&s)[PAIRS / 2]) const {
    float cc[NP], ss[NP], cs[PAIRS], sn[PAIRS];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const unsigned long long turn = (unsigned long long)(long long)pos * frac[i];
      sincospif((float)(int)(turn >> 32) * 0x1p-31f, &ss[i], &cc[i]);
      cc[i] *= h.rot_scale;
      ss[i] *= h.rot_scale;
    }
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      cs[j] = __shfl_sync(0xFFFFFFFFu, cc[j % NP], j / NP * LPR + li);
      sn[j] = __shfl_sync(0xFFFFFFFFu, ss[j % NP], j / NP * LPR + li);
    }
#pragma unroll
    for (int j = 0; j < PAIRS / 2; ++j) {
      c[j] = make_float2(cs[2 * j], cs[2 * j + 1]);
      s[j] = make_float2(sn[2 * j], sn[2 * j + 1]);
    }
  }
  __device__ __forceinline__ void weights(const kv_qkv_heads &h, int which, Pairs &w) const {
    const float plus = h.flags & KV_ROPE_ONE_PLUS ? 1.f : 0.f;
    const T *p = static_cast<const T *>(which ? h.k_weight : h.q_weight);
    if (p) {
      Raw<T> x;
      load_row<T, MODE, false>(p, a, b, h.rot, x);
      unpack<MODE>(x, w);
    }
#pragma unroll
    for (int j = 0; j < PAIRS / 2; ++j) {
      w.a[j] = p ? make_float2(w.a[j].x + plus, w.a[j].y + plus) : make_float2(1.f, 1.f);
      w.b[j] = p ? make_float2(w.b[j].x + plus, w.b[j].y + plus) : make_float2(1.f, 1.f);
    }
  }
  // A group's rows normalised and turned.  The two elements of a pair that does not turn have nothing to do with one
  // another: each is only scaled, and stays as it was without the norm (a turn by 0 would hand an infinity or a NaN on
  // to the other and lose the sign of a zero).
  __device__ __forceinline__ void turn(Raw<T> &raw, bool norm, float eps, const Pairs &w, const float2 (&c)[PAIRS / 2],
                                       const float2 (&s)[PAIRS / 2]) const {
    Pairs x;
    unpack<MODE>(raw, x);
    float f = 1.f;
    if (norm) {
      float2 q = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < PAIRS / 2; ++j) q = __ffma2_rn(x.a[j], x.a[j], __ffma2_rn(x.b[j], x.b[j], q));
      float sum = q.x + q.y;
#pragma unroll
      for (int o = LPR / 2; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      f = rsqrtf(sum * (1.f / D) + eps);
    }
    const float2 f2 = make_float2(f, f), n2 = make_float2(-f, -f);
#pragma unroll
    for (int j = 0; j < PAIRS / 2; ++j) {
      float2 p = x.a[j], r = x.b[j];
      if (norm) {
        p = __fmul2_rn(p, w.a[j]);
        r = __fmul2_rn(r, w.b[j]);
      }
      const float2 cf = __fmul2_rn(c[j], f2), sf = __fmul2_rn(s[j], f2), nf = __fmul2_rn(s[j], n2);
      x.a[j] = __ffma2_rn(r, nf, __fmul2_rn(p, cf));
      x.b[j] = __ffma2_rn(p, sf, __fmul2_rn(r, cf));
      if constexpr (PART) {
        const float2 ps = __fmul2_rn(p, f2), rs = __fmul2_rn(r, f2);
        if (2 * j >= turning) x.a[j].x = ps.x, x.b[j].x = rs.x;
        if (2 * j + 1 >= turning) x.a[j].y = ps.y, x.b[j].y = rs.y;
      }
    }
    pack<MODE>(x, raw);
  }
};

// The tensors' rows of token t of batch row bi: this lane's first input and output row (the latter at row 0 of
// the token axis).
template <typename T>
__device__ __forceinline__ const T *input(const kv_qkv_heads &h, int which, int bi, int t, int head) {
  const int64_t *st = h.strides + 3 * which;
  return static_cast<const T *>(which == 0 ? h.q : which == 1 ? h.k : h.v) + bi * st[0] + t * st[2] + head * st[1];
}
template <typename T>
__device__ __forceinline__ T *output(const kv_qkv_heads &h, int which, int bi, int head) {
  const int64_t *st = h.strides + 9 + 3 * which;
  return static_cast<T *>(which == 0 ? h.q_out : which == 1 ? h.k_out : h.v_out) + bi * st[0] + head * st[1];
}

// ---- few tokens, or rows that the ring below does not hold: an item is some groups of a token ----
template <typename T, int D, int MODE, bool PART>
__global__ void __launch_bounds__(NT, kPerSm) rope_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int U = 2;  // groups in flight
  using L = Lane<T, D, MODE, PART>;
  const kv_qkv_heads &h = A.h;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long items = (long)h.B * h.T * A.chunks, stride = (long)gridDim.x * NW;
  L l(h.rot);
  pdl_wait();
  pdl_launch();
  l.frequencies(h);
  const bool norm = h.flags & KV_ROPE_NORM;
#pragma unroll 1
  for (long item = (long)blockIdx.x * NW + warp; item < items; item += stride) {
    const int token = (int)(item / A.chunks), g0 = (int)(item - (long)token * A.chunks) * A.steps;
    const int bi = token / h.T, t = token - bi * h.T;
    const int pos = h.pos ? h.pos[token] : t;
    if (h.seq) {
      const int n = h.seq[bi];
      if (n < 0 || n > h.T) {
        if (lane == 0 && A.status) atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
        continue;
      }
      if (t >= n) continue;
    }
    float2 c[PAIRS / 2], s[PAIRS / 2];
    bool have_angles = false;
    int start = 0;  // the tensor's first group
#pragma unroll 1
    for (int which = 0; which < 3; start += A.groups[which], ++which) {
      const int lo = max(g0, start), n = min(g0 + A.steps, start + A.groups[which]) - lo;
      if (n <= 0) continue;
      const int head = (lo - start) * L::RPW + l.lr, left = (which ? h.Hkv : h.Hq) - head;  // this lane's first, and heads from there
      const T *in = input<T>(h, which, bi, t, head);
      T *out = output<T>(h, which, bi, head);
      const int32_t *slot = which && h.slot ? h.slot + bi * h.Hkv + head : nullptr;
      const long step_in = L::RPW * h.strides[3 * which + 1], step_out = L::RPW * h.strides[10 + 3 * which];
      const long token_out = h.strides[11 + 3 * which];
      const int cap = which ? h.cap : h.T;
      Pairs w;
      if (which < 2 && norm) l.weights(h, which, w);
#pragma unroll 1
      for (int g = 0; g < n; g += U) {
        Raw<T> raw[U];
        int row[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          row[u] = t;
          if (g + u < n && (g + u) * L::RPW < left) {
            load_row<T, MODE>(in, l.a, l.b, h.rot, raw[u]);
            if (slot) row[u] += slot[(g + u) * L::RPW];
          }
          in += step_in;
        }
        if (which < 2 && !have_angles) {
          l.angles(h, pos, c, s);
          have_angles = true;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (g + u >= n) break;
          if (which < 2) l.turn(raw[u], norm, h.eps, w, c, s);
          if ((g + u) * L::RPW < left) {
            if (row[u] >= 0 && row[u] < cap)
              store_row<T, MODE>(out + row[u] * token_out, l.a, l.b, h.rot, raw[u]);
            else if (l.li == 0 && A.status)
              atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
          }
          out += step_out;
        }
      }
    }
  }
}

// ---- many tokens: a warp has one token, all of whose rows are sent for at once ----
// Each lane copies what it reads itself into shared memory, so nothing is waited for but the copies.
// Warps that go on to other tokens, sending for a group of the next one as its place becomes free, are
// slower the more tokens they have (two 122 us, four 126, fourteen 141; one token and no more
// 124): tokens that are on their way together should lie together.
template <typename T, int D, int MODE, bool PART>
__global__ void __launch_bounds__(NT, kPerSm) rope_token_kernel(const __grid_constant__ RopeArgs A) {
  using L = Lane<T, D, MODE, PART>;
  constexpr int V = 2 * Raw<T>::H;  // 16-byte pieces of a lane and group
  extern __shared__ __align__(16) uint4 places[];
  const kv_qkv_heads &h = A.h;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = A.groups[0] + A.groups[1] + A.groups[2];
  uint4 *place = places + (size_t)warp * groups * V * 32 + lane;  // piece v of group g: place[(g V + v) 32]
  const int token = blockIdx.x * NW + warp;
  const bool deep = groups >= kDeep;
  L l(h.rot);
  pdl_wait();
  pdl_launch();
  if (token >= h.B * h.T) return;
  const int bi = token / h.T, t = token - bi * h.T;
  if (h.seq) {
    const int n = h.seq[bi];
    if (n < 0 || n > h.T) {
      if (lane == 0 && A.status) atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
      return;
    }
    if (t >= n) return;
  }
#pragma unroll 1
  for (int which = 0; which < 3; ++which) {
    const T *in = input<T>(h, which, bi, t, l.lr);
    const long step = L::RPW * h.strides[3 * which + 1];
    const int heads = (which ? h.Hkv : h.Hq) - l.lr;
#pragma unroll 1
    for (int g = 0; g < A.groups[which]; ++g, in += step, place += V * 32) {
      if (g * L::RPW < heads) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(place + v * 32)),
                       "l"(reinterpret_cast<const uint4 *>(in + (v < V / 2 ? l.a : l.b)) + v % (V / 2))
                       : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  place -= groups * V * 32;
  const int pos = h.pos ? h.pos[token] : t;
  l.frequencies(h);
  const bool norm = h.flags & KV_ROPE_NORM;
  float2 c[PAIRS / 2], s[PAIRS / 2];
  l.angles(h, pos, c, s);
#pragma unroll 1
  for (int which = 0; which < 3; ++which) {
    const int heads = (which ? h.Hkv : h.Hq) - l.lr, cap = which ? h.cap : h.T;
    const long step_out = L::RPW * h.strides[10 + 3 * which], token_out = h.strides[11 + 3 * which];
    T *out = output<T>(h, which, bi, l.lr);
    const int32_t *slot = which && h.slot ? h.slot + bi * h.Hkv + l.lr : nullptr;
    if (!slot) out += t * token_out;
    Pairs w;
    if (which < 2 && norm && A.groups[which]) l.weights(h, which, w);
#pragma unroll 1
    for (int g = 0; g < A.groups[which]; ++g) {
      const bool there = g * L::RPW < heads;
      int row = t;
      if (slot && there) row += slot[g * L::RPW];
      // the commits behind the last group keep the count: at most kDeep - 1 groups are left behind this one
      if (deep) asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 1) : "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
      asm volatile("cp.async.commit_group;" ::: "memory");
      Raw<T> raw;
#pragma unroll
      for (int v = 0; v < V; ++v) raw.v[v] = place[v * 32];
      if (which < 2) l.turn(raw, norm, h.eps, w, c, s);
      if (there) {
        if (row >= 0 && row < cap)
          store_row<T, MODE>(slot ? out + row * token_out : out, l.a, l.b, h.rot, raw);
        else if (l.li == 0 && A.status)
          atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
      }
      place += V * 32;
      out += step_out;
    }
  }
}

template <typename T, int D, int MODE, bool PART>
int run(RopeArgs A, cudaStream_t st) {
  constexpr int RPW = Lane<T, D, MODE, PART>::RPW;
  const long tokens = (long)A.h.B * A.h.T;
  A.groups[0] = A.h.q ? (A.h.Hq + RPW - 1) / RPW : 0;
  A.groups[1] = A.h.k ? (A.h.Hkv + RPW - 1) / RPW : 0;
  A.groups[2] = A.h.v ? (A.h.Hkv + RPW - 1) / RPW : 0;
  const int groups = A.groups[0] + A.groups[1] + A.groups[2];
  const long warps = (long)kPerSm * NW * kNumSmsHint;  // that run at once
  cudaError_t e;
  if constexpr (MODE != HALVES_ODD) {
    // As many tokens as warps run at once, with 12 KB each at most (four CTAs an SM); fewer tokens are
    // shared out over the warps (64 tokens 3.2 us, a warp each 5).
    const size_t bytes = (size_t)groups * RPW * D * sizeof(T);
    if (tokens >= warps && bytes <= 12 * 1024) {
      if (ensure_smem((const void *)rope_token_kernel<T, D, MODE, PART>, NW * bytes)) return KV_ERR_CUDA;
      e = launch_pdl(rope_token_kernel<T, D, MODE, PART>, (unsigned)((tokens + NW - 1) / NW), NT, NW * bytes, st, A);
      if (e != cudaSuccess) return cuda_failure(e, "norm and rotary positions");
      return launch_status();
    }
  }
  // A whole token per warp computes its angles once; fewer rows where that leaves warps idle.
  A.steps = (int)(tokens * groups / warps);
  A.steps = A.steps < 1 ? 1 : A.steps > groups ? groups : A.steps;
  A.chunks = (groups + A.steps - 1) / A.steps;
  const long ctas = (tokens * A.chunks + NW - 1) / NW, most = 4L * kPerSm * kNumSmsHint;
  e = launch_pdl(rope_kernel<T, D, MODE, PART>, (unsigned)(ctas < most ? ctas : most), NT, 0, st, A);
  if (e != cudaSuccess) return cuda_failure(e, "norm and rotary positions");
  return launch_status();
}

template <typename T, int D>
int run_mode(const RopeArgs &A, cudaStream_t st) {
  const bool part = A.h.rot < D;
  if (A.h.flags & KV_ROPE_INTERLEAVED) return part ? run<T, D, NEIGHBOURS, true>(A, st) : run<T, D, NEIGHBOURS, false>(A, st);
  if (A.h.rot % (2 * RUN)) return run<T, D, HALVES_ODD, true>(A, st);
  return part ? run<T, D, HALVES, true>(A, st) : run<T, D, HALVES, false>(A, st);
}

}  // namespace

int launch_qk_norm_rope(const kv_qkv_heads &h, int *status, cudaStream_t st) {
  const RopeArgs A{h, status, {}, 0, 0};
  if (h.dtype == KV_BF16) return h.d == 128 ? run_mode<__nv_bfloat16, 128>(A, st) : run_mode<__nv_bfloat16, 64>(A, st);
  return h.d == 128 ? run_mode<float, 128>(A, st) : run_mode<float, 64>(A, st);
}

// Frequencies in 64 bits on the host.
int rope_freqs(int rot, double theta, const kv_rope_scaling *s, double *f, float *rot_scale) {
  const int kind = s ? s->kind : KV_ROPE_PLAIN;
  const double two_pi = 6.283185307179586;
  const bool bands = kind == KV_ROPE_BANDS || kind == KV_ROPE_YARN;
  if (rot < 0 || rot % 2 || !(theta > 0) || !std::isfinite(theta) || (rot && !f) || kind < KV_ROPE_PLAIN || kind > KV_ROPE_YARN ||
      (kind != KV_ROPE_PLAIN && !(s->factor >= 1 && std::isfinite(s->factor))) ||
      (bands && !(s->low > 0 && s->high > s->low && std::isfinite(s->high) && s->context > 0 && std::isfinite(s->context))) ||
      (kind == KV_ROPE_YARN && theta == 1.0))
    return KV_ERR_INVALID_ARG;
  if (kind == KV_ROPE_BASE && rot > 2) theta *= std::pow(s->factor, (double)rot / (rot - 2));
  double first = 0, last = 0;  // YaRN: pair indices that turn `high` and `low` times within the context
  if (kind == KV_ROPE_YARN) {
    auto index = [&](double turns) { return rot * std::log(s->context / (turns * two_pi)) / (2 * std::log(theta)); };
    first = std::fmax(0.0, std::floor(index(s->high)));
    last = std::fmin(rot - 1.0, std::ceil(index(s->low)));
    if (!(last > first)) last = first + 1e-3;
  }
  for (int i = 0; i < rot / 2; ++i) {
    const double x = std::pow(theta, -2.0 * i / rot);
    double keep = 1;  // share of the unscaled frequency
    if (kind == KV_ROPE_LINEAR) keep = 0;
    if (kind == KV_ROPE_BANDS) keep = (s->context * x / two_pi - s->low) / (s->high - s->low);
    if (kind == KV_ROPE_YARN) keep = 1 - (i - first) / (last - first);
    keep = std::fmin(1.0, std::fmax(0.0, keep));
    f[i] = kind == KV_ROPE_PLAIN || kind == KV_ROPE_BASE ? x : x * keep + x / s->factor * (1 - keep);
  }
  if (rot_scale) *rot_scale = kind == KV_ROPE_YARN ? (float)(0.1 * std::log(s->factor) + 1) : 1.f;
  return KV_OK;
}

}  // namespace kvc

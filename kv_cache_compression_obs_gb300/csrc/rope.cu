// rope.cu -- RMS norm of query and key heads, rotary positions and the rows of the cache,
// in one pass over a projection.
//
// A row is one head of one token; its d elements are d / 16 lanes' 16 each, as 8 pairs
// (a, b) that turn together, so that a rotation needs no exchange.  Where in the row
// a lane's two runs of 8 elements lie depends on the pairing:
//   halves       8i and rot/2 + 8i below rot, neighbouring runs behind it;
//   neighbours   16i and 16i + 8;
// and when rot / 2 is no multiple of 8 (halves only) elements are read one by one.
// A warp takes some rows of one token (queries, keys, values in that order): cosines and
// sines are computed once for them all.
//
// Angles: a frequency in turns is held as a 64-bit fraction of a turn, so position x
// frequency modulo 1 is one wrapping integer product, exact at any position; the upper
// 32 bits go to sincospif.  The fraction is off by 2^-55, so the angle by
// |pos| 2^-55 turns, 2^-24 at the largest position; fp32 products would lose it
// from positions of a few thousand on.
//
// Bound by memory in long calls, by latency in short ones.
#include <cmath>

#include "kvc_internal.cuh"
#include "pdl.cuh"

namespace kvc {
namespace {

constexpr int NT = 256, NW = NT / 32;
enum { HALVES = 0, NEIGHBOURS = 1, HALVES_ODD = 2 };

struct RopeArgs {
  kv_qkv_heads h;
  int *status;
  int rows, nq, nk;  // heads of a token that take part; of them queries, keys
  int steps;         // row groups (what a warp holds at a time) per item
  int chunks;        // items per token
};

// 16 elements in two runs of 8.
template <typename T> struct Raw {
  static constexpr int H = sizeof(T) / 2;  // 16-byte vectors per run
  uint4 v[2 * H];
};

__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16> &r, float (&x)[16]) {
  Vec16<__nv_bfloat16>::unpack(r.v[0], x);
  Vec16<__nv_bfloat16>::unpack(r.v[1], x + 8);
}
__device__ __forceinline__ void unpack(const Raw<float> &r, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) Vec16<float>::unpack(r.v[i], x + 4 * i);
}
__device__ __forceinline__ void pack(const float (&x)[16], Raw<__nv_bfloat16> &r) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&p);
  }
  r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
  r.v[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void pack(const float (&x)[16], Raw<float> &r) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.v[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                        __float_as_uint(x[4 * i + 3]));
}

// Elements of pair x of a row whose rot / 2 is no multiple of 8.
__device__ __forceinline__ int2 odd_pair(int x, int rot) {
  return x < rot / 2 ? make_int2(x, x + rot / 2) : make_int2(2 * x, 2 * x + 1);
}

template <typename T, int MODE>
__device__ __forceinline__ void load_row(const T *p, int a, int b, int rot, Raw<T> &r) {
  if constexpr (MODE == HALVES_ODD) {
    T *e = reinterpret_cast<T *>(r.v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int2 at = odd_pair(a + j, rot);
      e[j] = p[at.x];
      e[8 + j] = p[at.y];
    }
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T>::H; ++i) {
      r.v[i] = __ldcs(reinterpret_cast<const uint4 *>(p + a) + i);
      r.v[Raw<T>::H + i] = __ldcs(reinterpret_cast<const uint4 *>(p + b) + i);
    }
  }
}
template <typename T, int MODE>
__device__ __forceinline__ void store_row(T *p, int a, int b, int rot, const Raw<T> &r) {
  if constexpr (MODE == HALVES_ODD) {
    const T *e = reinterpret_cast<const T *>(r.v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int2 at = odd_pair(a + j, rot);
      p[at.x] = e[j];
      p[at.y] = e[8 + j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T>::H; ++i) {
      reinterpret_cast<uint4 *>(p + a)[i] = r.v[i];
      reinterpret_cast<uint4 *>(p + b)[i] = r.v[Raw<T>::H + i];
    }
  }
}

template <typename T, int D, int MODE>
__global__ void __launch_bounds__(NT) rope_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;  // lanes per row, rows of a warp at a time
  constexpr int U = sizeof(T) == 2 ? 4 : 2;    // row groups in flight
  __shared__ unsigned long long frac[D / 2];
  __shared__ float wt[2][D];
  const kv_qkv_heads &h = A.h;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int li = lane % LPR, lr = lane / LPR;
  pdl_wait();
  pdl_launch();
  for (int i = threadIdx.x; i < h.rot / 2; i += NT) {
    double x = h.inv_freq[i] * 0.15915494309189535;  // turns per position
    x -= floor(x);
    frac[i] = (unsigned long long)(x * 18446744073709551616.0);
  }
  if (h.flags & KV_ROPE_NORM)
    for (int i = threadIdx.x; i < 2 * D; i += NT) {
      const T *w = static_cast<const T *>(i < D ? h.q_weight : h.k_weight);
      wt[i / D][i % D] = w ? to_f32(w[i % D]) + (h.flags & KV_ROPE_ONE_PLUS ? 1.f : 0.f) : 1.f;
    }
  __syncthreads();
  int a, b;  // this lane's runs
  if constexpr (MODE == HALVES) {
    const int turning = h.rot / 16;
    a = li < turning ? 8 * li : 16 * li;
    b = li < turning ? 8 * li + h.rot / 2 : 16 * li + 8;
  } else if constexpr (MODE == NEIGHBOURS) {
    a = 16 * li;
    b = a + 8;
  } else {
    a = 8 * li;
    b = 0;
  }
  const long items = (long)h.B * h.T * A.chunks;
  for (long item = (long)blockIdx.x * NW + warp; item < items; item += (long)gridDim.x * NW) {
    const int token = (int)(item / A.chunks), first = (int)(item - (long)token * A.chunks) * A.steps * RPW;
    const int bi = token / h.T, t = token - bi * h.T;
    if (h.seq) {
      const int n = h.seq[bi];
      if (n < 0 || n > h.T) {
        if (lane == 0 && A.status) atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
        continue;
      }
      if (t >= n) continue;
    }
    const int last = min(A.rows, first + A.steps * RPW);
    const int pos = h.pos ? h.pos[token] : t;
    float c[8], s[8];
    bool have_angles = false;
    for (int r0 = first; r0 < last; r0 += U * RPW) {
      Raw<T> raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * RPW + lr;
        if (r < last) {
          const bool isq = r < A.nq, isk = r < A.nq + A.nk;
          const int64_t *st = h.strides + (isq ? 0 : isk ? 3 : 6);
          const int head = r - (isq ? 0 : isk ? A.nq : A.nq + A.nk);
          load_row<T, MODE>(static_cast<const T *>(isq ? h.q : isk ? h.k : h.v) + bi * st[0] + head * st[1] + t * st[2], a, b,
                            h.rot, raw[u]);
        }
      }
      if (!have_angles && first < A.nq + A.nk) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int x = 8 * li + j;
          if (x < h.rot / 2) {
            const unsigned long long turn = (unsigned long long)(long long)pos * frac[x];
            sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s[j], &c[j]);
            s[j] *= h.rot_scale;
            c[j] *= h.rot_scale;
          } else {
            s[j] = 0.f;
            c[j] = 1.f;
          }
        }
        have_angles = true;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * RPW + lr;
        const bool isq = r < A.nq, isk = r < A.nq + A.nk;
        if (r0 + u * RPW < A.nq + A.nk && r0 + u * RPW < last) {  // some row of the group turns
          float x[16];
          unpack(raw[u], x);
          if (h.flags & KV_ROPE_NORM) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) sum += x[j] * x[j];
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            const float f = rsqrtf(sum * (1.f / D) + h.eps);
            const float *w = wt[isq ? 0 : 1];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int2 at = MODE == HALVES_ODD ? odd_pair(a + j, h.rot) : make_int2(a + j, b + j);
              x[j] = x[j] * f * w[at.x];
              x[8 + j] = x[8 + j] * f * w[at.y];
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            constexpr bool N = MODE == NEIGHBOURS;
            const float p = x[N ? 2 * j : j], q = x[N ? 2 * j + 1 : 8 + j];
            x[N ? 2 * j : j] = p * c[j] - q * s[j];
            x[N ? 2 * j + 1 : 8 + j] = q * c[j] + p * s[j];
          }
          if (isk) pack(x, raw[u]);
        }
        if (r < last) {
          const int64_t *st = h.strides + (isq ? 9 : isk ? 12 : 15);
          const int head = r - (isq ? 0 : isk ? A.nq : A.nq + A.nk);
          int row = t;
          bool ok = true;
          if (!isq) {
            if (h.slot) row += h.slot[bi * h.Hkv + head];
            ok = row >= 0 && row < h.cap;
            if (!ok && li == 0 && A.status) atomicExch(A.status, (int)KV_ERR_INVALID_ARG);
          }
          if (ok)
            store_row<T, MODE>(static_cast<T *>(isq ? h.q_out : isk ? h.k_out : h.v_out) + bi * st[0] + head * st[1] + row * st[2],
                               a, b, h.rot, raw[u]);
        }
      }
    }
  }
}

template <typename T, int D, int MODE>
int run(RopeArgs A, cudaStream_t st) {
  constexpr int RPW = 32 / (D / 16);
  const long tokens = (long)A.h.B * A.h.T;
  const int groups = (A.rows + RPW - 1) / RPW;
  // A whole token per warp computes its angles once; fewer rows where that leaves warps idle.
  const long want = 16L * kNumSmsHint;
  A.steps = (int)(tokens * groups / want);
  A.steps = A.steps < 1 ? 1 : A.steps > groups ? groups : A.steps;
  A.chunks = (groups + A.steps - 1) / A.steps;
  const long ctas = (tokens * A.chunks + NW - 1) / NW, most = 8L * kNumSmsHint;
  const cudaError_t e = launch_pdl(rope_kernel<T, D, MODE>, (unsigned)(ctas < most ? ctas : most), NT, 0, st, A);
  if (e != cudaSuccess) return cuda_failure(e, "norm and rotary positions");
  return launch_status();
}

template <typename T, int D>
int run_mode(const RopeArgs &A, cudaStream_t st) {
  if (A.h.flags & KV_ROPE_INTERLEAVED) return run<T, D, NEIGHBOURS>(A, st);
  return A.h.rot % 16 == 0 ? run<T, D, HALVES>(A, st) : run<T, D, HALVES_ODD>(A, st);
}

}  // namespace

int launch_qk_norm_rope(const kv_qkv_heads &h, int *status, cudaStream_t st) {
  RopeArgs A{h, status};
  A.nq = h.q ? h.Hq : 0;
  A.nk = h.k ? h.Hkv : 0;
  A.rows = A.nq + A.nk + (h.v ? h.Hkv : 0);
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

// q8_cache.cu -- writing the 8-bit slot cache: gather-compaction of a prompt's
// kept rows into codes, and eviction of the slots with the least accumulated
// attention (H2O page, 两套代码 and 贪心驱逐算法; formulas of the codes in
// q8_common.cuh).
//
//   compact  destination slot m takes prompt row idx[m];
//   evict    destination slot m takes the source cache's slot idx[m], idx chosen
//            here: the leading slots with pos < sink and the last `recent` slots
//            stay, and of the others the (acc, slot)-largest, in slot order.
// Either way a destination block's rows are read once into the registers of one CTA, each
// thread some pieces of 16 elements of K and of V, its largest magnitudes found across the
// CTA and its codes written from the registers.
// The rows of the unfinished block are copied (evict: decoded where they were
// codes, rounded to the cache's dtype, half a step at most).
//
// compact is bound by memory: a tenth of 32768 rows, 32 layers of 8 heads, 102 us, 0.95 of the
// copy rate.  evict by arithmetic (nine instructions a code) and by the selection's barriers:
// 64 units of 60000 to 65536 slots to 32768, 195 us for the move (0.82 of the copy rate) and
// 37 us for the selection; 32 heads of 2048 slots 17 us, all latency.
#include "pdl.cuh"
#include "q8_common.cuh"
#include "select_common.cuh"

namespace kvc {
namespace {

constexpr int NTS = 1024;  // threads of the selection
constexpr int NWS = NTS / 32;

__device__ __forceinline__ void flag_bad(int *status) {
  if (status) atomicExch(status, (int)KV_ERR_INVALID_ARG);
}

// ---- the block kernel ------------------------------------------------------------
struct BlockArgs {
  // source: a prompt (K, V [units][T][d]) or a cache
  const void *src[2];
  const float *s;        // prompt scores [units][T] (may be null)
  const int32_t *idx;    // [units][k] (null: row m is prompt row m)
  int T, k;
  kv_q8_cache from, out;
  int d_log2, b_log2;    // d and block are powers of two
  int nblk;              // blocks per unit that may be written (the unfinished one included)
  int *status;
};

// 16 source elements as they lie in memory: rows of T, or codes with their scale.
template <typename T>
struct Piece {
  static constexpr int NV = 16 / Vec16<T>::N;  // vectors of 16 elements of T
  uint4 v[NV];
  float a;     // scale, when v[0] holds 16 codes
  bool coded;
  __device__ __forceinline__ void load_rows(const T *p) {
    coded = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
  }
  __device__ __forceinline__ void store_rows(T *p) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) reinterpret_cast<uint4 *>(p)[i] = v[i];
  }
  __device__ __forceinline__ void zero() {
    coded = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  // the values; CODES: of codes as well as of rows
  template <int FMT, bool CODES>
  __device__ __forceinline__ void get(float2 (&x)[8]) const {
    if (CODES && coded) {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
      const float2 a2 = make_float2(a, a);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Q8<FMT>::unpack4(w[i], x[2 * i], x[2 * i + 1]);
        x[2 * i] = __fmul2_rn(x[2 * i], a2);
        x[2 * i + 1] = __fmul2_rn(x[2 * i + 1], a2);
      }
    } else {
      float y[16];
#pragma unroll
      for (int i = 0; i < NV; ++i) Vec16<T>::unpack(v[i], y + i * Vec16<T>::N);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = make_float2(y[2 * i], y[2 * i + 1]);
    }
  }
  // the bits of the largest magnitude of a piece of rows
  __device__ __forceinline__ uint32_t big() const {
    if constexpr (sizeof(T) == 2) {  // without the sign bf16 bits order like their values
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        m = __vimax3_u16x2(m, v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu);
        m = __vimax3_u16x2(m, v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu);
      }
      return max(m & 0xFFFFu, m >> 16) << 16;
    } else {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        m = max_nan(max_nan(m, fabsf(__uint_as_float(v[i].x))), fabsf(__uint_as_float(v[i].y)));
        m = max_nan(max_nan(m, fabsf(__uint_as_float(v[i].z))), fabsf(__uint_as_float(v[i].w)));
      }
      return __float_as_uint(m);
    }
  }
};

// The block's two scales and its codes, `bytes` of them for K and for V, from pieces of rows.
template <typename T, int FMT, int N>
__device__ __forceinline__ void quantise(const Piece<T> (&p)[2][N], const int (&at)[N], int bytes,
                                         uint8_t *const (&co)[2], float *const (&so)[2], uint32_t (&red)[2][16]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) big = max(big, p[kv][i].big());
    big = __reduce_max_sync(0xFFFFFFFFu, big);
    if (lane == 0) red[kv][warp] = big;
  }
  __syncthreads();
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, lane < (int)blockDim.x >> 5 ? red[kv][lane] : 0u);
    const float a = q8_scale<FMT>(m), inv = __fdiv_rn(1.f, a);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (at[i] >= bytes) continue;
      float2 x[8];
      p[kv][i].template get<FMT, false>(x);
      *reinterpret_cast<uint4 *>(co[kv] + at[i]) = q8_pack16<FMT>(x, inv);
    }
    if (threadIdx.x == 0) *so[kv] = a;
  }
}

constexpr int kCompactPieces = 2;  // of K and of V per thread, all loads in flight together

// One CTA per (unit, destination block) of a prompt's kept rows.
template <typename T, int FMT>
__global__ void __launch_bounds__(512) compact_block_kernel(const __grid_constant__ BlockArgs A) {
  constexpr int PP = kCompactPieces;
  __shared__ uint32_t red[2][16];
  __shared__ int src[128];
  pdl_wait();
  pdl_launch();
  const int block = A.out.block, d = A.out.d, bl = A.b_log2;
  const int u = (int)(blockIdx.x / (unsigned)A.nblk);
  const int b = (int)(blockIdx.x - (unsigned)u * (unsigned)A.nblk);
  const int m0 = b << bl;
  const int rows = min(block, A.k - m0);
  for (int r = threadIdx.x; r < rows; r += blockDim.x) {
    const int j = A.idx ? A.idx[(long)u * A.k + m0 + r] : m0 + r;
    src[r] = j >= 0 && j < A.T ? j : -1;
  }
  __syncthreads();
  const long src0 = (long)u * A.T;
  Piece<T> p[2][PP];
  int at[PP];  // first of the piece's 16 elements within the block
#pragma unroll
  for (int i = 0; i < PP; ++i) {
    at[i] = (i * (int)blockDim.x + (int)threadIdx.x) << 4;
    const int row = at[i] >> A.d_log2;
    const int j = row < rows ? src[row] : -1;
    if (j < 0) {
      p[0][i].zero();
      p[1][i].zero();
    } else {
      const long f = ((src0 + j) << A.d_log2) + (at[i] & (d - 1));
      p[0][i].load_rows(static_cast<const T *>(A.src[0]) + f);
      p[1][i].load_rows(static_cast<const T *>(A.src[1]) + f);
    }
  }
  // what moves beside K and V, while they are on their way
  const long to = (long)u * A.out.cap + m0;
  for (int r = threadIdx.x; r < rows; r += blockDim.x) {
    const int j = src[r];
    if (j < 0) flag_bad(A.status);
    A.out.pos[to + r] = j;
    if (A.out.acc) A.out.acc[to + r] = j >= 0 && A.s ? A.s[src0 + j] : 0.f;
  }
  if (b == 0 && threadIdx.x == 0) A.out.len[u] = A.k;
  if (rows < block) {  // the unfinished block keeps its rows
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int i = 0; i < PP; ++i)
        if (at[i] >> A.d_log2 < rows)
          p[kv][i].store_rows(static_cast<T *>(kv ? A.out.Vt : A.out.Kt) + (((long)u << bl) << A.d_log2) + at[i]);
    return;
  }
  float *const so[2] = {A.out.Ks + (to >> bl), A.out.Vs + (to >> bl)};
  uint8_t *const co[2] = {static_cast<uint8_t *>(A.out.K) + (to << A.d_log2),
                          static_cast<uint8_t *>(A.out.V) + (to << A.d_log2)};
  quantise<T, FMT>(p, at, block << A.d_log2, co, so, red);
}

// ---- moving a cache's kept slots -----------------------------------------------------
// One CTA per (unit, run of destination blocks).  The run's slots and their scales are read
// once, at its start; the rows then come through a ring of stages, every thread copying
// (16 bytes at a time, asynchronously) exactly the pieces that it will decode, so that the
// stages need no barrier and several blocks' rows are in flight while one is quantised.
constexpr int kRunRows = 512;  // rows of a run at most

__device__ __forceinline__ void copy16_async(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}

// A unit's last blocks: unfinished rows among the sources, or the new unfinished block.  Few,
// so each piece is read twice (magnitude, then code) rather than held in registers.
template <typename T, int FMT>
__device__ __forceinline__ void move_last_block(const BlockArgs &A, int u, int b, int rows, int nf, const int *src,
                                                const float2 *skv, uint32_t (&red)[2][16]) {
  const int block = A.out.block, d = A.out.d, bl = A.b_log2, bytes = rows << A.d_log2;
  const long src0 = (long)u * A.from.cap, to = (long)u * A.out.cap + ((long)b << bl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
  for (int kv = 0; kv < 2; ++kv) {
    auto piece = [&](int at, float2 (&x)[8]) {
      const int row = at >> A.d_log2, el = at & (d - 1), j = src[row];
      Piece<T> p;
      if (j < nf) {
        p.v[0] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(kv ? A.from.V : A.from.K) +
                                                       ((src0 + j) << A.d_log2) + el));
        p.a = kv ? skv[row].y : skv[row].x;
        p.coded = true;
      } else {
        p.load_rows(static_cast<const T *>(kv ? A.from.Vt : A.from.Kt) + ((((long)u << bl) + (j - nf)) << A.d_log2) + el);
      }
      p.template get<FMT, true>(x);
    };
    float2 x[8];
    if (rows < block) {  // the unfinished block keeps its rows
#pragma unroll 1
      for (int at = threadIdx.x << 4; at < bytes; at += blockDim.x << 4) {
        piece(at, x);
        float y[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[2 * e] = x[e].x;
          y[2 * e + 1] = x[e].y;
        }
        store16(static_cast<T *>(kv ? A.out.Vt : A.out.Kt) + (((long)u << bl) << A.d_log2) + at, y);
      }
      continue;
    }
    float big = 0.f;
#pragma unroll 1
    for (int at = threadIdx.x << 4; at < bytes; at += blockDim.x << 4) {
      piece(at, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) big = max_nan(big, max_nan(fabsf(x[e].x), fabsf(x[e].y)));
    }
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(big));
    if (lane == 0) red[kv][warp] = m;
    __syncthreads();
    uint32_t v = red[kv][0];
    for (int w = 1; w < (int)blockDim.x >> 5; ++w) v = max(v, red[kv][w]);
    const float a = q8_scale<FMT>(v), inv = __fdiv_rn(1.f, a);
    uint8_t *const co = static_cast<uint8_t *>(kv ? A.out.V : A.out.K) + (to << A.d_log2);
#pragma unroll 1
    for (int at = threadIdx.x << 4; at < bytes; at += blockDim.x << 4) {
      piece(at, x);
      *reinterpret_cast<uint4 *>(co + at) = q8_pack16<FMT>(x, inv);
    }
    if (threadIdx.x == 0) (kv ? A.out.Vs : A.out.Ks)[to >> bl] = a;
  }
}

// SQ: 16-byte pieces of a block (K or V) per thread; a block is NTM * SQ of them.
template <typename T, int FMT, int NTM, int SQ, int ST>
__global__ void __launch_bounds__(NTM, 1024 / NTM) evict_move_kernel(const __grid_constant__ BlockArgs A, int runs, int run_blocks) {
  constexpr int BYTES = NTM * SQ * 16;  // codes of a block of K or V
  extern __shared__ __align__(16) unsigned char ring[];  // ST stages of K codes, V codes
  __shared__ uint32_t red[2][2][16];
  __shared__ int src[kRunRows];
  __shared__ float2 skv[kRunRows];  // the rows' scales
  pdl_wait();
  pdl_launch();
  const int block = A.out.block, bl = A.b_log2;
  const int u = (int)(blockIdx.x / (unsigned)runs);
  const int b0 = (int)(blockIdx.x - (unsigned)u * (unsigned)runs) * run_blocks;
  const int n_src = A.from.len[u];
  if (n_src < 0 || n_src > A.from.cap) return;  // reported by the selection
  const int n_new = min(n_src, A.k);
  const int r0 = b0 << bl;
  if (r0 >= n_new) return;
  const int rows = min(run_blocks << bl, n_new - r0);  // of the run
  const int nblk = (rows + block - 1) >> bl;
  const int nf = n_src >> bl << bl;  // slots held as codes
  const long src0 = (long)u * A.from.cap;
  int coded = 0;  // rows whose source is codes: the first ones, slots ascend
  for (int r = threadIdx.x; r < rows; r += NTM) {
    // one of the unit's slots, by the selection; held to it all the same: it is an address
    const int j = max(0, min(n_src - 1, A.idx[(long)u * A.k + r0 + r]));
    src[r] = j;
    if (j < nf) {
      skv[r] = make_float2(__ldg(A.from.Ks + ((src0 + j) >> bl)), __ldg(A.from.Vs + ((src0 + j) >> bl)));
      coded = r + 1;
    }
  }
  const int nring = __reduce_max_sync(0xFFFFFFFFu, coded);
  if ((threadIdx.x & 31) == 0) red[0][0][threadIdx.x >> 5] = (uint32_t)nring;
  __syncthreads();
  int most = 0;
  for (int w = 0; w < NTM / 32; ++w) most = max(most, (int)red[0][0][w]);
  const int ring_blocks = most >> bl;  // blocks of codes alone go through the ring
  __syncthreads();
  // this thread's pieces: the same place in every block
  int prow[SQ];
  const uint8_t *kq[SQ], *vq[SQ];
#pragma unroll
  for (int q = 0; q < SQ; ++q) {
    const int at = (q * NTM + (int)threadIdx.x) << 4;
    prow[q] = at >> A.d_log2;
    const long f = (src0 << A.d_log2) + (at & (A.out.d - 1));
    kq[q] = static_cast<const uint8_t *>(A.from.K) + f;
    vq[q] = static_cast<const uint8_t *>(A.from.V) + f;
  }
  auto fetch = [&](int i, int stage) {
    if (i < ring_blocks) {
      unsigned char *to = ring + stage * 2 * BYTES + (threadIdx.x << 4);
#pragma unroll
      for (int q = 0; q < SQ; ++q) {
        const unsigned long long off = (unsigned long long)(unsigned)src[(i << bl) + prow[q]] * (unsigned)A.out.d;
        copy16_async(to + q * NTM * 16, kq[q] + off);
        copy16_async(to + q * NTM * 16 + BYTES, vq[q] + off);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) fetch(i, i);
  for (int r = threadIdx.x; r < rows; r += NTM) {
    const long to = (long)u * A.out.cap + r0 + r;
    A.out.pos[to] = A.from.pos[src0 + src[r]];
    A.out.acc[to] = A.from.acc[src0 + src[r]];
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long out0 = (long)u * A.out.cap + r0;
  uint8_t *ck = static_cast<uint8_t *>(A.out.K) + (out0 << A.d_log2) + (threadIdx.x << 4);
  uint8_t *cv = static_cast<uint8_t *>(A.out.V) + (out0 << A.d_log2) + (threadIdx.x << 4);
  float *sok = A.out.Ks + (out0 >> bl), *sov = A.out.Vs + (out0 >> bl);
  int stage = 0, turn = 0;
  for (int i = 0; i < ring_blocks; ++i, ck += BYTES, cv += BYTES) {
    fetch(i + ST - 1, stage == 0 ? ST - 1 : stage - 1);  // into the stage that this thread has just read
    asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
    const unsigned char *st = ring + stage * 2 * BYTES + (threadIdx.x << 4);
    stage = stage + 1 == ST ? 0 : stage + 1;
    const int row0 = i << bl;
    uint4 k[SQ], v[SQ];
    float2 a[SQ];
#pragma unroll
    for (int q = 0; q < SQ; ++q) {
      k[q] = *reinterpret_cast<const uint4 *>(st + q * NTM * 16);
      v[q] = *reinterpret_cast<const uint4 *>(st + q * NTM * 16 + BYTES);
      a[q] = skv[row0 + prow[q]];
    }
    const int j0 = src[row0];
    if ((j0 & (block - 1)) == 0 && src[row0 + block - 1] - j0 == block - 1) {
      // a whole block moves: its codes and its scale as they are
#pragma unroll
      for (int q = 0; q < SQ; ++q) {
        *reinterpret_cast<uint4 *>(ck + q * NTM * 16) = k[q];
        *reinterpret_cast<uint4 *>(cv + q * NTM * 16) = v[q];
      }
      if (threadIdx.x == 0) {
        sok[i] = a[0].x;
        sov[i] = a[0].y;
      }
      continue;
    }
    // rounding c a to fp32 keeps the order: a piece's largest code gives its largest value
    // (NaN with a NaN scale, whatever the code)
    float bk = 0.f, bv = 0.f;
#pragma unroll
    for (int q = 0; q < SQ; ++q) {
      bk = max_nan(bk, __fmul_rn(Q8<FMT>::big16(k[q]), a[q].x));
      bv = max_nan(bv, __fmul_rn(Q8<FMT>::big16(v[q]), a[q].y));
    }
    const uint32_t mk = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(bk));
    const uint32_t mv = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(bv));
    // Two buffers in turn over the blocks that get here, each with a barrier (a whole block
    // has none): who writes a buffer again knows that everybody has read it.
    uint32_t (&rd)[2][16] = red[turn];
    turn ^= 1;
    if (lane < 2) rd[lane][warp] = lane ? mv : mk;
    __syncthreads();
    // the lower half of a warp finds K's scale, the upper half V's
    uint32_t big = (lane & 15) < NTM / 32 ? rd[lane >> 4][lane & 15] : 0u;
#pragma unroll
    for (int o = 8; o; o >>= 1) big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
    const float mine = q8_scale<FMT>(big), minv = __fdiv_rn(1.f, mine);
    const float ik = __shfl_sync(0xFFFFFFFFu, minv, 0), iv = __shfl_sync(0xFFFFFFFFu, minv, 16);
    if (warp == 0 && (lane & 15) == 0) (lane ? sov : sok)[i] = mine;
#pragma unroll
    for (int q = 0; q < SQ; ++q) {
      *reinterpret_cast<uint4 *>(ck + q * NTM * 16) = q8_requantise16<FMT>(k[q], a[q].x, ik);
      *reinterpret_cast<uint4 *>(cv + q * NTM * 16) = q8_requantise16<FMT>(v[q], a[q].y, iv);
    }
  }
  for (int i = ring_blocks; i < nblk; ++i) {
    __syncthreads();
    move_last_block<T, FMT>(A, u, b0 + i, min(block, rows - (i << bl)), nf, src + (i << bl), skv + (i << bl), red[0]);
  }
}

// ---- which slots stay ------------------------------------------------------------
// Units of any length, one CTA each: exact radix select over the candidates' order-preserving keys
// (4 passes of 8 bits, per-warp histograms), then one ordered pass.  Of the slots
// that equal the threshold the last ones stay: eviction takes the smallest
// (acc, slot) first, as the decode step's single victim does.
__global__ void __launch_bounds__(NTS) evict_select_kernel(const float *__restrict__ acc_all,
                                                           const int32_t *__restrict__ pos_all,
                                                           const int32_t *__restrict__ len, int cap, int keep,
                                                           int recent, int sink, int32_t *__restrict__ idx,
                                                           int32_t *__restrict__ len_out, int *status) {
  __shared__ uint32_t hist[NWS][256];
  __shared__ uint32_t tot[256];
  __shared__ int warp_sums[NWS];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_need, sh_sinks, sh_equal;
  const long u = blockIdx.x;
  const float *acc = acc_all + u * (long)cap;
  int32_t *out = idx + u * (long)keep;
  const int n = len[u];
  if (n < 0 || n > cap) {
    if (threadIdx.x == 0) flag_bad(status);
    return;
  }
  if (threadIdx.x == 0) {
    len_out[u] = min(n, keep);
    sh_sinks = 0;
  }
  if (n <= keep) {
    for (int m = threadIdx.x; m < keep; m += NTS) out[m] = m < n ? m : -1;
    return;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int found = 0;
  for (int i = threadIdx.x; i < min(sink, n - recent); i += NTS) found += pos_all[u * (long)cap + i] < sink;
  for (int o = 16; o; o >>= 1) found += __shfl_xor_sync(0xFFFFFFFFu, found, o);
  if (lane == 0 && found) atomicAdd(&sh_sinks, found);
  __syncthreads();
  const int S = sh_sinks;
  const int nc = n - recent - S;          // candidates: slots S .. S + nc - 1
  const int nh = keep - recent - S;       // of which so many stay (1 <= nh < nc)
  const float *a = acc + S;
  uint32_t prefix = 0, mask = 0;
  int need = nh;
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int e = threadIdx.x; e < NWS * 256; e += NTS) (&hist[0][0])[e] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < nc; i += NTS) {
      const uint32_t key = order_key(a[i]);
      if ((key & mask) == prefix) atomicAdd(&hist[warp][(key >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (threadIdx.x < 256) {
      uint32_t t = 0;
      for (int w = 0; w < NWS; ++w) t += hist[w][threadIdx.x];
      tot[threadIdx.x] = t;
    }
    __syncthreads();
    if (warp == 0) {
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += tot[255 - 8 * lane - i];
      uint32_t incl = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += y;
      }
      uint32_t above = incl - mine;
      if (above < (uint32_t)need && (uint32_t)need <= incl) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const int dgt = 255 - 8 * lane - i;
          const uint32_t c = tot[dgt];
          if ((uint32_t)need <= above + c) {
            sh_prefix = prefix | ((uint32_t)dgt << shift);
            sh_need = need - (int)above;
            sh_equal = (int)c;
            break;
          }
          above += c;
        }
      }
    }
    __syncthreads();
    prefix = sh_prefix;
    need = sh_need;
    mask |= 255u << shift;
    __syncthreads();
  }
  const int skip = sh_equal - need;  // so many of the equal slots go, the first ones
  for (int m = threadIdx.x; m < S; m += NTS) out[m] = m;
  int carry_eq = 0, carry_keep = 0;
  for (int base = 0; base < nc; base += NTS) {
    const int i = base + threadIdx.x;
    const uint32_t key = i < nc ? order_key(a[i]) : 0u;
    const int gt = i < nc && key > prefix;
    const int eq = i < nc && key == prefix;
    int eq_total, keep_total;
    const int eq_rank = carry_eq + block_exclusive_scan<NTS>(eq, warp_sums, &eq_total);
    const int stay = gt || (eq && eq_rank >= skip);
    const int slot = carry_keep + block_exclusive_scan<NTS>(stay, warp_sums, &keep_total);
    if (stay && slot < nh) out[S + slot] = S + i;
    carry_eq += eq_total;
    carry_keep += keep_total;
  }
  for (int m = threadIdx.x; m < recent; m += NTS) out[S + nh + m] = S + nc + m;
}

// The same selection for units whose order keys fit on chip: a cluster of CTAs per unit,
// each with a slice of the slots in shared memory, so that acc is read once.  A protected
// slot gets the largest key (that of no acc: a NaN with it is held to the one below): the
// `keep` largest of all slots stay.
// Four passes find the threshold's key; of the slots that equal it the last ones stay, which
// takes no more passes but a count of the equal slots in front of each CTA, warp and slot.
constexpr int NTC = 512;
constexpr int NWC = NTC / 32;
constexpr int kHistCopies = 4;
constexpr int kMaxCl = 8;
constexpr int kSliceMax = 49152;  // keys per CTA at most (192 KB)

__global__ void __launch_bounds__(NTC) evict_select_resident_kernel(
    const float *__restrict__ acc_all, const int32_t *__restrict__ pos_all, const int32_t *__restrict__ len, int cap,
    int keep, int recent, int sink, int32_t *__restrict__ idx, int32_t *__restrict__ len_out, int *status) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ RadixScratch<NTC, kHistCopies> rx;
  __shared__ int2 wcnt[NWC], cnt[kMaxCl];  // slots above the threshold, slots equal to it
  pdl_wait();
  pdl_launch();
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  const int CL = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const long u = blockIdx.x / CL;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = len[u];
  int32_t *out = idx + u * (long)keep;
  if (n < 0 || n > cap) {
    if (rank == 0 && threadIdx.x == 0) flag_bad(status);
    return;
  }
  if (rank == 0 && threadIdx.x == 0) len_out[u] = min(n, keep);
  if (n <= keep) {
    for (int m = rank * NTC + threadIdx.x; m < keep; m += CL * NTC) out[m] = m < n ? m : -1;
    return;
  }
  const int per = ((n + CL - 1) / CL + 31) & ~31;  // at most the host's slice
  const int lo = min(n, rank * per), m = min(n, lo + per) - lo;
  for (int e = threadIdx.x; e < kHistCopies * 256; e += NTC) (&rx.hist[0][0])[e] = 0u;
  __syncthreads();
  const float *acc = acc_all + u * (long)cap + lo;
  const int32_t *pos = pos_all + u * (long)cap + lo;
  // The first digit (sign and seven bits of the exponent) is counted here.  Neighbouring
  // accumulators mostly share it: a thread adds up runs before it touches the histogram,
  // where equal bins would queue.
  uint32_t *const hist = rx.hist[warp & (kHistCopies - 1)];
  uint32_t bin = 0, count = 0;
  auto put = [&](int i, float a) {
    const bool safe = lo + i >= n - recent || (lo + i < sink && pos[i] < sink);
    const uint32_t k = safe ? 0xFFFFFFFFu : min(order_key(a), 0xFFFFFFFEu);
    keys[i] = k;
    if (k >> 24 != bin) {
      if (count) atomicAdd(hist + bin, count);
      bin = k >> 24;
      count = 0;
    }
    ++count;
  };
  if ((reinterpret_cast<uintptr_t>(acc) & 15) == 0) {
    const float4 *a4 = reinterpret_cast<const float4 *>(acc);
    for (int base = threadIdx.x; base < m >> 2; base += 4 * NTC) {
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (base + k * NTC < m >> 2) v[k] = __ldg(a4 + base + k * NTC);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = 4 * (base + k * NTC);
        if (i < (m & ~3)) {
          put(i, v[k].x);
          put(i + 1, v[k].y);
          put(i + 2, v[k].z);
          put(i + 3, v[k].w);
        }
      }
    }
    for (int i = (m & ~3) + threadIdx.x; i < m; i += NTC) put(i, acc[i]);
  } else {
    for (int i = threadIdx.x; i < m; i += NTC) put(i, acc[i]);
  }
  if (count) atomicAdd(hist + bin, count);
  cl.sync();  // slices loaded, and every CTA of the cluster is running
  const uint32_t thr = (uint32_t)(radix_select_ge<NTC, true>(
                                      rx, keep,
                                      [&](auto &&f) {
                                        for (int i = threadIdx.x; i < m; i += NTC) f((uint64_t)keys[i] << 32);
                                      },
                                      [&](auto &&f) {
                                        const uint4 *k4 = reinterpret_cast<const uint4 *>(keys);
                                        for (int i = threadIdx.x; i < m >> 2; i += NTC) {
                                          const uint4 q = k4[i];
                                          f(q.x);
                                          f(q.y);
                                          f(q.z);
                                          f(q.w);
                                        }
                                        for (int i = (m & ~3) + threadIdx.x; i < m; i += NTC) f(keys[i]);
                                      },
                                      true, 4) >>
                                  32);
  // all keys at or above thr stay, or of those that equal it only some
  const bool whole = rx.sh_done != 0;
  const int wanted = rx.sh_need;
  // counts per warp range, per CTA, then what stands in front of the CTA
  const int wper = ((m + NWC - 1) / NWC + 31) & ~31;
  const int wlo = min(m, warp * wper), whi = min(m, wlo + wper);
  int2 c = make_int2(0, 0);
  for (int i = wlo + lane; i < whi; i += 32) {
    c.x += whole ? keys[i] >= thr : keys[i] > thr;
    c.y += !whole && keys[i] == thr;
  }
  c.x = __reduce_add_sync(0xFFFFFFFFu, c.x);
  c.y = __reduce_add_sync(0xFFFFFFFFu, c.y);
  if (lane == 0) wcnt[warp] = c;
  __syncthreads();
  if ((int)threadIdx.x < CL) {
    int2 tot = make_int2(0, 0);
    for (int w = 0; w < NWC; ++w) {
      tot.x += wcnt[w].x;
      tot.y += wcnt[w].y;
    }
    cl.map_shared_rank(&cnt[0], threadIdx.x)[rank] = tot;
  }
  cl.sync();  // the last remote access is above
  int above = 0, equal = 0, all_equal = 0;
  for (int r = 0; r < CL; ++r) {
    if (r < rank) above += cnt[r].x, equal += cnt[r].y;
    all_equal += cnt[r].y;
  }
  for (int w = 0; w < warp; ++w) above += wcnt[w].x, equal += wcnt[w].y;
  const int skip = whole ? 0 : all_equal - wanted;  // so many of the equal slots go, the first ones
  const unsigned before = (1u << lane) - 1u;
  for (int i0 = wlo; i0 < whi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < whi ? keys[i] : 0u;
    const bool gt = i < whi && (whole ? k >= thr : k > thr), eq = i < whi && !whole && k == thr;
    const unsigned mg = __ballot_sync(0xFFFFFFFFu, gt), me = __ballot_sync(0xFFFFFFFFu, eq);
    const int rank_eq = equal + __popc(me & before);
    const int at = above + __popc(mg & before) + max(0, rank_eq - skip);
    if ((gt || (eq && rank_eq >= skip)) && at < keep) out[at] = lo + i;
    above += __popc(mg);
    equal += __popc(me);
  }
}

// CTAs per unit and slots per CTA (0: the unit does not fit).  About one CTA an SM over
// all units (more spend longer at the cluster's barriers), slices of at least 2048 slots.
void select_plan(long units, int cap, int *CL, int *slice) {
  const long want = (kNumSmsHint + units - 1) / units, most = (cap + 2047) / 2048;
  long cl = want < most ? want : most;
  const long least = (cap + kSliceMax - 33) / (kSliceMax - 32);
  if (cl < least) cl = least;
  if (cl > kMaxCl) cl = kMaxCl;
  if (cl < 1) cl = 1;
  *CL = (int)cl;
  *slice = least > kMaxCl ? 0 : (int)(((cap + cl - 1) / cl + 31) & ~31L);
}

int log2_of(int n) { return n == 128 ? 7 : n == 64 ? 6 : 5; }  // a head dim or a block

template <typename T, int FMT>
int launch_move(const BlockArgs &A, long units, cudaStream_t st) {
  // runs of blocks: about four CTAs an SM, several times over, at most kRunRows rows
  const long want = (12L * kNumSmsHint + units - 1) / units;
  int run = (int)((A.nblk + want - 1) / want);
  run = run < 1 ? 1 : run > (kRunRows >> A.b_log2) ? (kRunRows >> A.b_log2) : run;
  const int runs = (A.nblk + run - 1) / run;
  if (units * runs > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  const int bytes = A.out.block * A.out.d;
  auto go = [&](auto *fn, int threads, int stages) {
    const size_t smem = (size_t)stages * 2 * bytes;
    if (ensure_smem((const void *)fn, smem)) return cuda_failure(cudaErrorInvalidValue, "eviction: shared memory");
    const cudaError_t e = launch_pdl(fn, (unsigned)(units * runs), threads, smem, st, A, runs, run);
    if (e != cudaSuccess) return cuda_failure(e, "eviction: moving the slots");
    return launch_status();
  };
  if (bytes <= 2048) return go(evict_move_kernel<T, FMT, 128, 1, 4>, 128, 4);
  if (bytes <= 4096) return go(evict_move_kernel<T, FMT, 256, 1, 4>, 256, 4);
  if (bytes <= 8192) return go(evict_move_kernel<T, FMT, 256, 2, 3>, 256, 3);
  return go(evict_move_kernel<T, FMT, 512, 2, 3>, 512, 3);
}

}  // namespace

int launch_compact_q8(const void *K, const void *V, const float *s, const int32_t *idx, int T, int k,
                      const kv_q8_cache &out, int *status, cudaStream_t st) {
  BlockArgs A{};
  A.src[0] = K;
  A.src[1] = V;
  A.s = s;
  A.idx = idx;
  A.T = T;
  A.k = k;
  A.out = out;
  A.from = out;
  A.d_log2 = log2_of(out.d);
  A.b_log2 = log2_of(out.block);
  A.nblk = (k + out.block - 1) / out.block;
  A.status = status;
  const long ctas = (long)out.B * out.Hkv * A.nblk;
  if (ctas > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  const int nt = out.block * out.d / 16 / kCompactPieces;  // 64 .. 512 (d is 64 or 128)
  const bool bf = out.dtype == KV_BF16, s8 = out.format == KV_Q8_S8;
  auto *fn = bf && s8 ? compact_block_kernel<__nv_bfloat16, KV_Q8_S8>
             : bf     ? compact_block_kernel<__nv_bfloat16, KV_Q8_E4M3>
             : s8     ? compact_block_kernel<float, KV_Q8_S8>
                      : compact_block_kernel<float, KV_Q8_E4M3>;
  const cudaError_t e = launch_pdl(fn, (unsigned)ctas, nt, 0, st, A);
  if (e != cudaSuccess) return cuda_failure(e, "8-bit compaction");
  return launch_status();
}

int launch_evict_q8(const kv_q8_cache &from, int keep, int recent, int sink, int32_t *idx,
                    const kv_q8_cache &out, int *status, cudaStream_t st) {
  const long units = (long)from.B * from.Hkv;
  BlockArgs A{};
  A.idx = idx;
  A.T = from.cap;
  A.k = keep;
  A.from = from;
  A.out = out;
  A.d_log2 = log2_of(out.d);
  A.b_log2 = log2_of(out.block);
  A.nblk = (min(keep, from.cap) + out.block - 1) / out.block;
  A.status = status;
  int CL, slice;
  select_plan(units, from.cap, &CL, &slice);
  if (units * A.nblk > 0x7FFFFFFFL || units * CL > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;  // before the first launch
  if (slice > 0) {
    const size_t smem = (size_t)slice * 4;
    if (ensure_smem((const void *)evict_select_resident_kernel, smem))
      return cuda_failure(cudaErrorInvalidValue, "eviction: shared memory");
    const cudaError_t e = launch_pdl_cluster(evict_select_resident_kernel, (unsigned)(units * CL), NTC, smem, st, CL,
                                             from.acc, from.pos, from.len, from.cap, keep, recent, sink, idx, out.len,
                                             status);
    if (e != cudaSuccess) return cuda_failure(e, "eviction: selection");
  } else {
    evict_select_kernel<<<(unsigned)units, NTS, 0, st>>>(from.acc, from.pos, from.len, from.cap, keep, recent, sink,
                                                         idx, out.len, status);
  }
  const int rc = launch_status();
  if (rc != KV_OK) return rc;
  if (out.dtype == KV_BF16)
    return out.format == KV_Q8_S8 ? launch_move<__nv_bfloat16, KV_Q8_S8>(A, units, st)
                                  : launch_move<__nv_bfloat16, KV_Q8_E4M3>(A, units, st);
  return out.format == KV_Q8_S8 ? launch_move<float, KV_Q8_S8>(A, units, st)
                                : launch_move<float, KV_Q8_E4M3>(A, units, st);
}

}  // namespace kvc

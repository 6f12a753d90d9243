// q8_cache.cu -- writing the 8-bit slot cache: gather-compaction of a prompt's
// kept rows into codes, and eviction of the slots with the least accumulated
// attention (H2O page, 两套代码 and 贪心驱逐算法; formulas of the codes in
// q8_common.cuh).
//
//   compact  destination slot m takes prompt row idx[m];
//   evict    destination slot m takes the source cache's slot idx[m], idx chosen
//            here: the leading slots with pos < sink and the last `recent` slots
//            stay, and of the others the (acc, slot)-largest, in slot order.
// Both then run the same block kernel: one CTA per (unit, destination block, K or
// V), one thread per 16 elements of the block, so a block is read once, its
// largest magnitude found across the CTA and its codes written from registers.
// The rows of the unfinished block are copied (evict: decoded where they were
// codes, rounded to the cache's dtype, half a step at most).
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
  int d_log2, nblk;      // blocks per unit that may be written (the unfinished one included)
  int *status;
};

template <typename T, int FMT, bool EVICT>
__global__ void __launch_bounds__(1024) q8_block_kernel(const __grid_constant__ BlockArgs A) {
  __shared__ float red[32];
  __shared__ int src[128];
  const int block = A.out.block, d = A.out.d;
  const long u = blockIdx.x / (2 * A.nblk);
  const int rest = blockIdx.x % (2 * A.nblk);
  const int b = rest >> 1, kv = rest & 1;
  int n_new = A.k, n_src = A.T;
  if constexpr (EVICT) {
    n_src = A.from.len[u];
    if (n_src < 0 || n_src > A.from.cap) return;  // reported by the selection
    n_new = min(n_src, A.k);
  }
  const int m0 = b * block;
  if (m0 >= n_new) return;
  const int rows = min(block, n_new - m0);
  // the rows' sources, and what moves beside K and V
  if ((int)threadIdx.x < rows) {
    const int m = m0 + threadIdx.x;
    int j = A.idx ? A.idx[u * (long)A.k + m] : m;
    const bool ok = j >= 0 && j < n_src;
    src[threadIdx.x] = ok ? j : -1;
    if (kv == 0) {
      const long at = u * (long)A.out.cap + m;
      if constexpr (EVICT) {
        const long f = u * (long)A.from.cap + j;
        A.out.pos[at] = A.from.pos[f];
        A.out.acc[at] = A.from.acc[f];
      } else {
        if (!ok) flag_bad(A.status);
        A.out.pos[at] = ok ? j : -1;
        if (A.out.acc) A.out.acc[at] = ok && A.s ? A.s[u * (long)A.T + j] : 0.f;
        if (m == 0) A.out.len[u] = n_new;
      }
    }
  }
  __syncthreads();
  const int r = (int)(threadIdx.x << 4) >> A.d_log2;       // row of the block
  const int e = (int)(threadIdx.x << 4) & (d - 1);         // first of the thread's 16 elements
  const int j = r < rows ? src[r] : -1;
  float x[16];
  if constexpr (EVICT) {
    const int nf = n_src / block * block;  // slots held as codes
    const uint8_t *codes = static_cast<const uint8_t *>(kv ? A.from.V : A.from.K);
    const float *sc = (kv ? A.from.Vs : A.from.Ks) + u * (long)(A.from.cap / block);
    if (rows == block && src[block - 1] < nf && src[0] % block == 0 && src[block - 1] - src[0] == block - 1) {
      // a whole block moves: its codes and its scale as they are
      const long to = (u * (long)A.out.cap + m0 + r) * d + e;
      const long f = (u * (long)A.from.cap + j) * d + e;
      *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(kv ? A.out.V : A.out.K) + to) =
          __ldg(reinterpret_cast<const uint4 *>(codes + f));
      if (threadIdx.x == 0)
        (kv ? A.out.Vs : A.out.Ks)[u * (long)(A.out.cap / block) + b] = sc[src[0] / block];
      return;
    }
    if (j >= nf) {
      load16(static_cast<const T *>(kv ? A.from.Vt : A.from.Kt) + (u * (long)block + (j - nf)) * d + e, x);
    } else if (j >= 0) {
      const uint4 w = __ldg(reinterpret_cast<const uint4 *>(codes + (u * (long)A.from.cap + j) * d + e));
      const float a = __ldg(sc + j / block);
      Q8<FMT>::unpack4(w.x, x);
      Q8<FMT>::unpack4(w.y, x + 4);
      Q8<FMT>::unpack4(w.z, x + 8);
      Q8<FMT>::unpack4(w.w, x + 12);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], a);
    }
  } else {
    if (j >= 0) load16(static_cast<const T *>(A.src[kv]) + (u * (long)A.T + j) * d + e, x);
  }
  if (j < 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
  }
  if (rows < block) {  // the unfinished block keeps its rows
    if (r < rows) store16(static_cast<T *>(kv ? A.out.Vt : A.out.Kt) + (u * (long)block + r) * d + e, x);
    return;
  }
  const float a = q8_scale<FMT>(block_max(max_abs16(x), red));
  const float inv = __fdiv_rn(1.f, a);
  const long to = (u * (long)A.out.cap + m0 + r) * d + e;
  *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(kv ? A.out.V : A.out.K) + to) = q8_pack16<FMT>(x, inv);
  if (threadIdx.x == 0) (kv ? A.out.Vs : A.out.Ks)[u * (long)(A.out.cap / block) + b] = a;
}

// ---- which slots stay ------------------------------------------------------------
// One CTA per unit: exact radix select over the candidates' order-preserving keys
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

int log2_of(int d) { return d == 128 ? 7 : 6; }

template <bool EVICT>
int launch_blocks(const BlockArgs &A, long units, cudaStream_t st) {
  const long ctas = units * 2 * A.nblk;
  if (ctas > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  const int nt = A.out.block * A.out.d / 16;
  const unsigned grid = (unsigned)ctas;
  const bool bf = A.out.dtype == KV_BF16, s8 = A.out.format == KV_Q8_S8;
  if (bf && s8) q8_block_kernel<__nv_bfloat16, KV_Q8_S8, EVICT><<<grid, nt, 0, st>>>(A);
  else if (bf) q8_block_kernel<__nv_bfloat16, KV_Q8_E4M3, EVICT><<<grid, nt, 0, st>>>(A);
  else if (s8) q8_block_kernel<float, KV_Q8_S8, EVICT><<<grid, nt, 0, st>>>(A);
  else q8_block_kernel<float, KV_Q8_E4M3, EVICT><<<grid, nt, 0, st>>>(A);
  return launch_status();
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
  A.nblk = (k + out.block - 1) / out.block;
  A.status = status;
  return launch_blocks<false>(A, (long)out.B * out.Hkv, st);
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
  A.nblk = (min(keep, from.cap) + out.block - 1) / out.block;
  A.status = status;
  if (units * 2 * A.nblk > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  evict_select_kernel<<<(unsigned)units, NTS, 0, st>>>(from.acc, from.pos, from.len, from.cap, keep, recent, sink,
                                                       idx, out.len, status);
  const int rc = launch_status();
  if (rc != KV_OK) return rc;
  return launch_blocks<true>(A, units, st);
}

}  // namespace kvc

// attn_prompt_tc.cu -- prompt attention for bf16 on the tensor cores (tcgen05, TMA).
//
// One CTA takes two query tiles of 128 rows against the same keys: two query heads of
// one KV head at the same rows (G even), or the 256 rows of one head (G odd).  Per
// tile i and key tile j of 128 keys:
//     S = Q_i K_j^T (TMEM, fp32); P = 2^(c S - m) rounded to bf16 (its rounding is a
//     relative half step 2^-9 of each weight, which averages out in O; the row sums z
//     take P before the rounding); O_i += P V_j (TMEM, fp32), P read from TMEM.
// The reference m of a row moves only when a logit passes it by more than kLazy (log2
// units; weights stay below 2^kLazy): only then is O rescaled, by the softmax warps
// themselves, which know that the product before is complete because the commit that
// announces S_j covers it.
//
// Roles: warpgroup i (of two) is tile i's softmax, one thread a row; warp 8 issues the
// products, warp 9 the TMA loads.  The order P_0 V_j, Q_0 K_{j+1}, P_1 V_j,
// Q_1 K_{j+1} keeps the tensor pipe busy with one tile while the other's softmax
// runs; warp 10 clears V rows behind a sequence's end.  TMEM (512 columns): S_0, S_1, O_0, O_1; P_i lies over S_i's first 64 columns,
// whose logits are in registers by then (products execute in the order of issue, so
// Q_i K_{j+1} overwrites P_i only after P_i V_j has read it).
// K and V tiles share one ring of stages in the order K_0 V_0 K_1 V_1 ...  V is used
// as it lies in memory (the keys along k, d along n: a transposed operand).
// Keys behind a sequence's end belong to another sequence or to nobody: S there is
// replaced by -inf and the V rows are cleared in shared memory, so NaN in them
// cannot reach the result.
#include <cmath>

#include "attn_common.cuh"
#include "tc_common.cuh"

namespace kvc {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int NT = 384;
constexpr float kLazy = 8.f;
constexpr long long kWaitBudget = 4000000000LL;  // clock cycles (~2 s) before a wait gives up
constexpr long long kDrainBudget = 200000000LL;

template <int D>
struct Geo {
  static constexpr int NKB = D / 64;                    // 128-byte column blocks of a row
  static constexpr int SUB = 128 * 128;                 // one column block of a tile
  static constexpr int TILE = NKB * SUB;                // 128 rows
  static constexpr int STAGES = D == 128 ? 5 : 8;
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = 2 * TILE;
  static constexpr int BAR_OFF = KV_OFF + STAGES * TILE;
  static constexpr int SMEM_NEED = 1024 + BAR_OFF + 512;
  // more than half an SM's shared memory: a CTA takes all of TMEM, so one per SM
  static constexpr int SMEM = SMEM_NEED > 116 * 1024 ? SMEM_NEED : 116 * 1024;
};

struct Bars {
  uint64_t *qfull, *full, *empty, *sfull, *pfull, *ofull, *drain, *vreq, *vfix;
};

struct TcArgs {
  AttnArgs A;
  __nv_bfloat16 *O;
  int pair_rows;  // 1: the two tiles are the halves of 256 rows; 0: two heads
};

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
      "%5}], [%6];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(tc::smem_u32(bar))
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a));
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// V tile as the second operand of P V: n (d) is contiguous, 64 elements per 128-byte
// row, one row per key; 1024 bytes per group of 8 keys, `SUB` bytes to the next 64
// elements of d.
__device__ __forceinline__ uint64_t vdesc_sw128(uint32_t saddr, uint32_t sub) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(sub >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
constexpr uint32_t kTransposeB = 1u << 16;

// The work of one CTA.
struct Work {
  AttnTile t;
  int h[2], r0[2], rows[2], n[2];  // per tile: head, first row, rows, key tiles
  int nmax;
};

__device__ __forceinline__ Work make_work(const TcArgs &T, const AttnTile &t, int hi) {
  Work w;
  w.t = t;
  w.nmax = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w.h[i] = T.pair_rows ? hi : 2 * hi + i;
    w.r0[i] = t.r0 + (T.pair_rows ? i * BM : 0);
    w.rows[i] = max(0, min(BM, t.nq - w.r0[i]));
    // the tile's last row sees keys up to r0 + rows - 1 + nk - nq
    const int kend = w.rows[i] ? min(t.nk, max(0, w.r0[i] + w.rows[i] + t.nk - t.nq)) : 0;
    w.n[i] = (kend + BN - 1) / BN;
    w.nmax = max(w.nmax, w.n[i]);
  }
  return w;
}

template <int D>
__global__ void __launch_bounds__(NT, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TcArgs T) {
  using Gm = Geo<D>;
  constexpr int ST = Gm::STAGES;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char *sQ = sm + Gm::Q_OFF, *sKV = sm + Gm::KV_OFF;
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Gm::BAR_OFF);
  const Bars B{bars, bars + 1, bars + 1 + ST, bars + 1 + 2 * ST, bars + 3 + 2 * ST, bars + 5 + 2 * ST,
               bars + 7 + 2 * ST, bars + 8 + 2 * ST, bars + 9 + 2 * ST};
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + Gm::BAR_OFF + 8 * (10 + 2 * ST));
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  __shared__ AttnTile stile;
  const AttnShape &S = T.A.S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = T.pair_rows ? S.Hq : S.Hq / 2;
  const int index = blockIdx.x / groups;

  if (warp == 9) {
    const AttnTile t = attn_locate(S, index, T.pair_rows ? 2 * BM : BM, blockIdx.x == 0, T.A.status);
    if (lane == 0) stile = t;
  }
  if (threadIdx.x == 0) {
    tc::mbar_init(B.qfull, 1);
    tc::mbar_init(B.drain, 1);
    tc::mbar_init(B.vreq, 1);
    tc::mbar_init(B.vfix, 1);
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(B.full + i, 1);
      tc::mbar_init(B.empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(B.sfull + i, 1);
      tc::mbar_init(B.pfull + i, 4);
      tc::mbar_init(B.ofull + i, 1);
    }
    *abort_flag = 0;
    tc::mbar_fence_init();
  }
  if (warp == 8) tc::tmem_alloc(tmem_slot, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const AttnTile tile = stile;
  auto give_up = [&]() {
    *abort_flag = 1;
    if (T.A.status) atomicExch(T.A.status, (int)KV_ERR_TIMEOUT);
  };

  if (tile.nq > 0) {
    const Work w = make_work(T, tile, blockIdx.x % groups);
    // registers: 256 x 216 + 128 x 72 = the 384 x 168 of the launch
    if (warp >= 8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 9) {
      if (tc::elect_one() && w.nmax > 0) {
        // ---- loads ----
        const int hk = w.h[0] / (S.Hq / S.Hkv);
        tc::mbar_arrive_expect_tx(B.qfull, 2 * Gm::TILE);
        for (int i = 0; i < 2; ++i)
          for (int c = 0; c < Gm::NKB; ++c)
            tma_load_4d(sQ + i * Gm::TILE + c * Gm::SUB, &tmQ, c * 64, tile.q0 + w.r0[i], w.h[i], tile.b, B.qfull);
        const int total = 2 * w.nmax;  // K_0 V_0 K_1 V_1 ...
        int x = 0;
        for (; x < total; ++x) {
          const int st = x % ST;
          if (!tc::mbar_wait(B.empty + st, ((x / ST) & 1) ^ 1, kWaitBudget, abort_flag)) {
            give_up();
            break;
          }
          tc::mbar_arrive_expect_tx(B.full + st, Gm::TILE);
          for (int c = 0; c < Gm::NKB; ++c)
            tma_load_4d(sKV + st * Gm::TILE + c * Gm::SUB, (x & 1) ? &tmV : &tmK, c * 64,
                        tile.k0 + (x >> 1) * BN, hk, tile.b, B.full + st);
        }
        if (*abort_flag) {  // copies in flight land before the CTA may exit
          tc::mbar_wait(B.qfull, 0, kDrainBudget, nullptr);
          for (int k = 1; k <= ST && x - k >= 0; ++k)
            tc::mbar_wait(B.full + (x - k) % ST, ((x - k) / ST) & 1, kDrainBudget, nullptr);
        }
      }
    } else if (warp == 8) {
      // ---- products (one elected thread: the operands then stay in uniform registers) ----
      if (tc::elect_one() && w.nmax > 0) {
        const uint64_t qd = tc::sdesc_sw128(tc::smem_u32(sQ));
        const uint64_t kd0 = tc::sdesc_sw128(tc::smem_u32(sKV));
        const uint64_t vd0 = vdesc_sw128(tc::smem_u32(sKV), Gm::SUB);
        const uint32_t id_s = tc::idesc_bf16(BM, BN), id_o = tc::idesc_bf16(BM, D) | kTransposeB;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t ph) {
          if (!tc::mbar_wait(bar, ph, kWaitBudget, abort_flag)) {
            ok = false;
            give_up();
          }
          tc::fence_after_sync();
          return ok;
        };
        auto qk = [&](int i, int st) {  // S_i = Q_i K^T
          const uint64_t q = qd + (uint64_t)((i * Gm::TILE) >> 4), k = kd0 + (uint64_t)((st * Gm::TILE) >> 4);
          const uint32_t dst = tmem + i * 128;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t o = (uint64_t)(((kk / 4) * Gm::SUB + (kk % 4) * 32) >> 4);
            tc::umma_bf16(dst, q + o, k + o, id_s, kk > 0);
          }
        };
        if (wait(B.qfull, 0) && wait(B.full, 0)) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (w.n[i] > 0) {
              qk(i, 0);
              tc::umma_commit(B.sfull + i);
            }
          tc::umma_commit(B.empty);
          for (int j = 0; j < w.nmax && ok; ++j) {
            const int xv = 2 * j + 1, xk = 2 * j + 2;
            const int sv = xv % ST, sk = xk % ST;
            if (!wait(B.full + sv, (xv / ST) & 1)) break;
            if (tile.nk - j * BN < BN) {  // the sequence ends inside this tile, its last
              tc::mbar_arrive(B.vreq);
              if (!wait(B.vfix, 0)) break;
            }
            const uint64_t vd = vd0 + (uint64_t)((sv * Gm::TILE) >> 4);
            bool have_k = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (j < w.n[i]) {
                if (!wait(B.pfull + i, j & 1)) break;
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                  umma_ts(tmem + 256 + i * 128, tmem + i * 128 + kk * 8, vd + (uint64_t)((kk * 2048) >> 4), id_o,
                          (j > 0) | (kk > 0));
                if (j == w.n[i] - 1) tc::umma_commit(B.ofull + i);
              }
              if (j + 1 < w.n[i]) {
                if (!have_k && !wait(B.full + sk, (xk / ST) & 1)) break;
                have_k = true;
                qk(i, sk);
                tc::umma_commit(B.sfull + i);
              }
            }
            tc::umma_commit(B.empty + sv);
            if (j + 1 < w.nmax) tc::umma_commit(B.empty + sk);
          }
        }
        // every product is complete before TMEM is released
        tc::umma_commit(B.drain);
        tc::mbar_wait(B.drain, 0, kDrainBudget, nullptr);
      }
    } else if (warp == 10) {
      // ---- rows of V behind the sequence's end, in the one tile that it ends in ----
      const int j = w.nmax - 1, left = tile.nk - j * BN;
      if (w.nmax > 0 && left < BN) {
        const int sv = (2 * j + 1) % ST;
        if (tc::mbar_wait(B.vreq, 0, kWaitBudget, abort_flag)) {  // the tile has landed
          for (int e = lane; e < (BN - left) * 8 * Gm::NKB; e += 32) {
            const int cb = e / ((BN - left) * 8), r = e % ((BN - left) * 8);
            *reinterpret_cast<uint4 *>(sKV + sv * Gm::TILE + cb * Gm::SUB + left * 128 + r * 16) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(B.vfix);
        }
      }
    }
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      // ---- softmax of tile i: one thread a row ----
      const int i = warp >> 2;
      const int row = (warp & 3) * 32 + lane;
      const uint32_t ts = tmem + i * 128 + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t to = tmem + 256 + i * 128 + ((uint32_t)((warp & 3) * 32) << 16);
      const float c = T.A.c_log2;
      const int n = w.n[i];
      const int first = w.r0[i] + tile.nk - tile.nq;         // last key that the tile's first row sees
      const int mine = min(first + row, tile.nk - 1);        // ... that this row sees
      float m = -INFINITY;                                   // reference, log2 units
      float2 z2 = make_float2(0.f, 0.f);
      bool ok = true;
      for (int j = 0; j < n; ++j) {
        if (!tc::mbar_wait(B.sfull + i, j & 1, kWaitBudget, abort_flag)) {
          ok = false;
          give_up();
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc::fence_after_sync();
        uint32_t r[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(ts + q * 32, r + q * 32);
        tc::tmem_ld_wait();
        const int j0 = j * BN;
        if (j0 + BN - 1 > first) {  // some row sees only part of the tile
          const int lim = mine - j0;
#pragma unroll
          for (int x = 0; x < 128; ++x) r[x] = x <= lim ? r[x] : 0xFF800000u;
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) mx[q] = fmaxf(__uint_as_float(r[q]), __uint_as_float(r[q + 4]));
#pragma unroll
        for (int x = 8; x < 128; x += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(r[x + q]), __uint_as_float(r[x + q + 4])));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        const bool over = top > m + kLazy;
        if (__any_sync(0xFFFFFFFFu, over)) {
          const float f = over ? tc::ex2(m - top) : 1.f;
          if (over) m = top;
          z2.x *= f;
          z2.y *= f;
          if (j > 0) {
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld32(to + q * 32, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
              tmem_st32(to + q * 32, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : -m;  // a row that has seen no key yet
        const float2 c2 = make_float2(c, c), b2 = make_float2(base, base);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t p[32];
          float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const int s = hf * 64 + 2 * x;
            const float2 u = __ffma2_rn(make_float2(__uint_as_float(r[s]), __uint_as_float(r[s + 1])), c2, b2);
            const float2 v = __ffma2_rn(make_float2(__uint_as_float(r[s + 2]), __uint_as_float(r[s + 3])), c2, b2);
            const float2 eu = make_float2(tc::ex2(u.x), tc::ex2(u.y)), ev = make_float2(tc::ex2(v.x), tc::ex2(v.y));
            a0 = __fadd2_rn(a0, eu);
            a1 = __fadd2_rn(a1, ev);
            const __nv_bfloat162 h0 = __floats2bfloat162_rn(eu.x, eu.y), h1 = __floats2bfloat162_rn(ev.x, ev.y);
            p[x] = *reinterpret_cast<const uint32_t *>(&h0);
            p[x + 1] = *reinterpret_cast<const uint32_t *>(&h1);
          }
          z2 = __fadd2_rn(z2, __fadd2_rn(a0, a1));
          tmem_st32(ts + hf * 32, p);
        }
        tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(B.pfull + i);
      }
      // ---- O / z ----
      if (n > 0 && ok) {
        if (!tc::mbar_wait(B.ofull + i, 0, kWaitBudget, abort_flag)) {
          ok = false;
          give_up();
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc::fence_after_sync();
      }
      if (ok && w.rows[i] > 0) {
        const float z = z2.x + z2.y;
        const float inv = z > 0.f ? 1.f / z : 0.f;
        const long long at = (long long)tile.q0 + w.r0[i] + row;
        __nv_bfloat16 *dst = T.O + tile.b * S.o[0] + w.h[i] * S.o[1] + at * S.o[2];
        const bool live = row < w.rows[i];
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(to + q * 32, o);
            tc::tmem_ld_wait();
          }
          uint32_t p[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(z > 0.f ? __uint_as_float(o[2 * x]) * inv : 0.f,
                                                           z > 0.f ? __uint_as_float(o[2 * x + 1]) * inv : 0.f);
            p[x] = *reinterpret_cast<const uint32_t *>(&v);
          }
          if (live) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              reinterpret_cast<uint4 *>(dst + q * 32)[x] = make_uint4(p[4 * x], p[4 * x + 1], p[4 * x + 2], p[4 * x + 3]);
          }
        }
        if (live && T.A.lse)
          T.A.lse[((long long)tile.b * S.Hq + w.h[i]) * S.Tq + at] =
              z > 0.f ? (m + log2f(z)) * 0.6931471805599453f : -INFINITY;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 8) tc::tmem_dealloc(tmem, 512);
}

// [B][H][T][d] with free strides as a 4-D map of boxes of 64 elements x 128 tokens.
bool encode_heads(CUtensorMap *map, const void *base, int d, long T, long H, long B, const long long *st) {
  tc::EncodeTiledFn fn = tc::encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)H, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)st[2] * 2, (cuuint64_t)st[1] * 2, (cuuint64_t)st[0] * 2};
  cuuint32_t box[4] = {64, BN, 1, 1}, estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
int run(const void *Q, const void *K, const void *V, const TcArgs &T, cudaStream_t st) {
  const AttnShape &S = T.A.S;
  CUtensorMap tmQ, tmK, tmV;
  if (!encode_heads(&tmQ, Q, D, S.Tq, S.Hq, S.B, S.q) || !encode_heads(&tmK, K, D, S.Tk, S.Hkv, S.B, S.k) ||
      !encode_heads(&tmV, V, D, S.Tk, S.Hkv, S.B, S.v))
    return KV_ERR_CUDA;
  const long ctas = attn_tiles(S, T.pair_rows ? 2 * BM : BM) * (T.pair_rows ? S.Hq : S.Hq / 2);
  if (ctas > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  if (ensure_smem((const void *)attn_tc_kernel<D>, Geo<D>::SMEM)) return KV_ERR_CUDA;
  attn_tc_kernel<D><<<(unsigned)ctas, NT, Geo<D>::SMEM, st>>>(tmQ, tmK, tmV, T);
  return launch_status();
}

}  // namespace

// scale > 0: the running maximum is taken over the products before they are scaled.
bool attn_tc_eligible(const AttnShape &S, float scale, int dtype) {
  return dtype == KV_BF16 && S.Tk > 0 && scale > 0.f && std::isfinite(scale);
}

int launch_attn_prompt_tc(const void *Q, const void *K, const void *V, const AttnArgs &A, void *O, cudaStream_t st) {
  TcArgs T{A, static_cast<__nv_bfloat16 *>(O), (A.S.Hq / A.S.Hkv) % 2};
  return A.S.d == 128 ? run<128>(Q, K, V, T, st) : run<64>(Q, K, V, T, st);
}

}  // namespace kvc

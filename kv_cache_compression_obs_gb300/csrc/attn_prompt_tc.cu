// attn_prompt_tc.cu -- prompt attention for bf16 on the tensor cores (tcgen05, TMA).
//
// An item of work is two query tiles of 128 rows against the same keys: two query heads
// of one KV head at the same rows (G even), or the 256 rows of one head (G odd).  There
// is one CTA per item; a CTA that is done takes over the next one that has not started
// (cluster launch control), so that its loads and first products run behind the
// writing of the last result.  Per tile i and key tile j of 128 keys:
//     S = Q_i K_j^T (TMEM, fp32); P = 2^(c S - m) rounded to bf16; O_i += P V_j (TMEM,
//     fp32), P read from TMEM.
// P is rounded because the product takes both operands in V's type: each weight is off by at
// most a half step, 2^-8 of it, and O by about 1e-3 of its norm (1.5e-3 for rows behind
// 30000 keys), beside the 1.6e-3 of rounding O itself; hi + lo weights would be half as
// much tensor work again.  The row sums z take P before the rounding: lse is fp32 and needs
// them so, and sums of the rounded weights would change O's error little (in a float64 model
// 1.91e-3 of the norm in all for 1.92e-3 over 2048 tokens, 2.27e-3 for 2.26e-3 behind 11000 keys).
// The reference m of a row moves only when a logit passes it by more than kLazy (log2
// units; weights stay below 2^kLazy): only then is O rescaled, by the softmax warps
// themselves, which know that the product before is complete because the commit that
// announces S_j covers it.
//
// Roles: warpgroup i (of two) is tile i's softmax, one thread a row; warp 8 issues the
// products, warp 9 the TMA loads, warp 11 fetches the items, warp 10 clears V rows behind
// a sequence's end.  The order P_0 V_j, Q_0 K_{j+1}, P_1 V_j, Q_1 K_{j+1} keeps the tensor
// pipe busy with one tile while the other's softmax runs.  TMEM (512 columns): S_0, S_1,
// O_0, O_1; P_i lies over S_i's first 64 columns, whose logits are in registers by then
// (products execute in the order of issue, so Q_i K_{j+1} overwrites P_i only after
// P_i V_j has read it).
// K and V tiles share one ring of stages in the order K_0 V_0 K_1 V_1 ...  V is used
// as it lies in memory (the keys along k, d along n: a transposed operand).
// Keys behind a sequence's end belong to another sequence or to nobody: S there is
// replaced by -inf and the V rows are cleared in shared memory, so NaN in them
// cannot reach the result.
//
// Bound by the tensor pipe and, in long calls, by power: 32768 tokens of 32/8 heads 5.20 to
// 5.42 ms from one GPU to the next, 1690 to 1620 TFLOP/s over the causal half (0.87 to 0.83 of
// the library's burst rate, 0.97 to 0.93 of what it sustains); 8192 tokens 334 us with the tensor
// pipe active 71% of the time; 4096 tokens 99 to 102 us, where an item's end and the next one's start (2 to 3 us) weigh more.  Two threads a
// row (four softmax warpgroups) spilled; O out of TMEM in one go instead of by 32 columns
// changed nothing that could be measured.
#include <cmath>

#include "attn_common.cuh"
#include "attn_tc.cuh"
#include "pdl.cuh"

namespace kvc {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int NT = 384;
constexpr int W_SOFTMAX = 8, W_MMA = 8, W_TMA = 9, W_SCHED = 11;  // warps 0-7: softmax, 10: V's ends
constexpr int kMaxStages = 8;
// The next item is asked for when the loads are this many key tiles from the end of the one at hand
// (a layer of 4096 tokens: 0 tiles 103.3 us, 1 101.8, 2 100.9, 4 100.4, 6 100.8).
constexpr int kClaimTiles = 4;
constexpr int kCtrlBytes = 1024;
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
  static constexpr int CTRL_OFF = KV_OFF + STAGES * TILE;
  static constexpr int SMEM_NEED = CTRL_OFF + kCtrlBytes;
  // more than half an SM's shared memory: a CTA takes all of TMEM, so one per SM
  static constexpr int SMEM = SMEM_NEED > 116 * 1024 ? SMEM_NEED : 116 * 1024;
};

struct TcArgs {
  AttnArgs A;
  __nv_bfloat16 *O;
  int pair_rows;  // 1: the two tiles are the halves of 256 rows; 0: two heads
  int wide;       // O's rows start on 32-byte boundaries
  int whole;      // query tiles (in the order of attn_locate) whose items are not split
  int splits;     // the others' items: each with a share of its key tiles
  // splits > 1, one row for each row of a share (share_row):
  int by_tile;          // 1: [splits][split tiles][Hq][tile rows]; 0: [splits][B][Hq][Tq]
  long long share_rows; // rows of one share of everything that is split
  float *part;          // [splits][share_rows][D] sums of P V, not yet divided
  float2 *stat;         // [splits][share_rows] reference (log2 units) and sum of weights

  // Row `row` of split tile `tile`, token `tok` of batch row b, in the first share.
  __device__ __forceinline__ long long share_row(int b, int h, int tile, int row, long long tok) const {
    return by_tile ? ((long long)tile * A.S.Hq + h) * (pair_rows ? 2 * BM : BM) + row
                   : ((long long)b * A.S.Hq + h) * A.S.Tq + tok;
  }
};

// One item of work.
struct Work {
  AttnTile t;
  int h[2], r0[2], rows[2], n[2];  // per tile: head, first row, rows, key tiles
  int nmax;
  int split, j0;  // share of the key tiles (-1: all) and the first of them
  int tile;       // with a share: index among the split tiles
};

// CTA `block`'s item; executed by one whole warp.
__device__ __forceinline__ Work make_work(const TcArgs &T, int block, bool check_all, AttnScan &scan) {
  const int pairs = T.pair_rows ? T.A.S.Hq : T.A.S.Hq / 2;  // items per query tile, unsplit
  int index = block / pairs, hi = block - index * pairs;
  Work w;
  w.split = -1;
  w.tile = 0;
  if (index >= T.whole) {
    const int b = block - T.whole * pairs;
    index = b / (pairs * T.splits);
    const int part = b - index * pairs * T.splits;
    w.tile = index;
    index += T.whole;
    hi = part / T.splits;
    w.split = part - hi * T.splits;
  }
  const AttnTile t = attn_locate(T.A.S, index, T.pair_rows ? 2 * BM : BM, check_all, T.A.status, scan);
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
  w.j0 = 0;
  if (w.split >= 0) {
    const int per = (w.nmax + T.splits - 1) / T.splits;
    w.j0 = w.split * per;
#pragma unroll
    for (int i = 0; i < 2; ++i) w.n[i] = max(0, min(per, w.n[i] - w.j0));
    w.nmax = max(w.n[0], w.n[1]);
  }
  return w;
}

// Barriers and what else the roles share.
struct Ctrl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t qfull[2], qempty[2], sfull[2], pfull[4], pva[2], ofull[2], oempty[2], wfull[2], wempty[2];
  uint64_t clc, drain, vreq, vfix, want;
  uint4 reply;
  Work work[2];
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(Ctrl) <= kCtrlBytes, "control block");

// Ask the hardware for the index of a CTA of this grid that has not started; the
// 16-byte reply arrives on `bar`.
__device__ __forceinline__ void clc_request(uint4 &reply, uint64_t *bar) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the last reply has been read
  tc::mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          tc::smem_u32(&reply)),
      "r"(tc::smem_u32(bar))
      : "memory");
}
// That CTA's index (it will not start any more), or -1 when none was left.
__device__ __forceinline__ int clc_block(const uint4 &reply) {
  int got, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.s32 %0, 1, 0, p;\n\t"
      "mov.s32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(tc::smem_u32(&reply))
      : "memory");
  return got ? x : -1;
}

template <int D>
__global__ void __launch_bounds__(NT, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TcArgs T) {
  using Gm = Geo<D>;
  constexpr int ST = Gm::STAGES;
  extern __shared__ __align__(1024) unsigned char sm[];  // no static shared memory in front of it
  unsigned char *sQ = sm + Gm::Q_OFF, *sKV = sm + Gm::KV_OFF;
  Ctrl &C = *reinterpret_cast<Ctrl *>(sm + Gm::CTRL_OFF);
  const AttnShape &S = T.A.S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(C.full + i, 1);
      tc::mbar_init(C.empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(C.qfull + i, 1);
      tc::mbar_init(C.qempty + i, 1);
      tc::mbar_init(C.sfull + i, 1);
      tc::mbar_init(C.pfull + i, 4);
      tc::mbar_init(C.pfull + 2 + i, 4);
      tc::mbar_init(C.pva + i, 1);
      tc::mbar_init(C.ofull + i, 1);
      tc::mbar_init(C.oempty + i, 4);
      tc::mbar_init(C.wfull + i, 1);
      tc::mbar_init(C.wempty + i, 11);  // loads, products, V's ends, 8 softmax warps
    }
    tc::mbar_init(&C.clc, 1);
    tc::mbar_init(&C.drain, 1);
    tc::mbar_init(&C.vreq, 1);
    tc::mbar_init(&C.vfix, 1);
    tc::mbar_init(&C.want, 1);
    C.abort_flag = 0;
    tc::mbar_fence_init();
  }
  if (warp == W_MMA) tc::tmem_alloc(&C.tmem, 512);
  if (warp == W_TMA && lane == 0) {
    tc::tma_prefetch_desc(&tmQ);
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
  pdl_wait();
  pdl_launch();
  Work first_work{};
  AttnScan scan{0, 0};
  if (warp == W_SCHED)
    first_work = make_work(T, blockIdx.x, blockIdx.x == 0, scan);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = C.tmem;
  volatile int *abort_flag = &C.abort_flag;
  auto wait = [&](uint64_t *bar, uint32_t ph) -> bool {
    if (tc::mbar_wait(bar, ph & 1, kWaitBudget, abort_flag)) return true;
    *abort_flag = 1;
    if (T.A.status) atomicExch(T.A.status, (int)KV_ERR_TIMEOUT);
    return false;
  };
  // Item k of this CTA (false: there is none).  Every role walks the same items.
  auto have_item = [&](uint32_t k) -> bool { return wait(C.wfull + (k & 1), k >> 1) && C.work[k & 1].t.nq >= 0; };

  if (warp >= W_SOFTMAX) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == W_SCHED) {
      // ---- which work: the CTA's own index, then those of CTAs that have not started,
      // which the hardware hands over on request (in index order: long tiles first) ----
      // A request goes out when the loads of the item at hand are nearly all issued: early enough
      // for the reply and the next item's first loads, late enough that a CTA with a long item does
      // not sit on the next one.
      Work w = first_work;
      int pending = -1;  // the request whose reply was not waited for
      for (uint32_t k = 0;; ++k) {
        const bool ok = wait(C.wempty + (k & 1), (k >> 1) ^ 1);
        if (lane == 0) {
          C.work[k & 1] = w;
          tc::mbar_arrive(C.wfull + (k & 1));
        }
        if (!__all_sync(0xFFFFFFFFu, ok) || w.t.nq < 0) break;
        if (!__all_sync(0xFFFFFFFFu, wait(&C.want, k))) break;
        if (lane == 0) clc_request(C.reply, &C.clc);
        __syncwarp();
        int block = -1;
        if (wait(&C.clc, k))
          block = clc_block(C.reply);
        else
          pending = (int)k;
        block = __shfl_sync(0xFFFFFFFFu, block, 0);
        if (block >= 0)
          w = make_work(T, block, false, scan);
        else
          w.t.nq = -1;
      }
      // the reply lands before the CTA may exit
      if (pending >= 0) tc::mbar_wait(&C.clc, pending & 1, kDrainBudget, nullptr);
    } else if (warp == W_TMA) {
      // ---- loads: K_0 V_0 K_1 V_1 ... of every item through one ring, Q_0 and Q_1 ----
      if (tc::elect_one()) {
        uint32_t x = 0, qn[2] = {0, 0};
        bool ok = true;
        for (uint32_t k = 0; ok && have_item(k); ++k) {
          const Work &w = C.work[k & 1];
          const int hk = w.h[0] / (S.Hq / S.Hkv);
          const int ask = max(0, 2 * (w.nmax - kClaimTiles));
          auto kv = [&](int y) {
            if (y == ask) tc::mbar_arrive(&C.want);
            const int st = x % ST;
            if (!wait(C.empty + st, (x / ST) ^ 1)) return false;
            tc::mbar_arrive_expect_tx(C.full + st, Gm::TILE);
            for (int c = 0; c < Gm::NKB; ++c)
              tma_load_4d(sKV + st * Gm::TILE + c * Gm::SUB, (y & 1) ? &tmV : &tmK, c * 64, w.t.k0 + (w.j0 + (y >> 1)) * BN, hk,
                          w.t.b, C.full + st);
            ++x;
            return true;
          };
          // K_0 does not wait for Q's buffers; the loads behind Q wait until it has landed, as copies
          // in flight together share the way and Q is what the next product needs.
          if (w.nmax > 0) ok = kv(0);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (ok && w.n[i] > 0) {
              ok = wait(C.qempty + i, qn[i] ^ 1);
              if (!ok) continue;
              tc::mbar_arrive_expect_tx(C.qfull + i, Gm::TILE);
              for (int c = 0; c < Gm::NKB; ++c)
                tma_load_4d(sQ + i * Gm::TILE + c * Gm::SUB, &tmQ, c * 64, w.t.q0 + w.r0[i], w.h[i], w.t.b, C.qfull + i);
              ++qn[i];
            }
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (ok && w.n[i] > 0) ok = wait(C.qfull + i, qn[i] - 1);
          for (int y = 1; y < 2 * w.nmax && ok; ++y) ok = kv(y);
          if (w.nmax == 0) tc::mbar_arrive(&C.want);
          tc::mbar_arrive(C.wempty + (k & 1));
        }
        // copies in flight land before the CTA may exit (at once unless it gave up)
        for (int i = 0; i < 2; ++i)
          if (qn[i]) tc::mbar_wait(C.qfull + i, (qn[i] - 1) & 1, kDrainBudget, nullptr);
        for (uint32_t k = 1; k <= (uint32_t)ST && k <= x; ++k)
          tc::mbar_wait(C.full + (x - k) % ST, ((x - k) / ST) & 1, kDrainBudget, nullptr);
      }
    } else if (warp == W_MMA) {
      // ---- products (one elected thread: the operands then stay in uniform registers) ----
      if (tc::elect_one()) {
        const uint64_t qd = tc::sdesc_sw128(tc::smem_u32(sQ));
        const uint64_t kd0 = tc::sdesc_sw128(tc::smem_u32(sKV));
        const uint64_t vd0 = vdesc_sw128(tc::smem_u32(sKV), Gm::SUB);
        const uint32_t id_s = tc::idesc_bf16(BM, BN), id_o = tc::idesc_bf16(BM, D) | kTransposeB;
        auto qk = [&](int i, int st) {  // S_i = Q_i K^T
          const uint64_t q = qd + (uint64_t)((i * Gm::TILE) >> 4), k = kd0 + (uint64_t)((st * Gm::TILE) >> 4);
          const uint32_t dst = tmem + i * 128;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t o = (uint64_t)(((kk / 4) * Gm::SUB + (kk % 4) * 32) >> 4);
            tc::umma_bf16(dst, q + o, k + o, id_s, kk > 0);
          }
        };
        // Ring position and phases are counted here, not read from the items: values that
        // come from shared memory would not stay uniform.
        int st = 0;
        uint32_t ph = 0, fixes = 0, items[2] = {0, 0}, ps[2] = {0, 0};
        auto item = [&](const Work &w) -> bool {
          const int n[2] = {w.n[0], w.n[1]}, nmax = w.nmax, nk = w.t.nk - w.j0 * BN;
          if (nmax == 0) return true;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (n[i] > 0 && !wait(C.qfull + i, items[i])) return false;
          if (!wait(C.full + st, ph)) return false;
          tc::fence_after_sync();
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (n[i] > 0) {
              qk(i, st);
              tc::umma_commit(C.sfull + i);
              if (n[i] == 1) tc::umma_commit(C.qempty + i);
            }
          tc::umma_commit(C.empty + st);
          for (int j = 0; j < nmax; ++j) {
            if (++st == ST) st = 0, ph ^= 1;  // V_j
            const int sv = st;
            if (!wait(C.full + sv, ph)) return false;
            if (++st == ST) st = 0, ph ^= 1;  // K_{j+1}, if there is one
            if (nk - j * BN < BN) {           // the sequence ends inside this tile, its last
              tc::mbar_arrive(&C.vreq);
              if (!wait(&C.vfix, fixes++)) return false;
            }
            const uint64_t vd = vd0 + (uint64_t)((sv * Gm::TILE) >> 4);
            bool have_k = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (j < n[i]) {
                if (j == 0 && !wait(C.oempty + i, items[i] ^ 1)) return false;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {  // P comes in two halves of 64 keys
                  if (!wait(C.pfull + 2 * hf + i, ps[i])) return false;
                  tc::fence_after_sync();
#pragma unroll
                  for (int kk = hf * 4; kk < hf * 4 + 4; ++kk)
                    umma_ts(tmem + 256 + i * 128, tmem + i * 128 + kk * 8, vd + (uint64_t)((kk * 2048) >> 4), id_o,
                            (j > 0) | (kk > 0));
                  if (hf == 0) tc::umma_commit(C.pva + i);
                }
                ++ps[i];
                if (j == n[i] - 1) tc::umma_commit(C.ofull + i);
              }
              if (j + 1 < n[i]) {
                if (!have_k && !wait(C.full + st, ph)) return false;
                have_k = true;
                qk(i, st);
                tc::umma_commit(C.sfull + i);
                if (j + 2 == n[i]) tc::umma_commit(C.qempty + i);
              }
            }
            tc::umma_commit(C.empty + sv);
            if (j + 1 < nmax) tc::umma_commit(C.empty + st);
          }
          items[0] += n[0] > 0;
          items[1] += n[1] > 0;
          return true;
        };
        for (uint32_t it = 0; have_item(it); ++it) {
          if (!item(C.work[it & 1])) break;
          tc::mbar_arrive(C.wempty + (it & 1));
        }
        // every product is complete before TMEM is released
        tc::umma_commit(&C.drain);
        tc::mbar_wait(&C.drain, 0, kDrainBudget, nullptr);
      }
    } else {
      // ---- rows of V behind a sequence's end, in the one tile that it ends in ----
      uint32_t x = 0, fixes = 0;
      for (uint32_t k = 0; have_item(k); ++k) {
        const Work &w = C.work[k & 1];
        const int left = w.t.nk - (w.j0 + w.nmax - 1) * BN;
        x += 2 * w.nmax;
        if (w.nmax > 0 && left < BN) {
          unsigned char *v = sKV + ((x - 1) % ST) * Gm::TILE + left * 128;
          if (!__all_sync(0xFFFFFFFFu, wait(&C.vreq, fixes++))) break;  // the tile has landed
          for (int e = lane; e < (BN - left) * 8 * Gm::NKB; e += 32) {
            const int c = e / ((BN - left) * 8), r = e % ((BN - left) * 8);
            *reinterpret_cast<uint4 *>(v + c * Gm::SUB + r * 16) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&C.vfix);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(C.wempty + (k & 1));
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---- softmax of tile i: one thread a row ----
    const int i = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t ts = tmem + i * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = tmem + 256 + i * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    const float c = T.A.c_log2;
    uint32_t ss = 0, items = 0;
    for (uint32_t it = 0; have_item(it); ++it) {
      const Work &w = C.work[it & 1];
      const int n = w.n[i];
      const int first = w.r0[i] + w.t.nk - w.t.nq - w.j0 * BN;     // last key that the tile's first row sees
      const int mine = min(first + row, w.t.nk - 1 - w.j0 * BN);   // ... that this row sees
      float m = -INFINITY;                             // reference, log2 units
      float2 z2 = make_float2(0.f, 0.f);
      bool ok = true;
      for (int j = 0; j < n; ++j) {
        ok = __all_sync(0xFFFFFFFFu, wait(C.sfull + i, ss++));
        if (!ok) break;
        tc::fence_after_sync();
        // The tile in two steps of 64 keys: the second half's logits arrive and are searched for
        // their maximum while the first half's weights are computed, and the first half's
        // product runs while the second half's are.
        uint32_t r[128];
        tmem_ld32(ts, r);
        tmem_ld32(ts + 32, r + 32);
        tmem_landed<64>(r);
        tmem_ld32(ts + 64, r + 64);
        tmem_ld32(ts + 96, r + 96);
        const int lim = mine - j * BN;                   // last key of the tile that this row sees
        const bool part = j * BN + BN - 1 > first;       // some row sees only part of the tile
        float top[2];
        top[0] = half_max(r, part ? lim : BN) * c;
        tmem_landed<64>(r + 64);
        top[1] = half_max(r + 64, part ? lim - 64 : BN) * c;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const bool over = top[hf] > m + kLazy;
          if (__any_sync(0xFFFFFFFFu, over)) {
            const float f = over ? tc::ex2(m - top[hf]) : 1.f;
            if (over) m = top[hf];
            z2.x *= f;
            z2.y *= f;
            // O holds every product before this half: those of the tiles before are complete
            // (the commit that announced S covers them), the first half's has its own
            if (hf == 1) {
              ok = __all_sync(0xFFFFFFFFu, wait(C.pva + i, ss - 1));
              if (!ok) break;
              tc::fence_after_sync();
            }
            if (j > 0 || hf == 1) {
#pragma unroll
              for (int q = 0; q < D / 16; ++q) {
                uint32_t o[16];
                tc::tmem_ld16(to + q * 16, o);
                tc::tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                tmem_st16(to + q * 16, o);
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : -m;  // a row that has seen no key yet
          const float2 c2 = make_float2(c, c), b2 = make_float2(base, base);
#pragma unroll
          for (int q = 2 * hf; q < 2 * hf + 2; ++q) {
            uint32_t p[16];
            float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
            for (int x = 0; x < 16; x += 2) {
              const int s = q * 32 + 2 * x;
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
            tmem_st16(ts + q * 16, p);
          }
          tmem_st_wait();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(C.pfull + 2 * hf + i);
        }
        if (!ok) break;
      }
      if (!ok) break;
      // ---- O / z ----
      if (n > 0) {
        ok = __all_sync(0xFFFFFFFFu, wait(C.ofull + i, items++));
        if (!ok) break;
        tc::fence_after_sync();
      }
      if (w.split >= 0 && w.rows[i] > 0) {
        // this share of the keys, for attn_join_kernel
        const long long at = w.split * T.share_rows + T.share_row(w.t.b, w.h[i], w.tile, w.r0[i] - w.t.r0 + row,
                                                                  (long long)w.t.q0 + w.r0[i] + row);
        const bool live = row < w.rows[i];
        if (live) T.stat[at] = make_float2(m, z2.x + z2.y);
        if (n > 0) {
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(to + q * 32, o);
            tc::tmem_ld_wait();
            if (live) {
#pragma unroll
              for (int x = 0; x < 32; x += 8) st_global_32(T.part + at * D + q * 32 + x, o + x);
            }
          }
        }
      } else if (w.rows[i] > 0) {
        const float z = z2.x + z2.y;  // 0: no key seen; a NaN is passed on
        const float inv = z != 0.f ? 1.f / z : 0.f;
        const long long at = (long long)w.t.q0 + w.r0[i] + row;
        __nv_bfloat16 *dst = T.O + w.t.b * S.o[0] + w.h[i] * S.o[1] + at * S.o[2];
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
            const __nv_bfloat162 v = __floats2bfloat162_rn(z != 0.f ? __uint_as_float(o[2 * x]) * inv : 0.f,
                                                           z != 0.f ? __uint_as_float(o[2 * x + 1]) * inv : 0.f);
            p[x] = *reinterpret_cast<const uint32_t *>(&v);
          }
          // every lane writes its own row: whole 32-byte sectors where they are aligned
          if (live && T.wide) {
            st_global_32(dst + q * 32, p);
            st_global_32(dst + q * 32 + 16, p + 8);
          } else if (live) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              reinterpret_cast<uint4 *>(dst + q * 32)[x] = make_uint4(p[4 * x], p[4 * x + 1], p[4 * x + 2], p[4 * x + 3]);
          }
        }
        if (live && T.A.lse)
          T.A.lse[((long long)w.t.b * S.Hq + w.h[i]) * S.Tq + at] =
              z != 0.f ? (m + log2f(z)) * 0.6931471805599453f : -INFINITY;
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (n > 0) tc::mbar_arrive(C.oempty + i);
        tc::mbar_arrive(C.wempty + (it & 1));
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == W_MMA) tc::tmem_dealloc(tmem, 512);
}

// Joins the shares of the split tiles' rows: O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) z_s.  One CTA
// per (query tile, head); a row is D / 4 threads, all its shares in flight.
constexpr int kMaxSplits = 16;
constexpr int NTJ = 256, JM = 32;  // threads and rows of a CTA
template <int D>
__global__ void __launch_bounds__(NTJ) attn_join_kernel(const __grid_constant__ TcArgs T) {
  __shared__ AttnTile tile;
  const AttnShape &S = T.A.S;
  pdl_wait();
  pdl_launch();
  const int bm = T.pair_rows ? 2 * BM : BM, subs = bm / JM;
  const int h = blockIdx.x % S.Hq, sub = blockIdx.x / S.Hq % subs, split_tile = blockIdx.x / S.Hq / subs;
  if (threadIdx.x < 32) {
    const AttnTile t = attn_locate(S, T.whole + split_tile, bm, false, nullptr);
    if (threadIdx.x == 0) tile = t;
  }
  __syncthreads();
  AttnTile t = tile;
  t.r0 += sub * JM;
  const int rows = min(JM, t.nq - t.r0);
  const int lane = threadIdx.x % (D / 4);
  for (int r = threadIdx.x / (D / 4); r < rows; r += NTJ / (D / 4)) {
    const long long tok = (long long)t.q0 + t.r0 + r, at = T.share_row(t.b, h, split_tile, sub * JM + r, tok);
    float2 st[kMaxSplits];
    float M = -INFINITY;
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s)
      if (s < T.splits) {
        st[s] = T.stat[s * T.share_rows + at];
        if (st[s].y != 0.f) M = fmaxf(M, st[s].x);
      }
    float z = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s)
      if (s < T.splits && st[s].y != 0.f) {  // a share without a visible key was not written
        const float f = tc::ex2(st[s].x - M);
        const float4 x = __ldcs(reinterpret_cast<const float4 *>(T.part + (s * T.share_rows + at) * D) + lane);
        z += f * st[s].y;
        o.x += f * x.x;
        o.y += f * x.y;
        o.z += f * x.z;
        o.w += f * x.w;
      }
    const float inv = z != 0.f ? 1.f / z : 0.f;
    const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2 *>(T.O + t.b * S.o[0] + h * S.o[1] + tok * S.o[2] + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    if (T.A.lse && lane == 0) T.A.lse[((long long)t.b * S.Hq + h) * S.Tq + tok] = z != 0.f ? (M + log2f(z)) * 0.6931471805599453f : -INFINITY;
  }
}

// How the items are split over their keys: `whole` query tiles are not, the others in `splits`.
struct Plan {
  long tiles, pairs;  // query tiles, items per tile
  int whole, splits;
};

// A round of `items` equal items of `tiles` key tiles on all SMs, split in s, takes
// ceil(items s / SMs) (tiles / s + 2) steps of about 1.4 us (two are what an item costs
// besides its tiles); the shares' fp32 sums are written and read again by the join.
double round_steps(long items, int tiles, int s) {
  return (double)((items * s + kNumSmsHint - 1) / kNumSmsHint) * ((double)tiles / s + 2.) + (s > 1 ? 3. + items * s / 60. : 0.);
}

// Sizes alone decide (the lengths are on the device): Tk stands for every sequence's keys.
// Fewer items than SMs: all of them are split if that pays (16 rows of 32 heads over 32768
// keys, 16 items: 56 us against 352).  A few rounds of about equal items (a chunk behind
// many more keys): the tiles of the last, partial round are (2000 rows of 32 heads behind 30001
// keys, 256 items: 651 us against 672 on one GPU, to 683 on others; all in 4 shares 725).  Otherwise the items are
// many or shrink towards the end, and evening out is the claims' work.
Plan make_plan(const AttnShape &S) {
  const bool pair_rows = (S.Hq / S.Hkv) % 2;
  const int bm = pair_rows ? 2 * BM : BM, tiles = (S.Tk + BN - 1) / BN;
  Plan p{attn_tiles(S, bm), pair_rows ? S.Hq : S.Hq / 2, 0, 1};
  const long items = p.tiles * p.pairs;
  p.whole = (int)p.tiles;
  long rest = items;
  if (items >= kNumSmsHint) {
    if (items > 4 * kNumSmsHint || S.Tk < 2L * S.Tq) return p;
    p.whole = (int)(items / kNumSmsHint * kNumSmsHint / p.pairs);
    rest = items - p.whole * p.pairs;
  }
  const double one = round_steps(rest, tiles, 1);
  double least = one;
  for (int s = 2; s <= kMaxSplits && s * 4 <= tiles; ++s) {
    const double t = round_steps(rest, tiles, s);
    if (t < 0.85 * one && t < 0.95 * least) {
      p.splits = s;
      least = t;
    }
  }
  if (p.splits == 1) p.whole = (int)p.tiles;
  else if (items < kNumSmsHint) p.whole = 0;
  return p;
}

// Rows of one share: those of the split tiles (the last round of a chunk: few of all tokens), or
// every token's where the split tiles are not full (packed short sequences).
long long share_rows(const AttnShape &S, const Plan &p, bool *by_tile) {
  const long long tile = (p.tiles - p.whole) * ((S.Hq / S.Hkv) % 2 ? 2 * BM : BM), token = (long long)S.B * S.Tq;
  *by_tile = tile < token;
  return (*by_tile ? tile : token) * S.Hq;
}

template <int D>
int run(const void *Q, const void *K, const void *V, const TcArgs &T, cudaStream_t st) {
  const AttnShape &S = T.A.S;
  CUtensorMap tmQ, tmK, tmV;
  if (!encode_heads(&tmQ, Q, D, S.Tq, S.Hq, S.B, S.q) || !encode_heads(&tmK, K, D, S.Tk, S.Hkv, S.B, S.k) ||
      !encode_heads(&tmV, V, D, S.Tk, S.Hkv, S.B, S.v))
    return KV_ERR_CUDA;
  const Plan plan = make_plan(S);
  const long split = plan.tiles - plan.whole;  // split tiles
  const long ctas = (plan.whole + split * plan.splits) * plan.pairs;
  const long joins = plan.splits > 1 ? split * ((T.pair_rows ? 2 : 1) * BM / JM) * S.Hq : 0;
  if (ctas > 0x7FFFFFFFL || joins > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  if (ensure_smem((const void *)attn_tc_kernel<D>, Geo<D>::SMEM)) return KV_ERR_CUDA;
  const cudaError_t e = launch_pdl(attn_tc_kernel<D>, (unsigned)ctas, NT, Geo<D>::SMEM, st, tmQ, tmK, tmV, T);
  if (e != cudaSuccess) return cuda_failure(e, "prompt attention");
  if (joins > 0) {
    count_launches(1);
    const cudaError_t f = launch_pdl(attn_join_kernel<D>, (unsigned)joins, NTJ, 0, st, T);
    if (f != cudaSuccess) return cuda_failure(f, "prompt attention: joining the splits");
  }
  return launch_status();
}

}  // namespace

// scale > 0: the running maximum is taken over the products before they are scaled.
bool attn_tc_eligible(const AttnShape &S, float scale, int dtype) {
  return dtype == KV_BF16 && S.Tk > 0 && scale > 0.f && std::isfinite(scale);
}

size_t attn_tc_workspace_bytes(const AttnShape &S) {
  if (S.Tq <= 0 || S.Tk <= 0) return 0;
  const Plan plan = make_plan(S);
  bool by_tile;
  return plan.splits > 1 ? (size_t)plan.splits * share_rows(S, plan, &by_tile) * (S.d * sizeof(float) + sizeof(float2)) + 32 : 0;
}

int launch_attn_prompt_tc(const void *Q, const void *K, const void *V, const AttnArgs &A, void *O, void *ws,
                          cudaStream_t st) {
  bool wide = (reinterpret_cast<uintptr_t>(O) & 31) == 0;
  for (int i = 0; i < 3; ++i) wide = wide && A.S.o[i] % 16 == 0;
  const Plan plan = make_plan(A.S);
  bool by_tile;
  const long long rows = share_rows(A.S, plan, &by_tile);
  TcArgs T{A, static_cast<__nv_bfloat16 *>(O), (A.S.Hq / A.S.Hkv) % 2, wide, plan.whole, plan.splits, by_tile, rows,
           nullptr, nullptr};
  T.part = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(ws) + 31) & ~uintptr_t(31));  // 32-byte stores
  T.stat = reinterpret_cast<float2 *>(T.part + (size_t)T.splits * rows * A.S.d);
  return A.S.d == 128 ? run<128>(Q, K, V, T, st) : run<64>(Q, K, V, T, st);
}

}  // namespace kvc

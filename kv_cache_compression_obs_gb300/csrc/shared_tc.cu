// shared_tc.cu -- the common prefix of a batch on the tensor cores (tcgen05, TMA), bf16.
//
// The rows of all batch entries, group heads and new tokens that share a KV head are rows of one
// product: per head R = B G nq rows against the prefix's keys, which are read once for up to 256
// rows.  An item of work is two query tiles of 128 rows (R > 128) over a share of the keys, or
// one tile whose key tiles two softmax warpgroups take in turn (R <= 128; each then leaves a
// share of its own).  Per tile i and key tile j of 128 keys, as in prompt attention without the
// causal mask:
//     S = Q K_j^T (TMEM, fp32); P = 2^(c S - m) rounded to bf16; O_i += P V_j (TMEM, fp32),
// with a reference m that moves only when a logit passes it by kLazy.  One CTA per item and
// SM; O, m and the weights' sum go to the workspace undivided.
//
// Q's rows lie anywhere (batch, head and token strides), so the softmax warps place them in shared
// memory themselves; K and V come by TMA, whose fill makes rows behind the prefix 0.
//
// P is rounded to bf16 because the product takes both operands in V's type: each weight is off by at most
// half a step, 2^-8 of it.  2048 rows of 8 heads over 32768 keys: 31 us in a run of calls, of which the
// tiles take 20 (1.45 us each, 1.1 of them products), 5 pass until the first logits and 4 at the end
// until the shares (20 MB) are written.
#include "attn_tc.cuh"
#include "pdl.cuh"
#include "shared_common.cuh"

namespace kvc {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int NT = 384;
constexpr int W_MMA = 8, W_TMA = 9;  // warps 0-7: softmax; 10 and 11 only give up registers
constexpr int kMaxStages = 8;
constexpr int kCtrlBytes = 1024;
constexpr float kLazy = 8.f;
constexpr long long kWaitBudget = 4000000000LL;  // clock cycles (~2 s) before a wait gives up
constexpr long long kDrainBudget = 200000000LL;

template <int D>
struct Geo {
  static constexpr int NKB = D / 64;
  static constexpr int SUB = 128 * 128;
  static constexpr int TILE = NKB * SUB;
  static constexpr int STAGES = D == 128 ? 5 : 8;
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = 2 * TILE;
  static constexpr int CTRL_OFF = KV_OFF + STAGES * TILE;
  static constexpr int SMEM_NEED = CTRL_OFF + kCtrlBytes;
  // more than half an SM's shared memory: a CTA takes all of TMEM, so one per SM
  static constexpr int SMEM = SMEM_NEED > 116 * 1024 ? SMEM_NEED : 116 * 1024;
};

struct Ctrl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t qfull[2], sfull[2], pfull[4], pva[2], ofull[2], drain;
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(Ctrl) <= kCtrlBytes, "control block");

struct PrefixArgs {
  SharedArgs A;
  int pairs;   // items' row pairs per head
  int shares;  // of the keys
  int tiles;   // key tiles of a share
  int turn;    // 1: one row tile, key tiles in turn
};

template <int D>
__global__ void __launch_bounds__(NT, 1) prefix_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                                                          const __grid_constant__ PrefixArgs T) {
  using Gm = Geo<D>;
  constexpr int ST = Gm::STAGES;
  extern __shared__ __align__(1024) unsigned char sm[];  // no static shared memory in front of it
  unsigned char *sQ = sm + Gm::Q_OFF, *sKV = sm + Gm::KV_OFF;
  Ctrl &C = *reinterpret_cast<Ctrl *>(sm + Gm::CTRL_OFF);
  const SharedArgs &A = T.A;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(C.full + i, 1);
      tc::mbar_init(C.empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(C.qfull + i, 4);
      tc::mbar_init(C.sfull + i, 1);
      tc::mbar_init(C.pfull + i, 4);
      tc::mbar_init(C.pfull + 2 + i, 4);
      tc::mbar_init(C.pva + i, 1);
      tc::mbar_init(C.ofull + i, 1);
    }
    tc::mbar_init(&C.drain, 1);
    C.abort_flag = 0;
    tc::mbar_fence_init();
  }
  if (warp == W_MMA) tc::tmem_alloc(&C.tmem, 512);
  if (warp == W_TMA && lane == 0) {
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
  const int share = blockIdx.x % T.shares, rest = blockIdx.x / T.shares;
  const int h = rest % A.Hkv, pair = rest / A.Hkv;
  const int j0 = share * T.tiles;                        // first key tile
  const int n = min(T.tiles, (A.P + BN - 1) / BN - j0);  // at least 1
  const int row0 = pair * 2 * BM;                        // first row, of head h's
  const bool turn = T.turn;
  const bool two = turn || row0 + BM < A.rows;           // the second tile has work
  constexpr int CH = D / 8;                              // 16-byte pieces of a row
  struct {
    int b, g, t;
  } at{0, 0, 0};  // the first query row that a softmax lane fetches
  if (warp < 8) {
    const int gn = A.G * A.nq, r = row0 + (turn ? 0 : (warp >> 2) * BM) + (warp & 3) * 32 + lane / CH;
    at.b = r / gn;
    at.g = (r - at.b * gn) / A.nq;
    at.t = r - at.b * gn - at.g * A.nq;
  }
  pdl_wait();
  pdl_launch();  // in this order: the next launch takes it that what precedes the call is complete (pdl.cuh)
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = C.tmem;
  volatile int *abort_flag = &C.abort_flag;
  auto wait = [&](uint64_t *bar, uint32_t ph) -> bool {
    if (tc::mbar_wait(bar, ph & 1, kWaitBudget, abort_flag)) return true;
    *abort_flag = 1;
    if (A.status) atomicExch(A.status, (int)KV_ERR_TIMEOUT);
    return false;
  };
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == W_TMA) {
      // ---- loads: K one tile ahead of V (two, where the tiles take turns) ----
      if (tc::elect_one()) {
        uint32_t x = 0;
        auto load = [&](const CUtensorMap *map, int j) {
          const int st = x % ST;
          if (!wait(C.empty + st, (x / ST) ^ 1)) return false;
          tc::mbar_arrive_expect_tx(C.full + st, Gm::TILE);
          for (int c = 0; c < Gm::NKB; ++c)
            tma_load_4d(sKV + st * Gm::TILE + c * Gm::SUB, map, c * 64, (j0 + j) * BN, h, 0, C.full + st);
          ++x;
          return true;
        };
        const int lead = turn ? 2 : 1;
        bool ok = true;
        for (int j = 0; ok && j < min(lead, n); ++j) ok = load(&tmK, j);
        for (int j = 0; ok && j < n; ++j) {
          ok = load(&tmV, j);
          if (ok && j + lead < n) ok = load(&tmK, j + lead);
        }
        // copies in flight land before the CTA may exit (at once unless it gave up)
        for (uint32_t k = 1; k <= (uint32_t)ST && k <= x; ++k)
          tc::mbar_wait(C.full + (x - k) % ST, ((x - k) / ST) & 1, kDrainBudget, nullptr);
      }
    } else if (warp == W_MMA) {
      // ---- products ----
      if (tc::elect_one()) {
        const uint64_t qd = tc::sdesc_sw128(tc::smem_u32(sQ));
        const uint64_t kd0 = tc::sdesc_sw128(tc::smem_u32(sKV));
        const uint64_t vd0 = vdesc_sw128(tc::smem_u32(sKV), Gm::SUB);
        const uint32_t id_s = tc::idesc_bf16(BM, BN), id_o = tc::idesc_bf16(BM, D) | kTransposeB;
        int st = 0;
        uint32_t ph = 0, ps[2] = {0, 0};
        auto next = [&]() {  // the ring's next stage, once it is full
          const int s = st;
          if (!wait(C.full + s, ph)) return -1;
          if (++st == ST) st = 0, ph ^= 1;
          return s;
        };
        auto qk = [&](int i, int s) {  // S_i = Q_i K^T
          const uint64_t q = qd + (uint64_t)((i * Gm::TILE) >> 4), k = kd0 + (uint64_t)((s * Gm::TILE) >> 4);
          tc::fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t o = (uint64_t)(((kk / 4) * Gm::SUB + (kk % 4) * 32) >> 4);
            tc::umma_bf16(tmem + i * 128, q + o, k + o, id_s, kk > 0);
          }
          tc::umma_commit(C.sfull + i);
        };
        auto pv = [&](int i, int s, bool first, bool last) {  // O_i += P_i V, P in two halves of 64 keys
          const uint64_t vd = vd0 + (uint64_t)((s * Gm::TILE) >> 4);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            if (!wait(C.pfull + 2 * hf + i, ps[i])) return false;
            tc::fence_after_sync();
#pragma unroll
            for (int kk = hf * 4; kk < hf * 4 + 4; ++kk)
              umma_ts(tmem + 256 + i * 128, tmem + i * 128 + kk * 8, vd + (uint64_t)((kk * 2048) >> 4), id_o, !first | (kk > 0));
            if (hf == 0) tc::umma_commit(C.pva + i);
          }
          ++ps[i];
          if (last) tc::umma_commit(C.ofull + i);
          return true;
        };
        auto products = [&]() {
          if (!wait(C.qfull, 0) || (two && !wait(C.qfull + 1, 0))) return;
          if (turn) {
            for (int j = 0; j < min(2, n); ++j) {
              const int sk = next();
              if (sk < 0) return;
              if (j == 0) qk(0, sk); else qk(1, sk);
              tc::umma_commit(C.empty + sk);
            }
            for (int j = 0; j < n; ++j) {
              const int sv = next();
              if (sv < 0) return;
              const bool last = j + 2 >= n;
              if (!((j & 1) ? pv(1, sv, j < 2, last) : pv(0, sv, j < 2, last))) return;
              tc::umma_commit(C.empty + sv);
              if (last) continue;
              const int sk = next();
              if (sk < 0) return;
              if (j & 1) qk(1, sk); else qk(0, sk);
              tc::umma_commit(C.empty + sk);
            }
          } else {
            int sk = next();
            if (sk < 0) return;
            qk(0, sk);
            if (two) qk(1, sk);
            tc::umma_commit(C.empty + sk);
            for (int j = 0; j < n; ++j) {
              const int sv = next();
              if (sv < 0) return;
              const bool last = j + 1 == n;
              if (!pv(0, sv, j == 0, last)) return;
              if (!last) {
                sk = next();
                if (sk < 0) return;
                qk(0, sk);
              }
              if (two) {
                if (!pv(1, sv, j == 0, last)) return;
                if (!last) qk(1, sk);
              }
              tc::umma_commit(C.empty + sv);
              if (!last) tc::umma_commit(C.empty + sk);
            }
          }
        };
        products();
        // every product is complete before TMEM is released
        tc::umma_commit(&C.drain);
        tc::mbar_wait(&C.drain, 0, kDrainBudget, nullptr);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---- softmax of tile i: one thread a row ----
    const int i = warp >> 2;
    const int tile0 = row0 + (turn ? 0 : i * BM);  // first row
    const int row = (warp & 3) * 32 + lane;
    const int cnt = turn ? (n - i + 1) / 2 : (i == 0 || two ? n : 0);
    if (two || i == 0) {
      // this warp's rows of Q, 16 bytes a lane, where the swizzled layout wants them; rows that do not exist are 0
      // all on their way together: in four batches, each behind the ring's tiles, they took 12 us
      uint4 x[CH];
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        x[e] = make_uint4(0, 0, 0, 0);
        if (at.b < A.B)
          x[e] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(A.q) + at.b * A.sq[0] +
                                                  ((long)h * A.G + at.g) * A.sq[1] + at.t * A.sq[2] + lane % CH * 8);
        at.t += 32 / CH;
        while (at.t >= A.nq) at.t -= A.nq, ++at.g;
        while (at.g >= A.G) at.g -= A.G, ++at.b;
      }
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        const int r = (warp & 3) * 32 + (e * 32 + lane) / CH, c = lane % CH;
        *reinterpret_cast<uint4 *>(sQ + i * Gm::TILE + (c / 8) * Gm::SUB + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x[e];
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(C.qfull + i);
    }
    const uint32_t ts = tmem + i * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = tmem + 256 + i * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    const float c = A.c_log2;
    float m = -INFINITY;  // reference, log2 units
    float2 z2 = make_float2(0.f, 0.f);
    bool ok = true;
    for (int y = 0; y < cnt; ++y) {
      const int j = j0 + (turn ? 2 * y + i : y);
      ok = __all_sync(0xFFFFFFFFu, wait(C.sfull + i, y));
      if (!ok) break;
      tc::fence_after_sync();
      // the tile in two steps of 64 keys, as in prompt attention
      uint32_t r[128];
      tmem_ld32(ts, r);
      tmem_ld32(ts + 32, r + 32);
      tmem_landed<64>(r);
      tmem_ld32(ts + 64, r + 64);
      tmem_ld32(ts + 96, r + 96);
      const int lim = A.P - 1 - j * BN;  // last key of the tile that is there
      float top[2];
      top[0] = half_max(r, lim) * c;
      tmem_landed<64>(r + 64);
      top[1] = half_max(r + 64, lim - 64) * c;
      if (y == 0) top[0] = fmaxf(top[0], top[1]);  // not to wait for the first half's product, whose V may be far
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
            ok = __all_sync(0xFFFFFFFFu, wait(C.pva + i, y));
            if (!ok) break;
            tc::fence_after_sync();
          }
          if (y > 0 || hf == 1) {
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
        const float base = m == -INFINITY ? 0.f : -m;
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
    if (ok && cnt > 0) {
      ok = __all_sync(0xFFFFFFFFu, wait(C.ofull + i, 0));
      tc::fence_after_sync();
    }
    if (ok) {
      const bool live = tile0 + row < A.rows;
      const long at = ((long)(turn ? 2 * share + i : share) * A.Hkv + h) * A.rows + tile0 + row;
      if (live) A.stat[at] = make_float2(m, z2.x + z2.y);
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        if (cnt > 0) {
          tmem_ld32(to + q * 32, o);
          tc::tmem_ld_wait();
        } else {  // no key tile: sums of 0
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0u;
        }
        if (live) {
#pragma unroll
          for (int x = 0; x < 32; x += 8) st_global_32(A.part + at * D + q * 32 + x, o + x);
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == W_MMA) tc::tmem_dealloc(tmem, 512);
}

struct Plan {
  int turn, pairs, shares, tiles;
};

// Sizes alone decide.  A round of `items` on all SMs takes as long as its key tiles (about 1.3 us
// each) and what a CTA costs besides (3 us); the shares' fp32 sums are written and read again (from L2).
Plan make_plan(long rows, int Hkv, int P) {
  Plan p{};
  p.turn = rows <= BM;
  p.pairs = p.turn ? 1 : (int)((rows + 2 * BM - 1) / (2 * BM));
  const int all = (P + BN - 1) / BN;
  const long items = (long)p.pairs * Hkv;
  double least = 0;
  for (int s = 1; s <= 32 && s <= all; ++s) {
    const int tiles = (all + s - 1) / s;
    const double us = (double)((items * s + kNumSmsHint - 1) / kNumSmsHint) * (tiles * 1.3 + 3.) + (double)s * rows * Hkv * 1.3e-4;
    if (s == 1 || us < least) {
      least = us;
      p.tiles = tiles;
      p.shares = (all + tiles - 1) / tiles;  // none is empty
    }
  }
  return p;
}

template <int D>
int run(const PrefixArgs &T, cudaStream_t st) {
  const SharedArgs &A = T.A;
  const long long sk[3] = {A.skp[0], A.skp[0], A.skp[1]}, sv[3] = {A.svp[0], A.svp[0], A.svp[1]};  // one batch row: never stepped
  CUtensorMap tmK, tmV;
  if (!encode_heads(&tmK, A.Kp, D, A.P, A.Hkv, 1, sk) || !encode_heads(&tmV, A.Vp, D, A.P, A.Hkv, 1, sv)) return KV_ERR_CUDA;
  const long ctas = (long)T.pairs * A.Hkv * T.shares;
  if (ctas > 0x7FFFFFFFL) return KV_ERR_UNSUPPORTED;
  if (ensure_smem((const void *)prefix_tc_kernel<D>, Geo<D>::SMEM)) return KV_ERR_CUDA;
  const cudaError_t e = launch_pdl(prefix_tc_kernel<D>, (unsigned)ctas, NT, Geo<D>::SMEM, st, tmK, tmV, T);
  if (e != cudaSuccess) return cuda_failure(e, "shared prefix");
  count_launches(1);
  return KV_OK;
}

}  // namespace

SharedPlan shared_tc_plan(long rows, int Hkv, int P) {
  const Plan p = make_plan(rows, Hkv, P);
  return SharedPlan{p.shares * (p.turn ? 2 : 1), p.tiles * BN};
}

int launch_shared_prefix_tc(const SharedArgs &A, int d, cudaStream_t st) {
  const Plan p = make_plan(A.rows, A.Hkv, A.P);
  const PrefixArgs T{A, p.pairs, p.shares, p.tiles, p.turn};
  return d == 128 ? run<128>(T, st) : run<64>(T, st);
}

}  // namespace kvc

// attn_common.cuh -- what the two prompt attention kernels share: the call's
// shape and the walk from a query tile's index to its sequence.
#pragma once

#include "kvc_internal.cuh"

namespace kvc {

struct AttnArgs {
  AttnShape S;
  float c_log2;  // scale log2(e)
  float *lse;
  int *status;
};

// A query tile: rows [r0, r0 + bm) of a sequence of nq query rows and nk keys, whose
// first query row and key stand at tokens q0, k0 of batch row b.  nq = 0: no such tile.
struct AttnTile {
  int b, q0, k0, nq, nk, r0;
};

// Sequence i's rows; nq < 0 when its length or offsets are out of range.
__device__ __forceinline__ AttnTile attn_sequence(const AttnShape &S, int i) {
  AttnTile t{0, 0, 0, S.Tq, S.Tk, 0};
  if (S.n_seq > 0) {
    t.q0 = S.seq_q[i];
    t.k0 = S.seq_k[i];
    const int q1 = S.seq_q[i + 1], k1 = S.seq_k[i + 1];
    const bool ok = t.q0 >= 0 && q1 >= t.q0 && q1 <= S.Tq && t.k0 >= 0 && k1 >= t.k0 && k1 <= S.Tk;
    t.nq = ok ? q1 - t.q0 : -1;
    t.nk = ok ? k1 - t.k0 : 0;
  } else {
    t.b = i;
    if (S.seq_q) t.nq = S.seq_q[i];
    if (S.seq_k) t.nk = S.seq_k[i];
    if (t.nq < 0 || t.nq > S.Tq || t.nk < 0 || t.nk > S.Tk) t.nq = -1;
  }
  return t;
}

// How far a warp has walked the sequences: `before` tiles in those in front of `base`.
struct AttnScan {
  int base, before;
};

// The index-th query tile of bm rows over all sequences, a sequence's last rows
// (which see the most keys) first.  Executed by one whole warp; every lane gets the
// tile.  scan: where the last call found its tile; a later tile is looked for from there,
// so that a CTA walks thousands of short sequences once and not once per tile.
// check_all: also look at every sequence and report bad ones.
__device__ __forceinline__ AttnTile attn_locate(const AttnShape &S, int index, int bm, bool check_all, int *status,
                                                AttnScan &scan) {
  const int lane = threadIdx.x & 31;
  const int n = S.n_seq > 0 ? S.n_seq : S.B;
  AttnTile found{0, 0, 0, 0, 0, 0};
  bool have = false;
  const bool ahead = index >= scan.before;
  int before = ahead ? scan.before : 0;
  for (int base = ahead ? scan.base : 0; base < n && (!have || check_all); base += 32) {
    AttnTile t{0, 0, 0, 0, 0, 0};
    if (base + lane < n) {
      t = attn_sequence(S, base + lane);
      if (t.nq < 0) {
        if (check_all && status) atomicExch(status, (int)KV_ERR_INVALID_ARG);
        t.nq = 0;
      }
    }
    const int tiles = (t.nq + bm - 1) / bm;
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    const int first = before + incl - tiles;
    const bool mine = !have && index >= first && index < first + tiles;
    t.r0 = (tiles - 1 - (index - first)) * bm;
    const unsigned who = __ballot_sync(0xFFFFFFFFu, mine);
    if (who) {
      const int src = __ffs(who) - 1;
      found.b = __shfl_sync(0xFFFFFFFFu, t.b, src);
      found.q0 = __shfl_sync(0xFFFFFFFFu, t.q0, src);
      found.k0 = __shfl_sync(0xFFFFFFFFu, t.k0, src);
      found.nq = __shfl_sync(0xFFFFFFFFu, t.nq, src);
      found.nk = __shfl_sync(0xFFFFFFFFu, t.nk, src);
      found.r0 = __shfl_sync(0xFFFFFFFFu, t.r0, src);
      have = true;
      scan = AttnScan{base, before};
    }
    before += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  return found;
}

// The same for a warp that takes one tile only.
__device__ __forceinline__ AttnTile attn_locate(const AttnShape &S, int index, int bm, bool check_all, int *status) {
  AttnScan scan{0, 0};
  return attn_locate(S, index, bm, check_all, status, scan);
}

bool attn_tc_eligible(const AttnShape &S, float scale, int dtype);
size_t attn_tc_workspace_bytes(const AttnShape &S);
int launch_attn_prompt_tc(const void *Q, const void *K, const void *V, const AttnArgs &A, void *O, void *ws,
                          cudaStream_t st);

// Tiles at most: every sequence may end in a partial one.
inline long attn_tiles(const AttnShape &S, int bm) {
  if (S.n_seq == 0) return (long)S.B * ((S.Tq + bm - 1) / bm);
  return (long)S.Tq / bm + S.n_seq;
}

}  // namespace kvc

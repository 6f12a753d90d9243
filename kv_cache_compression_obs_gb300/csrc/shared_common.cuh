// shared_common.cuh -- what the two kernels over a shared prefix leave for the one that joins
// them with the rows' own slots.
#pragma once

#include "kvc_internal.cuh"

namespace kvc {

// The query rows of KV head h against the prefix: R = B G nq of them, row (b, g, t) at b G nq + g nq + t.
struct SharedArgs {
  const void *q, *Kp, *Vp, *K, *V;
  const int32_t *len;
  void *o;
  float *lse;
  int *status;
  long long sq[3], so[3], skp[2], svp[2];  // batch, head, token; head, token
  int B, Hq, Hkv, G, nq, P, cap;
  int rows;      // R
  int splits;    // shares of the prefix's keys (0: no prefix)
  float c_log2;
  float *part;   // [splits][Hkv][R][d] sums of P V, not yet divided
  float2 *stat;  // [splits][Hkv][R] reference (log2 units) and sum of weights
};

// Shares of the prefix and how many of its keys (whole tiles) each takes.
struct SharedPlan {
  int splits, per;
};
SharedPlan shared_tc_plan(long rows, int Hkv, int P);
int launch_shared_prefix_tc(const SharedArgs &A, int d, cudaStream_t st);

}  // namespace kvc

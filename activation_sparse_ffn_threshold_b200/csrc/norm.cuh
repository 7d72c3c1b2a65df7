// norm.cuh -- what the norms' kernels share (norm.cu, norm_ring.cu): their parameters, and the launchers
// of the kernels whose rows pass through shared memory.
#pragma once

#include "dense.cuh"

namespace sfnn {

struct NormParams {
  const void *x, *z, *gate, *w, *b, *wp, *bp;
  int64_t ldx, ldz, ldg;  // ldg 0: one gate row
  void *r, *h;
  int64_t ldr, ldh;
  float *stats;  // [T][4]: mean and reciprocal deviation of R, of Z; or null
  int T, d, x32, z32;
  int pre, post;  // sfnn_norm
  float eps, a, c, inv_d;
};

// What is summed over the rows.  Behind the post norm two sums serve five gradients, since a gate row,
// w_post and b_post are the same for every row (with p = D, or D gate where each token has its gate):
//
//     S1 = sum p Z^,  S0 = sum p:   dw_post = c gate S1,  db_post = c gate S0,  dgate = c (w_post S1 + b_post S0)
enum { kSumW, kSumB, kSum1, kSum0, kSums };
struct NormBackParams {
  NormParams f;
  const void *dr, *dh;
  int64_t lddr, lddh;
  void *dx, *dz, *dgate;  // contiguous; dgate: of a gate of every token
  float *part;            // [groups][sums][d], or null
  int32_t *err;
  int sums;       // that are asked for
  int at[kSums];  // their places in part, or -1
};

// Rows through shared memory (norm_ring.cu).  `fits` is false, and nothing was launched, where a row is
// too long for it; groups: of sums in part, no more than SMs or rows.
struct RingPlan {
  bool fits;
  int groups;
};
cudaError_t norm_forward_ring(const NormParams &P, int32_t *err, bool bf16, bool vec, int sms, cudaStream_t s,
                              RingPlan &plan);
cudaError_t norm_backward_ring(const NormBackParams &P, bool sums_all, bool bf16, bool vec, int sms, cudaStream_t s,
                               RingPlan &plan);

}  // namespace sfnn

// mx_grad.h -- host side of the dense gradient with its sum shared out (internal to libnf4).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nf4 {
namespace mx {

// parts[i][m][k] = the i-th part of sum_n dY[m][n] v(n,k), i < grad_splits(plan_M, plan_N, K);
// with `rescale` it is added to parts[i][m][k] * rescale[m].  Rows of dY are ld values apart, ld
// a multiple of 8, and zero from column N up to the next multiple of 8.  plan_M, plan_N: what the
// splits are planned for, one plan for all pieces of a sum.
struct GradParts {
  const uint8_t *codes, *scales;
  int64_t N, K, plan_M, plan_N;
  const uint16_t *dY;
  int64_t ld, M;
  float *parts;
  const float *rescale;
};
int grad_splits(int64_t M, int64_t N, int64_t K);
int launch_grad_parts(const GradParts &g, hipStream_t s);

}  // namespace mx
}  // namespace nf4

// nf4_check.h -- host-side argument checks shared by the MXFP4 and routing entry
// points (internal to libnf4).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/nf4.h"

namespace nf4 {

int device_status();  // NF4_OK on a gfx950 device (api.hip)

inline bool aligned_to(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline int launch_status(hipError_t e) { return e == hipSuccess ? NF4_OK : NF4_ELAUNCH; }

inline bool known_dtype(int dtype) { return dtype == NF4_F32 || dtype == NF4_BF16; }

// One packed MXFP4 matrix: K in whole blocks, codes below 2 GiB (32-bit byte
// offsets inside a matrix).
inline int check_mx_shape(int64_t N, int64_t K) {
  if (N <= 0 || K <= 0 || K % NF4_MX_BLOCK != 0) return NF4_EINVAL;
  if (K > NF4_MAX_K || N >= (int64_t(1) << 31)) return NF4_ERANGE;
  if (N * (K / 2) >= (int64_t(1) << 31)) return NF4_ERANGE;
  return NF4_OK;
}

}  // namespace nf4

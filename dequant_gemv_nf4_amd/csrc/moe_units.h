// moe_units.h -- which expert, rows and range of k a unit of the expert layer's second
// product is (gfx950; compiled for the host, too, where its bounds are tested).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/nf4.h"

namespace nf4 {
namespace mx {

// Tokens of each expert, a bit a token: what every workgroup makes of the routing.
struct Masks {
  uint32_t of[2 * NF4_MOE_MAX_E];
};

// The experts with a row, in order; entries from `count` on are never written.
struct ActiveExperts {
  Masks masks;
  uint16_t expert[NF4_MOE_MAX_E];
  uint16_t row0[NF4_MOE_MAX_E];
  int count;
};

struct Unit {  // past the last one all is 0: no rows, and empty buffers
  int e, row0, rows, cols, k0;
  uint64_t mask;
};

// Unit u of `units` (= count * ranges), range by range of each expert.  `uniform` passes on
// what is read, which is the same for the wave.  Nothing that is read past the last unit
// becomes an index: without any row not even entry 0 is written.
template <class UNIFORM>
__host__ __device__ __forceinline__ Unit unit_of(const ActiveExperts &act, int u, int units, int ranges, int range,
                                                 int cols, const UNIFORM &uniform) {
  if (u >= units) return Unit{0, 0, 0, 0, 0, 0};
  const int i = u / ranges;
  Unit v{uniform(act.expert[i]), uniform(act.row0[i]), 0, cols, (u - i * ranges) * range, 0};
  v.mask = (uint64_t)(uint32_t)uniform(act.masks.of[2 * v.e + 1]) << 32 | (uint32_t)uniform(act.masks.of[2 * v.e]);
  v.rows = __builtin_popcountll(v.mask);
  return v;
}

}  // namespace mx
}  // namespace nf4

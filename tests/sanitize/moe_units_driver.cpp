// Host run of the expert layer's unit lookup (moe_units.h) over lists of active experts whose
// unwritten entries hold the worst that LDS may: every index that comes out has to be one
// that the kernel may use.  Built with AddressSanitizer and UndefinedBehaviorSanitizer.
#include <cstdio>
#include <cstring>
#include <memory>

#include "moe_units.h"

using namespace nf4::mx;

int main() {
  int bad = 0;
  const auto same = [](int v) { return v; };
  for (int fill : {0x00, 0x5a, 0xff})
    for (int count : {0, 1, 2, 7, NF4_MOE_MAX_E})
      for (int ranges : {1, 2, 28, 64}) {
        // the list as the kernel writes it: entries from `count` on, and the masks of experts
        // past E, are whatever was there
        auto act = std::make_unique<ActiveExperts>();
        std::memset(act.get(), fill, sizeof(ActiveExperts));
        const int E = count == 0 ? 1 : count;
        std::memset(act->masks.of, 0, 8 * E);
        for (int i = 0; i < count; ++i) {
          act->masks.of[2 * i + (i & 1)] = 0x80000001u;  // two tokens each
          act->expert[i] = (uint16_t)i;
          act->row0[i] = (uint16_t)(2 * i);
        }
        act->count = count;
        const int units = count * ranges, range = 512, cols = 64;
        for (int u = 0; u < units + 3 * 2048; ++u) {
          const Unit v = unit_of(*act, u, units, ranges, range, cols, same);
          const bool in = u < units;
          const int i = in ? u / ranges : 0;
          const bool right = in ? v.e == i && v.row0 == 2 * i && v.rows == 2 && v.cols == cols &&
                                      v.k0 == (u - i * ranges) * range && v.mask != 0
                                : v.rows == 0 && v.cols == 0 && v.k0 == 0 && v.mask == 0;
          if (!right || v.e < 0 || v.e >= E || v.row0 < 0 || v.row0 > 2 * count) {
            std::printf("count %d ranges %d unit %d: expert %d row %d rows %d\n", count, ranges, u, v.e, v.row0, v.rows);
            bad = 1;
            break;
          }
        }
      }
  std::printf("moe units run: %s\n", bad ? "FAILED" : "ok");
  return bad;
}

// Exchanges between a warp's lanes.
#pragma once

#include <stdint.h>

namespace mla {

// Eight lanes with eight 16-byte pieces each exchange them: lane i gets piece i of each lane's.  Between
// a row a lane, as tensor memory has it, and 128 bytes of a row over eight lanes, as memory wants it:
// a warp's access then touches four lines, not 32 (which kept the store unit busy for 6,000 clocks for
// the 256 output rows of a prefill unit, and the load unit for 7,000 for the 128 rows of mla_expand).
__device__ __forceinline__ void transpose8(uint32_t (&v)[32], int lane) {
#pragma unroll
  for (int b = 1; b < 8; b <<= 1) {
    const bool up = lane & b;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      if (p & b) continue;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t &lo = v[4 * p + w], &hi = v[4 * (p | b) + w];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, b);
        if (up) lo = got;
        else hi = got;
      }
    }
  }
}

}  // namespace mla

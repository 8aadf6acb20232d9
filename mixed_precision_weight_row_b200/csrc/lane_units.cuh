// Exchange of register units among neighbouring lanes, so that the lanes of a
// store write neighbouring units.
#pragma once

#include <stdint.h>

namespace mpw {

// Transposes blocks of U x U units of W words among U neighbouring lanes: unit
// q of lane l goes to unit (l % U) of lane (l - l % U + q).
template <int U, int W>
__device__ __forceinline__ void transpose_units(uint32_t (&v)[U * W], int lane) {
#pragma unroll
  for (int s = U / 2; s > 0; s >>= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (q & s) continue;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t& a = v[q * W + w];
        uint32_t& b = v[(q | s) * W + w];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a : b, s);
        if (up) a = got;
        else b = got;
      }
    }
  }
}

}  // namespace mpw

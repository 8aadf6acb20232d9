// bf16 weights s * q from packed codes of up to 9 bits, two at a time.
//
// s is split into two bf16 values, s = hi + lo up to 2^-16 of it, and
// s q = fma(q, hi, q lo) in bf16x2 arithmetic: the product with hi is exact inside
// the fma, so the result is s q rounded to bf16 once, from a value that is off by
// at most 2^-16 of itself.  Two operations a pair, where going through fp32
// takes five.  (bf16 is what the tensor cores multiply: the operand is off by at
// most 2^-8 of itself, as the bf16 result is once more.)
//
// Below 2^-100 lo would lose bits, since bf16's steps get no smaller below 2^-126:
// there a power of two moves from the codes to the scale, s q = (s / p)(p q),
// exactly; the code's last fma takes its factor and its offset from registers.
// (One B200, dx of 48 x 17408 x 5120, b = 6: 34.8 us, 33.6 without p; multiplying the
// products of such rows by p in a branch took 34.8 as well.)
// hi is kept finite: a scale beyond bf16's largest number has the rest in lo.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include <utility>

#include "expand.cuh"

namespace mpw {
namespace dec {

// A row's scale: hi and lo of s / p; p, 128 p and the offset of a code times p.
struct PairScale {
  uint32_t hi2, lo2, one, high, off;
};

template <int B>
__device__ __forceinline__ PairScale split_scale(float s) {
  static_assert(B <= 9, "one exact bf16 value per code");
  const bool small = fabsf(s) < 0x1p-100f;
  if (small) s *= 0x1p64f;
  const float top = fminf(s, 0x1.FEp127f);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(top, top);
  const float rest = s - __low2float(hi);
  const __nv_bfloat162 lo = __floats2bfloat162_rn(rest, rest);
  // the factors and the offset of the expansion; p takes 64 from a bf16 exponent
  constexpr uint32_t p = 0x20002000u, one = pair_of(1), high = pair_of(128);
  constexpr uint32_t off = pair_of(B <= 7 ? -(128 + (1 << (B - 1))) : -128 * (129 + (1 << (B <= 7 ? 0 : B - 8))));
  PairScale r;
  r.hi2 = *reinterpret_cast<const uint32_t*>(&hi);
  r.lo2 = *reinterpret_cast<const uint32_t*>(&lo);
  r.one = small ? one - p : one;
  r.high = small ? high - p : high;
  r.off = small ? off - p : off;
  return r;
}

// Codes 2I and 2I+1 of a group times the scale.
template <int B, bool PAIRED, int I>
__device__ __forceinline__ uint32_t scaled_pair(const uint32_t (&w)[B + 1], const PairScale& s) {
  uint32_t q;
  if constexpr (B <= 7) {
    q = bf2_fma(field2<B, PAIRED, I, 0, B, true>(w), s.one, s.off);
  } else {
    // q = lo7 + 128 * hi: t = 128 * hi - 128, then (128 + lo7) + t
    const uint32_t t = bf2_fma(field2<B, PAIRED, I, 7, B - 7, true>(w), s.high, s.off);
    q = bf2_fma(field2<B, PAIRED, I, 0, 7, false>(w), s.one, t);
  }
  const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&q);
  const __nv_bfloat162 r = __hfma2(v, *reinterpret_cast<const __nv_bfloat162*>(&s.hi2),
                                   __hmul2(v, *reinterpret_cast<const __nv_bfloat162*>(&s.lo2)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int B, bool PAIRED, int... I>
__device__ __forceinline__ void scaled_all(const uint32_t (&w)[B + 1], const PairScale& s, uint32_t (&o)[16],
                                           std::integer_sequence<int, I...>) {
  ((o[I] = scaled_pair<B, PAIRED, I>(w, s)), ...);
}

// One 32-code group (B words, w[B] = 0) -> 16 pairs of weights.
template <int B, bool PAIRED>
__device__ __forceinline__ void scaled_group(const uint32_t (&w)[B + 1], const PairScale& s, uint32_t (&o)[16]) {
  scaled_all<B, PAIRED>(w, s, o, std::make_integer_sequence<int, 16>{});
}

}  // namespace dec
}  // namespace mpw

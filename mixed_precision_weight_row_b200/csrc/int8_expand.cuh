// Packed codes of 4..8 bits -> signed bytes for the int8 tensor cores and the
// integer dot product.
//
// A code's B two's-complement bits are moved to the top of a byte, the low
// 8 - B bits cleared: as a signed byte that is q * 2^(8-B), with no separate
// sign extension.  Every sum over k is then 2^(8-B) times the wanted one and
// the epilogue shifts it back, exactly.  |q * 2^(8-B)| <= 128 and |xq| <= 127,
// so a 32-bit sum cannot overflow for K <= kInt8MaxK.
#pragma once

#include <stdint.h>

#include <utility>

#include "expand.cuh"

namespace mpw {
namespace i8 {

// Byte mask of the left-justified field.
template <int B>
struct Just {
  static constexpr uint32_t kMask = ((0xFFu << (8 - B)) & 0xFFu) * 0x01010101u;
};

// Shift by a compile-time amount, left when positive.
template <int S>
__device__ __forceinline__ uint32_t shift(uint32_t v) {
  if constexpr (S > 0) return v << S;
  else if constexpr (S < 0) return v >> (-S);
  else return v;
}

// Codes 2I (low half) and 2I+1 (high half) of a paired group, each at the top
// of one byte of its half; `hi` tells which byte.
template <int B, int I>
struct PairedByte {
  static constexpr int o = I * B, h = o >> 4, r = o & 15;
  static constexpr bool cross = r + B > 16;
  static constexpr int rr = cross ? r - 8 : r;             // offset in the 16-bit window
  static constexpr bool hi = rr + B > 8;                   // ends in the window's upper byte
  static constexpr int sh = (hi ? 16 : 8) - B - rr;
  static __device__ __forceinline__ uint32_t get(const uint32_t (&w)[B + 1]) {
    uint32_t t = w[h];
    // a field that crosses a half-word lies in the window that starts at bit 8
    if constexpr (cross) t = __byte_perm(w[h], w[h + 1], 0x6341);
    return shift<sh>(t);
  }
};

// Codes 4I .. 4I+3 of a 32-code group as left-justified bytes in k order.
template <int B, bool PAIRED, int I>
__device__ __forceinline__ uint32_t quad(const uint32_t (&w)[B + 1]) {
  if constexpr (PAIRED) {
    using P0 = PairedByte<B, 2 * I>;
    using P1 = PairedByte<B, 2 * I + 1>;
    constexpr uint32_t sel = (P0::hi ? 0x0031u : 0x0020u) | (P1::hi ? 0x7500u : 0x6400u);
    const uint32_t v = __byte_perm(P0::get(w), P1::get(w), sel);
    return B == 8 ? v : v & Just<B>::kMask;
  } else if constexpr (B == 8) {
    return w[I];
  } else if constexpr (B == 4) {
    // word I/2 holds codes of even index in the low nibbles of its bytes and
    // codes of odd index in the high ones
    const uint32_t a = (w[I >> 1] << 4) & 0xF0F0F0F0u, b = w[I >> 1] & 0xF0F0F0F0u;
    return __byte_perm(a, b, (I & 1) ? 0x7362 : 0x5140);
  } else {
    // two codes to each half-word, then each to its byte
    const uint32_t t = dec::window<B>(w, 4 * I * B);
    constexpr uint32_t low = (1u << (2 * B)) - 1u;
    const uint32_t u = (t & low) | ((t << (16 - 2 * B)) & ~low);
    constexpr uint32_t m0 = (((1u << B) - 1u) << (8 - B)) * 0x00010001u;
    return ((u << (8 - B)) & m0) | ((u << (16 - 2 * B)) & (m0 << 8));
  }
}

template <int B, bool PAIRED, int... I>
__device__ __forceinline__ void group_all(const uint32_t (&w)[B + 1], uint32_t (&o)[8],
                                          std::integer_sequence<int, I...>) {
  ((o[I] = quad<B, PAIRED, I>(w)), ...);
}

// One 32-code group (B words, w[B] = 0) -> 32 left-justified bytes in k order.
template <int B, bool PAIRED>
__device__ __forceinline__ void group(const uint32_t (&w)[B + 1], uint32_t (&o)[8]) {
  group_all<B, PAIRED>(w, o, std::make_integer_sequence<int, 8>{});
}

}  // namespace i8
}  // namespace mpw

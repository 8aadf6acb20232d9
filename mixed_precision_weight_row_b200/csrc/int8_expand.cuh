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

// A row's scale s for y = sum * s * sx in fp32: before sx, or after it if s is so
// large that the sum (below 2^31) times it might overflow where y does not.  A whole
// number times a scale loses nothing to underflow.
struct RowScale {
  float before, after;
  static constexpr float kLarge = 0x1p64f;
  explicit __device__ RowScale(float s) : before(s > kLarge ? 1.0f : s), after(s > kLarge ? s : 1.0f) {}
  __device__ __forceinline__ float of(int32_t sum, float sx) const {
    return static_cast<float>(sum) * before * sx * after;
  }
};

// Byte mask of the left-justified field.
template <int B>
struct Just {
  static constexpr uint32_t kMask = ((0xFFu << (8 - B)) & 0xFFu) * 0x01010101u;
};

// The B words of a group from shared memory (w[B] = 0), in the widest loads its
// alignment allows.
template <int B>
__device__ __forceinline__ void lds_group(const uint8_t* p, uint32_t (&w)[B + 1]) {
  if constexpr (B % 4 == 0) {
#pragma unroll
    for (int i = 0; i < B / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  } else if constexpr (B % 2 == 0) {
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      const uint2 v = reinterpret_cast<const uint2*>(p)[i];
      w[2 * i] = v.x; w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < B; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
  w[B] = 0u;
}

// A canonical group re-ordered into two streams, codes 0..15 in the low and codes
// 16..31 in the high halves of its words (one byte permute a word): what the paired
// layout's expansion takes, which then yields the pairs (i, 16 + i).
template <int B>
__device__ __forceinline__ void halves_of(const uint32_t (&w)[B + 1], uint32_t (&z)[B + 1]) {
#pragma unroll
  for (int h = 0; h < B; ++h) {
    const uint32_t sel = ((h & 1) ? 0x0032u : 0x0010u) | (((B + h) & 1) ? 0x7600u : 0x5400u);
    z[h] = __byte_perm(w[h >> 1], w[(B + h) >> 1], sel);
  }
  z[B] = 0u;
}

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

// ---------------------------------------------------------------------------
// The same bytes in an order of k that takes fewer operations, for kernels
// that can order x to match.  Codes repeat against byte borders every
// U = 8 / gcd(8, B) codes (a unit of U * B / 8 bytes): byte p of four units
// side by side in one word (a "plane") lets one shift and one mask place the
// same code of all four, or two of each and an OR when it crosses a byte.
// A plane takes one byte permute of paired words, whose halves hold two
// streams already, and two or three of canonical ones; 4-bit codes need none and
// 8-bit codes are left as they are.
// ---------------------------------------------------------------------------

template <int B>
struct Unit {
  static constexpr int codes = B == 8 ? 1 : (B == 4 ? 2 : (B == 6 ? 4 : 8));
  static constexpr int bytes = codes * B / 8;
};

// Index in the group of the code in byte j of ordered word c.
template <int B, bool PAIRED>
__host__ __device__ constexpr int ordered_code(int c, int j) {
  constexpr int U = Unit<B>::codes;
  if (!PAIRED) {
    const int block = c / U, in = c % U;             // four units in a row make a block of U words
    return 4 * U * block + U * j + in;
  }
  // bytes 0, 1: two units of the even stream, bytes 2, 3: of the odd one
  const int block = c / U, in = c % U;
  return 2 * (2 * U * block + U * (j & 1) + in) + (j >> 1);
}

// Plane P of block K: byte P of its four units.
template <int B, bool PAIRED, int K, int P>
__device__ __forceinline__ uint32_t plane(const uint32_t (&w)[B + 1]) {
  constexpr int S = Unit<B>::bytes;
  if constexpr (PAIRED) {
    constexpr int a = 2 * S * K + P, b = a + S;      // stream bytes of the two units
    constexpr uint32_t sel = (a & 1) | (((b & 1) + 4) << 4) | (((a & 1) + 2) << 8) | (((b & 1) + 6) << 12);
    return __byte_perm(w[a >> 1], w[b >> 1], sel);
  } else {
    constexpr int a = 4 * S * K + P, b = a + S, c = b + S, d = c + S;
    constexpr uint32_t s1 = (a & 3) | (((b & 3) + 4) << 4), s2 = (c & 3) | (((d & 3) + 4) << 4);
    return __byte_perm(__byte_perm(w[a >> 2], w[b >> 2], s1), __byte_perm(w[c >> 2], w[d >> 2], s2), 0x5410);
  }
}

// Code C of the units whose planes are given, at the top of each byte.
template <int B, int C, int S>
__device__ __forceinline__ uint32_t from_planes(const uint32_t (&pl)[S]) {
  constexpr int p = C * B >> 3, r = C * B & 7;
  if constexpr (r + B <= 8) {
    return shift<8 - B - r>(pl[p]) & Just<B>::kMask;
  } else {
    constexpr int low = 8 - r, high = B - low;       // bits in byte p and in byte p + 1
    constexpr uint32_t ml = (((1u << low) - 1u) << (8 - B)) * 0x01010101u;
    constexpr uint32_t mh = ((0xFFu << (8 - high)) & 0xFFu) * 0x01010101u;
    return (shift<8 - B - r>(pl[p]) & ml) | (shift<8 - high>(pl[p + 1]) & mh);
  }
}

template <int B, bool PAIRED, int K, int... P>
__device__ __forceinline__ void block_planes(const uint32_t (&w)[B + 1], uint32_t (&pl)[Unit<B>::bytes],
                                             std::integer_sequence<int, P...>) {
  ((pl[P] = plane<B, PAIRED, K, P>(w)), ...);
}

template <int B, int K, int... C>
__device__ __forceinline__ void block_codes(const uint32_t (&pl)[Unit<B>::bytes], uint32_t (&o)[8],
                                            std::integer_sequence<int, C...>) {
  ((o[K * Unit<B>::codes + C] = from_planes<B, C>(pl)), ...);
}

template <int B, bool PAIRED, int... K>
__device__ __forceinline__ void ordered_all(const uint32_t (&w)[B + 1], uint32_t (&o)[8],
                                            std::integer_sequence<int, K...>) {
  (([&] {
     uint32_t pl[Unit<B>::bytes];
     block_planes<B, PAIRED, K>(w, pl, std::make_integer_sequence<int, Unit<B>::bytes>{});
     block_codes<B, K>(pl, o, std::make_integer_sequence<int, Unit<B>::codes>{});
   }()),
   ...);
}

// One 32-code group -> 32 left-justified bytes, byte j of word c being code
// ordered_code<B, PAIRED>(c, j).
template <int B, bool PAIRED>
__device__ __forceinline__ void group_ordered(const uint32_t (&w)[B + 1], uint32_t (&o)[8]) {
  ordered_all<B, PAIRED>(w, o, std::make_integer_sequence<int, 8 / Unit<B>::codes>{});
}

// The bytes of x of one group (v in k order) in that order.
template <int B, bool PAIRED>
__device__ __forceinline__ void order_x(const uint32_t (&v)[8], uint32_t (&o)[8]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = ordered_code<B, PAIRED>(c, j);
      r |= ((v[k >> 2] >> (8 * (k & 3))) & 0xFFu) << (8 * j);
    }
    o[c] = r;
  }
}

}  // namespace i8
}  // namespace mpw

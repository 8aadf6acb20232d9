// bf16 weights s * q from exact bf16 codes, two at a time.
//
// s is split into two bf16 values, s = hi + lo up to 2^-16 of it, and
// s q = fma(q, hi, q lo) in bf16x2 arithmetic: the product with hi is exact inside
// the fma, so the result is s q rounded to bf16 once, from a value that is off by
// at most 2^-16 of itself.  Two operations a pair, where going through fp32
// takes five.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace mpw {
namespace dec {

__device__ __forceinline__ void split_scale(float s, uint32_t& hi2, uint32_t& lo2) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(s);
  const __nv_bfloat16 lo = __float2bfloat16_rn(s - __bfloat162float(hi));
  hi2 = static_cast<uint32_t>(__bfloat16_as_ushort(hi)) * 0x10001u;
  lo2 = static_cast<uint32_t>(__bfloat16_as_ushort(lo)) * 0x10001u;
}

__device__ __forceinline__ uint32_t scale_pair(uint32_t q, uint32_t hi2, uint32_t lo2) {
  const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&q);
  const __nv_bfloat162 r = __hfma2(v, *reinterpret_cast<const __nv_bfloat162*>(&hi2),
                                   __hmul2(v, *reinterpret_cast<const __nv_bfloat162*>(&lo2)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

}  // namespace dec
}  // namespace mpw

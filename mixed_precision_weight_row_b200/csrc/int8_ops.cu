// Per-token 8-bit activations, and the passes that lay operands out for the
// dense GEMMs of the int8 linear and of the gradients.
//
// The quantization tutorial's symmetric per-channel formula ("How quantization
// works") applied to each token with max_int = 127: sx = max|x| / 127,
// xq = round(x / sx).  The codes are stored as canonical 8-bit packed rows, so
// mpw_unpack and mpw_dequantize read them, and they serve as the operand of
// the int8 product and as an 8-bit checkpoint of x for the backward pass.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "expand.cuh"
#include "int8_expand.cuh"
#include "int8_internal.h"
#include "lane_units.cuh"
#include "mpw_internal.h"
#include "scale_pair.cuh"
#include "tc_ptx.cuh"

namespace mpw {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_val(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

unsigned grid_for(int64_t work) {
  const int64_t blocks = (work + kThreads - 1) / kThreads;
  const int64_t cap = static_cast<int64_t>(device_info().num_sms) * 16;
  return static_cast<unsigned>(blocks < cap ? (blocks > 0 ? blocks : 1) : cap);
}

// xq = clamp(rint(fl32(x / s)), -127, 127), IEEE quotient, ties to even.
__device__ __forceinline__ uint32_t code8(float x, float s) {
  const int q = __float2int_rn(__fdiv_rn(x, s));
  return static_cast<uint32_t>(max(-127, min(127, q))) & 0xFFu;
}

// |x| as ordered integer bits: the maximum of these is the maximum magnitude,
// and a value above 0x7F80 (bf16 infinity) means a NaN was seen.
__device__ __forceinline__ uint32_t mag2(uint32_t v) { return v & 0x7FFF7FFFu; }

// One CTA per token.  Two passes over the row, the second from L1 / L2.  The
// next launch may start at once (the decode kernel reads weights before it waits
// for this one).
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
quantize_x_int8_kernel(const uint16_t* __restrict__ x, int K, int stride, uint8_t* __restrict__ xq,
                       float* __restrict__ sx) {
  ptx::grid_dep_wait_then_release();
  __shared__ uint32_t red[kThreads / 32];
  const size_t m = blockIdx.x;
  const uint16_t* row = x + m * static_cast<size_t>(K);
  uint32_t top = 0;   // two 16-bit maxima
  if constexpr (VEC) {
    const uint4* r8 = reinterpret_cast<const uint4*>(row);
    for (int i = threadIdx.x; i < (K >> 3); i += kThreads) {
      const uint4 v = __ldg(r8 + i);
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(mag2(v.x), mag2(v.y)), __vmaxu2(mag2(v.z), mag2(v.w))));
    }
  } else {
    for (int k = threadIdx.x; k < K; k += kThreads) top = __vmaxu2(top, row[k] & 0x7FFFu);
  }
  uint32_t mx = max(top & 0xFFFFu, top >> 16);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
  __syncthreads();
  mx = red[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) mx = max(mx, red[i]);
  const bool finite = mx < 0x7F80u;
  const float amax = __uint_as_float(mx << 16);
  // a token with an infinity or NaN: scale NaN, codes 0, so that what is computed from it is NaN
  const float s = !finite ? __uint_as_float(0x7FC00000u) : __fdiv_rn(mx == 0 ? 1.0f : amax, 127.0f);
  if (threadIdx.x == 0) sx[m] = s;
  uint8_t* out = xq + m * static_cast<size_t>(stride);
  if constexpr (VEC) {
    const uint4* r8 = reinterpret_cast<const uint4*>(row);
    uint2* o8 = reinterpret_cast<uint2*>(out);
    for (int i = threadIdx.x; i < (stride >> 3); i += kThreads) {
      uint2 o = make_uint2(0u, 0u);
      if (finite && i < (K >> 3)) {
        const uint4 v = __ldg(r8 + i);
        o.x = code8(bf16_lo(v.x), s) | (code8(bf16_hi(v.x), s) << 8) | (code8(bf16_lo(v.y), s) << 16) |
              (code8(bf16_hi(v.y), s) << 24);
        o.y = code8(bf16_lo(v.z), s) | (code8(bf16_hi(v.z), s) << 8) | (code8(bf16_lo(v.w), s) << 16) |
              (code8(bf16_hi(v.w), s) << 24);
      }
      o8[i] = o;
    }
  } else {
    for (int k = threadIdx.x; k < stride; k += kThreads)
      out[k] = finite && k < K ? static_cast<uint8_t>(code8(bf16_val(row[k]), s)) : 0;
  }
}

// Words of the 32-code group g of a row (words past the row read as zero).
template <int B>
__device__ __forceinline__ void load_group(const uint32_t* row, int g, int rw, uint32_t (&w)[B + 1]) {
#pragma unroll
  for (int i = 0; i < B; ++i) w[i] = g * B + i < rw ? __ldg(row + g * B + i) : 0u;
  w[B] = 0u;
}

// The group of element idx of N x G, or nothing past the end.
struct Group {
  int64_t n;
  int g;
  bool in;
  __device__ Group(int64_t idx, int64_t total, int G) : n(idx / G), g(static_cast<int>(idx - n * G)), in(idx < total) {}
};

// Stores U 16-byte units per lane to its own dst (units q < have); the lanes of a
// group of U change units first, so that they write one lane's units side by
// side (a lane writing its own leaves half a sector at a time).
template <int U>
__device__ __forceinline__ void store_units(uint32_t (&o)[4 * U], uint4* dst, int have, int lane) {
  transpose_units<U, 4>(o, lane);
  const int q = lane % U, base = lane - q;
#pragma unroll
  for (int t = 0; t < U; ++t) {
    uint4* d = reinterpret_cast<uint4*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), base + t));
    const int h = __shfl_sync(0xffffffffu, have, base + t);
    if (q < h) d[q] = make_uint4(o[4 * t], o[4 * t + 1], o[4 * t + 2], o[4 * t + 3]);
  }
}

// One thread per (row, 32-code group); whole warps stay in the loop.
template <int B, bool PAIRED>
__global__ void __launch_bounds__(kThreads)
expand_i8_kernel(const uint32_t* __restrict__ packed, int64_t N, int G, int rw, int stride,
                 uint8_t* __restrict__ out) {
  const int64_t total = N * G;
  const int lane = threadIdx.x & 31;
  for (int64_t w0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x - lane; w0 < total;
       w0 += static_cast<int64_t>(gridDim.x) * kThreads) {
    const Group e(w0 + lane, total, G);
    uint32_t w[B + 1] = {}, o[8];
    if (e.in) load_group<B>(packed + e.n * rw, e.g, rw, w);
    i8::group<B, PAIRED>(w, o);
    uint4* dst = reinterpret_cast<uint4*>(out + e.n * stride + 32 * static_cast<int64_t>(e.g));
    store_units<2>(o, dst, !e.in ? 0 : (32 * e.g + 16 < stride ? 2 : 1), lane);
  }
}

template <int B, bool PAIRED>
__global__ void __launch_bounds__(kThreads)
expand_bf16_kernel(const uint32_t* __restrict__ packed, const float* __restrict__ scales, int64_t N, int G, int rw,
                   int stride, uint16_t* __restrict__ out) {
  constexpr int P = dec::GemmParts<B>::parts;
  const int64_t total = N * G;
  const int lane = threadIdx.x & 31;
  for (int64_t w0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x - lane; w0 < total;
       w0 += static_cast<int64_t>(gridDim.x) * kThreads) {
    const Group e(w0 + lane, total, G);
    uint32_t w[B + 1] = {}, v[P][16], o[16];
    if (e.in) load_group<B>(packed + e.n * rw, e.g, rw, w);
    dec::gemm_expand_group<B, PAIRED>(w, v);
    const float s = e.in ? __ldg(scales + e.n) : 0.0f;
    uint32_t hi, lo;
    dec::split_scale(s, hi, lo);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (P == 1) {
        o[i] = dec::scale_pair(v[0][i], hi, lo);
      } else {
        // the parts' sum is exact in fp32: the code has at most 15 bits
        const __nv_bfloat162 r = __floats2bfloat162_rn((bf16_lo(v[0][i]) + bf16_lo(v[1][i])) * s,
                                                       (bf16_hi(v[0][i]) + bf16_hi(v[1][i])) * s);
        o[i] = *reinterpret_cast<const uint32_t*>(&r);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(out + e.n * stride + 32 * static_cast<int64_t>(e.g));
    store_units<4>(o, dst, e.in ? min(4, (stride - 32 * e.g) >> 3) : 0, lane);
  }
}

// One thread per (token, 8 codes).
template <int PARTS>
__global__ void __launch_bounds__(kThreads)
expand_x_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ sx, int64_t M, int xstride, int stride,
                uint16_t* __restrict__ out) {
  const int G = stride >> 3;
  const int64_t total = M * G;
  for (int64_t idx = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; idx < total;
       idx += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t m = idx / G;
    const int g = static_cast<int>(idx - m * G);
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(xq + m * xstride) + g);
    const float s = __ldg(sx + m);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = i < 2 ? v.x : v.y;
      const int sh = 16 * (i & 1);
      const float a = s * static_cast<float>(static_cast<int8_t>(u >> sh));
      const float b = s * static_cast<float>(static_cast<int8_t>(u >> (sh + 8)));
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      hi[i] = *reinterpret_cast<const uint32_t*>(&h);
      if constexpr (PARTS == 2) {
        const __nv_bfloat162 l = __floats2bfloat162_rn(a - bf16_lo(hi[i]), b - bf16_hi(hi[i]));
        lo[i] = *reinterpret_cast<const uint32_t*>(&l);
      }
    }
    reinterpret_cast<uint4*>(out + m * stride)[g] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if constexpr (PARTS == 2)
      reinterpret_cast<uint4*>(out + (M + m) * stride)[g] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

__global__ void __launch_bounds__(kThreads)
pad_bf16_kernel(const uint16_t* __restrict__ in, int64_t rows, int cols, int stride, uint16_t* __restrict__ out) {
  const int G = stride >> 3;
  const int64_t total = rows * G;
  for (int64_t idx = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; idx < total;
       idx += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t r = idx / G;
    const int g = static_cast<int>(idx - r * G);
    const uint16_t* src = in + r * cols + 8 * static_cast<int64_t>(g);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = 8 * g + 2 * i < cols ? __ldg(src + 2 * i) : 0u;
      const uint32_t b = 8 * g + 2 * i + 1 < cols ? __ldg(src + 2 * i + 1) : 0u;
      o[i] = a | (b << 16);
    }
    reinterpret_cast<uint4*>(out + r * stride)[g] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int B>
cudaError_t run_expand_i8(const uint8_t* packed, int64_t N, int64_t K, int layout, uint8_t* out,
                          cudaStream_t stream) {
  const int G = static_cast<int>((K + 31) / 32), rw = static_cast<int>(row_words(K, B));
  const int stride = static_cast<int>(stride_i8(K));
  const uint32_t* src = reinterpret_cast<const uint32_t*>(packed);
  if (layout == kLayoutPaired)
    expand_i8_kernel<B, true><<<grid_for(N * G), kThreads, 0, stream>>>(src, N, G, rw, stride, out);
  else
    expand_i8_kernel<B, false><<<grid_for(N * G), kThreads, 0, stream>>>(src, N, G, rw, stride, out);
  return cudaGetLastError();
}

template <int B>
cudaError_t run_expand_bf16(const uint8_t* packed, const float* scales, int64_t N, int64_t K, int layout,
                            uint16_t* out, cudaStream_t stream) {
  const int G = static_cast<int>((K + 31) / 32), rw = static_cast<int>(row_words(K, B));
  const int stride = static_cast<int>(stride_bf16(K));
  const uint32_t* src = reinterpret_cast<const uint32_t*>(packed);
  if (layout == kLayoutPaired)
    expand_bf16_kernel<B, true><<<grid_for(N * G), kThreads, 0, stream>>>(src, scales, N, G, rw, stride, out);
  else
    expand_bf16_kernel<B, false><<<grid_for(N * G), kThreads, 0, stream>>>(src, scales, N, G, rw, stride, out);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_x_int8(const uint16_t* x, int64_t M, int64_t K, uint8_t* xq, float* sx,
                                   cudaStream_t stream) {
  const int stride = static_cast<int>(stride_i8(K));
  if (K % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0)
    quantize_x_int8_kernel<true><<<static_cast<unsigned>(M), kThreads, 0, stream>>>(x, static_cast<int>(K), stride,
                                                                                    xq, sx);
  else
    quantize_x_int8_kernel<false><<<static_cast<unsigned>(M), kThreads, 0, stream>>>(x, static_cast<int>(K), stride,
                                                                                     xq, sx);
  return cudaGetLastError();
}

cudaError_t launch_expand_i8(const uint8_t* packed, int64_t N, int64_t K, int bits, int layout, uint8_t* out,
                             cudaStream_t stream) {
  switch (bits) {
    case 4: return run_expand_i8<4>(packed, N, K, layout, out, stream);
    case 5: return run_expand_i8<5>(packed, N, K, layout, out, stream);
    case 6: return run_expand_i8<6>(packed, N, K, layout, out, stream);
    case 7: return run_expand_i8<7>(packed, N, K, layout, out, stream);
    case 8: return run_expand_i8<8>(packed, N, K, layout, out, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_expand_bf16(const uint8_t* packed, const float* scales, int64_t N, int64_t K, int bits, int layout,
                               uint16_t* out, cudaStream_t stream) {
  switch (bits) {
    case 4: return run_expand_bf16<4>(packed, scales, N, K, layout, out, stream);
    case 5: return run_expand_bf16<5>(packed, scales, N, K, layout, out, stream);
    case 6: return run_expand_bf16<6>(packed, scales, N, K, layout, out, stream);
    case 7: return run_expand_bf16<7>(packed, scales, N, K, layout, out, stream);
    case 8: return run_expand_bf16<8>(packed, scales, N, K, layout, out, stream);
    case 9: return run_expand_bf16<9>(packed, scales, N, K, layout, out, stream);
    case 10: return run_expand_bf16<10>(packed, scales, N, K, layout, out, stream);
    case 11: return run_expand_bf16<11>(packed, scales, N, K, layout, out, stream);
    case 12: return run_expand_bf16<12>(packed, scales, N, K, layout, out, stream);
    case 13: return run_expand_bf16<13>(packed, scales, N, K, layout, out, stream);
    case 14: return run_expand_bf16<14>(packed, scales, N, K, layout, out, stream);
    case 15: return run_expand_bf16<15>(packed, scales, N, K, layout, out, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_expand_x(const uint8_t* xq, const float* sx, int64_t M, int64_t K, int parts, uint16_t* out,
                            cudaStream_t stream) {
  const int xstride = static_cast<int>(stride_i8(K)), stride = static_cast<int>(stride_bf16(K));
  const unsigned grid = grid_for(M * (stride / 8));
  if (parts == 2) expand_x_kernel<2><<<grid, kThreads, 0, stream>>>(xq, sx, M, xstride, stride, out);
  else expand_x_kernel<1><<<grid, kThreads, 0, stream>>>(xq, sx, M, xstride, stride, out);
  return cudaGetLastError();
}

cudaError_t launch_pad_bf16(const uint16_t* in, int64_t rows, int64_t cols, uint16_t* out, cudaStream_t stream) {
  const int stride = static_cast<int>(stride_bf16(cols));
  pad_bf16_kernel<<<grid_for(rows * (stride / 8)), kThreads, 0, stream>>>(in, rows, static_cast<int>(cols), stride,
                                                                        out);
  return cudaGetLastError();
}

}  // namespace mpw

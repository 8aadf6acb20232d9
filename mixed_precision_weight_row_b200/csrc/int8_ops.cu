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

// Block-wide maximum over T threads.
template <int T>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < T / 32 ? red[threadIdx.x & 31] : 0u);
}

// Scale of a token whose largest magnitude has the bf16 bits mx; NaN (and codes
// 0) with an infinity or NaN, so that what is computed from the token is NaN.
__device__ __forceinline__ float scale8(uint32_t mx) {
  if (mx >= 0x7F80u) return __uint_as_float(0x7FC00000u);
  return __fdiv_rn(mx == 0 ? 1.0f : __uint_as_float(mx << 16), 127.0f);
}

__device__ __forceinline__ uint2 codes8_exact(const uint4& v, float s) {
  return make_uint2(code8(bf16_lo(v.x), s) | (code8(bf16_hi(v.x), s) << 8) | (code8(bf16_lo(v.y), s) << 16) |
                        (code8(bf16_hi(v.y), s) << 24),
                    code8(bf16_lo(v.z), s) | (code8(bf16_hi(v.z), s) << 8) | (code8(bf16_lo(v.w), s) << 16) |
                        (code8(bf16_hi(v.w), s) << 24));
}

// The codes of eight values without a division where the nearest whole number is
// not in doubt: with r = fl32(1 / s), x r and fl32(x / s) are each within 2^-17 of
// x / s (|x / s| < 128, relative errors of 2^-24), so a whole number that x r is
// within 1/2 - 2^-14 of is the one nearest to both.  Closer to a tie (about 1 value
// in 8000) the quotient decides.  Needs a normal 1 / s.
__device__ __forceinline__ uint2 codes8(const uint4& v, float s, float r) {
  constexpr float kMagic = 12582912.0f;          // 1.5 * 2^23: adding it rounds to a whole number, in the low bits
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  float t[8], far = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = (i & 1) ? bf16_hi(u[i >> 1]) : bf16_lo(u[i >> 1]);
    t[i] = __fmaf_rn(x, r, kMagic);
    far = fmaxf(far, fabsf(__fmaf_rn(x, r, -(t[i] - kMagic))));
  }
  if (far > 0.5f - 0x1p-14f) return codes8_exact(v, s);
  uint32_t o[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    o[h] = __byte_perm(__byte_perm(__float_as_uint(t[4 * h]), __float_as_uint(t[4 * h + 1]), 0x0040),
                       __byte_perm(__float_as_uint(t[4 * h + 2]), __float_as_uint(t[4 * h + 3]), 0x0040), 0x5410);
  return make_uint2(o[0], o[1]);
}

// One CTA of T threads per token.  It never lets the next launch start ahead of
// its end: its results are packed rows and scales, which the kernels that take
// rows read before they wait.
// KEEP > 0: rows of whole 16-byte units, of which a thread keeps up to KEEP in
// registers between the maximum and the codes (one read of x); KEEP = 0: any rows,
// two passes, the second from L1 / L2.
template <int T, int KEEP>
__global__ void __launch_bounds__(T)
quantize_x_int8_kernel(const uint16_t* __restrict__ x, int K, int stride, uint8_t* __restrict__ xq,
                       float* __restrict__ sx) {
  __shared__ uint32_t red[T / 32];
  const size_t m = blockIdx.x;
  const uint16_t* row = x + m * static_cast<size_t>(K);
  uint8_t* out = xq + m * static_cast<size_t>(stride);
  if constexpr (KEEP > 0) {
    const uint4* r8 = reinterpret_cast<const uint4*>(row);
    uint4 v[KEEP];
    uint32_t top = 0;   // two 16-bit maxima
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
      const int i = threadIdx.x + j * T;
      v[j] = i < (K >> 3) ? __ldg(r8 + i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(mag2(v[j].x), mag2(v[j].y)), __vmaxu2(mag2(v[j].z), mag2(v[j].w))));
    const uint32_t mx = block_max<T>(max(top & 0xFFFFu, top >> 16), red);
    const float s = scale8(mx);
    if (threadIdx.x == 0) sx[m] = s;
    const bool plain = s > 0x1p-120f;      // 1 / s is far from overflow (false for NaN)
    const float r = plain ? __fdiv_rn(1.0f, s) : 0.0f;
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
      const int i = threadIdx.x + j * T;
      if (i >= (stride >> 3)) continue;      // zeros past K give the zero padding
      reinterpret_cast<uint2*>(out)[i] =
          plain ? codes8(v[j], s, r) : (mx < 0x7F80u ? codes8_exact(v[j], s) : make_uint2(0u, 0u));
    }
  } else {
    uint32_t top = 0;
    for (int k = threadIdx.x; k < K; k += T) top = max(top, row[k] & 0x7FFFu);
    const uint32_t mx = block_max<T>(top, red);
    const float s = scale8(mx);
    if (threadIdx.x == 0) sx[m] = s;
    for (int k = threadIdx.x; k < stride; k += T)
      out[k] = mx < 0x7F80u && k < K ? static_cast<uint8_t>(code8(bf16_val(row[k]), s)) : 0;
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
  ptx::grid_dep_wait_then_release();
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
  ptx::grid_dep_wait_then_release();
  const int64_t total = N * G;
  const int lane = threadIdx.x & 31;
  for (int64_t w0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x - lane; w0 < total;
       w0 += static_cast<int64_t>(gridDim.x) * kThreads) {
    const Group e(w0 + lane, total, G);
    uint32_t w[B + 1] = {}, o[16];
    if (e.in) load_group<B>(packed + e.n * rw, e.g, rw, w);
    const float s = e.in ? __ldg(scales + e.n) : 0.0f;
    if constexpr (B <= 9) {
      dec::scaled_group<B, PAIRED>(w, dec::split_scale<B>(s), o);
    } else {
      uint32_t v[2][16];
      dec::gemm_expand_group<B, PAIRED>(w, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        // the parts' sum is exact in fp32: the code has at most 15 bits (and the
        // product rounded once, to the bf16 that the tensor cores multiply)
        const __nv_bfloat162 r = __floats2bfloat162_rn((bf16_lo(v[0][i]) + bf16_lo(v[1][i])) * s,
                                                       (bf16_hi(v[0][i]) + bf16_hi(v[1][i])) * s);
        o[i] = *reinterpret_cast<const uint32_t*>(&r);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(out + e.n * stride + 32 * static_cast<int64_t>(e.g));
    store_units<4>(o, dst, e.in ? min(4, (stride - 32 * e.g) >> 3) : 0, lane);
  }
}

// a as three bf16 values of its sign, all 24 bits of it (in steps of 2^-133, the
// smallest bf16): the first 8 bits, the next 8, the rest.  Where a part would be
// zero the part before it gives up its last step, so that none is (from 2^-124
// on): the sum over the parts of an infinite dy times each must be an infinity,
// not inf - inf or inf * 0.
__device__ __forceinline__ void split3(float a, float (&part)[3]) {
  uint32_t h = __float_as_uint(a) & 0xFFFF0000u;
  float rest = a - __uint_as_float(h);
  if (fabsf(rest) < 0x1p-132f && (h << 1) != 0u) {
    h -= 0x10000u;
    rest = a - __uint_as_float(h);
  }
  uint32_t m = __float_as_uint(rest) & 0xFFFF0000u;
  float last = rest - __uint_as_float(m);
  if (fabsf(last) < 0x1p-133f && (m << 1) != 0u) {
    m -= 0x10000u;
    last = rest - __uint_as_float(m);
  }
  part[0] = __uint_as_float(h);
  part[1] = __uint_as_float(m);
  part[2] = last;
}

// One thread per (token, 8 codes).  One part: sx xq rounded to bf16, what the
// tensor cores multiply (off by at most 2^-8 of it, as the bf16 result once more).
template <int PARTS>
__global__ void __launch_bounds__(kThreads)
expand_x_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ sx, int64_t M, int xstride, int stride,
                uint16_t* __restrict__ out) {
  ptx::grid_dep_wait_then_release();
  const int G = stride >> 3;
  const int64_t total = M * G;
  for (int64_t idx = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; idx < total;
       idx += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t m = idx / G;
    const int g = static_cast<int>(idx - m * G);
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(xq + m * xstride) + g);
    const float s = __ldg(sx + m);
    uint32_t part[PARTS][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = i < 2 ? v.x : v.y;
      const int sh = 16 * (i & 1);
      float a[PARTS], b[PARTS];
      a[0] = s * static_cast<float>(static_cast<int8_t>(u >> sh));
      b[0] = s * static_cast<float>(static_cast<int8_t>(u >> (sh + 8)));
      if constexpr (PARTS == 3) {
        split3(a[0], a);
        split3(b[0], b);
      }
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a[p], b[p]);
        part[p][i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
      reinterpret_cast<uint4*>(out + (p * M + m) * stride)[g] =
          make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
  }
}

__global__ void __launch_bounds__(kThreads)
pad_bf16_kernel(const uint16_t* __restrict__ in, int64_t rows, int cols, int stride, uint16_t* __restrict__ out) {
  ptx::grid_dep_wait_then_release();
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
    return launch_behind(expand_i8_kernel<B, true>, grid_for(N * G), kThreads, 0, stream, src, N, G, rw, stride, out);
  return launch_behind(expand_i8_kernel<B, false>, grid_for(N * G), kThreads, 0, stream, src, N, G, rw, stride, out);
}

template <int B>
cudaError_t run_expand_bf16(const uint8_t* packed, const float* scales, int64_t N, int64_t K, int layout,
                            uint16_t* out, cudaStream_t stream) {
  const int G = static_cast<int>((K + 31) / 32), rw = static_cast<int>(row_words(K, B));
  const int stride = static_cast<int>(stride_bf16(K));
  const uint32_t* src = reinterpret_cast<const uint32_t*>(packed);
  if (layout == kLayoutPaired)
    return launch_behind(expand_bf16_kernel<B, true>, grid_for(N * G), kThreads, 0, stream, src, scales, N, G, rw,
                         stride, out);
  return launch_behind(expand_bf16_kernel<B, false>, grid_for(N * G), kThreads, 0, stream, src, scales, N, G, rw,
                       stride, out);
}

}  // namespace

cudaError_t launch_quantize_x_int8(const uint16_t* x, int64_t M, int64_t K, uint8_t* xq, float* sx,
                                   cudaStream_t stream) {
  const int stride = static_cast<int>(stride_i8(K)), k = static_cast<int>(K);
  const unsigned grid = static_cast<unsigned>(M);
  const int units = stride / 8;                    // 16-byte units of x, the padding's included
  const bool whole = K % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
  // as few threads as hold a row in few registers (one B200, 2048 x 5120: 256 threads
  // x 3 units 10.0 us, 512 x 2 11.3, 1024 x 1 15.6; 2048 x 17408: 512 x 5 30.7 us, 1024
  // x 3 44.7), more where a token's latency is what counts (1 x 5120: 512 x 2 3.1 us,
  // 256 x 3 3.4)
  if (whole && units <= 256 * 3 && M >= device_info().num_sms)
    quantize_x_int8_kernel<256, 3><<<grid, 256, 0, stream>>>(x, k, stride, xq, sx);
  else if (whole && units <= 512 * 2)
    quantize_x_int8_kernel<512, 2><<<grid, 512, 0, stream>>>(x, k, stride, xq, sx);
  else if (whole && units <= 512 * 5)
    quantize_x_int8_kernel<512, 5><<<grid, 512, 0, stream>>>(x, k, stride, xq, sx);
  else if (whole && units <= 1024 * 8)
    quantize_x_int8_kernel<1024, 8><<<grid, 1024, 0, stream>>>(x, k, stride, xq, sx);
  else
    quantize_x_int8_kernel<256, 0><<<grid, 256, 0, stream>>>(x, k, stride, xq, sx);
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
  auto kern = parts == 3 ? expand_x_kernel<3> : expand_x_kernel<1>;
  return launch_behind(kern, grid, kThreads, 0, stream, xq, sx, M, xstride, stride, out);
}

cudaError_t launch_pad_bf16(const uint16_t* in, int64_t rows, int64_t cols, uint16_t* out, cudaStream_t stream) {
  const int stride = static_cast<int>(stride_bf16(cols));
  return launch_behind(pad_bf16_kernel, grid_for(rows * (stride / 8)), kThreads, 0, stream, in, rows,
                       static_cast<int>(cols), stride, out);
}

}  // namespace mpw

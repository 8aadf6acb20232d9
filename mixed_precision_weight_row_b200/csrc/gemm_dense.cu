// Dense products behind the int8 linear and the gradients.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "int8_internal.h"
#include "mpw_internal.h"

namespace mpw {
namespace {

constexpr int T = 32;   // tile edge and depth

__device__ __forceinline__ float bf16_val(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// c[i, j] = sum_r a(i, r) b(j, r), a 32 x 32 tile per block, operands through shared memory.
template <typename Acc, typename LoadA, typename LoadB, typename Store>
__device__ __forceinline__ void tile_product(int64_t I, int64_t J, int64_t R, LoadA la, LoadB lb, Store store) {
  __shared__ Acc sa[T][T + 1], sb[T][T + 1];
  const int64_t jt = (J + T - 1) / T, tiles = jt * ((I + T - 1) / T);
  const int tx = threadIdx.x, ty = threadIdx.y;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t i0 = t / jt * T, j0 = t % jt * T;
    Acc acc[4] = {0, 0, 0, 0};
    for (int64_t r0 = 0; r0 < R; r0 += T) {
      for (int y = ty; y < T; y += 8) {
        sa[y][tx] = la(i0 + y, r0 + tx);
        sb[y][tx] = lb(j0 + y, r0 + tx);
      }
      __syncthreads();
      for (int r = 0; r < T; ++r)
        for (int u = 0; u < 4; ++u) acc[u] += sa[ty + 8 * u][r] * sb[tx][r];
      __syncthreads();
    }
    for (int u = 0; u < 4; ++u)
      if (i0 + ty + 8 * u < I && j0 + tx < J) store(i0 + ty + 8 * u, j0 + tx, acc[u]);
  }
}

__global__ void dense_i8_kernel(const int8_t* a, const int8_t* b, const float* sx, const float* scales, int shift,
                                int64_t M, int64_t N, int64_t K, int64_t stride, uint16_t* y) {
  tile_product<int32_t>(
      M, N, K, [&](int64_t m, int64_t k) { return m < M && k < K ? int32_t(a[m * stride + k]) : 0; },
      [&](int64_t n, int64_t k) { return n < N && k < K ? int32_t(b[n * stride + k]) : 0; },
      [&](int64_t m, int64_t n, int32_t v) {
        y[m * N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(static_cast<float>(v >> shift) * scales[n] * sx[m]));
      });
}

__global__ void dense_grad_x_kernel(const uint16_t* dy, const uint16_t* w, int64_t M, int64_t N, int64_t K,
                                    int64_t ys, int64_t ws, uint16_t* dx) {
  tile_product<float>(
      M, K, N, [&](int64_t m, int64_t n) { return m < M && n < N ? bf16_val(dy[m * ys + n]) : 0.0f; },
      [&](int64_t k, int64_t n) { return k < K && n < N ? bf16_val(w[n * ws + k]) : 0.0f; },
      [&](int64_t m, int64_t k, float v) { dx[m * K + k] = __bfloat16_as_ushort(__float2bfloat16_rn(v)); });
}

__global__ void dense_grad_w_kernel(const uint16_t* dy, const uint16_t* x, int parts, int64_t M, int64_t N, int64_t K,
                                    int64_t ys, int64_t xs, void* dw, bool f32, bool accumulate) {
  tile_product<float>(
      N, K, parts * M,
      [&](int64_t n, int64_t m) { return n < N && m < parts * M ? bf16_val(dy[m % M * ys + n]) : 0.0f; },
      [&](int64_t k, int64_t m) { return k < K && m < parts * M ? bf16_val(x[m * xs + k]) : 0.0f; },
      [&](int64_t n, int64_t k, float v) {
        if (f32) {
          float* p = static_cast<float*>(dw) + n * K + k;
          *p = accumulate ? *p + v : v;
        } else {
          static_cast<uint16_t*>(dw)[n * K + k] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        }
      });
}

unsigned grid_for_tiles(int64_t I, int64_t J) {
  const int64_t tiles = ((I + T - 1) / T) * ((J + T - 1) / T);
  return static_cast<unsigned>(tiles < 65535 ? tiles : 65535);
}

}  // namespace

cudaError_t launch_dense_i8(const uint8_t* a, const uint8_t* b, const float* sx, const float* scales, int shift,
                            int64_t M, int64_t N, int64_t K, uint16_t* y, cudaStream_t stream) {
  dense_i8_kernel<<<grid_for_tiles(M, N), dim3(T, 8), 0, stream>>>(
      reinterpret_cast<const int8_t*>(a), reinterpret_cast<const int8_t*>(b), sx, scales, shift, M, N, K,
      stride_i8(K), y);
  return cudaGetLastError();
}

cudaError_t launch_dense_grad_x(const uint16_t* dy, const uint16_t* w, int64_t M, int64_t N, int64_t K, uint16_t* dx,
                                cudaStream_t stream) {
  dense_grad_x_kernel<<<grid_for_tiles(M, K), dim3(T, 8), 0, stream>>>(dy, w, M, N, K, stride_bf16(N), stride_bf16(K),
                                                                      dx);
  return cudaGetLastError();
}

cudaError_t launch_dense_grad_w(const uint16_t* dy, const uint16_t* x, int parts, int64_t M, int64_t N, int64_t K,
                                void* dw, bool f32, bool accumulate, cudaStream_t stream) {
  dense_grad_w_kernel<<<grid_for_tiles(N, K), dim3(T, 8), 0, stream>>>(dy, x, parts, M, N, K, stride_bf16(N),
                                                                      stride_bf16(K), dw, f32, accumulate);
  return cudaGetLastError();
}

}  // namespace mpw

// Internal declarations of the int8 linear and of the gradients of packed
// linears.  As in mpw_internal.h, the C-ABI layer has checked every argument.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mpw {

// Largest K of an int8 product: 128 * 127 * K < 2^31.
constexpr int64_t kInt8MaxK = 131071;

// Row strides of the operands the dense GEMM reads by TMA: whole 16 bytes.
inline int64_t stride_i8(int64_t K) { return (K + 15) / 16 * 16; }   // bytes
inline int64_t stride_bf16(int64_t K) { return (K + 7) / 8 * 8; }    // elements

// Launches a kernel that may start while the one before it on the stream ends
// (programmatic dependent launch): it waits for it (griddepcontrol.wait) before
// it reads results or writes anything.  (One B200, the weight gradient's two
// kernels, us: 64 x 4096 x 4096 11.9 against 13.6, 64 x 17408 x 5120 36.1 / 37.5.
// Not for gradx_kernel, whose early CTAs would take their weights from the CTAs
// still at work: 5120 x 6144 64 tokens 19.2 / 20.9, but 4096 x 4096 768 tokens
// 34.5 / 29.4.)
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// int8_ops.cu
cudaError_t launch_quantize_x_int8(const uint16_t* x, int64_t M, int64_t K, uint8_t* xq, float* sx,
                                   cudaStream_t stream);
// Packed rows (4..8 bits) -> left-justified bytes, rows of stride_i8(K).
cudaError_t launch_expand_i8(const uint8_t* packed, int64_t N, int64_t K, int bits, int layout, uint8_t* out,
                             cudaStream_t stream);
// Packed rows (4..15 bits) -> bf16_rn(s_n * q), rows of stride_bf16(K).
cudaError_t launch_expand_bf16(const uint8_t* packed, const float* scales, int64_t N, int64_t K, int bits,
                               int layout, uint16_t* out, cudaStream_t stream);
// 8-bit activations -> bf16 rows of stride_bf16(K): bf16_rn(sx * xq), or, with
// parts == 3, three blocks of M rows whose sum is fl32(sx * xq): its first 8
// bits, the next 8 and the rest, all of its sign.
cudaError_t launch_expand_x(const uint8_t* xq, const float* sx, int64_t M, int64_t K, int parts, uint16_t* out,
                            cudaStream_t stream);
// bf16 [rows, cols] -> the same with rows of stride_bf16(cols).
cudaError_t launch_pad_bf16(const uint16_t* in, int64_t rows, int64_t cols, uint16_t* out, cudaStream_t stream);

// gemv_int8.cu: the int8 linear for up to 4 tokens, packed rows streamed once;
// for shapes whose x and the slots of eight warps fit in shared memory.
bool gemv_i8_fits(int bits, int64_t M, int64_t K);
cudaError_t launch_gemv_i8(const uint8_t* xq, const float* sx, const uint8_t* packed, const float* scales, int bits,
                           int layout, int64_t M, int64_t N, int64_t K, uint16_t* y, cudaStream_t stream);

// gemm_int8.cu: the int8 linear with packed rows expanded on the way to the
// tensor cores, in tiles of up to 256 tokens.
bool gemm_i8_fits(int64_t M, int64_t N);
cudaError_t launch_gemm_i8(const uint8_t* xq, const float* sx, const uint8_t* packed, const float* scales, int bits,
                           int layout, int64_t M, int64_t N, int64_t K, uint16_t* y, cudaStream_t stream);

// gradx_fused.cu: the gradient of x for up to a few hundred tokens, packed rows
// expanded on the way to the tensor cores; dy rows of stride_bf16(N).
bool gradx_fused_fits(int bits, int64_t M, int64_t N, int64_t K);
cudaError_t launch_gradx_fused(const uint16_t* dy, const uint8_t* packed, const float* scales, int bits, int layout,
                               int64_t M, int64_t N, int64_t K, uint16_t* dx, cudaStream_t stream);

// gemm_dense.cu: products of operands laid out for TMA (rows of a stride that
// is a multiple of 16 bytes, 16-byte aligned).
//   y[m, n] = bf16(s_n * sx_m * (sum_k a[m, k] b[n, k]) / 2^shift), a and b signed bytes
cudaError_t launch_dense_i8(const uint8_t* a, const uint8_t* b, const float* sx, const float* scales, int shift,
                            int64_t M, int64_t N, int64_t K, uint16_t* y, cudaStream_t stream);
// The gradients take a workspace (dense_workspace_bytes of the result's rows
// and columns, of the length of the summed axis and of the parts of x;
// unprepared).
size_t dense_workspace_bytes(int64_t I, int64_t J, int64_t depth, int parts);
//   dx[m, k] = bf16(sum_n dy[m, n] w[n, k])
cudaError_t launch_dense_grad_x(const uint16_t* dy, const uint16_t* w, int64_t M, int64_t N, int64_t K, uint16_t* dx,
                                void* ws, cudaStream_t stream);
//   dw[n, k] (+)= sum_m dy[m, n] (x[m, k] [+ x[M + m, k] + x[2 M + m, k] with parts == 3])
cudaError_t launch_dense_grad_w(const uint16_t* dy, const uint16_t* x, int parts, int64_t M, int64_t N, int64_t K,
                                void* dw, bool f32, bool accumulate, void* ws, cudaStream_t stream);

}  // namespace mpw

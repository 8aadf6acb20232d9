// C ABI of the int8 linear and of the gradients of packed linears: argument
// validation, workspace layout and kernel dispatch.  See mpw.h for the
// contract of every entry point.
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "int8_internal.h"
#include "mpw.h"
#include "mpw_internal.h"

using namespace mpw;

namespace {

constexpr int64_t kMaxDim = 0x3fffffff;   // rows, columns and tokens (tensor-map coordinates are 32-bit)

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
mpw_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MPW_OK : MPW_E_CUDA; }
bool layout_ok(int layout) { return layout == MPW_LAYOUT_CANONICAL || layout == MPW_LAYOUT_PAIRED; }
bool bits_ok(int bits, int most) { return bits >= kMinBits && bits <= most; }
bool dims_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 1 && N >= 1 && K >= 1 && M <= kMaxDim && N <= kMaxDim && K <= kMaxDim;
}
// Result tiles are counted in 32 bits: up to 2^44 results, far beyond any memory.
bool result_ok(int64_t I, int64_t J) { return I <= (int64_t{1} << 44) / J; }
size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

// Memory of an argument, and whether `out` shares no byte with any of the others.
struct Span {
  const void* p;
  size_t bytes;
};
bool apart(const Span& out, std::initializer_list<Span> others) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(out.p);
  for (const Span& o : others) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(o.p);
    if (out.bytes != 0 && o.bytes != 0 && a < b + o.bytes && b < a + out.bytes) return false;
  }
  return true;
}
Span span(const void* p, int64_t rows, int64_t row_bytes) {
  return {p, static_cast<size_t>(rows) * static_cast<size_t>(row_bytes)};
}
Span rows_span(const uint8_t* packed, int bits, int64_t N, int64_t K) { return span(packed, N, 4 * row_words(K, bits)); }

// Canonical 8-bit rows already are rows of signed bytes.
bool rows_are_bytes(int bits, int layout) { return bits == 8 && layout == MPW_LAYOUT_CANONICAL; }

// How a call of the int8 linear runs: a few tokens on the kernel that streams
// packed rows, up to a thousand on the one that expands them on the way to the
// tensor cores, more on expanded rows (the only one that takes a workspace).
// One B200, us: 5120 x 6144, b = 6: 4 tokens 9.6 / 10.4 (first / second);
// 5120 x 17408, b = 5: 2 tokens 14.7 / 19.5, 4 tokens 26.8 / 19.5; 17408 x 5120,
// b = 8: 4 tokens 20.1 / 17.3.  b = 6, second / third: 512 tokens 17408 x 5120
// 51 / 66, 5120 x 6144 22 / 26; 1024 tokens 93 / 85, 42 / 36, 4096 x 4096 18 / 21,
// 1024 x 17408 22 / 30 (mixed there); 1280 tokens 111 / 97, 44 / 37, 33 / 25.  Rows that already are bytes need no
// expansion: 5120 x 6144, b = 8: 128 tokens 12.7 / 14.0, 256 tokens 16.6 / 14.1, 512
// tokens 20.6 / 17.9.
// The third kernel sums a tile's K in one place, so the second, which shares it
// among four SMs, goes on where there are few tiles (256 tokens x 128 rows):
// b = 6, 256 x 17408, 1025 tokens (10 tiles) 15.2 / 25.9, 4096 (32) 22.2 / 28.7, 8192
// (64) 41.5 / 38.3; 512 x 5120, 2048 (32) 12.9 / 13.3, 4096 (64) 16.6 / 14.9; 128 x 4096,
// 8192 (32) 11.6 / 10.9.  Bytes, if K is long enough to share: 256 x 17408, 193 tokens
// (2 tiles) 10.6 / 25.4; 128 x 4096, 193 (1) 7.3 / 8.5; 512 x 5120, 1024 (16)
// 9.9 / 10.7, 2048 (32) 11.3 / 10.7; but 512 x 2560, 193 (4) 8.1 / 7.2.
enum class Int8Path { kGemv, kFused, kDense };
Int8Path int8_path(int bits, int layout, int64_t M, int64_t N, int64_t K) {
  if ((M <= 2 || (M <= 4 && K <= 8192 && bits <= 7)) && gemv_i8_fits(bits, M, K)) return Int8Path::kGemv;
  if (!gemm_i8_fits(M, N)) return Int8Path::kDense;
  const int64_t tiles = ((M + 255) / 256) * ((N + 127) / 128);
  const bool fused = rows_are_bytes(bits, layout) ? M <= 192 || (K >= 4096 && tiles <= 16) : M <= 1024 || tiles <= 32;
  return fused ? Int8Path::kFused : Int8Path::kDense;
}

// Room for the expanded rows of the int8 linear.
size_t int8_rows_bytes(int bits, int layout, int64_t N, int64_t K) {
  return rows_are_bytes(bits, layout) ? 0 : round256(static_cast<size_t>(N) * static_cast<size_t>(stride_i8(K)));
}

size_t expanded_bf16_bytes(int64_t rows, int64_t cols) {
  return round256(static_cast<size_t>(rows) * static_cast<size_t>(stride_bf16(cols)) * 2);
}

// TMA reads rows of whole 16 bytes: dy is copied to padded rows when N % 8 != 0.
size_t padded_dy_bytes(int64_t M, int64_t N) { return N % 8 == 0 ? 0 : expanded_bf16_bytes(M, N); }
bool dy_aligned(const uint16_t* dy, int64_t N) { return aligned(dy, N % 8 == 0 ? 16 : 2); }
mpw_status padded_dy(const uint16_t** dy, int64_t M, int64_t N, uint8_t* room, cudaStream_t s) {
  if (N % 8 == 0) return MPW_OK;
  uint16_t* out = reinterpret_cast<uint16_t*>(room);
  const mpw_status st = from_cuda(launch_pad_bf16(*dy, M, N, out, s));
  *dy = out;
  return st;
}

// How grad_x runs: rows expanded on the way to the tensor cores, or first.  One
// B200, us, b = 6: 256 tokens 17408 x 5120 47 / 90, 4096 x 4096 18 / 26; 768 tokens
// 112 / 138, 31 / 33, 5120 x 6144 41 / 47; 1024 tokens 174 / 165, 32 / 33, 71 / 63.
bool gradx_fused(int bits, int64_t M, int64_t N, int64_t K) { return M <= 768 && gradx_fused_fits(bits, M, N, K); }

}  // namespace

extern "C" {

mpw_status mpw_quantize_x_int8(const uint16_t* x, int64_t M, int64_t K, uint8_t* xq, float* sx, mpw_stream_t stream) {
  if (x == nullptr || xq == nullptr || sx == nullptr || !dims_ok(M, 1, K)) return MPW_E_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(xq, 16) || !aligned(sx, 4)) return MPW_E_MISALIGNED;
  const Span in = span(x, M, 2 * K), scales = span(sx, M, 4);
  if (!apart(scales, {in}) || !apart(span(xq, M, stride_i8(K)), {in, scales})) return MPW_E_INVALID_ARG;
  return from_cuda(launch_quantize_x_int8(x, M, K, xq, sx, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mpw_qlinear_int8_workspace_bytes(int bits, int layout, int64_t M, int64_t N, int64_t K) {
  if (!bits_ok(bits, 8) || !layout_ok(layout) || !dims_ok(M, N, K) || K > kInt8MaxK) return 0;
  return int8_path(bits, layout, M, N, K) == Int8Path::kDense ? int8_rows_bytes(bits, layout, N, K) : 0;
}

mpw_status mpw_qlinear_int8(const uint8_t* xq, const float* sx, const uint8_t* packed, const float* scales, int bits,
                            int layout, int64_t M, int64_t N, int64_t K, uint16_t* y, void* workspace,
                            size_t workspace_bytes, mpw_stream_t stream) {
  if (!bits_ok(bits, 8)) return MPW_E_UNSUPPORTED_BITS;
  if (xq == nullptr || sx == nullptr || packed == nullptr || scales == nullptr || y == nullptr) return MPW_E_INVALID_ARG;
  if (!dims_ok(M, N, K) || K > kInt8MaxK || !layout_ok(layout) || !result_ok(M, N)) return MPW_E_INVALID_ARG;
  if (layout == MPW_LAYOUT_PAIRED && K % 32 != 0) return MPW_E_INVALID_ARG;
  if (!aligned(xq, 16) || !aligned(packed, 16) || !aligned(sx, 4) || !aligned(scales, 4) || !aligned(y, 2))
    return MPW_E_MISALIGNED;
  const size_t need = mpw_qlinear_int8_workspace_bytes(bits, layout, M, N, K);
  if (need != 0 && (workspace == nullptr || workspace_bytes < need)) return MPW_E_INVALID_ARG;
  if (need != 0 && !aligned(workspace, 16)) return MPW_E_MISALIGNED;
  const Span in[4] = {span(xq, M, stride_i8(K)), span(sx, M, 4), rows_span(packed, bits, N, K), span(scales, N, 4)};
  const Span scratch{workspace, need}, out = span(y, M, 2 * N);
  if (!apart(out, {in[0], in[1], in[2], in[3], scratch}) || !apart(scratch, {in[0], in[1], in[2], in[3]}))
    return MPW_E_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (int8_path(bits, layout, M, N, K)) {
    case Int8Path::kGemv: return from_cuda(launch_gemv_i8(xq, sx, packed, scales, bits, layout, M, N, K, y, s));
    case Int8Path::kFused: return from_cuda(launch_gemm_i8(xq, sx, packed, scales, bits, layout, M, N, K, y, s));
    case Int8Path::kDense: break;
  }
  uint8_t* rows = static_cast<uint8_t*>(workspace);
  if (need != 0) {
    const cudaError_t e = launch_expand_i8(packed, N, K, bits, layout, rows, s);
    if (e != cudaSuccess) return MPW_E_CUDA;
  }
  return from_cuda(launch_dense_i8(xq, need != 0 ? rows : packed, sx, scales, 8 - bits, M, N, K, y, s));
}

size_t mpw_qlinear_grad_x_workspace_bytes(int bits, int layout, int64_t M, int64_t N, int64_t K) {
  if (!bits_ok(bits, kMaxBits) || !layout_ok(layout) || !dims_ok(M, N, K)) return 0;
  if (gradx_fused(bits, M, N, K)) return padded_dy_bytes(M, N);
  return expanded_bf16_bytes(N, K) + padded_dy_bytes(M, N) + dense_workspace_bytes(M, K, N, 1);
}

mpw_status mpw_qlinear_grad_x(const uint16_t* dy, const uint8_t* packed, const float* scales, int bits, int layout,
                              int64_t M, int64_t N, int64_t K, uint16_t* dx, void* workspace, size_t workspace_bytes,
                              mpw_stream_t stream) {
  if (!bits_ok(bits, kMaxBits)) return MPW_E_UNSUPPORTED_BITS;
  if (dy == nullptr || packed == nullptr || scales == nullptr || dx == nullptr) return MPW_E_INVALID_ARG;
  if (!dims_ok(M, N, K) || !layout_ok(layout) || !result_ok(M, K)) return MPW_E_INVALID_ARG;
  if (layout == MPW_LAYOUT_PAIRED && K % 32 != 0) return MPW_E_INVALID_ARG;
  if (!dy_aligned(dy, N) || !aligned(packed, 16) || !aligned(scales, 4) || !aligned(dx, 2)) return MPW_E_MISALIGNED;
  const size_t need = mpw_qlinear_grad_x_workspace_bytes(bits, layout, M, N, K);
  if (need != 0 && (workspace == nullptr || workspace_bytes < need)) return MPW_E_INVALID_ARG;
  if (need != 0 && !aligned(workspace, 16)) return MPW_E_MISALIGNED;
  const Span in[3] = {span(dy, M, 2 * N), rows_span(packed, bits, N, K), span(scales, N, 4)};
  const Span scratch{workspace, need}, out = span(dx, M, 2 * K);
  if (!apart(out, {in[0], in[1], in[2], scratch}) || !apart(scratch, {in[0], in[1], in[2]})) return MPW_E_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (gradx_fused(bits, M, N, K)) {
    const mpw_status st = padded_dy(&dy, M, N, ws, s);
    if (st != MPW_OK) return st;
    return from_cuda(launch_gradx_fused(dy, packed, scales, bits, layout, M, N, K, dx, s));
  }
  uint16_t* w = reinterpret_cast<uint16_t*>(ws);
  uint8_t* room = ws + expanded_bf16_bytes(N, K);
  mpw_status st = from_cuda(launch_expand_bf16(packed, scales, N, K, bits, layout, w, s));
  if (st == MPW_OK) st = padded_dy(&dy, M, N, room, s);
  if (st != MPW_OK) return st;
  return from_cuda(launch_dense_grad_x(dy, w, M, N, K, dx, room + padded_dy_bytes(M, N), s));
}

size_t mpw_qlinear_grad_w_int8_workspace_bytes(int dW_type, int64_t M, int64_t N, int64_t K) {
  if ((dW_type != MPW_GRAD_BF16 && dW_type != MPW_GRAD_F32) || !dims_ok(M, N, K)) return 0;
  const int parts = dW_type == MPW_GRAD_F32 ? 3 : 1;
  return expanded_bf16_bytes(parts * M, K) + padded_dy_bytes(M, N) +
         dense_workspace_bytes(N, K, M, parts);
}

mpw_status mpw_qlinear_grad_w_int8(const uint16_t* dy, const uint8_t* xq, const float* sx, int64_t M, int64_t N,
                                   int64_t K, void* dW, int dW_type, int accumulate, void* workspace,
                                   size_t workspace_bytes, mpw_stream_t stream) {
  if (dy == nullptr || xq == nullptr || sx == nullptr || dW == nullptr) return MPW_E_INVALID_ARG;
  if (!dims_ok(M, N, K) || (dW_type != MPW_GRAD_BF16 && dW_type != MPW_GRAD_F32) || !result_ok(N, K))
    return MPW_E_INVALID_ARG;
  const bool f32 = dW_type == MPW_GRAD_F32;
  if (accumulate != 0 && !f32) return MPW_E_INVALID_ARG;
  if (!dy_aligned(dy, N) || !aligned(xq, 16) || !aligned(sx, 4) || !aligned(dW, f32 ? 4 : 2)) return MPW_E_MISALIGNED;
  const size_t need = mpw_qlinear_grad_w_int8_workspace_bytes(dW_type, M, N, K);
  if (workspace == nullptr || workspace_bytes < need) return MPW_E_INVALID_ARG;
  if (!aligned(workspace, 16)) return MPW_E_MISALIGNED;
  const Span in[3] = {span(dy, M, 2 * N), span(xq, M, stride_i8(K)), span(sx, M, 4)};
  const Span scratch{workspace, need}, out = span(dW, N, (f32 ? 4 : 2) * K);
  if (!apart(out, {in[0], in[1], in[2], scratch}) || !apart(scratch, {in[0], in[1], in[2]})) return MPW_E_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int parts = f32 ? 3 : 1;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint16_t* x = reinterpret_cast<uint16_t*>(ws);
  uint8_t* room = ws + expanded_bf16_bytes(parts * M, K);
  mpw_status st = from_cuda(launch_expand_x(xq, sx, M, K, parts, x, s));
  if (st == MPW_OK) st = padded_dy(&dy, M, N, room, s);
  if (st != MPW_OK) return st;
  return from_cuda(launch_dense_grad_w(dy, x, parts, M, N, K, dW, f32, accumulate != 0, room + padded_dy_bytes(M, N),
                                       s));
}

}  // extern "C"

// Dense products behind the int8 linear and the gradients, on tcgen05 tensor
// cores:  d[i, j] = sum_r a(i, r) b(j, r).
//
//   int8 linear:  i = token, j = row of W, r = k; signed bytes, int32 sums;
//   grad_x:       i = token, j = k, r = row of W; bf16, fp32 sums.  dy has r
//                 contiguous (K-major), the weights j (MN-major);
//   grad_w:       i = row of W, j = k, r = token; bf16, fp32 sums, both
//                 operands MN-major.
// No operand is transposed in memory: tcgen05 reads either order from shared
// memory, and every result is written row by row as the caller wants it.
//
// One CTA per SM walks over tiles of 128 x BN results.  Warp 0 fills a ring of
// stages by TMA (128 bytes of r, or 64 steps of r, per stage and operand, in
// the 128-byte swizzle), one thread of warp 1 issues the products into one of
// two accumulators in tensor memory, and four warps write the other one out
// meanwhile.  Tiles run in groups of kGroup along i, so that the CTAs
// working at one time share operand rows in L2.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "int8_internal.h"
#include "mpw_internal.h"
#include "tc_ptx.cuh"

namespace mpw {
namespace {

constexpr int BM = 128;
constexpr int kThreads = 256;
constexpr int kEpiWarp0 = 4;
constexpr int kGroup = 16;               // tiles along i that share rows of b
constexpr uint32_t kTmemCols = 512;      // two accumulators of up to 256 columns
constexpr uint32_t kABytes = BM * 128;   // one stage of a

enum Op { kLinearI8, kGradX, kGradWBf16, kGradWF32 };

template <Op OP>
struct OpTraits {
  static constexpr bool i8 = OP == kLinearI8;
  static constexpr bool a_mn = OP == kGradWBf16 || OP == kGradWF32;
  static constexpr bool b_mn = !i8;
  static constexpr int depth = i8 ? 128 : 64;      // steps of r per stage
};

template <int BN>
struct Tile {
  static constexpr uint32_t kBBytes = BN * 128;
  static constexpr uint32_t kStage = kABytes + kBBytes;
  static constexpr int S = static_cast<int>((232448 - 1024 - 256) / kStage);
  static constexpr size_t SMEM = S * kStage + 1024 /*align*/ + 256 /*barriers*/;
};

struct Args {
  int64_t I, J;          // results
  int blocks;            // stages along r per part
  int parts;             // passes over r, part p reading slice p of b
  void* out;             // [I, J]
  const float* row_scale;
  const float* col_scale;
  int shift;
  bool accumulate;
  bool vec;              // rows of out are whole, aligned 16-byte units
};

// 32 columns of one result row, c0 .. c0 + 31 (those below J are written).
template <Op OP>
__device__ __forceinline__ void store_row(const Args& p, int64_t i, int64_t c0, const uint32_t (&v)[32], float rs) {
  const int64_t left = p.J - c0;
  if constexpr (OP == kGradWF32) {
    float* out = static_cast<float*>(p.out) + i * p.J + c0;
    if (p.vec) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (4 * q >= left) break;
        float4 o = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                               __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
        float4* dst = reinterpret_cast<float4*>(out) + q;
        if (p.accumulate) {
          const float4 old = *dst;
          o = make_float4(old.x + o.x, old.y + o.y, old.z + o.z, old.w + o.w);
        }
        *dst = o;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c < left) out[c] = p.accumulate ? out[c] + __uint_as_float(v[c]) : __uint_as_float(v[c]);
    }
  } else {
    uint32_t o[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      float a, b;
      if constexpr (OP == kLinearI8) {
        const float sa = 2 * c < left ? __ldg(p.col_scale + c0 + 2 * c) : 0.0f;
        const float sb = 2 * c + 1 < left ? __ldg(p.col_scale + c0 + 2 * c + 1) : 0.0f;
        a = static_cast<float>(static_cast<int32_t>(v[2 * c]) >> p.shift) * sa * rs;
        b = static_cast<float>(static_cast<int32_t>(v[2 * c + 1]) >> p.shift) * sb * rs;
      } else {
        a = __uint_as_float(v[2 * c]);
        b = __uint_as_float(v[2 * c + 1]);
      }
      const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
      o[c] = *reinterpret_cast<const uint32_t*>(&r);
    }
    uint16_t* out = static_cast<uint16_t*>(p.out) + i * p.J + c0;
    if (p.vec) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (8 * q < left)
          reinterpret_cast<uint4*>(out)[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c < left) out[c] = static_cast<uint16_t>(o[c >> 1] >> (16 * (c & 1)));
    }
  }
}

template <Op OP, int BN>
__global__ void __launch_bounds__(kThreads, 1)
dense_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
             const __grid_constant__ Args p, int32_t* err) {
  using T = OpTraits<OP>;
  using C = Tile<BN>;
  constexpr int S = C::S;
  constexpr int32_t kW = ptx::kWaitDense;
  extern __shared__ uint8_t dsmem_raw[];
  const uint32_t raw = ptx::smem_addr(dsmem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;       // 1024-aligned for the 128-byte swizzle
  uint64_t* bars = reinterpret_cast<uint64_t*>(dsmem_raw + (base - raw) + S * C::kStage);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
  const uint32_t bar0 = ptx::smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (S + s); };
  auto acc_full = [&](int s) { return bar0 + 8u * (2 * S + s); };
  auto acc_empty = [&](int s) { return bar0 + 8u * (2 * S + 2 + s); };
  const uint32_t drain = bar0 + 8u * (2 * S + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(acc_full(s), 1);
      ptx::mbar_init(acc_empty(s), 128);
    }
    ptx::mbar_init(drain, 1);
    ptx::mbar_fence_init();
    ptx::prefetch_tmap(&tmap_a);
    ptx::prefetch_tmap(&tmap_b);
  }
  if (warp == 2) {
    ptx::tmem_alloc(ptx::smem_addr(tmem_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int64_t IT = (p.I + BM - 1) / BM, JT = (p.J + BN - 1) / BN, tiles = IT * JT;
  const int total = p.blocks * p.parts;     // stages per tile
  auto place = [&](int64_t t, int64_t& i0, int64_t& j0) {
    const int64_t g = t / (kGroup * JT), in = t - g * kGroup * JT;
    const int64_t rows = min(static_cast<int64_t>(kGroup), IT - g * kGroup);
    i0 = (g * kGroup + in % rows) * BM;
    j0 = in / rows * BN;
  };

  if (warp == 0) {
    // ---------------- producer ----------------
    if (lane == 0) {
      bool ok = true;
      uint32_t n = 0;                       // stages filled so far
      for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        int64_t i64, j64;
        place(t, i64, j64);
        const int i0 = static_cast<int>(i64), j0 = static_cast<int>(j64);
        for (int rb = 0; rb < total; ++rb, ++n) {
          const int s = n % S;
          ok = ptx::mbar_wait(empty(s), ((n / S) & 1) ^ 1, err, ptx::wait_code(kW, ptx::kWaitXEmpty));
          if (!ok) break;
          const int part = rb / p.blocks, r0 = (rb - part * p.blocks) * T::depth;
          const uint32_t sa = base + s * C::kStage, sb = sa + kABytes;
          ptx::mbar_arrive_expect_tx(full(s), C::kStage);
          if constexpr (T::a_mn) {
#pragma unroll
            for (int c = 0; c < BM / 64; ++c) ptx::tma_load_2d(sa + c * 8192, &tmap_a, full(s), i0 + 64 * c, r0);
          } else {
            ptx::tma_load_2d(sa, &tmap_a, full(s), r0, i0);
          }
          if constexpr (T::b_mn) {
#pragma unroll
            for (int c = 0; c < BN / 64; ++c)
              ptx::tma_load_3d(sb + c * 8192, &tmap_b, full(s), j0 + 64 * c, r0, part);
          } else {
            ptx::tma_load_2d(sb, &tmap_b, full(s), r0, j0);
          }
        }
      }
      // nothing may still be landing in shared memory when the CTA exits
      for (uint32_t k = n > S ? n - S : 0; k < n; ++k)
        ptx::mbar_wait(full(k % S), (k / S) & 1, err, ptx::wait_code(kW, ptx::kWaitXTail));
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      constexpr uint32_t idesc =
          T::i8 ? ptx::idesc_i8_s32(BM, BN) : ptx::idesc_bf16_f32_major(BM, BN, T::a_mn, T::b_mn);
      bool ok = true;
      uint32_t n = 0, u = 0;
      for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++u) {
        const uint32_t acc = tmem + (u & 1) * 256u;
        ok = ptx::mbar_wait(acc_empty(u & 1), ((u >> 1) & 1) ^ 1, err, ptx::wait_code(kW, ptx::kWaitAccEmpty));
        if (!ok) break;
        ptx::tc_fence_after();
        for (int rb = 0; rb < total; ++rb, ++n) {
          const int s = n % S;
          ok = ptx::mbar_wait(full(s), (n / S) & 1, err, ptx::wait_code(kW, ptx::kWaitFull));
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t sa = base + s * C::kStage, sb = sa + kABytes;
          const uint64_t ad = T::a_mn ? ptx::sw128_mnmajor_desc(sa, 8192) : ptx::sw128_kmajor_desc(sa);
          const uint64_t bd = T::b_mn ? ptx::sw128_mnmajor_desc(sb, 8192) : ptx::sw128_kmajor_desc(sb);
          // a step is 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major operand
          constexpr uint64_t da = T::a_mn ? 128 : 2, db = T::b_mn ? 128 : 2;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (T::i8) ptx::mma_ss_i8(acc, ad + da * k, bd + db * k, idesc, (rb | k) != 0);
            else ptx::mma_ss_bf16(acc, ad + da * k, bd + db * k, idesc, (rb | k) != 0);
          }
          ptx::mma_commit(empty(s));
        }
        ptx::mma_commit(acc_full(u & 1));
      }
      // tensor memory is given back only when no product is under way
      ptx::mma_commit(drain);
      ptx::mbar_wait(drain, 0, err, ptx::wait_code(kW, ptx::kWaitDrain));
    }
  } else if (warp >= kEpiWarp0) {
    // ---------------- epilogue ----------------
    const int quad = warp & 3;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t u = 0;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, ++u) {
      int64_t i0, j0;
      place(t, i0, j0);
      const int64_t i = i0 + quad * 32 + lane;
      const float rs = OP == kLinearI8 && i < p.I ? __ldg(p.row_scale + i) : 0.0f;
      if (!ptx::mbar_wait(acc_full(u & 1), (u >> 1) & 1, err, ptx::wait_code(kW, ptx::kWaitAcc))) break;
      ptx::tc_fence_after();
      const uint32_t acc = tmem + (u & 1) * 256u + lane_addr;
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        if (j0 + 32 * c >= p.J) break;
        uint32_t v[32];
        ptx::tmem_ld32(acc + 32 * c, v);
        ptx::tmem_wait_ld(v);
        if (i < p.I) store_row<OP>(p, i, j0 + 32 * c, v, rs);
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(acc_empty(u & 1));
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// A K-major operand: rows of `cols` values (dense in r), box of one stage.
bool map_kmajor(CUtensorMap* m, const void* p, bool i8, int64_t rows, int64_t cols, int64_t stride_bytes, int box_rows) {
  auto encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride_bytes)};
  const cuuint32_t box[2] = {i8 ? 128u : 64u, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m, i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p),
                dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An MN-major bf16 operand: `slices` of `steps` rows (r) of `cols` values (i or
// j); box of 64 values x 64 rows.  rank 2 has no slices.
bool map_mnmajor(CUtensorMap* m, const uint16_t* p, int rank, int64_t slices, int64_t steps, int64_t cols) {
  auto encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t stride = static_cast<cuuint64_t>(stride_bf16(cols)) * 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(steps),
                              static_cast<cuuint64_t>(slices)};
  const cuuint64_t strides[2] = {stride, stride * static_cast<cuuint64_t>(steps)};
  const cuuint32_t box[3] = {64, 64, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<uint16_t*>(p), dims,
                strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Op OP, int BN>
cudaError_t run(const CUtensorMap& a, const CUtensorMap& b, const Args& p, cudaStream_t stream) {
  auto kern = dense_kernel<OP, BN>;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), Tile<BN>::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((p.I + BM - 1) / BM) * ((p.J + BN - 1) / BN);
  const int64_t sms = device_info().num_sms;
  kern<<<static_cast<unsigned>(tiles < sms ? tiles : sms), kThreads, Tile<BN>::SMEM, stream>>>(a, b, p,
                                                                                             device_error_word());
  return cudaGetLastError();
}

bool whole16(const void* out, int64_t row_bytes) {
  return row_bytes % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
}

}  // namespace

cudaError_t launch_dense_i8(const uint8_t* a, const uint8_t* b, const float* sx, const float* scales, int shift,
                            int64_t M, int64_t N, int64_t K, uint16_t* y, cudaStream_t stream) {
  const int64_t stride = stride_i8(K);
  CUtensorMap ma, mb;
  if (!map_kmajor(&ma, a, true, M, stride, stride, BM) || !map_kmajor(&mb, b, true, N, stride, stride, 256))
    return cudaErrorInvalidValue;
  Args p{M, N, static_cast<int>((K + 127) / 128), 1, y, sx, scales, shift, false, whole16(y, 2 * N)};
  return run<kLinearI8, 256>(ma, mb, p, stream);
}

cudaError_t launch_dense_grad_x(const uint16_t* dy, const uint16_t* w, int64_t M, int64_t N, int64_t K, uint16_t* dx,
                                cudaStream_t stream) {
  CUtensorMap ma, mb;
  if (!map_kmajor(&ma, dy, false, M, N, 2 * stride_bf16(N), BM) || !map_mnmajor(&mb, w, 3, 1, N, K))
    return cudaErrorInvalidValue;
  Args p{M, K, static_cast<int>((N + 63) / 64), 1, dx, nullptr, nullptr, 0, false, whole16(dx, 2 * K)};
  return run<kGradX, 256>(ma, mb, p, stream);
}

cudaError_t launch_dense_grad_w(const uint16_t* dy, const uint16_t* x, int parts, int64_t M, int64_t N, int64_t K,
                                void* dw, bool f32, bool accumulate, cudaStream_t stream) {
  CUtensorMap ma, mb;
  if (!map_mnmajor(&ma, dy, 2, 1, M, N) || !map_mnmajor(&mb, x, 3, parts, M, K)) return cudaErrorInvalidValue;
  Args p{N, K, static_cast<int>((M + 63) / 64), parts, dw, nullptr, nullptr, 0, accumulate,
         whole16(dw, (f32 ? 4 : 2) * K)};
  return f32 ? run<kGradWF32, 256>(ma, mb, p, stream) : run<kGradWBf16, 256>(ma, mb, p, stream);
}

}  // namespace mpw

// Int8 linear for tens to hundreds of tokens (more, where the rows are few): packed rows expanded on the way
// to the tensor cores, y[m, n] = bf16(s_n sx_m sum_k xq[m, k] q[n, k]).
//
// DynaQuant, "Custom kernel architecture": packed codes are read from memory,
// expanded in registers to a tensor-core format and multiplied.  With few
// tokens the packed bytes are the cost (each row tile reads its rows once for
// all of them); a copy of the expanded rows would be written and read again.
//
// One CTA computes 128 rows of W x BN tokens (y^T) over one of S slices of K with
// tcgen05.mma.kind::i8:
//   * packed rows move in blocks of 128 codes (16 B bytes per row) by TMA into
//     a ring of SW stages, deep enough to cover the latency of memory;
//   * A = 128 rows x 128 signed bytes per block in tensor memory (32 columns):
//     groups of four converter warps take the blocks in turn, one row per
//     thread (int8_expand.cuh);
//   * B = BN tokens x 128 bytes of xq by TMA, in the 128-byte swizzle;
//   * D = 32-bit sums, BN columns of tensor memory.
// When the row tiles do not fill the SMs, a cluster of S CTAs shares a tile:
// each leaves its sums in shared memory and writes its share of the tokens from
// all of them.  Whole numbers: the split does not change a result.
// The weights do not depend on the launch before; their loads start ahead of
// the wait for it (programmatic dependent launch).  Every mbarrier wait is bounded.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "int8_expand.cuh"
#include "int8_internal.h"
#include "mpw_internal.h"
#include "tc_ptx.cuh"
#include "tile_choice.h"

namespace mpw {
namespace {

constexpr int BM = 128;                    // weight rows per CTA
constexpr int BK = 128;                    // codes per block
constexpr int kConvWarp0 = 4;
constexpr uint32_t kACols = BK / 4;        // tensor-memory columns of one A stage

template <int B, int BN>
struct Code {
  // groups of four converter warps: with many tokens a block's products take
  // long enough for four groups to pay (17408 x 5120, b = 6, 256 tokens: 27.2 to
  // 24.8 us), and with 64 for the widths whose codes cross bytes, which take the
  // most operations (5120 x 17408, b = 6: 22.8 to 21.0; b = 4: 16.8, 17.1); with few
  // the threads' start costs more than it gives (4096 x 4096, 32 tokens, b = 4: 7.7
  // against 8.7, b = 6: 8.9 against 9.4)
  static constexpr int G = BN >= 128 || (BN == 64 && B > 4 && B < 8) ? 4 : 2;
  static constexpr int kThreads = (kConvWarp0 + 4 * G) * 32;
  static constexpr uint32_t kXStage = BN * BK;
  static constexpr uint32_t PITCH = 16u * B;
  static constexpr uint32_t kWStage = BM * PITCH;
  // a stage of xq takes over a microsecond to come: enough of them to cover it
  static constexpr int SX = BN == 16 ? 16 : (BN == 32 ? 12 : (BN == 64 ? 8 : (BN < 256 ? 6 : 5)));
  static constexpr int SW = BN >= 192 ? 4 : 8;
  static constexpr uint32_t kCols = BN <= 32 ? 256 : 512;                 // tensor memory
  static constexpr int SA_all = static_cast<int>((kCols - BN) / kACols);
  static constexpr int SA = SA_all > 8 ? 8 : SA_all;
  static constexpr CUtensorMapSwizzle WSWZ =
      B == 8 ? CU_TENSOR_MAP_SWIZZLE_128B : (B == 4 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE);
  // byte offset of 16-byte unit u of row r inside a weight stage
  static __device__ __forceinline__ uint32_t unit(int r, int u) {
    if constexpr (B == 8) return r * 128u + 16u * (static_cast<uint32_t>(u) ^ (r & 7));
    else if constexpr (B == 4) return r * 64u + 16u * (static_cast<uint32_t>(u) ^ ((r >> 1) & 3));
    else return r * PITCH + 16u * u;
  }
  static constexpr size_t SMEM = SX * kXStage + SW * kWStage + 1024 /*align*/ + 640 /*barriers*/;
  static_assert(SMEM + 1024 <= 232448, "shared memory per block");
  // A stage is always read by the same group: were it another one's turn, that
  // group could find the stage's previous fill, not yet complete, to have the
  // parity it waits for.
  static_assert(SW % G == 0 && SA >= G, "whole turns of the groups per ring");
  // the sums of a split tile take the place of the x ring
  static_assert(SX * kXStage >= BM * BN * 4, "room for the sums");
};

template <int B, bool PAIRED, int BN>
__global__ void __launch_bounds__(Code<B, BN>::kThreads, 1)
gemm_i8_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
               const float* __restrict__ scales, const float* __restrict__ sx, uint16_t* __restrict__ y, int M,
               int64_t N, int KB, int splits, int32_t* err) {
  using C = Code<B, BN>;
  constexpr int SX = C::SX, SW = C::SW, SA = C::SA, kGroups = C::G;
  extern __shared__ uint8_t fsmem_raw[];
  __shared__ float sx_s[BN];
  const uint32_t raw = ptx::smem_addr(fsmem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;       // 1024-aligned for the 128-byte swizzle
  uint8_t* fsmem = fsmem_raw + (base - raw);
  const uint32_t xs0 = base, ws0 = base + SX * C::kXStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(fsmem + SX * C::kXStage + SW * C::kWStage);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * SX + 2 * SW + 2 * SA + 1);
  const uint32_t bar0 = ptx::smem_addr(bars);
  auto full_x = [&](int s) { return bar0 + 8u * s; };
  auto empty_x = [&](int s) { return bar0 + 8u * (SX + s); };
  auto full_w = [&](int s) { return bar0 + 8u * (2 * SX + s); };
  auto empty_w = [&](int s) { return bar0 + 8u * (2 * SX + SW + s); };
  auto full_a = [&](int s) { return bar0 + 8u * (2 * SX + 2 * SW + s); };
  auto empty_a = [&](int s) { return bar0 + 8u * (2 * SX + 2 * SW + SA + s); };
  const uint32_t acc_full = bar0 + 8u * (2 * SX + 2 * SW + 2 * SA);
  constexpr int32_t kW = ptx::kWaitGemmI8;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the CTAs of a cluster are the K slices of one tile; token tiles run next
  const int part = blockIdx.x % splits;
  const int m0 = blockIdx.x / splits * BN;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * BM;
  const int kb0 = static_cast<int>(static_cast<int64_t>(KB) * part / splits);
  const int kbs = static_cast<int>(static_cast<int64_t>(KB) * (part + 1) / splits) - kb0;    // blocks of this CTA

  if (threadIdx.x == 0) {
    for (int s = 0; s < SX; ++s) {
      ptx::mbar_init(full_x(s), 1);
      ptx::mbar_init(empty_x(s), 1);
    }
    for (int s = 0; s < SW; ++s) {
      ptx::mbar_init(full_w(s), 1);
      ptx::mbar_init(empty_w(s), 4);        // one converter group, a lane for a warp
    }
    for (int s = 0; s < SA; ++s) {
      ptx::mbar_init(full_a(s), 4);
      ptx::mbar_init(empty_a(s), 1);
    }
    ptx::mbar_init(acc_full, 1);
    ptx::mbar_fence_init();
    ptx::prefetch_tmap(&tmap_x);
    ptx::prefetch_tmap(&tmap_w);
  }
  if (warp == 2) {
    ptx::tmem_alloc(ptx::smem_addr(tmem_slot), C::kCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_a = tmem + BN;

  bool ok = true;
  if (warp == 0) {
    // ---------------- x producer ----------------
    ptx::grid_dep_wait_then_release();
    if (ptx::elect_one()) {
      int issued = 0;
      for (int kb = 0; kb < kbs; ++kb) {
        const int s = kb % SX;
        if (!ptx::mbar_wait(empty_x(s), ((kb / SX) & 1) ^ 1, err, ptx::wait_code(kW, ptx::kWaitXEmpty))) break;
        ptx::mbar_arrive_expect_tx(full_x(s), C::kXStage);
        ptx::tma_load_2d(xs0 + s * C::kXStage, &tmap_x, full_x(s), (kb0 + kb) * BK, m0);
        issued = kb + 1;
      }
      // nothing may still be landing in shared memory when the CTA exits
      for (int kb = max(0, issued - SX); kb < issued; ++kb)
        ptx::mbar_wait(full_x(kb % SX), (kb / SX) & 1, err, ptx::wait_code(kW, ptx::kWaitXTail));
    }
  } else if (warp == 3) {
    // ---------------- weight producer ----------------
    if (ptx::elect_one()) {
      int issued = 0;
      for (int wb = 0; wb < kbs; ++wb) {
        const int s = wb % SW;
        if (!ptx::mbar_wait(empty_w(s), ((wb / SW) & 1) ^ 1, err, ptx::wait_code(kW, ptx::kWaitWEmpty))) break;
        ptx::mbar_arrive_expect_tx(full_w(s), C::kWStage);
        ptx::tma_load_2d(ws0 + s * C::kWStage, &tmap_w, full_w(s), (kb0 + wb) * 16 * B, static_cast<int>(n0));
        issued = wb + 1;
      }
      for (int wb = max(0, issued - SW); wb < issued; ++wb)
        ptx::mbar_wait(full_w(wb % SW), (wb / SW) & 1, err, ptx::wait_code(kW, ptx::kWaitWTail));
    }
    __syncwarp();
    ptx::grid_dep_wait_then_release();
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    ptx::grid_dep_wait_then_release();
    if (ptx::elect_one()) {
      constexpr uint32_t idesc = ptx::idesc_i8_s32(BM, BN);
      for (int kb = 0; kb < kbs && ok; ++kb) {
        const int s = kb % SX, sa = kb % SA;
        ok = ptx::mbar_wait(full_x(s), (kb / SX) & 1, err, ptx::wait_code(kW, ptx::kWaitFull));
        if (ok) ok = ptx::mbar_wait(full_a(sa), (kb / SA) & 1, err, ptx::wait_code(kW, ptx::kWaitAFull));
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t bdesc = ptx::sw128_kmajor_desc(xs0 + s * C::kXStage);
        const uint32_t a_cols = tmem_a + sa * kACols;
#pragma unroll
        for (int k = 0; k < BK / 32; ++k)
          ptx::mma_ts_i8(tmem, a_cols + k * 8, bdesc + static_cast<uint64_t>(2 * k), idesc, (kb | k) != 0);
        ptx::mma_commit(empty_x(s));
        ptx::mma_commit(empty_a(sa));
      }
      ptx::mma_commit(acc_full);
      // tensor memory is given back only when no product is under way
      ptx::mbar_wait(acc_full, 0, err, ptx::wait_code(kW, ptx::kWaitDrain));
    }
  } else if (warp == 2) {
    ptx::grid_dep_wait_then_release();
  } else {
    // ---------------- converters ----------------
    const int wg = (warp - kConvWarp0) >> 2;       // which blocks
    const int quad = warp & 3;                     // tensor-memory lane quadrant
    const int r = quad * 32 + lane;                // weight row within the tile
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    for (int wb = wg; wb < kbs; wb += kGroups) {
      const int ws = wb % SW, sa = wb % SA;
      ok = ptx::mbar_wait(full_w(ws), (wb / SW) & 1, err, ptx::wait_code(kW, ptx::kWaitWFull));
      if (!ok) break;
      uint32_t w[4 * B + 1];
      const uint8_t* stage = fsmem + SX * C::kXStage + ws * C::kWStage;
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(stage + C::unit(r, i));
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
      w[4 * B] = 0u;
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty_w(ws));
      ok = ptx::mbar_wait(empty_a(sa), ((wb / SA) & 1) ^ 1, err, ptx::wait_code(kW, ptx::kWaitAEmpty));
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t col = tmem_a + lane_addr + sa * kACols;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t o[16];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t gw[B + 1], og[8];
#pragma unroll
          for (int i = 0; i <= B; ++i) gw[i] = w[(2 * h + g) * B + i];
          i8::group<B, PAIRED>(gw, og);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[8 * g + i] = og[i];
        }
        ptx::tmem_st16(col + 16 * h, o);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(full_a(sa));
    }
    ptx::grid_dep_wait_then_release();
    // ---------------- epilogue: this warp's rows, a share of the tokens ----------------
    const int ct = threadIdx.x - kConvWarp0 * 32;
    for (int t = ct; t < BN; t += kGroups * 128) sx_s[t] = m0 + t < M ? __ldg(sx + m0 + t) : 0.0f;
    asm volatile("bar.sync 1, %0;" ::"n"(kGroups * 128) : "memory");
    if (ok) ok = ptx::mbar_wait(acc_full, 0, err, ptx::wait_code(kW, ptx::kWaitAcc));
    if (ok) {
      ptx::tc_fence_after();
      const int64_t n = n0 + r;
      const i8::RowScale sn(n < N ? __ldg(scales + n) : 0.0f);
      constexpr int CH = BN < 32 ? BN : 32;        // tokens per step
      for (int c = wg; c < BN / CH; c += kGroups) {
        uint32_t v[32];
        ptx::tmem_ld32(tmem + lane_addr + c * CH, v);
        ptx::tmem_wait_ld(v);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int t = c * CH + i;
          if (splits > 1) {
            reinterpret_cast<int32_t*>(fsmem)[t * BM + r] = static_cast<int32_t>(v[i]);
          } else if (m0 + t < M && n < N) {
            const float o = sn.of(static_cast<int32_t>(v[i]) >> (8 - B), sx_s[t]);
            y[static_cast<size_t>(m0 + t) * N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
          }
        }
      }
    }
  }
  __syncwarp();
  if (splits > 1) {
    ptx::cluster_sync();       // the sums of every slice are in shared memory
    if (warp >= kConvWarp0) {
      // this CTA's share of the tokens, eight of them at a time, so that the
      // reads of one slice's sums overlap
      constexpr int E = 8;
      const int r = threadIdx.x & 127;
      const int64_t n = n0 + r;
      const int t1 = min(BN, M - m0);
      const i8::RowScale sn(n < N ? __ldg(scales + n) : 0.0f);
      for (int t0 = E * (part * kGroups + ((warp - kConvWarp0) >> 2)); t0 < t1; t0 += E * splits * kGroups) {
        int32_t sum[E];
#pragma unroll
        for (int i = 0; i < E; ++i) sum[i] = 0;
        for (int c = 0; c < splits; ++c) {
          const uint32_t a = ptx::cluster_addr(base + 4u * (t0 * BM + r), c);
          int32_t v[E];
#pragma unroll
          for (int i = 0; i < E; ++i) v[i] = ptx::ld_cluster_s32(a + 4u * BM * i);
#pragma unroll
          for (int i = 0; i < E; ++i) sum[i] += v[i];
        }
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (t0 + i < t1 && n < N) {
            const float o = sn.of(sum[i] >> (8 - B), sx_s[t0 + i]);
            y[static_cast<size_t>(m0 + t0 + i) * N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
          }
      }
    }
    __syncwarp();
    ptx::cluster_sync();       // nobody reads this CTA's sums any more
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kCols);
  }
}

template <int B, bool PAIRED, int BN>
cudaError_t run(const uint8_t* xq, const float* sx, const uint8_t* packed, const float* scales, int64_t M, int64_t N,
                int64_t K, uint16_t* y, int splits, cudaStream_t stream) {
  using C = Code<B, BN>;
  auto encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint32_t estr[2] = {1, 1};
  CUtensorMap mx, mw;
  {
    const int64_t stride = stride_i8(K);
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(stride), static_cast<cuuint64_t>(M)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
    const cuuint32_t box[2] = {BK, BN};
    if (encode(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(xq), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  {
    const int64_t rb = 4 * row_words(K, B);
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(rb), static_cast<cuuint64_t>(N)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(rb)};
    const cuuint32_t box[2] = {16 * B, BM};
    if (encode(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(packed), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, C::WSWZ, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  auto kern = gemm_i8_kernel<B, PAIRED, BN>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((M + BN - 1) / BN * splits), static_cast<unsigned>((N + BM - 1) / BM));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, mx, mw, scales, sx, y, static_cast<int>(M), N,
                            static_cast<int>((K + BK - 1) / BK), splits, device_error_word());
}

// A tile width, its slices and the time they promise.
struct Choice {
  int bn = 0, slices = 1;
  double us = 0.0;
};

// Takes tiles of BN tokens when they promise 7% less than the wider ones before
// them (narrow tiles read more).  (One B200, a block 0.29 us with up to 128 tokens,
// 0.36 us with 192 and 0.42 us with 256; for instance 4096 x 4096, b = 4, 256 tokens:
// 128-token tiles 10.9 us, 256 in four slices 13.0, 256 whole 15.8; 1024 x 5120,
// b = 5, 128 tokens: tiles of 64 in four slices 6.9, 128 in four 7.9, 128 whole
// 14.1; 17408 x 5120, b = 7, 300 tokens: 192 41.7, 256 44.0.)
template <int B, bool PAIRED, int BN>
cudaError_t consider(int64_t M, int64_t N, int64_t K, Choice* best) {
  using C = Code<B, BN>;
  auto kern = gemm_i8_kernel<B, PAIRED, BN>;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  const ClusterCapacity cap = cluster_capacity<gemm_i8_kernel<B, PAIRED, BN>>(C::kThreads, C::SMEM);
  const int64_t tiles = (M + BN - 1) / BN * ((N + BM - 1) / BM), blocks = (K + BK - 1) / BK;
  Choice c;
  for (int i = 1; i <= kMaxSlices && (i == 1 || i * 4 <= blocks); ++i) {
    if (cap.ctas[i] == 0) continue;
    const double block = BN == 256 ? 0.42 : (BN == 192 ? 0.36 : 0.29);
    const double t = tile_time(tiles * i, cap.ctas[i], blocks, i, BN, block, 1.7);
    if (c.bn == 0 || t < 0.95 * c.us) c = Choice{BN, i, t};
  }
  if (best->bn == 0 || c.us < 0.93 * best->us) *best = c;
  return cudaSuccess;
}

// The widest tile that M fills, or a narrower one.
template <int B, bool PAIRED, int... BN>
cudaError_t run_best(const uint8_t* xq, const float* sx, const uint8_t* packed, const float* scales, int64_t M,
                     int64_t N, int64_t K, uint16_t* y, cudaStream_t stream) {
  Choice best;
  cudaError_t e = cudaSuccess;
  ((e = e == cudaSuccess ? consider<B, PAIRED, BN>(M, N, K, &best) : e), ...);
  if (e != cudaSuccess) return e;
  ((e = best.bn == BN ? run<B, PAIRED, BN>(xq, sx, packed, scales, M, N, K, y, best.slices, stream) : e), ...);
  return e;
}

template <int B, bool PAIRED>
cudaError_t run_bn(const uint8_t* xq, const float* sx, const uint8_t* packed, const float* scales, int64_t M,
                   int64_t N, int64_t K, uint16_t* y, cudaStream_t stream) {
  if (M <= 16) return run_best<B, PAIRED, 16>(xq, sx, packed, scales, M, N, K, y, stream);
  if (M <= 32) return run_best<B, PAIRED, 32, 16>(xq, sx, packed, scales, M, N, K, y, stream);
  if (M <= 64) return run_best<B, PAIRED, 64, 32, 16>(xq, sx, packed, scales, M, N, K, y, stream);
  if (M <= 128) return run_best<B, PAIRED, 128, 64, 32>(xq, sx, packed, scales, M, N, K, y, stream);
  return run_best<B, PAIRED, 256, 192, 128, 64>(xq, sx, packed, scales, M, N, K, y, stream);
}

template <int B>
cudaError_t run_layout(const uint8_t* xq, const float* sx, const uint8_t* packed, const float* scales, int layout,
                       int64_t M, int64_t N, int64_t K, uint16_t* y, cudaStream_t stream) {
  return layout == kLayoutPaired ? run_bn<B, true>(xq, sx, packed, scales, M, N, K, y, stream)
                                 : run_bn<B, false>(xq, sx, packed, scales, M, N, K, y, stream);
}

}  // namespace

bool gemm_i8_fits(int64_t M, int64_t N) {
  return (N + BM - 1) / BM <= 65535 && M <= (int64_t{1} << 24);
}

cudaError_t launch_gemm_i8(const uint8_t* xq, const float* sx, const uint8_t* packed, const float* scales, int bits,
                           int layout, int64_t M, int64_t N, int64_t K, uint16_t* y, cudaStream_t stream) {
  switch (bits) {
    case 4: return run_layout<4>(xq, sx, packed, scales, layout, M, N, K, y, stream);
    case 5: return run_layout<5>(xq, sx, packed, scales, layout, M, N, K, y, stream);
    case 6: return run_layout<6>(xq, sx, packed, scales, layout, M, N, K, y, stream);
    case 7: return run_layout<7>(xq, sx, packed, scales, layout, M, N, K, y, stream);
    case 8: return run_layout<8>(xq, sx, packed, scales, layout, M, N, K, y, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mpw

// Gradient of x through packed rows for up to a few hundred tokens: rows
// expanded on the way to the tensor cores,
//   dx[m, k] = bf16(sum_n dy[m, n] w[n, k]),  w[n, k] = s_n q[n, k] in bf16.
//
// The packed rows are the cost when there are few tokens; expanding them into
// memory writes and reads three to five times their bytes.  Here the sum runs
// over the rows, so the expanded tile is used with its n axis as the depth of the
// product: tcgen05 takes it MN-major from shared memory, as the rows lie.
//
// One CTA computes 128 inputs k x BN tokens (dx^T) over one of S slices of n:
//   * packed rows move in blocks of 64 rows x 128 codes (16 B bytes per row) by
//     TMA into a ring of SW stages;
//   * A: groups of four converter warps take the blocks in turn; a thread
//     expands 32 codes of a row to bf16, scales them and writes 64 bytes into
//     the 128-byte swizzle (two chunks of 64 k x 64 rows, 16 KB).  The codes of a
//     canonical group are left in the order that takes the fewest operations;
//     the writer of dx knows which input a lane holds;
//   * B: BN tokens x 64 values of dy by TMA;
//   * D: fp32, BN columns of tensor memory.
// A cluster of S CTAs shares a tile when the tiles do not fill the SMs: each
// leaves its sums in shared memory and writes its share of the tokens from all
// of them, added in order.  Every mbarrier wait is bounded.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "int8_expand.cuh"
#include "int8_internal.h"
#include "mpw_internal.h"
#include "scale_pair.cuh"
#include "tc_ptx.cuh"
#include "tile_choice.h"

namespace mpw {
namespace {

constexpr int BM = 128;                    // inputs k per CTA
constexpr int BK = 64;                     // rows n per block
constexpr int kGroups = 4;                 // groups of four converter warps
constexpr int kConvWarp0 = 4;
constexpr int kThreads = (kConvWarp0 + 4 * kGroups) * 32;
constexpr uint32_t kAStage = BM * BK * 2;  // two chunks of 64 k
constexpr int SA = 4;

template <int B, int BN>
struct Code {
  static constexpr uint32_t kXStage = BN * BK * 2;
  static constexpr uint32_t PITCH = 16u * B;
  static constexpr uint32_t kWStage = BK * PITCH;
  // a stage of dy takes over a microsecond to come: enough of them to cover it
  // (four of 64 tokens bound the kernel to 0.35 us a block)
  static constexpr int SX = BN == 32 ? 12 : (BN == 64 ? 8 : (BN == 128 ? 6 : 4));
  static constexpr int SW = BN == 256 ? 4 : 8;
  static constexpr uint32_t kCols = BN;                       // tensor memory
  static constexpr CUtensorMapSwizzle WSWZ =
      B == 8 ? CU_TENSOR_MAP_SWIZZLE_128B : (B == 4 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE);
  // the B words of group g of row r of a weight stage
  static __device__ __forceinline__ void load(const uint8_t* stage, int r, int g, uint32_t (&w)[B + 1]) {
    if constexpr (B == 8) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + 16 * ((2 * g + u) ^ (r & 7)));
        w[4 * u] = v.x; w[4 * u + 1] = v.y; w[4 * u + 2] = v.z; w[4 * u + 3] = v.w;
      }
      w[8] = 0u;
    } else if constexpr (B == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 64 + 16 * (g ^ ((r >> 1) & 3)));
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w; w[4] = 0u;
    } else {
      i8::lds_group<B>(stage + r * PITCH + g * 4 * B, w);
    }
  }
  // A stage is always read, and one of A always written, by groups that are at
  // most one fill behind: whole turns of the groups per weight ring, and a ring
  // of A of at least one turn.
  static_assert(SW % kGroups == 0 && SA >= kGroups, "rings and turns");
  static constexpr size_t SMEM = SA * kAStage + SX * kXStage + SW * kWStage + 1024 /*align*/ + 512 /*barriers*/;
  static_assert(SMEM + BN * 4 <= 232448, "shared memory per block");
  // the sums of a split tile take the place of the rings of A and B
  static_assert(SA * kAStage + SX * kXStage >= BM * BN * 4, "room for the sums");
};

// The input that lane r of a tile holds.
template <bool PAIRED>
__device__ __forceinline__ int input_of(int r) {
  return PAIRED ? r : (r & ~31) + ((r & 31) >> 1) + 16 * (r & 1);
}

template <int B, bool PAIRED, int BN>
__global__ void __launch_bounds__(kThreads, 1)
gradx_kernel(const __grid_constant__ CUtensorMap tmap_dy, const __grid_constant__ CUtensorMap tmap_w,
             const float* __restrict__ scales, uint16_t* __restrict__ dx, int M, int64_t N, int64_t K, int NB,
             int splits, int32_t* err) {
  using C = Code<B, BN>;
  constexpr int SX = C::SX, SW = C::SW;
  extern __shared__ uint8_t gsmem_raw[];
  const uint32_t raw = ptx::smem_addr(gsmem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;       // 1024-aligned for the 128-byte swizzle
  uint8_t* gsmem = gsmem_raw + (base - raw);
  const uint32_t as0 = base, xs0 = base + SA * kAStage, ws0 = xs0 + SX * C::kXStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(gsmem + SA * kAStage + SX * C::kXStage + SW * C::kWStage);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * SX + 2 * SW + 2 * SA + 1);
  const uint32_t bar0 = ptx::smem_addr(bars);
  auto full_x = [&](int s) { return bar0 + 8u * s; };
  auto empty_x = [&](int s) { return bar0 + 8u * (SX + s); };
  auto full_w = [&](int s) { return bar0 + 8u * (2 * SX + s); };
  auto empty_w = [&](int s) { return bar0 + 8u * (2 * SX + SW + s); };
  auto full_a = [&](int s) { return bar0 + 8u * (2 * SX + 2 * SW + s); };
  auto empty_a = [&](int s) { return bar0 + 8u * (2 * SX + 2 * SW + SA + s); };
  const uint32_t acc_full = bar0 + 8u * (2 * SX + 2 * SW + 2 * SA);
  constexpr int32_t kW = ptx::kWaitGradX;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the CTAs of a cluster are the slices of one tile; token tiles run next
  const int part = blockIdx.x % splits;
  const int m0 = blockIdx.x / splits * BN;
  const int64_t k0 = static_cast<int64_t>(blockIdx.y) * BM;
  const int nb0 = static_cast<int>(static_cast<int64_t>(NB) * part / splits);
  const int nbs = static_cast<int>(static_cast<int64_t>(NB) * (part + 1) / splits) - nb0;    // blocks of this CTA

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
    ptx::prefetch_tmap(&tmap_dy);
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

  bool ok = true;
  if (warp == 0) {
    // ---------------- dy producer ----------------
    if (ptx::elect_one()) {
      int issued = 0;
      for (int b = 0; b < nbs; ++b) {
        const int s = b % SX;
        if (!ptx::mbar_wait(empty_x(s), ((b / SX) & 1) ^ 1, err, ptx::wait_code(kW, ptx::kWaitXEmpty))) break;
        ptx::mbar_arrive_expect_tx(full_x(s), C::kXStage);
        ptx::tma_load_2d(xs0 + s * C::kXStage, &tmap_dy, full_x(s), (nb0 + b) * BK, m0);
        issued = b + 1;
      }
      // nothing may still be landing in shared memory when the CTA exits
      for (int b = max(0, issued - SX); b < issued; ++b)
        ptx::mbar_wait(full_x(b % SX), (b / SX) & 1, err, ptx::wait_code(kW, ptx::kWaitXTail));
    }
  } else if (warp == 3) {
    // ---------------- weight producer ----------------
    if (ptx::elect_one()) {
      int issued = 0;
      for (int b = 0; b < nbs; ++b) {
        const int s = b % SW;
        if (!ptx::mbar_wait(empty_w(s), ((b / SW) & 1) ^ 1, err, ptx::wait_code(kW, ptx::kWaitWEmpty))) break;
        ptx::mbar_arrive_expect_tx(full_w(s), C::kWStage);
        ptx::tma_load_2d(ws0 + s * C::kWStage, &tmap_w, full_w(s), static_cast<int>(k0 >> 7) * 16 * B, (nb0 + b) * BK);
        issued = b + 1;
      }
      for (int b = max(0, issued - SW); b < issued; ++b)
        ptx::mbar_wait(full_w(b % SW), (b / SW) & 1, err, ptx::wait_code(kW, ptx::kWaitWTail));
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (ptx::elect_one()) {
      constexpr uint32_t idesc = ptx::idesc_bf16_f32_major(BM, BN, true, false);
      for (int b = 0; b < nbs && ok; ++b) {
        const int s = b % SX, sa = b % SA;
        ok = ptx::mbar_wait(full_x(s), (b / SX) & 1, err, ptx::wait_code(kW, ptx::kWaitFull));
        if (ok) ok = ptx::mbar_wait(full_a(sa), (b / SA) & 1, err, ptx::wait_code(kW, ptx::kWaitAFull));
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t ad = ptx::sw128_mnmajor_desc(as0 + sa * kAStage, BK * 128);
        const uint64_t bd = ptx::sw128_kmajor_desc(xs0 + s * C::kXStage);
#pragma unroll
        for (int k = 0; k < BK / 16; ++k)
          ptx::mma_ss<1, false>(tmem, ad + static_cast<uint64_t>(128 * k), bd + static_cast<uint64_t>(2 * k), idesc,
                                (b | k) != 0);
        ptx::mma_commit(empty_x(s));
        ptx::mma_commit(empty_a(sa));
      }
      ptx::mma_commit(acc_full);
      // tensor memory is given back only when no product is under way
      ptx::mbar_wait(acc_full, 0, err, ptx::wait_code(kW, ptx::kWaitDrain));
    }
  } else if (warp >= kConvWarp0) {
    // ---------------- converters ----------------
    const int wg = (warp - kConvWarp0) >> 2;       // which blocks
    // 32-code group of the tile, and rows r0 and r0 + 32 of the block: the eight
    // lanes that store together hold eight rows, whose swizzled units cover
    // every bank once
    const int g = lane >> 3, r0 = (warp & 3) * 8 + (lane & 7);
    auto scale_of = [&](int b, int h) {
      const int64_t n = static_cast<int64_t>(nb0 + b) * BK + r0 + 32 * h;
      return b < nbs && n < N ? __ldg(scales + n) : 0.0f;
    };
    float next[2] = {scale_of(wg, 0), scale_of(wg, 1)};     // read a turn ahead
    for (int b = wg; b < nbs; b += kGroups) {
      const int ws = b % SW, sa = b % SA;
      dec::PairScale s2[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s2[h] = dec::split_scale<B>(next[h]);
        next[h] = scale_of(b + kGroups, h);
      }
      ok = ptx::mbar_wait(full_w(ws), (b / SW) & 1, err, ptx::wait_code(kW, ptx::kWaitWFull));
      if (!ok) break;
      const uint8_t* stage = gsmem + SA * kAStage + SX * C::kXStage + ws * C::kWStage;
      uint32_t o[2][16];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[B + 1];
        C::load(stage, r0 + 32 * h, g, w);
        if constexpr (PAIRED) {
          dec::scaled_group<B, true>(w, s2[h], o[h]);
        } else {
          uint32_t z[B + 1];
          i8::halves_of<B>(w, z);
          dec::scaled_group<B, true>(z, s2[h], o[h]);
        }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty_w(ws));
      ok = ptx::mbar_wait(empty_a(sa), ((b / SA) & 1) ^ 1, err, ptx::wait_code(kW, ptx::kWaitAEmpty));
      if (!ok) break;
      uint8_t* a = gsmem + sa * kAStage + (g >> 1) * (BK * 128);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = r0 + 32 * h;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(a + r * 128 + 16 * ((4 * (g & 1) + j) ^ (r & 7))) =
              make_uint4(o[h][4 * j], o[h][4 * j + 1], o[h][4 * j + 2], o[h][4 * j + 3]);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(full_a(sa));
    }
    // ---------------- epilogue: 32 inputs a warp, a share of the tokens ----------------
    const int quad = warp & 3;                     // tensor-memory lane quadrant
    const int r = quad * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    if (ok) ok = ptx::mbar_wait(acc_full, 0, err, ptx::wait_code(kW, ptx::kWaitAcc));
    if (ok) {
      ptx::tc_fence_after();
      const int64_t k = k0 + input_of<PAIRED>(r);
      for (int c = wg; c < BN / 32; c += kGroups) {
        uint32_t v[32];
        ptx::tmem_ld32(tmem + lane_addr + c * 32, v);
        ptx::tmem_wait_ld(v);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int t = c * 32 + i;
          if (splits > 1) reinterpret_cast<uint32_t*>(gsmem)[t * BM + r] = v[i];
          else if (m0 + t < M && k < K)
            dx[static_cast<size_t>(m0 + t) * K + k] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[i])));
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
      const int64_t k = k0 + input_of<PAIRED>(r);
      const int t1 = min(BN, M - m0);
      for (int t0 = E * (part * kGroups + ((warp - kConvWarp0) >> 2)); t0 < t1; t0 += E * splits * kGroups) {
        float sum[E];
#pragma unroll
        for (int i = 0; i < E; ++i) sum[i] = 0.0f;
        for (int c = 0; c < splits; ++c) {
          const uint32_t a = ptx::cluster_addr(base + 4u * (t0 * BM + r), c);
          int32_t v[E];
#pragma unroll
          for (int i = 0; i < E; ++i) v[i] = ptx::ld_cluster_s32(a + 4u * BM * i);
#pragma unroll
          for (int i = 0; i < E; ++i) sum[i] += __int_as_float(v[i]);
        }
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (t0 + i < t1 && k < K)
            dx[static_cast<size_t>(m0 + t0 + i) * K + k] = __bfloat16_as_ushort(__float2bfloat16_rn(sum[i]));
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
cudaError_t run(const uint16_t* dy, const uint8_t* packed, const float* scales, int64_t M, int64_t N, int64_t K,
                uint16_t* dx, int splits, cudaStream_t stream) {
  using C = Code<B, BN>;
  auto encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint32_t estr[2] = {1, 1};
  CUtensorMap my, mw;
  {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride_bf16(N)) * 2};
    const cuuint32_t box[2] = {BK, BN};
    if (encode(&my, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(dy), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  {
    const int64_t rb = 4 * row_words(K, B);
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(rb), static_cast<cuuint64_t>(N)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(rb)};
    const cuuint32_t box[2] = {16 * B, BK};
    if (encode(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(packed), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, C::WSWZ, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  auto kern = gradx_kernel<B, PAIRED, BN>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((M + BN - 1) / BN * splits), static_cast<unsigned>((K + BM - 1) / BM));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, my, mw, scales, dx, static_cast<int>(M), N, K,
                            static_cast<int>((N + BK - 1) / BK), splits, device_error_word());
}

// Slices for tiles of BN tokens and the time they promise.  (One B200, a block 0.33 us
// with up to 128 tokens and 0.43 us with 256; 17408 x 5120, b = 6, 48 tokens, 40
// tiles: one to four slices 95, 54, 40, 59 us; 4096 x 4096, b = 4, 128 tokens: 29,
// 21, 17, 15 us.)
template <int B, bool PAIRED, int BN>
cudaError_t slices(int64_t M, int64_t N, int64_t K, int* s, double* us) {
  using C = Code<B, BN>;
  auto kern = gradx_kernel<B, PAIRED, BN>;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  const ClusterCapacity cap = cluster_capacity<gradx_kernel<B, PAIRED, BN>>(kThreads, C::SMEM);
  const int64_t tiles = (M + BN - 1) / BN * ((K + BM - 1) / BM), blocks = (N + BK - 1) / BK;
  *s = 1;
  *us = 0.0;
  for (int i = 1; i <= kMaxSlices && (i == 1 || i * 4 <= blocks); ++i) {
    if (cap.ctas[i] == 0) continue;
    const double t = tile_time(tiles * i, cap.ctas[i], blocks, i, BN, BN == 256 ? 0.43 : 0.33, 2.0);
    if (*us == 0.0 || t < 0.95 * *us) {
      *us = t;
      *s = i;
    }
  }
  return cudaSuccess;
}

template <int B, bool PAIRED, int BN>
cudaError_t run_tile(const uint16_t* dy, const uint8_t* packed, const float* scales, int64_t M, int64_t N, int64_t K,
                     uint16_t* dx, cudaStream_t stream) {
  int s = 1, s2 = 1;
  double us = 0.0, us2 = 0.0;
  cudaError_t e = slices<B, PAIRED, BN>(M, N, K, &s, &us);
  if (e != cudaSuccess) return e;
  if constexpr (BN == 256) {
    // two tiles of 128 expand the rows twice, but may fill the SMs better
    e = slices<B, PAIRED, 128>(M, N, K, &s2, &us2);
    if (e != cudaSuccess) return e;
    if (us2 < 0.93 * us) return run<B, PAIRED, 128>(dy, packed, scales, M, N, K, dx, s2, stream);
  }
  return run<B, PAIRED, BN>(dy, packed, scales, M, N, K, dx, s, stream);
}

template <int B, bool PAIRED>
cudaError_t run_bn(const uint16_t* dy, const uint8_t* packed, const float* scales, int64_t M, int64_t N, int64_t K,
                   uint16_t* dx, cudaStream_t stream) {
  if (M <= 32) return run_tile<B, PAIRED, 32>(dy, packed, scales, M, N, K, dx, stream);
  if (M <= 64) return run_tile<B, PAIRED, 64>(dy, packed, scales, M, N, K, dx, stream);
  if (M <= 128) return run_tile<B, PAIRED, 128>(dy, packed, scales, M, N, K, dx, stream);
  return run_tile<B, PAIRED, 256>(dy, packed, scales, M, N, K, dx, stream);
}

template <int B>
cudaError_t run_layout(const uint16_t* dy, const uint8_t* packed, const float* scales, int layout, int64_t M, int64_t N,
                       int64_t K, uint16_t* dx, cudaStream_t stream) {
  return layout == kLayoutPaired ? run_bn<B, true>(dy, packed, scales, M, N, K, dx, stream)
                                 : run_bn<B, false>(dy, packed, scales, M, N, K, dx, stream);
}

}  // namespace

bool gradx_fused_fits(int bits, int64_t M, int64_t N, int64_t K) {
  return bits <= 8 && (K + BM - 1) / BM <= 65535 && M <= (int64_t{1} << 24);
}

cudaError_t launch_gradx_fused(const uint16_t* dy, const uint8_t* packed, const float* scales, int bits, int layout,
                               int64_t M, int64_t N, int64_t K, uint16_t* dx, cudaStream_t stream) {
  switch (bits) {
    case 4: return run_layout<4>(dy, packed, scales, layout, M, N, K, dx, stream);
    case 5: return run_layout<5>(dy, packed, scales, layout, M, N, K, dx, stream);
    case 6: return run_layout<6>(dy, packed, scales, layout, M, N, K, dx, stream);
    case 7: return run_layout<7>(dy, packed, scales, layout, M, N, K, dx, stream);
    case 8: return run_layout<8>(dy, packed, scales, layout, M, N, K, dx, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mpw

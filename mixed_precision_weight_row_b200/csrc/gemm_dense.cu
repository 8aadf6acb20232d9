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
// Two CTAs on neighbouring SMs (cta_group::2) compute tiles of 256 x BN
// results, each holding 128 rows of a, half of b's rows and its own 128 rows of
// the result; one CTA per SM walks over the tiles.  Warp 0 of each fills a ring
// of stages by TMA (128 bytes of r, or 64 steps of r, per stage and operand, in
// the 128-byte swizzle), one thread of the first CTA issues the products for
// both into one of two accumulators in tensor memory, and four warps of each
// write the other one out meanwhile.  Tiles run in groups of kGroup along i,
// so that the CTAs working at one time share operand rows in L2.
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
constexpr int kGroup = 8;                // tiles of 256 rows along i that share rows of b
constexpr uint32_t kTmemCols = 512;      // two accumulators of up to 256 columns
constexpr uint32_t kABytes = BM * 128;   // one stage of a

// The second CTA waits for the first one's last signal for as long as the
// kernel runs: well beyond any tile loop that makes progress.
constexpr uint64_t kDrainNs = 20000000000ull;

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
  static constexpr int rows_b = BN / 2;                  // rows of b per CTA
  static constexpr int chunks_b = (rows_b + 63) / 64;    // 64-wide chunks of an MN-major b
  template <bool MN>
  static constexpr uint32_t b_bytes() { return MN ? chunks_b * 8192u : rows_b * 128u; }
  template <bool MN>
  static constexpr uint32_t stage() { return kABytes + b_bytes<MN>(); }
  static constexpr uint32_t budget = 232448 - 1024 /*align*/ - 256 /*barriers*/;
  template <bool MN>
  static constexpr int stages() { return static_cast<int>(budget / stage<MN>()); }
  template <bool MN>
  static constexpr size_t smem() { return stages<MN>() * stage<MN>() + 1024 + 256; }
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

// Transposes blocks of U x U units of W words among U neighbouring lanes: unit
// q of lane l goes to unit (l % U) of lane (l - l % U + q).
template <int U, int W>
__device__ __forceinline__ void transpose_units(uint32_t (&v)[U * W], int lane) {
#pragma unroll
  for (int s = U / 2; s > 0; s >>= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (q & s) continue;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t& a = v[q * W + w];
        uint32_t& b = v[(q | s) * W + w];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a : b, s);
        if (up) a = got;
        else b = got;
      }
    }
  }
}

// Writes 32 columns c0 .. c0 + 31 of the 32 result rows i0 .. i0 + 31, of which
// this lane holds row i0 + lane.  A lane writing its own row would scatter a
// store over 32 rows; the values change lanes first, so that neighbouring
// lanes write neighbouring 16-byte units (rows of whole, aligned units) or
// neighbouring values (any other rows).
template <Op OP>
__device__ __forceinline__ void store_block(const Args& p, int64_t i0, int64_t c0, uint32_t (&v)[32], float rs,
                                            int lane) {
  const int64_t left = p.J - c0, rows = p.I - i0;
  if constexpr (OP == kGradWF32) {
    float* out = static_cast<float*>(p.out) + i0 * p.J + c0;
    if (p.vec) {
      transpose_units<8, 4>(v, lane);
      const int q = lane & 7, r0 = lane & ~7;
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        if (r0 + t >= rows || 4 * q >= left) continue;
        float4 o = make_float4(__uint_as_float(v[4 * t]), __uint_as_float(v[4 * t + 1]),
                               __uint_as_float(v[4 * t + 2]), __uint_as_float(v[4 * t + 3]));
        float4* dst = reinterpret_cast<float4*>(out + (r0 + t) * p.J) + q;
        if (p.accumulate) {
          const float4 old = *dst;
          o = make_float4(old.x + o.x, old.y + o.y, old.z + o.z, old.w + o.w);
        }
        *dst = o;
      }
    } else {
      transpose_units<32, 1>(v, lane);
#pragma unroll
      for (int t = 0; t < 32; ++t) {
        if (t >= rows || lane >= left) continue;
        float* dst = out + t * p.J + lane;
        *dst = p.accumulate ? *dst + __uint_as_float(v[t]) : __uint_as_float(v[t]);
      }
    }
  } else {
    if constexpr (OP == kLinearI8) {
      const float mine = lane < left ? __ldg(p.col_scale + c0 + lane) : 0.0f;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float cs = __shfl_sync(0xffffffffu, mine, c);
        v[c] = __float_as_uint(static_cast<float>(static_cast<int32_t>(v[c]) >> p.shift) * cs * rs);
      }
    }
    uint16_t* out = static_cast<uint16_t*>(p.out) + i0 * p.J + c0;
    if (p.vec) {
      uint32_t o[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1]));
        o[c] = *reinterpret_cast<const uint32_t*>(&r);
      }
      transpose_units<4, 4>(o, lane);
      const int q = lane & 3, r0 = lane & ~3;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (r0 + t < rows && 8 * q < left)
          reinterpret_cast<uint4*>(out + (r0 + t) * p.J)[q] =
              make_uint4(o[4 * t], o[4 * t + 1], o[4 * t + 2], o[4 * t + 3]);
    } else {
      transpose_units<32, 1>(v, lane);
#pragma unroll
      for (int t = 0; t < 32; ++t)
        if (t < rows && lane < left)
          out[t * p.J + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[t])));
    }
  }
}

template <Op OP, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
dense_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
             const __grid_constant__ Args p, int32_t* err) {
  using T = OpTraits<OP>;
  using C = Tile<BN>;
  constexpr uint32_t kStage = C::template stage<T::b_mn>();
  constexpr int S = C::template stages<T::b_mn>();
  constexpr int32_t kW = ptx::kWaitDense;
  extern __shared__ uint8_t dsmem_raw[];
  const uint32_t raw = ptx::smem_addr(dsmem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;       // 1024-aligned for the 128-byte swizzle
  uint64_t* bars = reinterpret_cast<uint64_t*>(dsmem_raw + (base - raw) + S * kStage);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
  const uint32_t bar0 = ptx::smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (S + s); };
  auto acc_full = [&](int s) { return bar0 + 8u * (2 * S + s); };
  auto acc_empty = [&](int s) { return bar0 + 8u * (2 * S + 2 + s); };
  const uint32_t drain = bar0 + 8u * (2 * S + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(acc_full(s), 1);
      ptx::mbar_init(acc_empty(s), 256);     // both CTAs' epilogues
    }
    ptx::mbar_init(drain, 1);
    ptx::mbar_fence_init();
    ptx::prefetch_tmap(&tmap_a);
    ptx::prefetch_tmap(&tmap_b);
  }
  if (warp == 2) {
    ptx::tmem_alloc_pair(ptx::smem_addr(tmem_slot), kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();     // barriers and tensor memory of both CTAs are ready
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int64_t IT = (p.I + 2 * BM - 1) / (2 * BM), JT = (p.J + BN - 1) / BN, tiles = IT * JT;
  const int total = p.blocks * p.parts;     // stages per tile
  auto place = [&](int64_t t, int64_t& i0, int64_t& j0) {
    const int64_t g = t / (kGroup * JT), in = t - g * kGroup * JT;
    const int64_t rows = min(static_cast<int64_t>(kGroup), IT - g * kGroup);
    i0 = (g * kGroup + in % rows) * 2 * BM + rank * BM;     // this CTA's rows
    j0 = in / rows * BN;
  };
  const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (warp == 0) {
    // ---------------- producer ----------------
    if (ptx::elect_one()) {
      // both CTAs' loads complete on the first one's barriers, where the
      // products are issued
      bool ok = true;
      uint32_t n = 0;                       // stages filled so far
      for (int64_t t = first; t < tiles && ok; t += step) {
        int64_t i64, j64;
        place(t, i64, j64);
        const int i0 = static_cast<int>(i64), j0 = static_cast<int>(j64) + static_cast<int>(rank) * C::rows_b;
        for (int rb = 0; rb < total; ++rb, ++n) {
          const int s = n % S;
          ok = ptx::mbar_wait(empty(s), ((n / S) & 1) ^ 1, err, ptx::wait_code(kW, ptx::kWaitXEmpty));
          if (!ok) break;
          const int part = rb / p.blocks, r0 = (rb - part * p.blocks) * T::depth;
          const uint32_t sa = base + s * kStage, sb = sa + kABytes;
          if (rank == 0) ptx::mbar_arrive_expect_tx(full(s), 2 * kStage);
          const uint32_t bar = ptx::cluster_addr(full(s), 0);
          if constexpr (T::a_mn) {
#pragma unroll
            for (int c = 0; c < BM / 64; ++c) ptx::tma_load_2d_pair(sa + c * 8192, &tmap_a, bar, i0 + 64 * c, r0);
          } else {
            ptx::tma_load_2d_pair(sa, &tmap_a, bar, r0, i0);
          }
          if constexpr (T::b_mn) {
#pragma unroll
            for (int c = 0; c < C::chunks_b; ++c)
              ptx::tma_load_3d_pair(sb + c * 8192, &tmap_b, bar, j0 + 64 * c, r0, part);
          } else {
            ptx::tma_load_2d_pair(sb, &tmap_b, bar, r0, j0);
          }
        }
      }
      // nothing may still be landing in shared memory when the CTA exits: the
      // first CTA sees the barriers of both, the other one leaves after it
      if (rank == 0)
        for (uint32_t k = n > S ? n - S : 0; k < n; ++k)
          ptx::mbar_wait(full(k % S), (k / S) & 1, err, ptx::wait_code(kW, ptx::kWaitXTail));
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (rank == 0) {
      constexpr uint32_t idesc =
          T::i8 ? ptx::idesc_i8_s32(2 * BM, BN) : ptx::idesc_bf16_f32_major(2 * BM, BN, T::a_mn, T::b_mn);
      if (ptx::elect_one()) {
        bool ok = true;
        int s = 0;
        uint32_t phase = 0, u = 0;
        for (int64_t t = first; t < tiles && ok; t += step, ++u) {
          const uint32_t acc = tmem + (u & 1) * 256u;
          ok = ptx::mbar_wait(acc_empty(u & 1), ((u >> 1) & 1) ^ 1, err, ptx::wait_code(kW, ptx::kWaitAccEmpty));
          if (!ok) break;
          ptx::tc_fence_after();
          for (int rb = 0; rb < total; ++rb) {
            ok = ptx::mbar_wait(full(s), phase, err, ptx::wait_code(kW, ptx::kWaitFull));
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t sa = base + s * kStage, sb = sa + kABytes;
            const uint64_t ad = T::a_mn ? ptx::sw128_mnmajor_desc(sa, 8192) : ptx::sw128_kmajor_desc(sa);
            const uint64_t bd = T::b_mn ? ptx::sw128_mnmajor_desc(sb, 8192) : ptx::sw128_kmajor_desc(sb);
            // a step is 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major operand
            constexpr uint64_t da = T::a_mn ? 128 : 2, db = T::b_mn ? 128 : 2;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ptx::mma_ss<2, T::i8>(acc, ad + da * k, bd + db * k, idesc, (rb | k) != 0);
            ptx::mma_commit_pair(empty(s));
            if (++s == S) {
              s = 0;
              phase ^= 1;
            }
          }
          ptx::mma_commit_pair(acc_full(u & 1));
        }
        // tensor memory is given back only when no product is under way
        ptx::mma_commit_pair(drain);
        ptx::mbar_wait(drain, 0, err, ptx::wait_code(kW, ptx::kWaitDrain));
      }
    } else if (lane == 0) {
      // no signal of the first CTA may reach this one after its exit
      ptx::mbar_wait(drain, 0, err, ptx::wait_code(kW, ptx::kWaitDrain), kDrainNs);
    }
  } else if (warp >= kEpiWarp0) {
    // ---------------- epilogue ----------------
    const int quad = warp & 3;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t u = 0;
    for (int64_t t = first; t < tiles; t += step, ++u) {
      int64_t i0, j0;
      place(t, i0, j0);
      const int64_t iw = i0 + quad * 32;      // the warp's first row
      const float rs = OP == kLinearI8 && iw + lane < p.I ? __ldg(p.row_scale + iw + lane) : 0.0f;
      if (!ptx::mbar_wait(acc_full(u & 1), (u >> 1) & 1, err, ptx::wait_code(kW, ptx::kWaitAcc))) break;
      ptx::tc_fence_after();
      const uint32_t acc = tmem + (u & 1) * 256u + lane_addr;
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        if (j0 + 32 * c >= p.J) break;
        uint32_t v[32];
        ptx::tmem_ld32(acc + 32 * c, v);
        ptx::tmem_wait_ld(v);
        if (iw < p.I) store_block<OP>(p, iw, j0 + 32 * c, v, rs, lane);
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive_cluster(ptx::cluster_addr(acc_empty(u & 1), 0));
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  ptx::cluster_sync();     // the other CTA neither reads nor signals this one any more
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, kTmemCols);
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
  constexpr size_t smem = Tile<BN>::template smem<OpTraits<OP>::b_mn>();
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((p.I + 2 * BM - 1) / (2 * BM)) * ((p.J + BN - 1) / BN);
  const int64_t pairs = device_info().num_sms / 2;
  kern<<<static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)), kThreads, smem, stream>>>(a, b, p,
                                                                                             device_error_word());
  return cudaGetLastError();
}

// Columns per tile: the width whose tiles fill the SM pairs in whole rounds
// with the least padding.  A round's time goes with the width down to about
// 180 columns, below which the loads of a bound it (one B200, int8, 2048 x 5120
// x 17408: three rounds of 256 take 168 us, three of 192 129 us, five of 128
// 203 us).  Wide tiles read less of a, so 256 unless a narrower one promises
// more than 12% (2048 x 17408 x 5120: 256 takes 126 us, 192 133 us for a
// promise of 6%).
int tile_columns(int64_t I, int64_t J) {
  const int64_t pairs = device_info().num_sms / 2, it = (I + 2 * BM - 1) / (2 * BM);
  auto cost = [&](int bn) {
    return static_cast<double>((it * ((J + bn - 1) / bn) + pairs - 1) / pairs) * (bn > 180 ? bn : 180);
  };
  int best = 256;
  for (int bn : {192, 128})
    if (cost(bn) < 0.88 * cost(256) && cost(bn) < cost(best)) best = bn;
  return best;
}

template <Op OP>
cudaError_t run_bn(int bn, const CUtensorMap& a, const CUtensorMap& b, const Args& p, cudaStream_t stream) {
  switch (bn) {
    case 128: return run<OP, 128>(a, b, p, stream);
    case 192: return run<OP, 192>(a, b, p, stream);
    default: return run<OP, 256>(a, b, p, stream);
  }
}

bool whole16(const void* out, int64_t row_bytes) {
  return row_bytes % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
}

}  // namespace

cudaError_t launch_dense_i8(const uint8_t* a, const uint8_t* b, const float* sx, const float* scales, int shift,
                            int64_t M, int64_t N, int64_t K, uint16_t* y, cudaStream_t stream) {
  const int64_t stride = stride_i8(K);
  CUtensorMap ma, mb;
  const int bn = tile_columns(M, N);
  if (!map_kmajor(&ma, a, true, M, stride, stride, BM) || !map_kmajor(&mb, b, true, N, stride, stride, bn / 2))
    return cudaErrorInvalidValue;
  Args p{M, N, static_cast<int>((K + 127) / 128), 1, y, sx, scales, shift, false, whole16(y, 2 * N)};
  return run_bn<kLinearI8>(bn, ma, mb, p, stream);
}

cudaError_t launch_dense_grad_x(const uint16_t* dy, const uint16_t* w, int64_t M, int64_t N, int64_t K, uint16_t* dx,
                                cudaStream_t stream) {
  CUtensorMap ma, mb;
  if (!map_kmajor(&ma, dy, false, M, N, 2 * stride_bf16(N), BM) || !map_mnmajor(&mb, w, 3, 1, N, K))
    return cudaErrorInvalidValue;
  Args p{M, K, static_cast<int>((N + 63) / 64), 1, dx, nullptr, nullptr, 0, false, whole16(dx, 2 * K)};
  return run_bn<kGradX>(tile_columns(M, K), ma, mb, p, stream);
}

cudaError_t launch_dense_grad_w(const uint16_t* dy, const uint16_t* x, int parts, int64_t M, int64_t N, int64_t K,
                                void* dw, bool f32, bool accumulate, cudaStream_t stream) {
  CUtensorMap ma, mb;
  if (!map_mnmajor(&ma, dy, 2, 1, M, N) || !map_mnmajor(&mb, x, 3, parts, M, K)) return cudaErrorInvalidValue;
  Args p{N, K, static_cast<int>((M + 63) / 64), parts, dw, nullptr, nullptr, 0, accumulate,
         whole16(dw, (f32 ? 4 : 2) * K)};
  const int bn = tile_columns(N, K);
  return f32 ? run_bn<kGradWF32>(bn, ma, mb, p, stream) : run_bn<kGradWBf16>(bn, ma, mb, p, stream);
}

}  // namespace mpw

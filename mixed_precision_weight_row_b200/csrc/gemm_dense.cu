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
// Two CTAs on neighbouring SMs (cta_group::2) compute tiles of 256 x BN results,
// each holding 128 rows of a, half of b's rows and its own 128 rows of the
// result; one CTA per SM walks over the tiles.  Warp 0 of each fills a ring of
// stages by TMA (128 bytes of r, or 64 steps of r, per stage and operand, in the
// 128-byte swizzle), one thread of the first CTA issues the products for both
// into one of two accumulators in tensor memory, and eight warps of each (two per
// 32 rows) write the other one out meanwhile: bf16 rows of whole, aligned 16-byte units by TMA
// from a block of 32 rows x 128 bytes per warp in shared memory, others by the
// lanes, which exchange values for coalesced stores in eight times the
// instructions (grad_w of 64 x 17408 x 5120, which writes 178 MB: 37 us by TMA,
// 48 by lanes).  fp32 results stay with the lanes, which add to memory as well
// and leave the ring its last stage: by TMA 16 x 5120 x 17408 took 77 us against
// 81, but 256 x 4096 x 4096 39 against 33 and 1000 x 4096 x 4096 107 against 87.
// Tiles run in groups of kGroup along i, so that the CTAs working at one time
// share operand rows in L2.
//
// Tiles that do not fill a last round of the SM pairs are cut into slices of r
// for all of them: a slice leaves its sums in a workspace, and a second kernel
// adds the slices of a tile in their order and writes it.  (Letting the slice
// that arrives last do so cost 40 us where this takes 5: one CTA pair reads what
// here the whole GPU reads.)
//
// The fp32 result of grad_w is meant to hold fp32 accuracy.  Its operand x comes
// as three bf16 values whose products are summed one after another, the
// smallest first, and since tensor cores truncate a sum at every step (2048
// tokens in one go are off by 2.1e-6 of the norm, 8192 by 9e-6, operands of one
// sign by 5.6e-6 and 35e-6), the sum runs over equal chunks of at most 768 tokens
// that the epilogue adds, rounding to nearest, to the tile in memory (it stays in
// L2).  Off by 0.45e-6 with 1000 tokens, 0.6e-6 with 2048, 0.7e-6 with 8192;
// operands of one sign 0.9e-6, 1.2e-6, 1.3e-6.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "int8_expand.cuh"
#include "int8_internal.h"
#include "lane_units.cuh"
#include "mpw_internal.h"
#include "tc_ptx.cuh"

namespace mpw {
namespace {

constexpr int BM = 128;                  // rows of a tile per CTA of a pair
constexpr int kThreads = 384;
constexpr int kEpiWarp0 = 4;            // eight epilogue warps: two per 32 rows
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
  static constexpr int chunk = OP == kGradWF32 ? 12 : 0;    // stages along r per chunk at most (0: all of them)
};

constexpr uint32_t kOutBlock = 32 * 128;        // 32 rows x 128 bytes of a result, per epilogue warp

template <Op OP, int BN>
struct Tile {
  static constexpr uint32_t kStage = kABytes + BN / 2 * 128;     // half of the pair's rows of b
  static constexpr uint32_t kOutBytes = OP == kGradWF32 ? 0 : 8 * kOutBlock;
  static constexpr int S = static_cast<int>((232448 - 1024 /*align*/ - kOutBytes - 256 /*barriers*/) / kStage);
  static constexpr size_t kSmem = S * kStage + 1024 + kOutBytes + 256;
};
constexpr int kSlicedBN = 256;                                   // the width of tiles that may be sliced
constexpr uint32_t kPartialWords = BM * kSlicedBN;               // sums of one CTA's half of a tile

struct Args {
  int64_t I, J;          // results
  int blocks;            // stages along r
  int parts;             // slices of b (with chunks), each read over all of r
  int whole;             // tiles done in one piece; those behind them in slices
  int slices;
  uint32_t* partial;     // sums of slices: [tile - whole][slice][256 rows x BN]
  void* out;             // [I, J]
  const float* row_scale;
  const float* col_scale;
  int shift;
  bool accumulate;
  bool vec;              // rows of out are whole, aligned 16-byte units (tmap_out is then valid for bf16)
};

// C columns of a row, scaled (int8 linear) and rounded to bf16, as pairs.
template <Op OP, int C>
__device__ __forceinline__ void bf16_pairs(const Args& p, int64_t c0, uint32_t (&v)[C], float rs, int lane,
                                           uint32_t (&o)[C / 2]) {
  if constexpr (OP == kLinearI8) {
    const int64_t left = p.J - c0;
#pragma unroll
    for (int h = 0; h < C / 32; ++h) {
      const float mine = 32 * h + lane < left ? __ldg(p.col_scale + c0 + 32 * h + lane) : 0.0f;
      auto scale = [&](auto of) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float cs = __shfl_sync(0xffffffffu, mine, c);
          uint32_t& d = v[32 * h + c];
          d = __float_as_uint(of(static_cast<int32_t>(d) >> p.shift, cs));
        }
      };
      // as a rule no column's scale is large (i8::RowScale)
      if (__any_sync(0xffffffffu, mine > i8::RowScale::kLarge))
        scale([&](int32_t sum, float cs) { return i8::RowScale(cs).of(sum, rs); });
      else
        scale([&](int32_t sum, float cs) { return static_cast<float>(sum) * cs * rs; });
    }
  }
#pragma unroll
  for (int c = 0; c < C / 2; ++c) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1]));
    o[c] = *reinterpret_cast<const uint32_t*>(&r);
  }
}

// Writes 64 columns c0 .. c0 + 63 of the 32 bf16 rows i0 .. i0 + 31, of which this
// lane holds row i0 + lane, by TMA from `block` (this warp's 4 KB of shared memory,
// in the 128-byte swizzle).
template <Op OP>
__device__ __forceinline__ void store_block_tma(const Args& p, const void* tmap, uint8_t* block, int64_t i0, int64_t c0,
                                                uint32_t (&v)[64], float rs, int lane) {
  uint32_t o[32];
  bf16_pairs<OP, 64>(p, c0, v, rs, lane, o);
  if (lane == 0) ptx::bulk_wait_read();      // the block's last store has read it
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 8; ++q)
    *reinterpret_cast<uint4*>(block + lane * 128 + 16 * (q ^ (lane & 7))) =
        make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
  ptx::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    ptx::tma_store_2d(tmap, ptx::smem_addr(block), static_cast<int32_t>(c0), static_cast<int32_t>(i0));
    ptx::bulk_commit();
  }
}

// Writes C columns c0 .. c0 + C - 1 of the 32 result rows i0 .. i0 + 31, of which
// this lane holds row i0 + lane (C = 32, or 64 for bf16: 128 bytes of a row
// either way).  A lane writing its own row would scatter a store over 32
// rows; the values change lanes first, so that neighbouring lanes write
// neighbouring 16-byte units (rows of whole, aligned units) or neighbouring
// values (any other rows).
template <Op OP, int C>
__device__ __forceinline__ void store_block(const Args& p, int64_t i0, int64_t c0, uint32_t (&v)[C], float rs,
                                            bool add, int lane) {
  const int64_t left = p.J - c0, rows = p.I - i0;
  if constexpr (OP == kGradWF32) {
    static_assert(C == 32, "fp32 blocks");
    float* out = static_cast<float*>(p.out) + i0 * p.J + c0;
    if (p.vec) {
      transpose_units<8, 4>(v, lane);
      const int q = lane & 7, r0 = lane & ~7;
      auto unit = [&](int t) { return reinterpret_cast<float4*>(out + (r0 + t) * p.J) + q; };
      const bool mine = 4 * q < left;
      if (add) {      // every read before the first write, so that they overlap
        float4 old[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) old[t] = mine && r0 + t < rows ? *unit(t) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          v[4 * t] = __float_as_uint(old[t].x + __uint_as_float(v[4 * t]));
          v[4 * t + 1] = __float_as_uint(old[t].y + __uint_as_float(v[4 * t + 1]));
          v[4 * t + 2] = __float_as_uint(old[t].z + __uint_as_float(v[4 * t + 2]));
          v[4 * t + 3] = __float_as_uint(old[t].w + __uint_as_float(v[4 * t + 3]));
        }
      }
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (mine && r0 + t < rows)
          *unit(t) = make_float4(__uint_as_float(v[4 * t]), __uint_as_float(v[4 * t + 1]),
                                 __uint_as_float(v[4 * t + 2]), __uint_as_float(v[4 * t + 3]));
    } else {
      transpose_units<32, 1>(v, lane);
      float* dst = out + lane;
      if (add) {
#pragma unroll
        for (int h = 0; h < 32; h += 8) {      // eight rows' reads at a time
          float old[8];
#pragma unroll
          for (int t = 0; t < 8; ++t) old[t] = h + t < rows && lane < left ? dst[(h + t) * p.J] : 0.0f;
#pragma unroll
          for (int t = 0; t < 8; ++t) v[h + t] = __float_as_uint(old[t] + __uint_as_float(v[h + t]));
        }
      }
#pragma unroll
      for (int t = 0; t < 32; ++t)
        if (t < rows && lane < left) dst[t * p.J] = __uint_as_float(v[t]);
    }
  } else {
    uint32_t o[C / 2];
    bf16_pairs<OP, C>(p, c0, v, rs, lane, o);
    uint16_t* out = static_cast<uint16_t*>(p.out) + i0 * p.J + c0;
    if (p.vec) {
      constexpr int U = C / 8;
      transpose_units<U, 4>(o, lane);
      const int q = lane % U, r0 = lane - q;
#pragma unroll
      for (int t = 0; t < U; ++t)
        if (r0 + t < rows && 8 * q < left)
          reinterpret_cast<uint4*>(out + (r0 + t) * p.J)[q] =
              make_uint4(o[4 * t], o[4 * t + 1], o[4 * t + 2], o[4 * t + 3]);
    } else {
      // C / 2 lanes end up with a pair of columns each, of C / 2 rows at a time
      constexpr int U = C / 2;
      transpose_units<U, 1>(o, lane);
      const int q = lane % U, r0 = lane - q;
#pragma unroll
      for (int t = 0; t < U; ++t) {
        if (r0 + t >= rows) continue;
        uint16_t* dst = out + (r0 + t) * p.J + 2 * q;
        if (2 * q < left) dst[0] = static_cast<uint16_t>(o[t]);
        if (2 * q + 1 < left) dst[1] = static_cast<uint16_t>(o[t] >> 16);
      }
    }
  }
}

// First row (of CTA `rank`'s half) and column of tile t.
template <int BN>
__device__ __forceinline__ void tile_place(const Args& p, int t, int rank, int64_t& i0, int64_t& j0) {
  const int IT = static_cast<int>((p.I + 2 * BM - 1) / (2 * BM)), JT = static_cast<int>((p.J + BN - 1) / BN);
  const int g = t / (kGroup * JT), in = t - g * kGroup * JT;
  const int rows = min(kGroup, IT - g * kGroup);
  i0 = static_cast<int64_t>(g * kGroup + in % rows) * (2 * BM) + rank * BM;
  j0 = static_cast<int64_t>(in / rows) * BN;
}

// Where the sums of 32 rows (quad) x 32 columns (c) of a slice are kept: 16-byte
// unit q of lane l at 32 q + l.
__device__ __forceinline__ uint4* partial_block(const Args& p, int64_t item, int rank, int quad, int c) {
  return reinterpret_cast<uint4*>(p.partial + (item * 2 + rank) * kPartialWords) + (quad * (kSlicedBN / 32) + c) * 256;
}

template <Op OP, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
dense_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
             const __grid_constant__ CUtensorMap tmap_out, const __grid_constant__ Args p, int32_t* err) {
  using T = OpTraits<OP>;
  static_assert(!T::b_mn || BN % 128 == 0, "whole chunks of an MN-major b per CTA");
  constexpr uint32_t kStage = Tile<OP, BN>::kStage;
  constexpr int S = Tile<OP, BN>::S;
  constexpr int32_t kW = ptx::kWaitDense;
  extern __shared__ uint8_t dsmem_raw[];
  const uint32_t raw = ptx::smem_addr(dsmem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;       // 1024-aligned for the 128-byte swizzle
  uint8_t* out_blocks = dsmem_raw + (base - raw) + S * kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(out_blocks + Tile<OP, BN>::kOutBytes);
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
      ptx::mbar_init(acc_empty(s), 16);      // both CTAs' epilogues, a lane for a warp
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
  ptx::grid_dep_wait_then_release();

  const int tiles = static_cast<int>(((p.I + 2 * BM - 1) / (2 * BM)) * ((p.J + BN - 1) / BN));
  // work items: whole tiles, then slices of the others; an item is a range of
  // chunks of r, or, of the only one, a range of its stages
  const int items = p.whole + (tiles - p.whole) * p.slices;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  auto slice_of = [&](int it, int n, int& n0, int& n1) {
    n0 = 0;
    n1 = n;
    if (it >= p.whole) {
      const int64_t slice = (it - p.whole) % p.slices;
      n0 = static_cast<int>(n * slice / p.slices);
      n1 = static_cast<int>(n * (slice + 1) / p.slices);
    }
  };
  const int chunks = T::chunk > 0 ? (p.blocks + T::chunk - 1) / T::chunk : 1;      // of equal length
  auto chunks_of = [&](int it, int& c0, int& c1) {
    c0 = 0;
    c1 = 1;
    if constexpr (T::chunk > 0) slice_of(it, chunks, c0, c1);
  };
  // first stage along r and number of stages (all parts) of a chunk of an item
  auto stages_of = [&](int it, int c, int& rb0, int& n) {
    if constexpr (T::chunk > 0) {
      rb0 = static_cast<int>(static_cast<int64_t>(p.blocks) * c / chunks);
      n = (static_cast<int>(static_cast<int64_t>(p.blocks) * (c + 1) / chunks) - rb0) * p.parts;
    } else {
      int rb1;
      slice_of(it, p.blocks, rb0, rb1);
      n = rb1 - rb0;
    }
  };
  auto place = [&](int it, int64_t& i0, int64_t& j0) {
    tile_place<BN>(p, it < p.whole ? it : p.whole + (it - p.whole) / p.slices, static_cast<int>(rank), i0, j0);
  };

  if (warp == 0) {
    // ---------------- producer ----------------
    if (ptx::elect_one()) {
      // both CTAs' loads complete on the first one's barriers, where the
      // products are issued
      bool ok = true;
      uint32_t n = 0;                       // stages filled so far
      for (int it = first; it < items && ok; it += step) {
        int64_t i64, j64;
        int c0, c1;
        place(it, i64, j64);
        chunks_of(it, c0, c1);
        const int i0 = static_cast<int>(i64), j0 = static_cast<int>(j64) + static_cast<int>(rank) * (BN / 2);
        for (int ch = c0; ch < c1 && ok; ++ch) {
          int rb0, stages;
          stages_of(it, ch, rb0, stages);
          const int each = T::chunk > 0 ? stages / p.parts : stages;
          for (int st = 0, pass = 0, in = 0; st < stages; ++st, ++n) {
            const int s = n % S;
            ok = ptx::mbar_wait(empty(s), ((n / S) & 1) ^ 1, err, ptx::wait_code(kW, ptx::kWaitXEmpty));
            if (!ok) break;
            const int r0 = (rb0 + in) * T::depth, part = p.parts - 1 - pass;
            if (++in == each) {
              in = 0;
              ++pass;
            }
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
              for (int c = 0; c < BN / 128; ++c)
                ptx::tma_load_3d_pair(sb + c * 8192, &tmap_b, bar, j0 + 64 * c, r0, part);
            } else {
              ptx::tma_load_2d_pair(sb, &tmap_b, bar, r0, j0);
            }
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
        for (int it = first; it < items && ok; it += step) {
          int c0, c1;
          chunks_of(it, c0, c1);
          for (int ch = c0; ch < c1; ++ch, ++u) {
            int rb0, stages;
            stages_of(it, ch, rb0, stages);
            const uint32_t acc = tmem + (u & 1) * 256u;
            ok = ptx::mbar_wait(acc_empty(u & 1), ((u >> 1) & 1) ^ 1, err, ptx::wait_code(kW, ptx::kWaitAccEmpty));
            if (!ok) break;
            ptx::tc_fence_after();
            for (int st = 0; st < stages; ++st) {
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
                ptx::mma_ss<2, T::i8>(acc, ad + da * k, bd + db * k, idesc, (st | k) != 0);
              ptx::mma_commit_pair(empty(s));
              if (++s == S) {
                s = 0;
                phase ^= 1;
              }
            }
            ptx::mma_commit_pair(acc_full(u & 1));
            if (!ok) break;
          }
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
    const int quad = warp & 3, half = (warp - kEpiWarp0) >> 2;     // rows, and which blocks of columns
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t u = 0;
    bool ok = true;
    for (int it = first; it < items && ok; it += step) {
      int64_t i0, j0;
      int c0, c1;
      place(it, i0, j0);
      chunks_of(it, c0, c1);
      const int64_t iw = i0 + quad * 32;      // the warp's first row
      const float rs = OP == kLinearI8 && iw + lane < p.I ? __ldg(p.row_scale + iw + lane) : 0.0f;
      for (int ch = c0; ch < c1; ++ch, ++u) {
        ok = ptx::mbar_wait(acc_full(u & 1), (u >> 1) & 1, err, ptx::wait_code(kW, ptx::kWaitAcc));
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t acc = tmem + (u & 1) * 256u + lane_addr;
        const bool sliced = it >= p.whole;
        const int tail = it - p.whole;
        constexpr int C = OP == kGradWF32 ? 32 : 64;      // columns per step
        const int cols = static_cast<int>(min(static_cast<int64_t>(BN / C), (p.J - j0 + C - 1) / C));
#pragma unroll 1
        for (int c = half; c < cols; c += 2) {
          uint32_t v[C];
#pragma unroll
          for (int h = 0; h < C / 32; ++h) ptx::tmem_ld32(acc + C * c + 32 * h, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * h));
#pragma unroll
          for (int h = 0; h < C / 32; ++h) ptx::tmem_wait_ld(*reinterpret_cast<uint32_t(*)[32]>(v + 32 * h));
          if (iw >= p.I) continue;
          if (OP != kGradWF32 && !sliced && p.vec) {
            if constexpr (OP != kGradWF32)
              store_block_tma<OP>(p, &tmap_out, out_blocks + (warp - kEpiWarp0) * kOutBlock, iw, j0 + C * c, v, rs, lane);
          } else if (!sliced) {
            store_block<OP, C>(p, iw, j0 + C * c, v, rs, p.accumulate || ch > c0, lane);
          } else {
#pragma unroll
            for (int h = 0; h < C / 32; ++h) {
              uint4* dst = partial_block(p, tail, static_cast<int>(rank), quad, C / 32 * c + h) + lane;
              uint32_t* w = v + 32 * h;
              if (T::chunk > 0 && ch > c0) {        // this lane's own words of the chunk before
                uint4 old[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) old[q] = dst[32 * q];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                  const uint32_t x[4] = {old[q].x, old[q].y, old[q].z, old[q].w};
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    w[4 * q + k] = __float_as_uint(__uint_as_float(x[k]) + __uint_as_float(w[4 * q + k]));
                }
              }
#pragma unroll
              for (int q = 0; q < 8; ++q) dst[32 * q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
            }
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(ptx::cluster_addr(acc_empty(u & 1), 0));
      }
    }
    if (lane == 0) ptx::bulk_wait();
  }
  __syncwarp();
  ptx::tc_fence_before();
  ptx::cluster_sync();     // the other CTA neither reads nor signals this one any more
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// Adds the slices of the tiles behind the whole ones: a warp for 32 rows x 32
// columns.
constexpr int kJoinThreads = 128;
constexpr int kJoinBlocks = 2 * 4 * (kSlicedBN / 32) * 32 / kJoinThreads;     // per tile
template <Op OP>
__global__ void __launch_bounds__(kJoinThreads)
dense_join_kernel(const __grid_constant__ Args p) {
  ptx::grid_dep_wait_then_release();
  constexpr int BN = kSlicedBN;
  const int lane = threadIdx.x & 31;
  const int tail = static_cast<int>(blockIdx.x) / kJoinBlocks;
  const int block = (blockIdx.x % kJoinBlocks) * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const int c = block % (BN / 32), quad = block / (BN / 32) % 4, rank = block / (BN / 32) / 4;
  int64_t i0, j0;
  tile_place<BN>(p, p.whole + tail, rank, i0, j0);
  i0 += quad * 32;
  j0 += 32 * c;
  if (i0 >= p.I || j0 >= p.J) return;
  uint32_t v[32];
#pragma unroll 2
  for (int s = 0; s < p.slices; ++s) {
    const uint4* src = partial_block(p, static_cast<int64_t>(tail) * p.slices + s, rank, quad, c) + lane;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint4 w = src[32 * q];
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t& d = v[4 * q + k];
        d = s == 0 ? x[k] : __float_as_uint(__uint_as_float(d) + __uint_as_float(x[k]));
      }
    }
  }
  store_block<OP, 32>(p, i0, j0, v, 0.0f, p.accumulate, lane);
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

int64_t sm_pairs() {
  const int64_t pairs = device_info().num_sms / 2;
  return pairs < 1 ? 1 : pairs;
}
int64_t tile_count(int64_t I, int64_t J, int bn) { return ((I + 2 * BM - 1) / (2 * BM)) * ((J + bn - 1) / bn); }

// Columns per tile of the int8 product: the width whose tiles fill the SM pairs
// in whole rounds with the least padding.  A round's time goes with the width
// down to about 180 columns, below which the loads of a bound it (one B200,
// 2048 x 5120 x 17408: three rounds of 256 take 168 us, three of 192 129 us, five
// of 128 203 us).  Wide tiles read less of a, so 256 unless a narrower one
// promises more than 12% (2048 x 17408 x 5120: 256 takes 126 us, 192 133 us for
// a promise of 6%).
int tile_columns(int64_t I, int64_t J) {
  auto cost = [&](int bn) {
    return static_cast<double>((tile_count(I, J, bn) + sm_pairs() - 1) / sm_pairs()) * (bn > 180 ? bn : 180);
  };
  int best = 256;
  for (int bn : {192, 128})
    if (cost(bn) < 0.88 * cost(256) && cost(bn) < cost(best)) best = bn;
  return best;
}

// How the tiles of a bf16 product run (always 256 wide: a half of 192 columns of
// an MN-major b would be one and a half chunks, loaded as two): `whole` of them in
// rounds of one per pair of SMs, the rest in slices.  A stage takes a pair
// about 0.38 us, leaving the sums of slices and adding them about 10 us (one
// B200, grad_x of 2048 x 17408 x 5120: 330 us with 192-wide tiles in three
// rounds, 262 us with two rounds of 256 and 12 tiles in six slices).
struct Plan {
  int64_t tiles, whole;
  int slices;
};
Plan plan_tiles(int64_t I, int64_t J, int64_t stages, int64_t most_slices) {
  const int64_t pairs = sm_pairs(), tiles = tile_count(I, J, kSlicedBN), rest = tiles % pairs;
  Plan p{tiles, tiles, 1};
  if (rest == 0) return p;
  double best = static_cast<double>(stages) * 0.38;
  for (int64_t s = 2; s * rest <= pairs && s <= most_slices; ++s) {
    const double us = static_cast<double>((stages + s - 1) / s) * 0.38 + 10.0;
    if (us < best) {
      best = us;
      p.slices = static_cast<int>(s);
    }
  }
  if (p.slices > 1) p.whole = tiles - rest;
  return p;
}

bool whole_units(const void* out, int64_t row_bytes) {
  return row_bytes % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
}

// The bf16 result, for stores of 32 rows x 128 bytes.
bool map_out(CUtensorMap* m, void* out, int64_t rows, int64_t cols) {
  auto encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  const cuuint32_t box[2] = {64, 32};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Slices of at least four stages, or (fp32 grad_w, three parts) of whole chunks.
Plan plan_for(int64_t I, int64_t J, int64_t blocks, int parts) {
  constexpr int64_t chunk = OpTraits<kGradWF32>::chunk;
  return plan_tiles(I, J, blocks * parts, parts > 1 ? (blocks + chunk - 1) / chunk : blocks / 4);
}

template <Op OP, int BN>
cudaError_t run(const CUtensorMap& a, const CUtensorMap& b, Args p, const Plan& plan, cudaStream_t stream) {
  CUtensorMap out = a;      // unused unless rows are written by TMA
  p.vec = whole_units(p.out, p.J * (OP == kGradWF32 ? 4 : 2));
  if (OP != kGradWF32 && p.vec && !map_out(&out, p.out, p.I, p.J)) return cudaErrorInvalidValue;
  auto kern = dense_kernel<OP, BN>;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), Tile<OP, BN>::kSmem);
  if (e != cudaSuccess) return e;
  p.whole = static_cast<int>(plan.whole);
  p.slices = plan.slices;
  const int64_t items = plan.whole + (plan.tiles - plan.whole) * plan.slices, pairs = sm_pairs();
  return launch_behind(kern, static_cast<unsigned>(2 * (items < pairs ? items : pairs)), kThreads, Tile<OP, BN>::kSmem,
                       stream, a, b, out, p, device_error_word());
}

template <Op OP>
cudaError_t run_sliced(const CUtensorMap& a, const CUtensorMap& b, Args p, void* ws, cudaStream_t stream) {
  const Plan plan = plan_for(p.I, p.J, p.blocks, p.parts);
  p.partial = static_cast<uint32_t*>(ws);
  const cudaError_t e = run<OP, kSlicedBN>(a, b, p, plan, stream);
  if (e != cudaSuccess || plan.slices == 1) return e;
  p.vec = whole_units(p.out, p.J * (OP == kGradWF32 ? 4 : 2));
  p.whole = static_cast<int>(plan.whole);
  p.slices = plan.slices;
  return launch_behind(dense_join_kernel<OP>, static_cast<unsigned>((plan.tiles - plan.whole) * kJoinBlocks),
                       kJoinThreads, 0, stream, p);
}

}  // namespace

size_t dense_workspace_bytes(int64_t I, int64_t J, int64_t depth, int parts) {
  const Plan p = plan_for(I, J, (depth + 63) / 64, parts);
  if (p.slices == 1) return 0;
  return static_cast<size_t>(p.tiles - p.whole) * static_cast<size_t>(p.slices) * 2 * kPartialWords * 4;
}

cudaError_t launch_dense_i8(const uint8_t* a, const uint8_t* b, const float* sx, const float* scales, int shift,
                            int64_t M, int64_t N, int64_t K, uint16_t* y, cudaStream_t stream) {
  const int64_t stride = stride_i8(K);
  const int bn = tile_columns(M, N);
  CUtensorMap ma, mb;
  if (!map_kmajor(&ma, a, true, M, stride, stride, BM) || !map_kmajor(&mb, b, true, N, stride, stride, bn / 2))
    return cudaErrorInvalidValue;
  Args p{};
  p.I = M;
  p.J = N;
  p.blocks = static_cast<int>((K + 127) / 128);
  p.parts = 1;
  p.out = y;
  p.row_scale = sx;
  p.col_scale = scales;
  p.shift = shift;
  const int64_t tiles = tile_count(M, N, bn);
  const Plan plan{tiles, tiles, 1};
  switch (bn) {
    case 128: return run<kLinearI8, 128>(ma, mb, p, plan, stream);
    case 192: return run<kLinearI8, 192>(ma, mb, p, plan, stream);
    default: return run<kLinearI8, 256>(ma, mb, p, plan, stream);
  }
}

cudaError_t launch_dense_grad_x(const uint16_t* dy, const uint16_t* w, int64_t M, int64_t N, int64_t K, uint16_t* dx,
                                void* ws, cudaStream_t stream) {
  CUtensorMap ma, mb;
  if (!map_kmajor(&ma, dy, false, M, N, 2 * stride_bf16(N), BM) || !map_mnmajor(&mb, w, 3, 1, N, K))
    return cudaErrorInvalidValue;
  Args p{};
  p.I = M;
  p.J = K;
  p.blocks = static_cast<int>((N + 63) / 64);
  p.parts = 1;
  p.out = dx;
  return run_sliced<kGradX>(ma, mb, p, ws, stream);
}

cudaError_t launch_dense_grad_w(const uint16_t* dy, const uint16_t* x, int parts, int64_t M, int64_t N, int64_t K,
                                void* dw, bool f32, bool accumulate, void* ws, cudaStream_t stream) {
  CUtensorMap ma, mb;
  if (!map_mnmajor(&ma, dy, 2, 1, M, N) || !map_mnmajor(&mb, x, 3, parts, M, K)) return cudaErrorInvalidValue;
  Args p{};
  p.I = N;
  p.J = K;
  p.blocks = static_cast<int>((M + 63) / 64);
  p.parts = parts;
  p.out = dw;
  p.accumulate = accumulate;
  return f32 ? run_sliced<kGradWF32>(ma, mb, p, ws, stream) : run_sliced<kGradWBf16>(ma, mb, p, ws, stream);
}

}  // namespace mpw

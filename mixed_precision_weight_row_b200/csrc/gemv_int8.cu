// Int8 linear for a few tokens: y[m, n] = bf16(s_n sx_m sum_k xq[m, k] q[n, k]).
//
// The packed rows are the cost (N * K * b / 8 bytes, read once); a row's codes
// meet M tokens, so the work is the expansion plus M integer dot products.
// Expanding four codes to signed bytes takes 4 to 7 integer operations
// (int8_expand.cuh) and one dp4a per token multiplies them.
//
// A CTA owns a contiguous share of the rows (c N / G .. (c + 1) N / G) and its
// warps take units of R rows in turn.  Every warp streams its own units: one
// lane keeps P row segments (whole rows up to kSegment codes) in flight as
// untiled bulk copies into slots that only this warp reads, and refills a slot
// as soon as the warp has read it, so no warp waits for another and the copies
// of an SM are issued by all of its warps (one thread issuing for all of
// them managed one copy per 130 ns and bound the kernel).  Lane l takes the
// 32-code groups l, l + 32, ... of a segment, x comes from shared memory, and
// one warp-wide integer reduction per result ends a row.  The weights do not
// depend on the launch before, so their first copies start before the wait
// for it (programmatic dependent launch); x is read after it, and like the
// other decode kernels this one lets its successor start only after its own
// wait.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "int8_expand.cuh"
#include "int8_internal.h"
#include "mpw_internal.h"
#include "tc_ptx.cuh"

namespace mpw {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kMaxSlots = 4;                      // per warp
constexpr int kSegment = 8192;                    // codes per slot and row at most
constexpr uint32_t kSmemTwo = 104 * 1024;         // per CTA, two on an SM
constexpr uint32_t kSmemMax = 220 * 1024;

struct Args {
  const uint8_t* xq;
  const float* sx;
  const uint8_t* packed;
  const float* scales;
  uint16_t* y;
  int64_t N;
  int M, K;
  int xstride;      // bytes between tokens of xq
  int rb;           // bytes of a packed row
  int segments;     // per row
  int seg_codes;    // codes per segment (a multiple of 1024; the last one shorter)
  int slots;        // per warp
};

__host__ __device__ constexpr uint32_t x_bytes(int MT, int K) {
  return static_cast<uint32_t>(MT) * static_cast<uint32_t>((K + 31) / 32) * 32u;
}

// MT: tokens (M <= MT, the others are zero), R: rows per unit.
template <int B, bool PAIRED, int MT, int R>
__global__ void __launch_bounds__(kMaxWarps * 32, 2)
gemv_i8_kernel(const __grid_constant__ Args p, int32_t* err) {
  extern __shared__ __align__(128) uint8_t vsmem[];
  __shared__ uint64_t bars[kMaxWarps * kMaxSlots];
  constexpr int32_t kW = ptx::kWaitGemvI8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int G = (p.K + 31) >> 5;
  const int seg_bytes = p.seg_codes / 8 * B;
  // x: two planes of 16 bytes per group and token, so that the lanes of a warp
  // read consecutive 16-byte units
  uint8_t* xs = vsmem;
  uint8_t* ring = vsmem + x_bytes(MT, p.K) + static_cast<uint32_t>(warp * p.slots * R) * seg_bytes;
  const uint32_t bar0 = ptx::smem_addr(bars + warp * kMaxSlots);
  const int64_t row0 = p.N * blockIdx.x / gridDim.x, row1 = p.N * (blockIdx.x + 1) / gridDim.x;
  const int units = static_cast<int>((row1 - row0 + R - 1) / R);
  const int mine = warp < units ? (units - 1 - warp) / warps + 1 : 0;
  const int steps = mine * p.segments;          // slots this warp fills and reads

  // step i of this warp: segment i % segments of unit warp + (i / segments) * warps
  auto fill = [&](int i, int slot) {
    const int seg = i % p.segments;
    const int64_t r = row0 + static_cast<int64_t>(warp + i / p.segments * warps) * R;
    const uint32_t bytes = static_cast<uint32_t>(min(seg_bytes, p.rb - seg * seg_bytes));
    const int rows = static_cast<int>(min(static_cast<int64_t>(R), row1 - r));
    const uint32_t bar = bar0 + 8u * slot, dst = ptx::smem_addr(ring) + static_cast<uint32_t>(slot * R) * seg_bytes;
    const uint8_t* src = p.packed + r * p.rb + static_cast<int64_t>(seg) * seg_bytes;
    ptx::mbar_arrive_expect_tx(bar, rows * bytes);
    for (int j = 0; j < rows; ++j) ptx::bulk_load(dst + j * seg_bytes, src + static_cast<int64_t>(j) * p.rb, bytes, bar);
  };
  if (lane == 0) {
    for (int s = 0; s < p.slots; ++s) ptx::mbar_init(bar0 + 8u * s, 1);
    ptx::mbar_fence_init();
    for (int i = 0; i < min(p.slots, steps); ++i) fill(i, i);
  }

  ptx::grid_dep_wait_then_release();
  // x into shared memory, zero past K and for tokens past M
  for (int i = threadIdx.x; i < MT * G; i += blockDim.x) {
    const int t = i / G, g = i - t * G;
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    const uint4* src = reinterpret_cast<const uint4*>(p.xq + static_cast<int64_t>(t) * p.xstride) + 2 * g;
    if (t < p.M) {
      lo = __ldg(src);
      if (32 * g + 16 < p.xstride) hi = __ldg(src + 1);
    }
    const uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t o[8];
    i8::order_x<B, PAIRED>(v, o);
    reinterpret_cast<uint4*>(xs)[(t * 2) * G + g] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(xs)[(t * 2 + 1) * G + g] = make_uint4(o[4], o[5], o[6], o[7]);
  }
  const float sx = lane < p.M ? __ldg(p.sx + lane) : 0.0f;
  __syncthreads();

  int slot = 0;
  uint32_t phase = 0;
  int32_t acc[R][MT];
  float sn[R];
  for (int i = 0, seg = 0; i < steps; ++i) {
    const int64_t r0 = row0 + static_cast<int64_t>(warp + i / p.segments * warps) * R;
    if (seg == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        sn[r] = r0 + r < row1 ? __ldg(p.scales + r0 + r) : 0.0f;
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[r][t] = 0;
      }
    }
    if (!ptx::mbar_wait(bar0 + 8u * slot, phase, err, ptx::wait_code(kW, ptx::kWaitWFull))) {
      // nothing may still be landing in shared memory when the CTA exits
      for (int j = i + 1; j < min(i + p.slots, steps); ++j) {
        if (++slot == p.slots) {
          slot = 0;
          phase ^= 1;
        }
        ptx::mbar_wait(bar0 + 8u * slot, phase, err, ptx::wait_code(kW, ptx::kWaitWTail));
      }
      break;
    }
    const uint8_t* w0 = ring + static_cast<uint32_t>(slot * R) * seg_bytes;
    const int g0 = seg * (p.seg_codes >> 5), g1 = min(G, g0 + (p.seg_codes >> 5));
#pragma unroll 1
    for (int g = g0 + lane; g < g1; g += 32) {
      uint32_t o[R][8];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        // a last group may reach past its row (and a last unit hold fewer than
        // R rows): what is read there meets zeros of x or is not written
        uint32_t w[B + 1];
        i8::lds_group<B>(w0 + r * seg_bytes + (g - g0) * 4 * B, w);
        i8::group_ordered<B, PAIRED>(w, o[r]);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint4 a = reinterpret_cast<const uint4*>(xs)[(t * 2) * G + g];
        const uint4 b = reinterpret_cast<const uint4*>(xs)[(t * 2 + 1) * G + g];
        const uint32_t xv[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            acc[r][t] = __dp4a(static_cast<int>(o[r][k]), static_cast<int>(xv[k]), acc[r][t]);
      }
    }
    __syncwarp();
    if (lane == 0 && i + p.slots < steps) {
      // the async-proxy refill of this slot must not overtake these reads
      ptx::fence_proxy_async_smem();
      fill(i + p.slots, slot);
    }
    if (++slot == p.slots) {
      slot = 0;
      phase ^= 1;
    }
    if (++seg < p.segments) continue;
    seg = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      int32_t sum = 0;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int32_t all = __reduce_add_sync(0xffffffffu, acc[r][t]);
        if (lane == t) sum = all;
      }
      if (lane < p.M && r0 + r < row1)
        p.y[static_cast<int64_t>(lane) * p.N + r0 + r] =
            __bfloat16_as_ushort(__float2bfloat16_rn(i8::RowScale(sn[r]).of(sum >> (8 - B), sx)));
    }
  }
}

// Shared memory past the last slot that a last group's read may touch.
constexpr uint32_t kTail = 64;

// Segments of a row: equal ones of at most kSegment codes, in whole rounds of
// a warp (32 lanes x 32 codes).
void segments_of(int K, int* count, int* codes) {
  const int n = (K + kSegment - 1) / kSegment;
  *codes = ((K + n - 1) / n + 1023) / 1024 * 1024;
  *count = (K + *codes - 1) / *codes;
}

template <int B, bool PAIRED, int MT, int R>
cudaError_t run(Args p, cudaStream_t stream) {
  const uint32_t xb = x_bytes(MT, p.K);
  const int64_t ctas = 2 * static_cast<int64_t>(device_info().num_sms);
  const unsigned grid = static_cast<unsigned>(p.N < ctas ? p.N : ctas);
  const int64_t units = (p.N / grid + 1 + R - 1) / R;
  segments_of(p.K, &p.segments, &p.seg_codes);
  const uint32_t slot = static_cast<uint32_t>(R) * (p.seg_codes / 8 * B);
  // two CTAs per SM when each then has room for eight warps, else one
  int64_t room = (static_cast<int64_t>(kSmemTwo) - xb - kTail) / slot;
  if (room < 8) room = (static_cast<int64_t>(kSmemMax) - xb - kTail) / slot;
  const int warps = static_cast<int>(units < room ? (units < kMaxWarps ? units : kMaxWarps)
                                                  : (room < kMaxWarps ? room : kMaxWarps));
  const int64_t steps = (units + warps - 1) / warps * p.segments;      // slots a warp can use at all
  const int64_t each = room / warps < steps ? room / warps : steps;
  p.slots = static_cast<int>(each < kMaxSlots ? each : kMaxSlots);
  const size_t smem = xb + kTail + static_cast<size_t>(warps * p.slots) * slot;
  auto kern = gemv_i8_kernel<B, PAIRED, MT, R>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), kSmemMax);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p, device_error_word());
}

template <int B, bool PAIRED>
cudaError_t run_m(const Args& p, cudaStream_t stream) {
  // two rows of a unit share the reads of x, once a CTA's share is several units
  const bool two = p.N >= 16 * static_cast<int64_t>(device_info().num_sms);
  if (p.M == 1) return two ? run<B, PAIRED, 1, 2>(p, stream) : run<B, PAIRED, 1, 1>(p, stream);
  if (p.M == 2) return two ? run<B, PAIRED, 2, 2>(p, stream) : run<B, PAIRED, 2, 1>(p, stream);
  return two ? run<B, PAIRED, 4, 2>(p, stream) : run<B, PAIRED, 4, 1>(p, stream);
}

template <int B>
cudaError_t run_layout(const Args& p, bool paired, cudaStream_t stream) {
  return paired ? run_m<B, true>(p, stream) : run_m<B, false>(p, stream);
}

}  // namespace

bool gemv_i8_fits(int bits, int64_t M, int64_t K) {
  if (M > 4 || K > kInt8MaxK) return false;
  const int mt = M <= 2 ? static_cast<int>(M) : 4;
  int n, codes;
  segments_of(static_cast<int>(K), &n, &codes);
  return x_bytes(mt, static_cast<int>(K)) + kTail + 8u * 2u * static_cast<uint32_t>(codes / 8 * bits) <= kSmemMax;
}

cudaError_t launch_gemv_i8(const uint8_t* xq, const float* sx, const uint8_t* packed, const float* scales, int bits,
                           int layout, int64_t M, int64_t N, int64_t K, uint16_t* y, cudaStream_t stream) {
  Args p{xq, sx, packed, scales, y, N, static_cast<int>(M), static_cast<int>(K), static_cast<int>(stride_i8(K)),
         static_cast<int>(4 * row_words(K, bits)), 0, 0, 0};
  const bool paired = layout == kLayoutPaired;
  switch (bits) {
    case 4: return run_layout<4>(p, paired, stream);
    case 5: return run_layout<5>(p, paired, stream);
    case 6: return run_layout<6>(p, paired, stream);
    case 7: return run_layout<7>(p, paired, stream);
    case 8: return run_layout<8>(p, paired, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mpw

// Int8 linear for a few tokens: y[m, n] = bf16(s_n sx_m sum_k xq[m, k] q[n, k]).
//
// The packed rows are the cost (N * K * b / 8 bytes, read once); a row's codes
// meet M tokens, so the work is the expansion plus M integer dot products.
// Expanding four codes to signed bytes takes 4 to 7 integer operations
// (int8_expand.cuh) and one dp4a per token multiplies them.
//
// Rows are contiguous, so one CTA per SM streams its share of them (rows
// c N / G .. (c + 1) N / G) as untiled bulk copies of R rows into a ring of
// slots, issued by one thread well ahead of their use; warps take the
// slots in turn (always the same warp a slot, so that nobody waits for a fill
// two ahead), lane l the 32-code groups l, l + 32, ... of each row, with x
// in shared memory, and one warp-wide integer reduction per result ends a
// row.  The weights do not depend on the launch before, so their copies
// start before the wait for it (programmatic dependent launch); x is read
// after it, and like the other decode kernels this one lets its successor
// start only after its own wait.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "int8_expand.cuh"
#include "int8_internal.h"
#include "mpw_internal.h"
#include "tc_ptx.cuh"

namespace mpw {
namespace {

constexpr int kWarps = 16;                        // consumers
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kMaxSlots = 64;
constexpr uint32_t kSmemTwo = 104 * 1024;         // two CTAs (this call's and the next one's) per SM
constexpr uint32_t kSmemOne = 220 * 1024;

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
  int slots;        // a multiple of warps
  int warps;        // consumers that take slots
};

__host__ __device__ constexpr uint32_t x_bytes(int MT, int K) {
  return static_cast<uint32_t>(MT) * static_cast<uint32_t>((K + 31) / 32) * 32u;
}

template <int B>
__device__ __forceinline__ void lds_group(const uint8_t* p, uint32_t (&w)[B + 1]) {
  if constexpr (B % 4 == 0) {
#pragma unroll
    for (int i = 0; i < B / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  } else if constexpr (B % 2 == 0) {
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      const uint2 v = reinterpret_cast<const uint2*>(p)[i];
      w[2 * i] = v.x; w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < B; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
  w[B] = 0u;
}

// MT: tokens (M <= MT, the others are zero), R: rows per slot.
template <int B, bool PAIRED, int MT, int R>
__global__ void __launch_bounds__(kThreads, 1)
gemv_i8_kernel(const __grid_constant__ Args p, int32_t* err) {
  extern __shared__ __align__(128) uint8_t vsmem[];
  __shared__ uint64_t bars[2 * kMaxSlots];
  constexpr int32_t kW = ptx::kWaitGemvI8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = (p.K + 31) >> 5;
  const uint32_t slot_bytes = static_cast<uint32_t>(R) * p.rb;
  // x: two planes of 16 bytes per group and token, so that the lanes of a warp
  // read consecutive 16-byte units
  uint8_t* xs = vsmem;
  uint8_t* ring = vsmem + x_bytes(MT, p.K);
  const uint32_t bar0 = ptx::smem_addr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxSlots + s); };
  const int64_t row0 = p.N * blockIdx.x / gridDim.x, row1 = p.N * (blockIdx.x + 1) / gridDim.x;
  const int units = static_cast<int>((row1 - row0 + R - 1) / R);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.slots; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    ptx::mbar_fence_init();
  }
  __syncthreads();

  if (warp == kWarps) {
    if (lane == 0) {
      int s = 0, issued = 0;
      uint32_t phase = 1;
      for (int u = 0; u < units; ++u) {
        if (!ptx::mbar_wait(empty(s), phase, err, ptx::wait_code(kW, ptx::kWaitWEmpty))) break;
        const int64_t r = row0 + static_cast<int64_t>(u) * R;
        const uint32_t bytes = static_cast<uint32_t>(min(static_cast<int64_t>(R), row1 - r)) * p.rb;
        ptx::mbar_arrive_expect_tx(full(s), bytes);
        ptx::bulk_load(ptx::smem_addr(ring) + s * slot_bytes, p.packed + r * p.rb, bytes, full(s));
        issued = u + 1;
        if (++s == p.slots) {
          s = 0;
          phase ^= 1;
        }
      }
      // nothing may still be landing in shared memory when the CTA exits
      for (int u = max(0, issued - p.slots); u < issued; ++u)
        ptx::mbar_wait(full(u % p.slots), (u / p.slots) & 1, err, ptx::wait_code(kW, ptx::kWaitWTail));
    }
    __syncwarp();
    ptx::grid_dep_wait_then_release();
    return;
  }

  ptx::grid_dep_wait_then_release();
  // x into shared memory, zero past K and for tokens past M
  for (int i = threadIdx.x; i < MT * G * 2; i += kWarps * 32) {
    const int t = i / (2 * G), j = i - t * 2 * G;         // token, 16-byte unit of it
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (t < p.M && 16 * j < p.xstride)
      v = __ldg(reinterpret_cast<const uint4*>(p.xq + static_cast<int64_t>(t) * p.xstride) + j);
    reinterpret_cast<uint4*>(xs)[(t * 2 + (j & 1)) * G + (j >> 1)] = v;
  }
  float sx[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) sx[t] = t < p.M ? __ldg(p.sx + t) : 0.0f;
  asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");

  if (warp >= p.warps) return;
  for (int u = warp; u < units; u += p.warps) {
    const int s = u % p.slots;
    if (!ptx::mbar_wait(full(s), (u / p.slots) & 1, err, ptx::wait_code(kW, ptx::kWaitWFull))) break;
    const uint8_t* slot = ring + s * slot_bytes;
    const int64_t r0 = row0 + static_cast<int64_t>(u) * R;
    int32_t acc[R][MT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[r][t] = 0;
    for (int g = lane; g < G; g += 32) {
      uint32_t o[R][8];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        // a last group may reach past its row (and a last slot hold fewer than
        // R rows): what is read there meets zeros of x or is not written
        uint32_t w[B + 1];
        lds_group<B>(slot + r * p.rb + g * 4 * B, w);
        i8::group<B, PAIRED>(w, o[r]);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint4 a = reinterpret_cast<const uint4*>(xs)[(t * 2) * G + g];
        const uint4 b = reinterpret_cast<const uint4*>(xs)[(t * 2 + 1) * G + g];
        const uint32_t xv[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            acc[r][t] = __dp4a(static_cast<int>(o[r][i]), static_cast<int>(xv[i]), acc[r][t]);
      }
    }
    __syncwarp();
    if (lane == 0) {
      // the async-proxy refill of this slot must not overtake these reads
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(empty(s));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float out = 0.0f;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int32_t sum = __reduce_add_sync(0xffffffffu, acc[r][t]);
        if (lane == t) out = static_cast<float>(sum >> (8 - B));
      }
      if (lane < p.M && r0 + r < row1) {
        float st = 0.0f;
#pragma unroll
        for (int t = 0; t < MT; ++t)
          if (lane == t) st = sx[t];
        p.y[static_cast<int64_t>(lane) * p.N + r0 + r] =
            __bfloat16_as_ushort(__float2bfloat16_rn(out * __ldg(p.scales + r0 + r) * st));
      }
    }
  }
}

// Shared memory past the last slot that a last group's read may touch.
constexpr uint32_t kTail = 64;

template <int B, bool PAIRED, int MT, int R>
cudaError_t run(Args p, cudaStream_t stream) {
  const uint32_t xb = x_bytes(MT, p.K), slot = static_cast<uint32_t>(R) * p.rb;
  const int64_t sms = device_info().num_sms;
  const unsigned grid = static_cast<unsigned>(p.N < sms ? p.N : sms);
  const int64_t units = (p.N / grid + 1 + R - 1) / R;
  // as many slots as leave room for the next call's CTA, if those keep every
  // warp busy; else as many as fit
  int64_t n = xb + kTail + kWarps * slot <= kSmemTwo ? (kSmemTwo - xb - kTail) / slot : (kSmemOne - xb - kTail) / slot;
  n = n < units ? n : units;
  n = n < kMaxSlots ? n : kMaxSlots;
  p.warps = static_cast<int>(n < kWarps ? n : kWarps);
  p.slots = static_cast<int>(n / p.warps) * p.warps;
  const size_t smem = xb + kTail + static_cast<size_t>(p.slots) * slot;
  auto kern = gemv_i8_kernel<B, PAIRED, MT, R>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), kSmemOne);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
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
  // two rows share the reads of x when every warp gets several slots of two
  const bool two = p.N >= static_cast<int64_t>(device_info().num_sms) * kWarps * 2 &&
                   gemv_i8_fits(p.M, p.K, 2 * p.rb);
  if (p.M == 1) return two ? run<B, PAIRED, 1, 2>(p, stream) : run<B, PAIRED, 1, 1>(p, stream);
  if (p.M == 2) return two ? run<B, PAIRED, 2, 2>(p, stream) : run<B, PAIRED, 2, 1>(p, stream);
  if (p.M <= 4) return two ? run<B, PAIRED, 4, 2>(p, stream) : run<B, PAIRED, 4, 1>(p, stream);
  return two ? run<B, PAIRED, 8, 2>(p, stream) : run<B, PAIRED, 8, 1>(p, stream);
}

template <int B>
cudaError_t run_layout(const Args& p, bool paired, cudaStream_t stream) {
  return paired ? run_m<B, true>(p, stream) : run_m<B, false>(p, stream);
}

}  // namespace

bool gemv_i8_fits(int64_t M, int64_t K, int64_t slot_bytes) {
  const int mt = M <= 1 ? 1 : (M <= 2 ? 2 : (M <= 4 ? 4 : 8));
  return M <= 8 && K <= kInt8MaxK && x_bytes(mt, static_cast<int>(K)) + kTail + 4 * slot_bytes <= kSmemOne;
}

cudaError_t launch_gemv_i8(const uint8_t* xq, const float* sx, const uint8_t* packed, const float* scales, int bits,
                           int layout, int64_t M, int64_t N, int64_t K, uint16_t* y, cudaStream_t stream) {
  Args p{xq, sx, packed, scales, y, N, static_cast<int>(M), static_cast<int>(K), static_cast<int>(stride_i8(K)),
         static_cast<int>(4 * row_words(K, bits)), 0, 0};
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

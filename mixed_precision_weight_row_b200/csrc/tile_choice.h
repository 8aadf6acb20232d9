// Token tiles and slices for the kernels that expand packed rows on the way to
// the tensor cores (one CTA per SM, a cluster of up to four CTAs sharing a
// tile's depth).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "mpw_internal.h"

namespace mpw {

constexpr int kMaxSlices = 4;

// CTAs of kernel KERN that run at once in clusters of 1 .. kMaxSlices: not every SM
// can take part in larger clusters.  Asked of the runtime once per kernel and
// device, so that a kernel's choices do not depend on what ran before.
struct ClusterCapacity {
  int ctas[kMaxSlices + 1] = {};
};
template <auto KERN>
ClusterCapacity cluster_capacity(int threads, size_t smem) {
  constexpr int kDevices = 64;
  static std::mutex mutex;
  static ClusterCapacity cache[kDevices];
  const DeviceInfo& d = device_info();
  std::lock_guard<std::mutex> lock(mutex);
  ClusterCapacity& c = cache[d.device >= 0 && d.device < kDevices ? d.device : 0];
  if (c.ctas[1] == 0) {
    c.ctas[1] = d.num_sms;
    for (int s = 2; s <= kMaxSlices; ++s) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(s));
      cfg.blockDim = dim3(static_cast<unsigned>(threads));
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = static_cast<unsigned>(s);
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, KERN, &cfg) == cudaSuccess)
        c.ctas[s] = n * s < d.num_sms ? n * s : d.num_sms;
      else
        (void)cudaGetLastError();
    }
  }
  return c;
}

// Time of a launch, us: a CTA spends `block` us a block of the depth and `fixed` us
// to start and end, joining S slices of a tile of BN tokens costs 2 us and
// S * BN / 128 more; the CTAs run in rounds of as many as fit.
inline double tile_time(int64_t ctas, int capacity, int64_t blocks, int slices, int bn, double block, double fixed) {
  const int64_t rounds = (ctas + capacity - 1) / capacity;
  return static_cast<double>(rounds) *
         (static_cast<double>((blocks + slices - 1) / slices) * block + fixed +
          (slices > 1 ? 2.0 + slices * bn / 128.0 : 0.0));
}

}  // namespace mpw

// Indexes that kernels check on the device, and a scan that several share.
#pragma once
#include "sm103_ptx.cuh"

namespace fa {

// First index error of a kernel (code 1), for fa_check_errors: which check
// (site), the CTA, and the request or token it concerns.
__device__ __forceinline__ void record_index_error(DevError* err, unsigned site, unsigned item) {
  if (atomicCAS(&err->code, 0u, 1u) == 0u) {
    err->site = site;
    err->block = blockIdx.x;
    err->tile = item;
    __threadfence();
  }
}

enum : unsigned { kSiteAppendSlot = 601, kSiteFwdBlock = 611, kSiteFwdLen = 612, kSiteFwdRows = 613,
                  kSiteFwdScale = 614, kSiteRopePosition = 621, kSiteReadSlot = 631 };

// Inclusive scan over the CTA (1024 threads) of one value per thread;
// `total` is the sum.  `tmp` holds 33 values.
__device__ __forceinline__ long long cta_scan(long long x, long long* tmp, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < static_cast<int>(blockDim.x >> 5) ? tmp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    tmp[lane] = w;
  }
  __syncthreads();
  total = tmp[31];
  if (warp > 0) x += tmp[warp - 1];
  __syncthreads();  // tmp may be reused
  return x;
}

}  // namespace fa

// What fa_fwd.cu shares with the library's other translation units: the error
// state, the tensor-map cache and the device's records.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>

#include "sm103_ptx.cuh"

namespace fa {
namespace host {

struct Device {
  int dev, sms;
  DevError* err;        // expired waits
  DevError* index_err;  // indexes out of range
};

int fail(cudaError_t e);  // keeps e for fa_get_last_cuda_error; FA_ERR_CUDA
bool overlap(const void* a, size_t na, const void* b, size_t nb);
// The current device, set up on first use.
int device(Device* out);
// A cached 3-D tensor map (128-byte swizzle, zero fill, boxes one deep).
int tensor_map(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, cuuint64_t d0, cuuint64_t d1,
               cuuint64_t d2, cuuint64_t stride1, cuuint64_t stride2, cuuint32_t box0, cuuint32_t box1);

}  // namespace host
}  // namespace fa

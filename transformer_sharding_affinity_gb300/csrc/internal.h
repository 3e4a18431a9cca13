// internal.h -- helpers shared by the translation units behind the C ABI
// (not part of include/affinity.h).
#pragma once

#include "affinity.h"

#include <cuda.h>
#include <cuda_runtime.h>

namespace aff {

// Records "<where>: <CUDA error name> (<text>)" for affinity_last_cuda_error()
// on this thread and returns AFF_ERR_CUDA.
aff_status cuda_fail(cudaError_t e, const char* where);

// AFF_OK with the SM count when the current device is an sm_103 part;
// AFF_ERR_ARCH otherwise (also when there is no device).
aff_status check_device(int* sm_count);

// Tensor map of a 16-bit tensor of `rank` dims (dims[0] innermost, contiguous; strides in bytes),
// 128 B swizzle, box = 64 innermost elements x box1 in dimension box1_dim (x box2 in box2_dim, if given);
// out of bounds reads zero.
aff_status map_16bit_sw128(CUtensorMap* m, const void* ptr, int rank, const uint64_t* dims, const uint64_t* strides,
                           uint32_t box1, int box1_dim, uint32_t box2 = 1, int box2_dim = -1);

}  // namespace aff

#define AFF_CUDA(call)                                        \
  do {                                                        \
    cudaError_t e_ = (call);                                  \
    if (e_ != cudaSuccess) return ::aff::cuda_fail(e_, #call); \
  } while (0)

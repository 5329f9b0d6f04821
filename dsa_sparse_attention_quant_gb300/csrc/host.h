// host.h — helpers of the C entry points (host code, internal to the library).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dsa {

// SM count of the current device; DSA_ENODEV unless it is an sm_103 part.
int device_sms(int* sms);

// DSA_* status of a CUDA runtime error.
int from_cuda(cudaError_t e);

// The driver's tensor-map encoder, looked up once.
int tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* out);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

}  // namespace dsa

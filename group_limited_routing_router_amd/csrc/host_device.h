// host_device.h -- functions that the kernels and a plain C++ compiler take, so
// that their arithmetic is tested on the CPU.
#pragma once

#ifdef __HIP__
#include <hip/hip_runtime.h>

#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

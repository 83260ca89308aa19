// Shared pieces of the logits operators' kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "spec_logits.h"

namespace sl {

// float32 to the output type, rounded to nearest even (bf16 by the hardware's conversion).
__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void store_out(uint16_t* p, float v) { *p = to_bf16(v); }
__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ float load_in(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float load_in(const float* p) { return *p; }

}  // namespace sl

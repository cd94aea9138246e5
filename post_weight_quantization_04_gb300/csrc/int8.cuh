// int8.cuh — the 8-bit integer form: whole numbers with one fp32 scale per row.
//
// A matrix (rows, cols) is stored as codes (rows, 16 * ceil(cols / 16)) int8, zeros past cols, so that
// every row starts where a 16-byte load or a TMA copy can, and scales (rows) fp32: value = code * scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gptq {

__host__ __device__ inline int64_t int8_pitch(int64_t cols) { return (cols + 15) / 16 * 16; }

__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// max and min that keep a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

}  // namespace gptq

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

// A unit of N consecutive elements of a row as fp32: one access of 16, 4 or 2 bytes (N sizeof(T)).
template <typename T, int N>
__device__ __forceinline__ void load_unit(const T* x, float (&v)[N]) {
    if constexpr (N == 1) {
        if constexpr (sizeof(T) == 2) v[0] = __bfloat162float(*x);
        else v[0] = *x;
    } else {
        constexpr int WORDS = N * sizeof(T) / 4;
        uint32_t u[WORDS];
        if constexpr (WORDS == 1) {
            u[0] = *reinterpret_cast<const uint32_t*>(x);
        } else {
            const uint4 w = *reinterpret_cast<const uint4*>(x);
            u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
        }
#pragma unroll
        for (int e = 0; e < WORDS; ++e) {
            if constexpr (sizeof(T) == 2) {
                v[2 * e] = __uint_as_float(u[e] << 16);
                v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
            } else {
                v[e] = __uint_as_float(u[e]);
            }
        }
    }
}

template <typename T, int N>
__device__ __forceinline__ void store_unit(T* y, const float (&v)[N]) {
    if constexpr (N == 1) {
        if constexpr (sizeof(T) == 2) *y = __float2bfloat16_rn(v[0]);
        else *y = v[0];
    } else {
        constexpr int WORDS = N * sizeof(T) / 4;
        uint32_t u[WORDS];
#pragma unroll
        for (int e = 0; e < WORDS; ++e) {
            if constexpr (sizeof(T) == 2) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                u[e] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                u[e] = __float_as_uint(v[e]);
            }
        }
        if constexpr (WORDS == 1) *reinterpret_cast<uint32_t*>(y) = u[0];
        else *reinterpret_cast<uint4*>(y) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

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

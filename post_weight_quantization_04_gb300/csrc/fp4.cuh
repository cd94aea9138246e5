// fp4.cuh — the microscaled 4-bit form: e2m1 codes with one scale per block of columns.
//
// e2m1 holds 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives. A matrix (rows, cols) is stored as
//   codes   (rows, 16 * ceil(cols / 32)) bytes: column 2i in the low half of byte i, zero
//           codes up to the pitch (a whole number of 32-column blocks, and of the 16 bytes a
//           TMA copy needs);
//   scales  one byte per block of 32 columns (GPTQ_MXFP4: e8m0, 2^(byte - 127)) or 16 columns
//           (GPTQ_NVFP4: e4m3, multiplied by one fp32 number for the whole matrix), in the
//           order the tensor core reads them: tiles of 128 rows x 4 blocks, 512 bytes each,
//           scale b of row r at byte (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4 of tile
//           (r / 128, b / 4), tiles of one row block adjacent.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gptq {

constexpr int kFp4Tile = 512;   // bytes of one scale tile: 128 rows x 4 blocks

__host__ __device__ inline int64_t fp4_pitch(int64_t cols) { return (cols + 31) / 32 * 16; }
__host__ __device__ inline int fp4_block(int format) { return format == GPTQ_MXFP4 ? 32 : 16; }
// scale tiles along the columns
__host__ __device__ inline int64_t fp4_tiles(int64_t cols, int format) {
    const int64_t span = 4 * fp4_block(format);
    return (cols + span - 1) / span;
}
// byte of scale b of row r, tiles_k scale tiles per row block
__host__ __device__ inline int64_t fp4_scale_at(int64_t r, int64_t b, int64_t tiles_k) {
    return ((r >> 7) * tiles_k + (b >> 2)) * kFp4Tile + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

// 2^(byte - 127), 255 = NaN
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    return b == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(b ? b << 23 : 0x00400000u);
}

__device__ __forceinline__ float e4m3_value(uint32_t b) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3)));
}

// two codes of one byte (column order) as exact fp32 values
__device__ __forceinline__ float2 e2m1_values(uint32_t byte) {
    return __half22float2(__half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)byte, __NV_E2M1)));
}

}  // namespace gptq

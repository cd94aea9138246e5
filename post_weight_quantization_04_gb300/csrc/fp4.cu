// fp4.cu — quantisation to the microscaled 4-bit form (fp4.cuh) and its inverse.
//
// For a block of B columns with a = max|x| (the last block of a row padded with zeros):
//   MX (B = 32): s = 2^(floor(log2 a) - 2), the power of two that brings a into [4, 8), as the
//                OCP microscaling format defines it; values above 6 saturate.
//   NV (B = 16): s = e4m3(a / (6 g)) * g with the matrix's fp32 scale g, so a maps to about 6.
//   code = e2m1 nearest to x / s, ties to the even code, saturating at 6; s = 0 gives zeros.
#include <algorithm>

#include "common.cuh"
#include "fp4.cuh"

namespace gptq {

namespace {

struct QParams {
    const void* X;
    int64_t rows, cols, ldx;
    int64_t src_rows;        // rows of X
    const int32_t* index;    // row r reads X row index[r] / per (negative: zeros); null: row r
    int per;
    const float* g;          // NV: the matrix's scale
    uint8_t* codes;
    uint8_t* scales;
    int64_t pitch, tiles_k;
    int* status;
};

constexpr int Q_THREADS = 128;
constexpr int Q_COLS = 16;   // columns per thread: one NV block, half an MX block

__device__ __forceinline__ float load_elem(const float* p) { return *p; }
__device__ __forceinline__ float load_elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// 16 consecutive values of one row as fp32, zeros past `n`. Returns the greatest magnitude's bits: exact,
// and a NaN or infinity stays visible (bf16 pairs are compared two at a time).
template <typename T, bool VEC>
__device__ __forceinline__ uint32_t load16(const T* x, int64_t n, float (&v)[Q_COLS]) {
    uint32_t m = 0;
    if (VEC && n >= Q_COLS) {
        constexpr int PER = 16 / sizeof(T);
#pragma unroll
        for (int q = 0; q < Q_COLS / PER; ++q) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(x) + q);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (sizeof(T) == 4) {
                    v[4 * q + e] = __uint_as_float(u[e]);
                    m = max(m, u[e] & 0x7FFFFFFFu);
                } else {
                    v[8 * q + 2 * e] = __uint_as_float(u[e] << 16);
                    v[8 * q + 2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
                    m = __vmaxu2(m, u[e] & 0x7FFF7FFFu);
                }
            }
        }
        return sizeof(T) == 4 ? m : max(m << 16, m & 0xFFFF0000u);
    }
#pragma unroll
    for (int e = 0; e < Q_COLS; ++e) {
        v[e] = e < n ? load_elem(x + e) : 0.0f;
        m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    }
    return m;
}

// The same for a row that 16-byte loads cannot take: the warp reads its 512 columns (x, n: those of its
// lane 0, which is column `col` of the row) in order, 4 bytes at a time, and hands each lane its 16
// through shared memory, one word left out after every 16 (fp32) or 8 (pairs of bf16) so that
// neither side has conflicts. Loading 16 neighbours per lane took twice as long.
constexpr int Q_BUF = 17 * 32;   // words per warp
__device__ __forceinline__ uint32_t load16_turned(const float* x, int64_t, int64_t n, float (&v)[Q_COLS], uint32_t* buf) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int e = 0; e < Q_COLS; ++e) {
        const int c = lane + 32 * e;
        v[e] = c < n ? x[c] : 0.0f;
    }
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < Q_COLS; ++e) {
        const int c = lane + 32 * e;
        buf[c + (c >> 4)] = __float_as_uint(v[e]);
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < Q_COLS; ++e) {
        v[e] = __uint_as_float(buf[17 * lane + e]);
        m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    }
    return m;
}

// bf16: whole aligned words, which for a row on an odd element hold its columns shifted by one; the
// words at the row's ends that are not all its own are put together from single elements
__device__ __forceinline__ uint32_t load16_turned(const __nv_bfloat16* x, int64_t col, int64_t n, float (&v)[Q_COLS], uint32_t* buf) {
    const int lane = threadIdx.x & 31;
    const int odd = (int)(reinterpret_cast<uintptr_t>(x) >> 1) & 1;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(x) & ~uintptr_t(3));
    const uint16_t* halves = reinterpret_cast<const uint16_t*>(x);
    auto word = [&](int i) -> uint32_t {   // columns c and c + 1
        const int c = 2 * i - odd;
        if (c + 1 < n && (c >= 0 || col > 0)) return words[i];
        return (c >= 0 && c < n ? (uint32_t)halves[c] : 0u) | (c + 1 < n ? (uint32_t)halves[c + 1] << 16 : 0u);
    };
    __syncwarp();
    uint32_t u[9];
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = word(lane + 32 * e);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = lane + 32 * e;
        buf[i + (i >> 3)] = u[e];
    }
    if (odd && lane == 0) buf[256 + 32] = word(256);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] = buf[9 * lane + k];
    u[8] = odd ? buf[9 * lane + 9] : 0u;
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t pair = odd ? __funnelshift_r(u[k], u[k + 1], 16) : u[k];
        v[2 * k] = __uint_as_float(pair << 16);
        v[2 * k + 1] = __uint_as_float(pair & 0xFFFF0000u);
        m = __vmaxu2(m, pair & 0x7FFF7FFFu);
    }
    return max(m << 16, m & 0xFFFF0000u);
}

// 8 values (already divided by their block's scale) to 8 codes: nearest, ties to even, saturating
__device__ __forceinline__ uint32_t to_codes(const float* y) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}

// One thread takes 16 columns of a row; an MX block's two threads share its maximum by one shuffle, and
// the scales of four blocks (one word of a scale tile) are stored together. Streams x once and writes
// 1/2 byte per value plus the scales: bound by memory. 16384 x 4096 fp32 to MX or NV in 48 us (6.3 TB/s);
// bf16 to MX 29 us (5.9 TB/s), to NV 33 (the division's instructions show). Two rows per thread in
// flight were slower (bf16 MX 35 us; fewer CTAs fit), and so were 8 fp32 columns per thread.
template <typename T, bool MX, bool VEC>
__global__ void __launch_bounds__(Q_THREADS) fp4_quantize_kernel(const QParams p) {
    const int64_t chunk = (int64_t)blockIdx.x * Q_THREADS + threadIdx.x;
    const int64_t c0 = chunk * Q_COLS;
    pdl_trigger();   // the product's or the inverse's prologue may begin
    const float g = MX ? 1.0f : *p.g, inv6g = MX ? 1.0f : 1.0f / (6.0f * g);
    const bool easy = (__float_as_uint(g) & 0x007FFFFFu) == 0 && g > 0x1p-40f && g < 0x1p40f;
    for (int64_t r = blockIdx.y; r < p.rows; r += gridDim.y) {
        int64_t sr = r;
        if (p.index) {
            const int k = p.index[r];
            sr = k < 0 ? -1 : k / p.per;
            if (sr >= p.src_rows) {
                sr = -1;
                set_status(p.status, GPTQ_ERR_INVALID_ARG);
            }
        }
        float y[Q_COLS];
        uint32_t m;
        if constexpr (VEC) {
            m = load16<T, true>(static_cast<const T*>(p.X) + (sr < 0 ? 0 : sr * p.ldx + c0), sr < 0 ? 0 : p.cols - c0, y);
        } else {
            __shared__ uint32_t buf[Q_THREADS / 32][Q_BUF];
            const int64_t cw = c0 - (int64_t)(threadIdx.x & 31) * Q_COLS;
            m = load16_turned(static_cast<const T*>(p.X) + (sr < 0 ? 0 : sr * p.ldx + cw), cw, sr < 0 ? 0 : p.cols - cw, y,
                              buf[threadIdx.x >> 5]);
        }
        if (MX) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const bool bad = m >= 0x7F800000u;
        if (bad) set_status(p.status, GPTQ_ERR_NONFINITE);
        uint32_t byte;
        if (MX) {
            // floor(log2 a) is a's exponent field; below 2^-125 the scale stays at 2^-127
            byte = bad ? 255u : (uint32_t)max((int)(m >> 23) - 2, 0);
            const float inv = __uint_as_float(byte < 254u ? (254u - byte) << 23 : 0x00400000u);
#pragma unroll
            for (int e = 0; e < Q_COLS; ++e) y[e] *= inv;   // exact: a power of two
        } else {
            const float a = __uint_as_float(m);
            // a / (6 g) and x / d correctly rounded (Markstein 1990: with the divisor's reciprocal correctly
            // rounded, one residual step on the product rounds the quotient correctly), so a value on
            // a midpoint of the grid is seen as one. x is first cut to 8 d, beyond which every
            // quotient saturates, and both are brought near 1 by a power of two where d is far from
            // it, so nothing overflows or vanishes on the way. A scale of zero (or past fp32) has zeros.
            const float aq = a * inv6g;
            const float ratio = aq > 0x1p-100f && aq < 0x1p100f && inv6g > 0x1p-60f && inv6g < 0x1p60f
                                    ? fmaf(fmaf(-aq, 6.0f * g, a), inv6g, aq) : a / (6.0f * g);
            // (a block of zeros has a scale of zero under any g: g = max|x| / 2688 of a matrix of zeros is 0)
            byte = bad ? 127u : a > 0.0f ? (uint32_t)__nv_cvt_float_to_fp8(ratio, __NV_SATFINITE, __NV_E4M3) : 0u;
            float d = e4m3_value(byte) * g;
            if (!(d >= 0x1p-60f && d <= 0x1p60f)) {
                const float f = d < 1.0f ? 0x1p64f : 0x1p-64f;
#pragma unroll
                for (int e = 0; e < Q_COLS; ++e) y[e] *= f;
                d = d < 0x1.fffffep127f ? d * f : d > 0.0f ? 0.0f : d;   // past fp32: none (a NaN stays)
            }
            const float inv = d != 0.0f ? 1.0f / d : 0.0f;
            if (sizeof(T) == 2 && easy) {
                // x has 8 significant bits and d 4 (g is a power of two): a quotient that is not a midpoint
                // is 2^-8 away from it, and for the eight d the reciprocals are exact or up to
                // 2^-24 too large, so the product cut towards zero is the midpoint where x / d is one
#pragma unroll
                for (int e = 0; e < Q_COLS; ++e) y[e] = __fmul_rz(y[e], inv);
            } else {
                const float most = 8.0f * d;
#pragma unroll
                for (int e = 0; e < Q_COLS; ++e) {
                    const float x = fminf(fmaxf(y[e], -most), most), q = x * inv;
                    y[e] = fmaf(fmaf(-q, d, x), inv, q);
                }
            }
        }
        if (c0 < 2 * p.pitch)
            *reinterpret_cast<uint2*>(p.codes + r * p.pitch + c0 / 2) = make_uint2(to_codes(y), to_codes(y + 8));
        // scales up to the end of the last tile: blocks past the columns get a zero byte
        constexpr int LANES = MX ? 2 : 1;   // threads per block
        const int64_t b = chunk / LANES;
        uint32_t word = b * (MX ? 32 : 16) < p.cols ? byte : 0u;
        word |= __shfl_down_sync(0xffffffffu, word, LANES) << 8;
        word |= __shfl_down_sync(0xffffffffu, word, 2 * LANES) << 16;
        if (chunk % (4 * LANES) == 0 && b < 4 * p.tiles_k)
            *reinterpret_cast<uint32_t*>(p.scales + fp4_scale_at(r, b, p.tiles_k)) = word;
    }
}

struct DqParams {
    const uint8_t* codes;
    const uint8_t* scales;
    const float* g;
    int64_t rows, cols, pitch, tiles_k;
    void* Y;
    int64_t ldy;
};

__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// One thread writes 16 consecutive bytes (4 fp32 or 8 bf16 columns), so a warp's store is one run of
// whole sectors; DQ_ROWS rows in flight. Bound by the bytes written: 14336 x 4096 NV to fp32, 268 MB, in
// 40 us (6.7 TB/s); 16 columns per thread, whose stores leave half sectors, took 61.
constexpr int DQ_ROWS = 4;
template <typename T, bool MX, bool VEC>
__global__ void __launch_bounds__(Q_THREADS) fp4_dequantize_kernel(const DqParams p) {
    constexpr int C = 16 / sizeof(T);
    const int64_t c0 = ((int64_t)blockIdx.x * Q_THREADS + threadIdx.x) * C, n = p.cols - c0;
    const int lane = threadIdx.x & 31;
    const int64_t cw = c0 - lane * C;   // the warp's first column
    if (cw >= p.cols) return;
    pdl_wait();
    const float g = MX ? 1.0f : *p.g;
    const int64_t b = c0 / (MX ? 32 : 16);
    for (int64_t r0 = (int64_t)blockIdx.y * DQ_ROWS; r0 < p.rows; r0 += (int64_t)gridDim.y * DQ_ROWS) {
        uint32_t w[DQ_ROWS], sb[DQ_ROWS];
#pragma unroll
        for (int i = 0; i < DQ_ROWS; ++i) {
            const int64_t r = min(r0 + i, p.rows - 1);
            const uint8_t* src = p.codes + r * p.pitch + min(c0 / 2, p.pitch - C / 2);   // (lanes past the row: any)
            w[i] = C == 8 ? *reinterpret_cast<const uint32_t*>(src) : *reinterpret_cast<const uint16_t*>(src);
            sb[i] = p.scales[fp4_scale_at(r, min(b, 4 * p.tiles_k - 1), p.tiles_k)];
        }
#pragma unroll
        for (int i = 0; i < DQ_ROWS; ++i) {
            if (r0 + i >= p.rows) break;
            const float s = MX ? e8m0_value(sb[i]) : e4m3_value(sb[i]) * g;
            float v[C];
#pragma unroll
            for (int e = 0; e < C / 2; ++e) {
                const float2 f = e2m1_values((w[i] >> (8 * e)) & 0xFFu);
                v[2 * e] = f.x * s;
                v[2 * e + 1] = f.y * s;
            }
            T* y = static_cast<T*>(p.Y) + (r0 + i) * p.ldy;
            if constexpr (VEC) {
                if (n >= C) {
                    if constexpr (C == 4)
                        *reinterpret_cast<float4*>(y + c0) = make_float4(v[0], v[1], v[2], v[3]);
                    else
                        *reinterpret_cast<uint4*>(y + c0) =
                            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
                } else {
#pragma unroll
                    for (int e = 0; e < C; ++e)
                        if (e < n) store_elem(y + c0 + e, v[e]);
                }
            } else {
                // in order through shared memory (a word left out after every 32, so no conflicts)
                __shared__ float buf[Q_THREADS / 32][33 * C];
                float* mine = buf[threadIdx.x >> 5];
                __syncwarp();
#pragma unroll
                for (int e = 0; e < C; ++e) mine[C * lane + e + ((C * lane + e) >> 5)] = v[e];
                __syncwarp();
#pragma unroll
                for (int e = 0; e < C; ++e) {
                    const int c = lane + 32 * e;
                    if (cw + c < p.cols) store_elem(y + cw + c, mine[c + (c >> 5)]);
                }
            }
        }
    }
}

// max|x| of a matrix, as the bits of an fp32 (ordered like the numbers, so an integer atomic
// maximum is exact and independent of order), into out[0], which starts at 0
template <typename T, bool VEC>
__global__ void __launch_bounds__(Q_THREADS) fp4_amax_kernel(const T* X, int64_t rows, int64_t cols, int64_t ldx,
                                                             uint32_t* out, int* status) {
    const int64_t c0 = ((int64_t)blockIdx.x * Q_THREADS + threadIdx.x) * Q_COLS;
    uint32_t m = 0;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        float v[Q_COLS];
        m = max(m, load16<T, VEC>(X + r * ldx + c0, cols - c0, v));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    __shared__ uint32_t part[Q_THREADS / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < Q_THREADS / 32; ++i) m = max(m, part[i]);
        if (m >= 0x7F800000u) set_status(status, GPTQ_ERR_NONFINITE);
        atomicMax(out, m);
    }
}

// the least normal power of two g with max|x| <= 448 * 6 * g, in place of the maximum (1 for all zeros)
__global__ void fp4_tensor_scale_kernel(uint32_t* out) {
    const float a = __uint_as_float(*out);
    int e = 0;
    if (a > 0.0f && a < __uint_as_float(0x7F800000u)) {
        frexpf(fmaxf(a / 2688.0f, 0x1p-126f), &e);   // (below that the quotient has few bits or is 0)
        if (ldexpf(0.5f, e) * 2688.0f >= a) --e;   // a / 2688 is a power of two itself
    }
    *out = __float_as_uint(ldexpf(1.0f, max(e, -126)));
}

__global__ void __launch_bounds__(256) fp4_tile_scales_kernel(const uint8_t* src, int64_t rows, int64_t blocks,
                                                              int64_t lds, int64_t tiles_k, uint8_t* dst, int64_t total) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t tile = i / kFp4Tile;
        const int at = (int)(i % kFp4Tile);
        const int64_t r = tile / tiles_k * 128 + (at >> 2 & 3) * 32 + (at >> 4), b = tile % tiles_k * 4 + (at & 3);
        dst[i] = r < rows && b < blocks ? src[r * lds + b] : (uint8_t)0;
    }
}

bool bad_format(int f) { return f != GPTQ_MXFP4 && f != GPTQ_NVFP4; }
bool bad_dtype(int t) { return t != GPTQ_F32 && t != GPTQ_BF16; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
constexpr int64_t kMaxDim = (1ll << 31) - 256;

// CTAs along the rows: enough to fill the device, each looping over the rest (a CTA per few rows spends
// as long starting as copying)
unsigned rows_grid(int64_t groups, int64_t ctas_x, int per_sm) {
    const int64_t want = std::max<int64_t>(1, ceil_div((int64_t)device_sm_count() * per_sm, ctas_x));
    return (unsigned)std::min<int64_t>(groups, std::min<int64_t>(want, 65535));
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" int64_t gptq_fp4_code_pitch(int64_t cols) { return cols < 0 ? 0 : fp4_pitch(cols); }

extern "C" int64_t gptq_fp4_scale_bytes(int64_t rows, int64_t cols, int format) {
    if (rows < 0 || cols < 0 || bad_format(format)) return 0;
    return ceil_div(rows, 128) * fp4_tiles(cols, format) * kFp4Tile;
}

extern "C" int gptq_fp4_tensor_scale(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ldx, float* g,
                                     void* stream) {
    if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim || bad_dtype(dtype) || !g || ldx < cols ||
        (!X && rows * cols > 0))
        return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    uint32_t* out = reinterpret_cast<uint32_t*>(g);
    GPTQ_CUDA_TRY(cudaMemsetAsync(out, 0, 4, s));
    if (rows > 0 && cols > 0) {
        const int64_t ctas_x = ceil_div(cols, Q_COLS * Q_THREADS);
        const dim3 grid((unsigned)ctas_x, rows_grid(rows, ctas_x, 16));
        const bool vec = aligned16(X) && (ldx * (dtype == GPTQ_BF16 ? 2 : 4)) % 16 == 0;
        auto go = [&](auto kern, auto* x) { GPTQ_LAUNCH(K_FP4_AMAX, s, kern<<<grid, Q_THREADS, 0, s>>>(x, rows, cols, ldx, out, st.word)); };
        if (dtype == GPTQ_BF16) {
            auto* x = static_cast<const __nv_bfloat16*>(X);
            vec ? go(fp4_amax_kernel<__nv_bfloat16, true>, x) : go(fp4_amax_kernel<__nv_bfloat16, false>, x);
        } else {
            auto* x = static_cast<const float*>(X);
            vec ? go(fp4_amax_kernel<float, true>, x) : go(fp4_amax_kernel<float, false>, x);
        }
        GPTQ_LAUNCH_CHECK();
    }
    GPTQ_LAUNCH(K_FP4_AMAX, s, fp4_tensor_scale_kernel<<<1, 1, 0, s>>>(out));
    GPTQ_LAUNCH_CHECK();
    return st.finish(s);
}

extern "C" int gptq_fp4_quantize(const void* X, int dtype, int64_t src_rows, int64_t cols, int64_t ldx,
                                 const int32_t* index, int64_t per, int64_t rows, int format, const float* g,
                                 uint8_t* codes, uint8_t* scales, void* stream) {
    if (rows < 0 || src_rows < 0 || cols < 0 || rows > kMaxDim || src_rows > kMaxDim || cols > kMaxDim || bad_dtype(dtype) ||
        bad_format(format))
        return GPTQ_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return GPTQ_OK;
    if ((!X && src_rows > 0) || !codes || !scales || ldx < cols || (index ? (per < 1 || per > kMaxDim) : rows != src_rows) ||
        (format == GPTQ_NVFP4 && !g) || !aligned16(codes) || !aligned16(scales))
        return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    QParams p{X, rows, cols, ldx, src_rows, index, (int)per, g, codes, scales, fp4_pitch(cols), fp4_tiles(cols, format), st.word};
    const int64_t chunks = ceil_div(p.tiles_k * 4 * fp4_block(format), Q_COLS);
    const dim3 grid((unsigned)ceil_div(chunks, Q_THREADS), rows_grid(rows, ceil_div(chunks, Q_THREADS), 64));
    const int64_t esize = dtype == GPTQ_BF16 ? 2 : 4;
    const bool vec = aligned16(X) && (ldx * esize) % 16 == 0, mx = format == GPTQ_MXFP4;
    auto go = [&](auto kern) { GPTQ_LAUNCH(K_FP4_QUANT, s, kern<<<grid, Q_THREADS, 0, s>>>(p)); };
    if (dtype == GPTQ_BF16) {
        if (mx) vec ? go(fp4_quantize_kernel<__nv_bfloat16, true, true>) : go(fp4_quantize_kernel<__nv_bfloat16, true, false>);
        else vec ? go(fp4_quantize_kernel<__nv_bfloat16, false, true>) : go(fp4_quantize_kernel<__nv_bfloat16, false, false>);
    } else {
        if (mx) vec ? go(fp4_quantize_kernel<float, true, true>) : go(fp4_quantize_kernel<float, true, false>);
        else vec ? go(fp4_quantize_kernel<float, false, true>) : go(fp4_quantize_kernel<float, false, false>);
    }
    GPTQ_LAUNCH_CHECK();
    return st.finish(s);
}

extern "C" int gptq_fp4_dequantize(const uint8_t* codes, const uint8_t* scales, const float* g, int64_t rows, int64_t cols,
                                   int format, void* Y, int dtype, int64_t ldy, void* stream) {
    if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim || bad_dtype(dtype) || bad_format(format))
        return GPTQ_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return GPTQ_OK;
    if (!codes || !scales || !Y || ldy < cols || (format == GPTQ_NVFP4 && !g) || !aligned16(codes) || !aligned16(scales))
        return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DqParams p{codes, scales, g, rows, cols, fp4_pitch(cols), fp4_tiles(cols, format), Y, ldy};
    const int64_t esize = dtype == GPTQ_BF16 ? 2 : 4;
    const dim3 grid((unsigned)ceil_div(cols * esize, 16 * Q_THREADS), rows_grid(ceil_div(rows, DQ_ROWS), ceil_div(cols * esize, 16 * Q_THREADS), 32));
    const bool vec = aligned16(Y) && (ldy * esize) % 16 == 0, mx = format == GPTQ_MXFP4;
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kern) { GPTQ_LAUNCH(K_FP4_DEQUANT, s, e = launch_pdl(kern, grid, dim3(Q_THREADS), 0, s, p)); };
    if (dtype == GPTQ_BF16) {
        if (mx) vec ? go(fp4_dequantize_kernel<__nv_bfloat16, true, true>) : go(fp4_dequantize_kernel<__nv_bfloat16, true, false>);
        else vec ? go(fp4_dequantize_kernel<__nv_bfloat16, false, true>) : go(fp4_dequantize_kernel<__nv_bfloat16, false, false>);
    } else {
        if (mx) vec ? go(fp4_dequantize_kernel<float, true, true>) : go(fp4_dequantize_kernel<float, true, false>);
        else vec ? go(fp4_dequantize_kernel<float, false, true>) : go(fp4_dequantize_kernel<float, false, false>);
    }
    GPTQ_CUDA_TRY(e);
    return GPTQ_OK;
}

extern "C" int gptq_fp4_tile_scales(const uint8_t* src, int64_t rows, int64_t cols, int64_t lds, int format,
                                    uint8_t* scales, void* stream) {
    if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim || bad_format(format)) return GPTQ_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return GPTQ_OK;
    const int64_t blocks = ceil_div(cols, fp4_block(format));
    if (!src || !scales || lds < blocks) return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t total = gptq_fp4_scale_bytes(rows, cols, format);
    GPTQ_LAUNCH(K_FP4_TILE, s, fp4_tile_scales_kernel<<<(unsigned)std::min<int64_t>(ceil_div(total, 256), 8 * 152), 256, 0, s>>>(
        src, rows, blocks, lds, fp4_tiles(cols, format), scales, total));
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

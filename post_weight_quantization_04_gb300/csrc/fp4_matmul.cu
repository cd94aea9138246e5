// fp4_matmul.cu — Y = X W^T for two matrices in the microscaled 4-bit form (fp4.cuh), dense or
// with one weight per expert over rows sorted by expert:
//   Y[t][o] = act(gx gw sum_b sx[t][b] sw[e(t)][o][b] sum_{k in b} x[t][k] w[e(t)][o][k])
// Products of two e2m1 values are exact; sums are fp32.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "fp4.cuh"

namespace gptq {

namespace {

struct MParams {
    const uint8_t *xc, *xs, *wc, *ws;
    const float *xg, *wg;
    int64_t T, N, K, pitch, tiles_k;
    int64_t w_codes_stride, w_scales_stride;   // bytes from one expert to the next
    int wg_stride;
    const int32_t* offsets;   // null: one expert, all rows
    int experts;
    int relu, bf16_out;
    void* Y;
    int64_t ldy;
    int* status;
};

// rows [lo, hi) of expert e, made safe: non-decreasing and within the rows of X
__device__ __forceinline__ void expert_rows(const MParams& p, int e, int64_t* lo, int64_t* hi) {
    if (!p.offsets) {
        *lo = 0;
        *hi = p.T;
        return;
    }
    const int64_t a = p.offsets[e], b = p.offsets[e + 1];
    const int64_t l = min(max(a, (int64_t)0), p.T), h = min(max(b, l), p.T);
    if (l != a || h != b) set_status(p.status, GPTQ_ERR_INVALID_ARG);
    *lo = l;
    *hi = h;
}

constexpr int B_T = 64, B_N = 64, B_K = 32;

// 64 x 64 outputs per CTA, 32 columns at a time expanded to fp32 in shared memory.
template <bool MX>
__global__ void __launch_bounds__(256) fp4_matmul_kernel(const MParams p) {
    __shared__ float xs[B_K][B_T + 1], ws[B_K][B_N + 1];
    // the CTA's expert and its first row: experts in order, ceil(rows / 64) tiles each
    int64_t tile = blockIdx.x, lo = 0, hi = 0;
    int e = 0;
    for (; e < p.experts; ++e) {
        expert_rows(p, e, &lo, &hi);
        const int64_t n = (hi - lo + B_T - 1) / B_T;
        if (tile < n) break;
        tile -= n;
    }
    const int64_t n0 = (int64_t)blockIdx.y * B_N;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    float acc[4][4] = {};
    int64_t t0;
    if (e < p.experts) {
        t0 = lo + tile * B_T;
        const uint8_t* wc = p.wc + e * p.w_codes_stride;
        const uint8_t* wsc = p.ws + e * p.w_scales_stride;
        const int r = tid >> 2, q = tid & 3;   // row of the tile, 8 columns of the step
        for (int64_t k0 = 0; k0 < p.K; k0 += B_K) {
            const int64_t b = k0 / (MX ? 32 : 16) + (MX ? 0 : q >> 1);
            uint32_t cx = 0, cw = 0;
            float sx = 0.0f, sw = 0.0f;
            if (t0 + r < hi) {
                cx = *reinterpret_cast<const uint32_t*>(p.xc + (t0 + r) * p.pitch + k0 / 2 + 4 * q);
                const uint32_t s = p.xs[fp4_scale_at(t0 + r, b, p.tiles_k)];
                sx = MX ? e8m0_value(s) : e4m3_value(s);
            }
            if (n0 + r < p.N) {
                cw = *reinterpret_cast<const uint32_t*>(wc + (n0 + r) * p.pitch + k0 / 2 + 4 * q);
                const uint32_t s = wsc[fp4_scale_at(n0 + r, b, p.tiles_k)];
                sw = MX ? e8m0_value(s) : e4m3_value(s);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = e2m1_values((cx >> (8 * i)) & 0xFFu), c = e2m1_values((cw >> (8 * i)) & 0xFFu);
                xs[8 * q + 2 * i][r] = a.x * sx;
                xs[8 * q + 2 * i + 1][r] = a.y * sx;
                ws[8 * q + 2 * i][r] = c.x * sw;
                ws[8 * q + 2 * i + 1][r] = c.y * sw;
            }
            __syncthreads();
#pragma unroll 8
            for (int k = 0; k < B_K; ++k) {
                float a[4], c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = xs[k][ty * 4 + i];
                    c[i] = ws[k][tx + 16 * i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], c[j], acc[i][j]);
            }
        }
    } else {
        // past the experts' tiles: rows that belong to none are zero
        t0 = hi + tile * B_T;
        hi = p.T;
        e = 0;
    }
    const float g = MX ? 1.0f : *p.xg * p.wg[e * p.wg_stride];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + ty * 4 + i;
        if (t >= hi) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t o = n0 + tx + 16 * j;
            if (o >= p.N) continue;
            float v = acc[i][j] * g;
            if (p.relu) v = fmaxf(v, 0.0f);
            if (p.bf16_out) static_cast<__nv_bfloat16*>(p.Y)[t * p.ldy + o] = __float2bfloat16_rn(v);
            else static_cast<float*>(p.Y)[t * p.ldy + o] = v;
        }
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
constexpr int64_t kMaxDim = (1ll << 31) - 256;

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" int gptq_fp4_matmul(const uint8_t* x_codes, const uint8_t* x_scales, const float* x_g, int64_t T,
                               const uint8_t* w_codes, const uint8_t* w_scales, const float* w_g, int64_t N, int64_t K,
                               int format, const int32_t* offsets, int64_t experts, int flags, void* Y, int64_t ldy,
                               void* stream) {
    if (T < 0 || N < 0 || K < 0 || T > kMaxDim || N > kMaxDim || K > kMaxDim || experts < 1 ||
        (format != GPTQ_MXFP4 && format != GPTQ_NVFP4) || (flags & ~(GPTQ_DQ_RELU | GPTQ_DQ_BF16_OUT | GPTQ_FP4_EXPERT_G)) ||
        (!offsets && experts != 1))
        return GPTQ_ERR_INVALID_ARG;
    if (experts > 65536) return GPTQ_ERR_UNSUPPORTED;
    if (T == 0 || N == 0) return GPTQ_OK;
    if (!Y || ldy < N || K < 1 || !x_codes || !x_scales || !w_codes || !w_scales || !aligned16(x_codes) || !aligned16(x_scales) ||
        !aligned16(w_codes) || !aligned16(w_scales) || (format == GPTQ_NVFP4 && (!x_g || !w_g)))
        return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    MParams p{};
    p.xc = x_codes;
    p.xs = x_scales;
    p.wc = w_codes;
    p.ws = w_scales;
    p.xg = x_g;
    p.wg = w_g;
    p.T = T;
    p.N = N;
    p.K = K;
    p.pitch = fp4_pitch(K);
    p.tiles_k = fp4_tiles(K, format);
    p.w_codes_stride = N * p.pitch;
    p.w_scales_stride = gptq_fp4_scale_bytes(N, K, format);
    p.wg_stride = (flags & GPTQ_FP4_EXPERT_G) ? 1 : 0;
    p.offsets = offsets;
    p.experts = (int)experts;
    p.relu = (flags & GPTQ_DQ_RELU) ? 1 : 0;
    p.bf16_out = (flags & GPTQ_DQ_BF16_OUT) ? 1 : 0;
    p.Y = Y;
    p.ldy = ldy;
    p.status = st.word;
    const dim3 grid((unsigned)(ceil_div(T, B_T) + (offsets ? experts : 0)), (unsigned)ceil_div(N, B_N));
    if (format == GPTQ_MXFP4) GPTQ_LAUNCH(K_FP4_MM, s, fp4_matmul_kernel<true><<<grid, 256, 0, s>>>(p));
    else GPTQ_LAUNCH(K_FP4_MM, s, fp4_matmul_kernel<false><<<grid, 256, 0, s>>>(p));
    GPTQ_LAUNCH_CHECK();
    return st.finish(s);
}

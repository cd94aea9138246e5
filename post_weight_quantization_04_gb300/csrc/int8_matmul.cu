// int8_matmul.cu — Y = X W^T for two matrices in the 8-bit integer form (int8.cuh), dense or with one
// weight per expert over rows sorted by expert:
//   Y[t][o] = act(sx[t] sw[e(t)][o] sum_k x[t][k] w[e(t)][o][k])
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "int8.cuh"
#include "tc_gemm.cuh"

namespace gptq {

namespace {

constexpr int I_MAX_EXPERTS = 1024;
// a sum of K products, each up to 2^14, has to fit 32 bits
constexpr int64_t I_MAX_K = (1 << 17) - 1;

struct IParams {
    const int8_t *xc, *wc;
    const float *xs, *ws;
    int T, N, K;
    int64_t pitch;
    const int32_t* offsets;   // null: one expert, all rows
    int experts;
    int relu, bf16_out;
    void* Y;
    int64_t ldy;
    int* status;
};

// rows [lo, hi) of expert e, made safe: within the rows of X
__device__ __forceinline__ void expert_rows(const IParams& p, int e, int* lo, int* hi) {
    if (!p.offsets) {
        *lo = 0;
        *hi = p.T;
        return;
    }
    const int a = p.offsets[e], b = p.offsets[e + 1];
    const int l = min(max(a, 0), p.T), h = min(max(b, l), p.T);
    if (l != a || h != b) set_status(p.status, GPTQ_ERR_INVALID_ARG);
    *lo = l;
    *hi = h;
}

// max(x, 0) that keeps a NaN
__device__ __forceinline__ float relu_of(float x) { return max_nan(x, 0.0f); }

// sum * sx * sw, the smaller scale first: with the sum a whole number that product is exact where it is
// subnormal, and past fp32 only if the result is
__device__ __forceinline__ float scaled(float sum, float a, float b) { return sum * min_nan(a, b) * max_nan(a, b); }

__device__ __forceinline__ void store_result(const IParams& p, int64_t row, int f, float v) {
    if (p.relu) v = relu_of(v);
    const int64_t at = row * p.ldy + f;
    if (p.bf16_out) static_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(v);
    else static_cast<float*>(p.Y)[at] = v;
}

// rows that belong to no expert are zero: those of [0, T) before the first range and after the last one
// (ranges that were clamped are an error)
__device__ __forceinline__ void zero_rest(const IParams& p, int cta, int ctas) {
    const int first = min(max(p.offsets[0], 0), p.T), last = max(min(p.offsets[p.experts], p.T), first);
    for (int r = cta; r < p.T - (last - first); r += ctas) {
        const int64_t row = r < first ? r : r + (last - first);
        for (int f = threadIdx.x; f < p.N; f += blockDim.x) store_result(p, row, f, 0.0f);
    }
}

// ------------------------------------------------------------------------------- few rows
// A CTA of 128 threads computes 8 features of up to 8 tokens: a thread takes 16 columns of each, every 128th
// such piece, and four products at a time go into 32-bit whole numbers (dp4a), which are exact. The
// sums are then added over the CTA.
constexpr int F_THREADS = 128, F_FEATURES = 8, F_TOKENS = 8;

template <int NT>
__device__ __forceinline__ void few_rows(const IParams& p, int e, int t0, int n, int f0, int (*part)[F_FEATURES * F_TOKENS]) {
    const int8_t* wc = p.wc + (int64_t)e * p.N * p.pitch;
    int acc[F_FEATURES][NT] = {};
    for (int64_t c = threadIdx.x * 16; c < p.pitch; c += F_THREADS * 16) {
        uint4 w[F_FEATURES], x[NT];
#pragma unroll
        for (int i = 0; i < F_FEATURES; ++i) w[i] = *reinterpret_cast<const uint4*>(wc + min(f0 + i, p.N - 1) * p.pitch + c);
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t] = *reinterpret_cast<const uint4*>(p.xc + (t0 + min(t, n - 1)) * p.pitch + c);
#pragma unroll
        for (int i = 0; i < F_FEATURES; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                int a = acc[i][t];
                a = __dp4a((int)w[i].x, (int)x[t].x, a);
                a = __dp4a((int)w[i].y, (int)x[t].y, a);
                a = __dp4a((int)w[i].z, (int)x[t].z, a);
                acc[i][t] = __dp4a((int)w[i].w, (int)x[t].w, a);
            }
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < F_FEATURES; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int v = __reduce_add_sync(0xffffffffu, acc[i][t]);
            if (lane == 0) part[warp][i * NT + t] = v;
        }
    __syncthreads();
    if (threadIdx.x < F_FEATURES * NT) {
        const int i = threadIdx.x / NT, t = threadIdx.x % NT, f = f0 + i;
        int v = 0;
#pragma unroll
        for (int k = 0; k < F_THREADS / 32; ++k) v += part[k][threadIdx.x];
        if (f < p.N && t < n) store_result(p, t0 + t, f, scaled((float)v, p.xs[t0 + t], p.ws[(int64_t)e * p.N + f]));
    }
    __syncthreads();
}

__global__ void __launch_bounds__(F_THREADS) int8_few_rows_kernel(const IParams p) {
    __shared__ int part[F_THREADS / 32][F_FEATURES * F_TOKENS];
    const int e = blockIdx.y;
    pdl_wait();
    if (e == p.experts) {   // (only with offsets)
        zero_rest(p, blockIdx.x, gridDim.x);
        return;
    }
    int lo, hi;
    expert_rows(p, e, &lo, &hi);
    const int f0 = blockIdx.x * F_FEATURES;
    for (int t = lo; t < hi;) {
        const int n = hi - t;
        if (n > 4) few_rows<8>(p, e, t, min(n, 8), f0, part);
        else if (n > 2) few_rows<4>(p, e, t, n, f0, part);
        else if (n == 2) few_rows<2>(p, e, t, 2, f0, part);
        else few_rows<1>(p, e, t, 1, f0, part);
        t += min(n, 8);
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
constexpr int64_t kMaxDim = (1ll << 31) - 512;

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" int gptq_int8_matmul(const int8_t* x_codes, const float* x_scales, int64_t T, const int8_t* w_codes, const float* w_scales,
                                int64_t N, int64_t K, const int32_t* offsets, int64_t experts, int flags, void* Y, int64_t ldy,
                                void* stream) {
    if (T < 0 || N < 0 || K < 0 || T > kMaxDim || N > kMaxDim || K > kMaxDim || experts < 1 ||
        (flags & ~(GPTQ_DQ_RELU | GPTQ_DQ_BF16_OUT)) || (!offsets && experts != 1))
        return GPTQ_ERR_INVALID_ARG;
    if (experts > I_MAX_EXPERTS || N > kMaxDim / experts || K > I_MAX_K) return GPTQ_ERR_UNSUPPORTED;
    if (T == 0 || N == 0) return GPTQ_OK;
    if (!Y || ldy < N || !x_scales || !w_scales || (K > 0 && (!x_codes || !w_codes || !aligned16(x_codes) || !aligned16(w_codes))))
        return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    IParams p{};
    p.xc = x_codes;
    p.wc = w_codes;
    p.xs = x_scales;
    p.ws = w_scales;
    p.T = (int)T;
    p.N = (int)N;
    p.K = (int)K;
    p.pitch = int8_pitch(K);
    p.offsets = offsets;
    p.experts = (int)experts;
    p.relu = (flags & GPTQ_DQ_RELU) ? 1 : 0;
    p.bf16_out = (flags & GPTQ_DQ_BF16_OUT) ? 1 : 0;
    p.Y = Y;
    p.ldy = ldy;
    p.status = st.word;
    cudaError_t e = cudaSuccess;
    const dim3 grid((unsigned)ceil_div(N, F_FEATURES), (unsigned)(experts + (offsets ? 1 : 0)));
    GPTQ_LAUNCH(K_INT8_MM, s, e = launch_pdl(int8_few_rows_kernel, grid, dim3(F_THREADS), 0, s, p));
    GPTQ_CUDA_TRY(e);
    return st.finish(s);
}

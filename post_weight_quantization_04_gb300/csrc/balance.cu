// balance.cu — the balance loss of a router, the experts' counts, and the loss's gradient.
//
//   p[t] = softmax(z[t]) over the E experts, n = the tokens that count (mask), c[e] = their slots with
//   ids = e:   L = E / (top n^2) sum_e c[e] sum_t p[t][e]     (1 where both are even)
//   dz[t][e] = dL E / (top n^2) p[t][e] (c[e] - sum_j p[t][j] c[j])
// Sums are fp32 in a fixed order; counts are whole numbers, so their atomics (in shared memory) give the same in any
// order.
#include <algorithm>

#include "common.cuh"
#include "int8.cuh"

namespace gptq {

namespace {

constexpr int L_THREADS = 256;          // 8 warps
constexpr int L_MAX_EXPERTS = 1024;
constexpr int L_MAX_CTAS = 152;
constexpr int L_AHEAD = 4;              // tokens in flight per group of lanes

struct LParams {
    const void* Z;
    int64_t tokens, ldz;
    int experts;
    int top;
    const int32_t* ids;
    const uint8_t* mask;     // null: every token counts
    float* sums;             // [cta][expert] sums of p
    int32_t* counts;         // [cta][expert + 1]; forward: per CTA; gradient: the call's
    const float* dloss;      // gradient
    void* dZ;
    int64_t lddz;
    float* loss;
    int* status;
};

__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// The softmax of a token over G lanes with V values each, lane l's v-th being expert l + G v (past the experts: 0).
// A row of nothing but -inf is 0. Returns the largest value's test: false where a NaN or +inf is among them.
template <int G, int V>
__device__ __forceinline__ bool softmax(float (&z)[V]) {
    float m = z[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = max_nan(m, z[v]);
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool none = m == -INFINITY;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        z[v] = none ? 0.0f : expf(z[v] - m);
        s += z[v];
    }
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float inv = none ? 0.0f : 1.0f / s;
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] *= inv;
    return m < INFINITY;
}

// the logits of token t, -inf where there is no expert or the token does not count
template <typename T, int G, int V>
__device__ __forceinline__ void load_logits(const LParams& p, int64_t t, bool live, float (&z)[V]) {
    const int l = threadIdx.x & (G - 1);
    const T* row = static_cast<const T*>(p.Z) + (live ? t * p.ldz : 0);
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = live && l + G * v < p.experts ? load_one(row + l + G * v) : -INFINITY;
}

template <typename T, int G, int V>
__global__ void __launch_bounds__(L_THREADS) balance_sums_kernel(const LParams p) {
    extern __shared__ float sh[];                               // [groups][experts], then counts [experts + 1]
    constexpr int GROUPS = L_THREADS / G;
    int32_t* cnt = reinterpret_cast<int32_t*>(sh + GROUPS * p.experts);
    for (int e = threadIdx.x; e <= p.experts; e += L_THREADS) cnt[e] = 0;
    pdl_wait();
    __syncthreads();
    const int64_t share = (p.tokens + gridDim.x - 1) / gridDim.x;
    const int64_t first = blockIdx.x * share, last = min(first + share, p.tokens);
    const int group = threadIdx.x / G, l = threadIdx.x & (G - 1);
    float acc[V] = {};
    int live_tokens = 0;
    bool fine = true;
    for (int64_t t0 = first; t0 < last; t0 += GROUPS * L_AHEAD) {   // (the same for the whole CTA)
        float z[L_AHEAD][V];
        bool live[L_AHEAD];
#pragma unroll
        for (int u = 0; u < L_AHEAD; ++u) {
            const int64_t t = t0 + u * GROUPS + group;
            live[u] = t < last && (!p.mask || p.mask[t]);
            load_logits<T, G, V>(p, t, live[u], z[u]);
        }
#pragma unroll
        for (int u = 0; u < L_AHEAD; ++u) {
            fine &= softmax<G, V>(z[u]);
            live_tokens += live[u] ? 1 : 0;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] += z[u][v];
        }
    }
    if (!fine) set_status(p.status, GPTQ_ERR_NONFINITE);
    if (l == 0 && live_tokens) atomicAdd(cnt + p.experts, live_tokens);
    for (int64_t i = first * p.top + threadIdx.x; i < last * p.top; i += L_THREADS) {
        const int e = p.ids[i];
        if (e < 0 || (p.mask && !p.mask[i / p.top])) continue;
        if (e < p.experts) atomicAdd(cnt + e, 1);
        else set_status(p.status, GPTQ_ERR_INVALID_ARG);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (l + G * v < p.experts) sh[group * p.experts + l + G * v] = acc[v];
    __syncthreads();
    for (int e = threadIdx.x; e <= p.experts; e += L_THREADS) {
        if (e < p.experts) {
            float s = 0.0f;
#pragma unroll 8
            for (int g = 0; g < GROUPS; ++g) s += sh[g * p.experts + e];
            p.sums[(int64_t)blockIdx.x * p.experts + e] = s;
        }
        p.counts[(int64_t)blockIdx.x * (p.experts + 1) + e] = cnt[e];
    }
}

// the CTAs' sums and counts to the loss and the counts: 32 experts x 32 shares of the CTAs at a time
__global__ void __launch_bounds__(1024) balance_loss_kernel(const LParams p, int ctas, int32_t* counts) {
    __shared__ float sums[32][33];
    __shared__ int32_t cnts[32][33];
    __shared__ float dots[32];
    __shared__ int32_t live;
    pdl_wait();
    float dot = 0.0f;
    for (int e0 = 0; e0 <= p.experts; e0 += 32) {
        const int e = e0 + threadIdx.x;
        float s = 0.0f;
        int32_t n = 0;
        if (e <= p.experts) {
#pragma unroll 4
            for (int k = threadIdx.y; k < ctas; k += 32) {
                if (e < p.experts) s += p.sums[(int64_t)k * p.experts + e];
                n += p.counts[(int64_t)k * (p.experts + 1) + e];
            }
        }
        sums[threadIdx.y][threadIdx.x] = s;
        cnts[threadIdx.y][threadIdx.x] = n;
        __syncthreads();
        s = sums[threadIdx.x][threadIdx.y];
        n = __reduce_add_sync(0xffffffffu, cnts[threadIdx.x][threadIdx.y]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const int mine = e0 + threadIdx.y;
        if (threadIdx.x == 0 && mine <= p.experts) {
            counts[mine] = n;
            if (mine == p.experts) live = n;
        }
        if (mine < p.experts) dot = fmaf((float)n, s, dot);
        __syncthreads();
    }
    if (threadIdx.x == 0) dots[threadIdx.y] = dot;
    __syncthreads();
    if (threadIdx.y == 0) {
        dot = dots[threadIdx.x];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float n = (float)max(live, 1);
        if (threadIdx.x == 0) *p.loss = (float)p.experts / (float)p.top * (dot / n / n);
    }
}

template <typename T, int G, int V>
__global__ void __launch_bounds__(L_THREADS) balance_grad_kernel(const LParams p) {
    constexpr int GROUPS = L_THREADS / G;
    pdl_wait();
    const int group = threadIdx.x / G, l = threadIdx.x & (G - 1);
    float c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = l + G * v < p.experts ? (float)p.counts[l + G * v] : 0.0f;
    const float n = (float)max(p.counts[p.experts], 1);
    const float k = (p.dloss ? *p.dloss : 1.0f) * ((float)p.experts / (float)p.top / n / n);
    for (int64_t t0 = (int64_t)blockIdx.x * GROUPS * L_AHEAD; t0 < p.tokens; t0 += (int64_t)gridDim.x * GROUPS * L_AHEAD) {
        float z[L_AHEAD][V];
        bool live[L_AHEAD];
#pragma unroll
        for (int u = 0; u < L_AHEAD; ++u) {
            const int64_t t = t0 + u * GROUPS + group;
            live[u] = t < p.tokens && (!p.mask || p.mask[t]);
            load_logits<T, G, V>(p, t, live[u], z[u]);
        }
#pragma unroll
        for (int u = 0; u < L_AHEAD; ++u) {
            const int64_t t = t0 + u * GROUPS + group;
            if (!softmax<G, V>(z[u])) set_status(p.status, GPTQ_ERR_NONFINITE);
            float mean = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) mean = fmaf(z[u][v], c[v], mean);
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
            if (t >= p.tokens) continue;
            T* out = static_cast<T*>(p.dZ) + t * p.lddz;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (l + G * v >= p.experts) continue;
                const float d[1] = {live[u] ? k * z[u][v] * (c[v] - mean) : 0.0f};
                store_unit<T, 1>(out + l + G * v, d);
            }
        }
    }
}

template <int A, int B>
struct GV {
    static constexpr int G = A, V = B;
};
// Calls f(GV): lanes per token and values per lane
template <typename F>
void with_lanes(int64_t experts, F f) {
    if (experts <= 4) f(GV<4, 1>());
    else if (experts <= 8) f(GV<8, 1>());
    else if (experts <= 16) f(GV<16, 1>());
    else if (experts <= 32) f(GV<32, 1>());
    else if (experts <= 64) f(GV<32, 2>());
    else if (experts <= 128) f(GV<32, 4>());
    else if (experts <= 256) f(GV<32, 8>());
    else if (experts <= 512) f(GV<32, 16>());
    else f(GV<32, 32>());
}

bool bad_dtype(int t) { return t != GPTQ_F32 && t != GPTQ_BF16; }
constexpr int64_t kMaxSlots = (1ll << 31) - 4096;
bool bad_shape(int64_t tokens, int64_t experts, int64_t top) {
    return tokens < 0 || experts < 1 || top < 1 || top > 65535 || tokens > kMaxSlots / top;
}
int64_t sum_ctas(int64_t tokens) { return std::min<int64_t>(std::max<int64_t>(ceil_div(tokens, 32), 1), L_MAX_CTAS); }

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" size_t gptq_expert_balance_workspace_bytes(int64_t tokens, int64_t experts) {
    if (tokens < 0 || experts < 1 || experts > L_MAX_EXPERTS) return 0;
    return (size_t)(sum_ctas(tokens) * (2 * experts + 1) * 4);
}

extern "C" int gptq_expert_balance(const void* Z, int dtype, int64_t tokens, int64_t experts, int64_t ldz, const int32_t* ids,
                                   int64_t top, const uint8_t* mask, float* loss, int32_t* counts, void* ws, size_t ws_bytes,
                                   void* stream) {
    if (bad_shape(tokens, experts, top) || bad_dtype(dtype)) return GPTQ_ERR_INVALID_ARG;
    if (experts > L_MAX_EXPERTS) return GPTQ_ERR_UNSUPPORTED;
    if (!loss || !counts || (tokens > 0 && (!Z || !ids || ldz < experts))) return GPTQ_ERR_INVALID_ARG;
    if (!ws || ws_bytes < gptq_expert_balance_workspace_bytes(tokens, experts)) return GPTQ_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) % 4 != 0) return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    const int64_t ctas = sum_ctas(tokens);
    LParams p{};
    p.Z = Z;
    p.tokens = tokens;
    p.ldz = ldz;
    p.experts = (int)experts;
    p.top = (int)top;
    p.ids = ids;
    p.mask = mask;
    p.sums = static_cast<float*>(ws);
    p.counts = reinterpret_cast<int32_t*>(p.sums + ctas * experts);
    p.loss = loss;
    p.status = st.word;
    cudaError_t e = cudaSuccess;
    with_lanes(experts, [&](auto gv) {
        constexpr int G = decltype(gv)::G, V = decltype(gv)::V;
        const size_t smem = 4 * ((size_t)(L_THREADS / G) * experts + experts + 1);   // at most 8 x 1024 words and 1025
        auto kern = dtype == GPTQ_BF16 ? balance_sums_kernel<__nv_bfloat16, G, V> : balance_sums_kernel<float, G, V>;
        GPTQ_LAUNCH(K_BALANCE, s, e = launch_pdl(kern, dim3((unsigned)ctas), dim3(L_THREADS), smem, s, p));
    });
    GPTQ_CUDA_TRY(e);
    GPTQ_LAUNCH(K_BALANCE, s, e = launch_pdl(balance_loss_kernel, dim3(1), dim3(32, 32), 0, s, p, (int)ctas, counts));
    GPTQ_CUDA_TRY(e);
    return st.finish(s);
}

extern "C" int gptq_expert_balance_grad(const float* dloss, const void* Z, int dtype, int64_t tokens, int64_t experts, int64_t ldz,
                                        const int32_t* counts, int64_t top, const uint8_t* mask, void* dZ, int64_t lddz, void* stream) {
    if (bad_shape(tokens, experts, top) || bad_dtype(dtype)) return GPTQ_ERR_INVALID_ARG;
    if (experts > L_MAX_EXPERTS) return GPTQ_ERR_UNSUPPORTED;
    if (tokens == 0) return GPTQ_OK;
    if (!Z || !counts || !dZ || ldz < experts || lddz < experts) return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    LParams p{};
    p.Z = Z;
    p.tokens = tokens;
    p.ldz = ldz;
    p.experts = (int)experts;
    p.top = (int)top;
    p.mask = mask;
    p.counts = const_cast<int32_t*>(counts);
    p.dloss = dloss;
    p.dZ = dZ;
    p.lddz = lddz;
    p.status = st.word;
    cudaError_t e = cudaSuccess;
    with_lanes(experts, [&](auto gv) {
        constexpr int G = decltype(gv)::G, V = decltype(gv)::V;
        const int64_t ctas = std::min<int64_t>(ceil_div(tokens, L_THREADS / G * L_AHEAD), 8 * kSMs);
        auto kern = dtype == GPTQ_BF16 ? balance_grad_kernel<__nv_bfloat16, G, V> : balance_grad_kernel<float, G, V>;
        GPTQ_LAUNCH(K_BALANCE, s, e = launch_pdl(kern, dim3((unsigned)ctas), dim3(L_THREADS), 0, s, p));
    });
    GPTQ_CUDA_TRY(e);
    return st.finish(s);
}

// balance.cu — the balance loss of a router, the experts' counts, and the loss's gradient.
//
//   p[t] = softmax(z[t]) over the E experts, n = the tokens that count (mask), c[e] = their slots with
//   ids = e:   L = E / (top n^2) sum_e c[e] sum_t p[t][e]     (1 where both are even)
//   dz[t][e] = dL E / (top n^2) p[t][e] (c[e] - sum_j p[t][j] c[j])
// (with counts taken from their mean, which changes nothing but the rounding: even counts give zeros)
// Sums are fp32 in a fixed order; counts are whole numbers, so their atomics (in shared memory) give the same in any
// order.
#include <algorithm>

#include "common.cuh"
#include "int8.cuh"
#include "pair.cuh"

namespace gptq {

namespace {

constexpr int L_THREADS = 256;          // of the gradient
constexpr int L_COUNTERS = 128;         // threads of the first kernel that count, besides those that take the softmax
constexpr int L_CLUSTER = 8;            // CTAs of the cluster that does all in one launch
constexpr int L_FEW = 128;              // tokens that never take two launches
// threads of the first kernel that take the softmax (their sums are in shared memory, by lanes and experts)
constexpr int summing_threads(int v) { return v <= 8 ? 512 : 256; }
constexpr int L_MAX_EXPERTS = 1024;
constexpr int L_MAX_CTAS = 304;
constexpr int L_SUMMERS = 1024;         // threads of a CTA of the second kernel
// tokens in flight per group of lanes, of V values per lane each
constexpr int ahead(int v) { return v <= 4 ? 4 : v <= 8 ? 2 : 1; }

struct LParams {
    const void* Z;
    int64_t tokens, ldz;
    int experts;
    int top;
    const int32_t* ids;
    const uint8_t* mask;     // null: every token counts
    float* sums;             // [cta][expert] sums of p
    int32_t* counts;         // [cta][expert + 1]; forward: per CTA; gradient: the call's
    int32_t* total;          // the call's counts
    const float* dloss;      // gradient
    void* dZ;
    int64_t lddz;
    float* loss;
    int together;            // the CTAs are one cluster, which leaves the results itself
    int* status;
};

// a word of another CTA's shared memory
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr, uint32_t rank) {
    uint32_t v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.u32 %0, [a];\n\t}"
                 : "=r"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

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

__device__ __forceinline__ float loss_of(const LParams& p, float dot, int32_t tokens) {
    const float n = (float)max(tokens, 1);
    return (float)p.experts / (float)p.top * (dot / n / n);
}

// Each CTA's sums of p and counts over a contiguous share of the tokens; with one CTA or one cluster of them the loss too. Bound by
// latency: a load, two trees of shuffles and a sum over the warps, then one over the CTAs, by their cluster or in a second launch.
// 16384 tokens x 64 experts fp32 11.3 us in two launches, 500 x 64 4.6 by a cluster (6.8 in two launches), 33 x 64 3.1 by one CTA,
// 16384 x 1024 48; with counting and softmax one after another in half the CTAs 16.7, 6.0 for 33 x 64, and 91.
template <typename T, int G, int V>
__global__ void __launch_bounds__(summing_threads(V) + L_COUNTERS) balance_sums_kernel(const LParams p) {
    extern __shared__ float sh[];                               // [groups][experts], then counts [experts + 1]
    constexpr int THREADS = summing_threads(V), ALL = THREADS + L_COUNTERS, GROUPS = THREADS / G, AHEAD = ahead(V);
    __shared__ float warp_dot[ALL / 32];
    __shared__ float dots;
    int32_t* cnt = reinterpret_cast<int32_t*>(sh + GROUPS * p.experts);
    for (int e = threadIdx.x; e <= p.experts; e += ALL) cnt[e] = 0;
    pdl_trigger();
    pdl_wait();
    __syncthreads();
    const int64_t share = (p.tokens + gridDim.x - 1) / gridDim.x;
    const int64_t first = blockIdx.x * share, last = min(first + share, p.tokens);
    if (threadIdx.x >= THREADS) {
        int live = 0;
        for (int64_t t = first + (threadIdx.x - THREADS); t < last; t += L_COUNTERS) {
            if (p.mask && !p.mask[t]) continue;
            ++live;
#pragma unroll 4
            for (int j = 0; j < p.top; ++j) {
                const int e = p.ids[t * p.top + j];
                if (e >= 0 && e < p.experts) atomicAdd(cnt + e, 1);
                else if (e >= 0) set_status(p.status, GPTQ_ERR_INVALID_ARG);
            }
        }
        if (live) atomicAdd(cnt + p.experts, live);
    } else {
        const int group = threadIdx.x / G, l = threadIdx.x & (G - 1);
        float acc[V] = {};
        bool fine = true;
        for (int64_t t0 = first; t0 < last; t0 += GROUPS * AHEAD) {   // (the same for all these threads)
            float z[AHEAD][V];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int64_t t = t0 + u * GROUPS + group;
                load_logits<T, G, V>(p, t, t < last && (!p.mask || p.mask[t]), z[u]);
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                fine &= softmax<G, V>(z[u]);
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] += z[u][v];
            }
        }
        if (!fine) set_status(p.status, GPTQ_ERR_NONFINITE);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (l + G * v < p.experts) sh[group * p.experts + l + G * v] = acc[v];
    }
    __syncthreads();
    float dot = 0.0f;
    for (int e = threadIdx.x; e <= p.experts; e += ALL) {
        float s = 0.0f;
        if (e < p.experts) {
#pragma unroll 8
            for (int g = 0; g < GROUPS; ++g) s += sh[g * p.experts + e];
        }
        if (p.together) {
            if (e < p.experts) sh[e] = s;   // (this thread's own column, which it has read)
        } else if (gridDim.x > 1) {
            if (e < p.experts) p.sums[(int64_t)blockIdx.x * p.experts + e] = s;
            p.counts[(int64_t)blockIdx.x * (p.experts + 1) + e] = cnt[e];
        } else {
            p.total[e] = cnt[e];
            if (e < p.experts) dot = fmaf((float)cnt[e], s, dot);
        }
    }
    if (gridDim.x > 1 && !p.together) return;
    if (p.together) {
        // the CTAs of the cluster share the experts (and, as one more, the tokens), each with the others' sums in their order
        cluster_sync();
        for (int e = blockIdx.x * ALL + threadIdx.x; e <= p.experts; e += gridDim.x * ALL) {
            float s = 0.0f;
            int32_t n = 0;
            for (uint32_t k = 0; k < gridDim.x; ++k) {
                if (e < p.experts) s += __uint_as_float(ld_cluster_u32(smem_u32(sh + e), k));
                n += (int32_t)ld_cluster_u32(smem_u32(cnt + e), k);
            }
            p.total[e] = n;
            if (e < p.experts) dot = fmaf((float)n, s, dot);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if ((threadIdx.x & 31) == 0) warp_dot[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
        dot = 0.0f;
        for (int w = 0; w < ALL / 32; ++w) dot += warp_dot[w];
        dots = dot;
        if (!p.together) *p.loss = loss_of(p, dot, cnt[p.experts]);
    }
    if (p.together) {
        cluster_sync();
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            int32_t tokens = 0;
            dot = 0.0f;
            for (uint32_t k = 0; k < gridDim.x; ++k) {
                dot += __uint_as_float(ld_cluster_u32(smem_u32(&dots), k));
                tokens += (int32_t)ld_cluster_u32(smem_u32(cnt + p.experts), k);
            }
            *p.loss = loss_of(p, dot, tokens);
        }
        cluster_sync();   // no CTA leaves while its sums are read
    }
}

// The CTAs' sums and counts to the counts and the loss. The CTAs of the cluster share the experts (and, as one more, the
// tokens), `wide` threads of each one's columns; its other threads share the rows. What they find is added in a
// fixed order.
__global__ void __launch_bounds__(L_SUMMERS) balance_loss_kernel(const LParams p, int rows, int wide) {
    __shared__ float sums[L_SUMMERS];
    __shared__ int32_t cnts[L_SUMMERS];
    __shared__ float warp_dot[L_SUMMERS / 32];
    __shared__ float dot;
    __shared__ int32_t live;
    pdl_wait();
    const int share = (p.experts + gridDim.x) / gridDim.x;   // of experts + 1 columns, rounded up
    const int c = threadIdx.x & (wide - 1), e = blockIdx.x * share + c, groups = L_SUMMERS / wide;
    const bool mine = c < share && e <= p.experts;
    float s = 0.0f;
    int32_t n = 0;
    if (mine) {
#pragma unroll 8
        for (int k = threadIdx.x / wide; k < rows; k += groups) {
            if (e < p.experts) s += p.sums[(int64_t)k * p.experts + e];
            n += p.counts[(int64_t)k * (p.experts + 1) + e];
        }
    }
    sums[threadIdx.x] = s;
    cnts[threadIdx.x] = n;
    __syncthreads();
    float d = 0.0f;
    if (threadIdx.x < wide && mine) {
        for (int g = 1; g < groups; ++g) {
            s += sums[g * wide + c];
            n += cnts[g * wide + c];
        }
        p.total[e] = n;
        if (e < p.experts) d = (float)n * s;
        else live = n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if ((threadIdx.x & 31) == 0) warp_dot[threadIdx.x >> 5] = d;
    __syncthreads();
    if (threadIdx.x == 0) {
        d = 0.0f;
        for (int w = 0; w < (wide + 31) / 32; ++w) d += warp_dot[w];
        dot = d;
    }
    if (gridDim.x > 1) cluster_sync();
    else __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        float all = dot;
        for (uint32_t r = 1; r < gridDim.x; ++r) all += __uint_as_float(ld_cluster_u32(smem_u32(&dot), r));
        const int32_t tokens = gridDim.x > 1 ? (int32_t)ld_cluster_u32(smem_u32(&live), p.experts / share) : live;
        *p.loss = loss_of(p, all, tokens);
    }
    if (gridDim.x > 1) cluster_sync();   // no CTA leaves while its sum is read
}

// 16384 tokens x 64 experts fp32 5.8 us, x 1024 32 us (4.2 TB/s): latency, then instructions.
template <typename T, int G, int V>
__global__ void __launch_bounds__(L_THREADS) balance_grad_kernel(const LParams p) {
    constexpr int GROUPS = L_THREADS / G;
    pdl_wait();
    constexpr int AHEAD = ahead(V);
    const int group = threadIdx.x / G, l = threadIdx.x & (G - 1);
    int n[V], sum = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        n[v] = l + G * v < p.experts ? p.counts[l + G * v] : 0;
        sum += n[v];
    }
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int mean_count = sum / p.experts;
    float c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = l + G * v < p.experts ? (float)(n[v] - mean_count) : 0.0f;
    const float tokens = (float)max(p.counts[p.experts], 1);
    const float k = (p.dloss ? *p.dloss : 1.0f) * ((float)p.experts / (float)p.top / tokens / tokens);
    for (int64_t t0 = (int64_t)blockIdx.x * GROUPS * AHEAD; t0 < p.tokens; t0 += (int64_t)gridDim.x * GROUPS * AHEAD) {
        float z[AHEAD][V];
        bool live[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int64_t t = t0 + u * GROUPS + group;
            live[u] = t < p.tokens && (!p.mask || p.mask[t]);
            load_logits<T, G, V>(p, t, live[u], z[u]);
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
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
                store_one(out + l + G * v, live[u] ? k * z[u][v] * (c[v] - mean) : 0.0f);
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
// CTAs of the first of two launches
int64_t sum_ctas(int64_t tokens) { return tokens <= L_FEW ? 1 : std::min<int64_t>(ceil_div(tokens, 32), L_MAX_CTAS); }
// CTAs of a launch that does all by itself: one, or one cluster; 0: too many tokens for that. A CTA takes
// (threads / lanes per token) x ahead tokens at a time, and more often than two or three times it is better to
// have all SMs at work and a second launch. (us, two launches / a cluster: 8 experts 2000 tokens 5.7 / 4.9, 4000 5.9 / 6.2; 64 experts 500
// 6.8 / 4.6, 1000 6.9 / 6.1, 2000 7.1 / 9.2; 256 experts 500 7.0 / 6.4, 1000 7.4 / 9.4; 1024 experts 200 13.6 / 11.3, 500 15.3 / 20.8; a
// launch less is 2.8 us of the call's time besides. One CTA: 64 experts 33 tokens 3.1.)
int alone_ctas(int64_t tokens, int64_t experts) {
    int64_t at_once = 0;
    with_lanes(experts, [&](auto gv) { at_once = summing_threads(gv.V) / gv.G * ahead(gv.V); });
    return tokens <= 2 * at_once ? 1 : tokens <= 3 * L_CLUSTER * at_once ? L_CLUSTER : 0;
}
// CTAs of the second kernel
unsigned summers(int64_t experts) { return experts >= 256 ? 8 : experts >= 32 ? 4 : 1; }

// A launch of `ctas` CTAs in clusters of `cluster`, which starts while the kernel before ends
struct Clustered {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    Clustered(unsigned ctas, unsigned cluster, dim3 block, size_t smem, cudaStream_t s) {
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = block;
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
};

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
    const int alone = alone_ctas(tokens, experts);
    const int64_t ctas = alone ? alone : sum_ctas(tokens);
    LParams p{};
    p.Z = Z;
    p.tokens = tokens;
    p.ldz = ldz;
    p.experts = (int)experts;
    p.top = (int)top;
    p.ids = ids;
    p.mask = mask;
    p.sums = static_cast<float*>(ws);
    if (!alone) p.counts = reinterpret_cast<int32_t*>(p.sums + ctas * experts);
    p.total = counts;
    p.loss = loss;
    p.together = alone > 1;
    p.status = st.word;
    cudaError_t e = cudaSuccess;
    with_lanes(experts, [&](auto gv) {
        constexpr int G = decltype(gv)::G, V = decltype(gv)::V;
        // at most 16 x 256 or 8 x 1024 words, and 1025
        const size_t smem = 4 * ((size_t)(summing_threads(V) / G) * experts + experts + 1);
        auto kern = dtype == GPTQ_BF16 ? balance_sums_kernel<__nv_bfloat16, G, V> : balance_sums_kernel<float, G, V>;
        const dim3 block(summing_threads(V) + L_COUNTERS);
        if (p.together) {
            const Clustered l(ctas, L_CLUSTER, block, smem, s);
            GPTQ_LAUNCH(K_BALANCE, s, e = cudaLaunchKernelEx(&l.cfg, kern, p));
        } else {
            GPTQ_LAUNCH(K_BALANCE, s, e = launch_pdl(kern, dim3((unsigned)ctas), block, smem, s, p));
        }
    });
    GPTQ_CUDA_TRY(e);
    if (alone) return st.finish(s);
    int wide = 1;
    while (wide < ceil_div(experts + 1, summers(experts))) wide <<= 1;
    const Clustered l(summers(experts), summers(experts), dim3(L_SUMMERS), 0, s);
    GPTQ_LAUNCH(K_BALANCE, s, e = cudaLaunchKernelEx(&l.cfg, balance_loss_kernel, p, (int)ctas, wide));
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
        const int64_t ctas = std::min<int64_t>(ceil_div(tokens, L_THREADS / G * ahead(V)), 8 * kSMs);
        auto kern = dtype == GPTQ_BF16 ? balance_grad_kernel<__nv_bfloat16, G, V> : balance_grad_kernel<float, G, V>;
        GPTQ_LAUNCH(K_BALANCE, s, e = launch_pdl(kern, dim3((unsigned)ctas), dim3(L_THREADS), 0, s, p));
    });
    GPTQ_CUDA_TRY(e);
    return st.finish(s);
}

// expert.cu — tokens sorted by expert and back: the routing around expert layers.
//
// A token t has `top` slots; slot i = t * top + j goes to expert ids[i], or nowhere (negative).
//   sort      pos[i] = offsets[ids[i]] + #{i' < i : ids[i'] = ids[i]} (-1: dropped), src its
//             inverse (-1 past the last live place); stable, so the order of results never
//             depends on timing
//   gather    xs[pos[t][j]] = x[t], rows past the last live place zero
//   combine   y[t] = sum_j w[t][j] ys[pos[t][j]] (w = 1: the gather's gradient)
//   gradient  dys[pos[t][j]] = w[t][j] dy[t] (past the last live place zero),
//             dw[t][j] = <dy[t], ys[pos[t][j]]>
// Sums are fp32 in a fixed order, rounded once.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"

namespace gptq {

namespace {

// ------------------------------------------------------------------------------------ sort
constexpr int S_WARPS = 8, S_THREADS = 32 * S_WARPS;
constexpr int S_CHUNK = 2048;          // least slots per CTA: below that one CTA does it all
constexpr int S_MAX_EXPERTS = 1024;    // S_WARPS counters per expert in shared memory
constexpr int S_MAX_CTAS = 152;        // every CTA reads every CTA's counts

struct SParams {
    const int32_t* ids;
    int64_t slots, chunk;      // chunk: slots per CTA
    int experts;
    int32_t *offsets, *src, *pos;
    int32_t* counts;           // [cta][expert], when there is more than one CTA
    int* status;
};

__device__ __forceinline__ int slot_expert(const SParams& p, int64_t i, int64_t end) {
    if (i >= end) return -1;
    const int e = p.ids[i];
    if (e >= p.experts) set_status(p.status, GPTQ_ERR_INVALID_ARG);
    return e >= 0 && e < p.experts ? e : -1;
}

// counts[w][e] += the slots of expert e that warp w of this CTA owns (its share is contiguous)
__device__ __forceinline__ void count_slots(const SParams& p, int64_t begin, int64_t end, int32_t* mine) {
    const int lane = threadIdx.x & 31;
    for (int64_t i0 = begin; i0 < end; i0 += 32) {
        const int e = slot_expert(p, i0 + lane, end);
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && (same & ((1u << lane) - 1u)) == 0) mine[e] += __popc(same);
        __syncwarp();
    }
}

__device__ __forceinline__ void warp_share(const SParams& p, int64_t* begin, int64_t* end) {
    const int64_t share = p.chunk / S_WARPS;
    *begin = (int64_t)blockIdx.x * p.chunk + (threadIdx.x >> 5) * share;
    *end = min(*begin + share, p.slots);
}

__global__ void __launch_bounds__(S_THREADS) expert_count_kernel(const SParams p) {
    extern __shared__ int32_t cnt[];   // [S_WARPS][experts]
    for (int i = threadIdx.x; i < S_WARPS * p.experts; i += S_THREADS) cnt[i] = 0;
    __syncthreads();
    int64_t b, e;
    warp_share(p, &b, &e);
    count_slots(p, b, e, cnt + (threadIdx.x >> 5) * p.experts);
    __syncthreads();
    for (int i = threadIdx.x; i < p.experts; i += S_THREADS) {
        int32_t n = 0;
        for (int w = 0; w < S_WARPS; ++w) n += cnt[w * p.experts + i];
        p.counts[(int64_t)blockIdx.x * p.experts + i] = n;
    }
}

// Places every slot. With one CTA the counts are its own; with more, each CTA sums the counts of
// all CTAs (totals, for the offsets) and of those before it.
__global__ void __launch_bounds__(S_THREADS) expert_place_kernel(const SParams p) {
    extern __shared__ int32_t cnt[];       // [S_WARPS][experts], then totals [experts]
    int32_t* total = cnt + S_WARPS * p.experts;
    __shared__ int32_t warp_sum[S_WARPS], carry;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < S_WARPS * p.experts; i += S_THREADS) cnt[i] = 0;
    if (threadIdx.x == 0) carry = 0;
    __syncthreads();
    int64_t b, e;
    warp_share(p, &b, &e);
    count_slots(p, b, e, cnt + warp * p.experts);
    __syncthreads();
    // exclusive prefix over the experts, S_THREADS at a time
    for (int e0 = 0; e0 < p.experts; e0 += S_THREADS) {
        const int x = e0 + threadIdx.x;
        int32_t all = 0, before = 0;
        if (x < p.experts) {
            if (gridDim.x > 1) {
                for (int c = 0; c < (int)gridDim.x; ++c) {
                    const int32_t n = p.counts[(int64_t)c * p.experts + x];
                    all += n;
                    if (c < (int)blockIdx.x) before += n;
                }
            } else {
                for (int w = 0; w < S_WARPS; ++w) all += cnt[w * p.experts + x];
            }
        }
        int32_t inc = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        int32_t first = carry + inc - all;
        for (int w = 0; w < warp; ++w) first += warp_sum[w];
        if (x < p.experts) {
            total[x] = first + all;
            if (blockIdx.x == 0) p.offsets[x] = first;
            // where each warp's slots of this expert start
            int32_t at = first + before;
            for (int w = 0; w < S_WARPS; ++w) {
                const int32_t n = cnt[w * p.experts + x];
                cnt[w * p.experts + x] = at;
                at += n;
            }
        }
        __syncthreads();
        if (threadIdx.x == S_THREADS - 1) carry = first + all;
        __syncthreads();
    }
    const int32_t live = total[p.experts - 1];
    if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[p.experts] = live;
    int32_t* mine = cnt + warp * p.experts;
    for (int64_t i0 = b; i0 < e; i0 += 32) {
        const int64_t i = i0 + lane;
        const int x = slot_expert(p, i, e);
        const uint32_t same = __match_any_sync(0xffffffffu, x);
        const int rank = __popc(same & ((1u << lane) - 1u));
        int32_t at = -1;
        if (x >= 0) at = mine[x] + rank;
        __syncwarp();
        if (x >= 0 && rank == 0) mine[x] += __popc(same);
        __syncwarp();
        if (i < e) {
            p.pos[i] = at;
            if (at >= 0) p.src[at] = (int32_t)i;
        }
    }
    for (int64_t i = live + (int64_t)blockIdx.x * S_THREADS + threadIdx.x; i < p.slots; i += (int64_t)gridDim.x * S_THREADS)
        p.src[i] = -1;
}

int64_t sort_chunk(int64_t slots) {
    const int64_t c = std::max<int64_t>(S_CHUNK, ceil_div(slots, S_MAX_CTAS));
    return ceil_div(c, 32 * S_WARPS) * (32 * S_WARPS);
}

// ---------------------------------------------------------------------------- rows there and back
constexpr int R_THREADS = 256;

struct RParams {
    const void* X;          // gather: x; combine: ys; gradient: ys
    int64_t ldx;
    const void* dY;         // gradient: dy
    int64_t lddy;
    void* Y;                // gather: xs; combine: y; gradient: dys
    int64_t ldy;
    int64_t tokens, slots;
    int top;
    int64_t d;
    const int32_t* pos;
    const int32_t* live;    // offsets + experts: the number of live rows
    const float* w;
    float* dw;
    int* status;
};

// the place of slot i, or -1 (a place past the rows is an error and counts as dropped)
__device__ __forceinline__ int64_t place(const RParams& p, int64_t i) {
    const int64_t at = p.pos[i];
    if (at >= p.slots) {
        set_status(p.status, GPTQ_ERR_INVALID_ARG);
        return -1;
    }
    return at;
}

__device__ __forceinline__ int64_t live_rows(const RParams& p) {
    const int64_t n = *p.live;
    return n < 0 ? 0 : n < p.slots ? n : p.slots;
}

// Rows are moved in units of U (16 bytes where pointers and strides allow, one element
// otherwise), `units` per row. Each row of x is read once and written `top` times.
template <typename U>
__global__ void __launch_bounds__(R_THREADS) expert_gather_kernel(const RParams p, int64_t units, int chunks, int64_t main_ctas) {
    const U* X = static_cast<const U*>(p.X);
    U* Y = static_cast<U*>(p.Y);
    if (blockIdx.x >= main_ctas) {   // the rows past the last live one
        const int64_t n = gridDim.x - main_ctas;
        const U zero = {};
        for (int64_t r = live_rows(p) + (blockIdx.x - main_ctas); r < p.slots; r += n)
            for (int64_t u = threadIdx.x; u < units; u += R_THREADS) Y[r * p.ldy + u] = zero;
        return;
    }
    const int64_t t = blockIdx.x / chunks;
    const int64_t u = (int64_t)(blockIdx.x % chunks) * R_THREADS + threadIdx.x;
    if (u >= units) return;
    const U v = X[t * p.ldx + u];
    for (int j = 0; j < p.top; ++j) {
        const int64_t at = place(p, t * p.top + j);
        if (at >= 0) Y[at * p.ldy + u] = v;
    }
}

// N consecutive elements as fp32
template <typename T, int N>
__device__ __forceinline__ void load_row(const T* x, float (&v)[N]) {
    if constexpr (N == 1) {
        if constexpr (sizeof(T) == 2) v[0] = __bfloat162float(*x);
        else v[0] = *x;
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(x);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
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
__device__ __forceinline__ void store_row(T* y, const float (&v)[N]) {
    if constexpr (N == 1) {
        if constexpr (sizeof(T) == 2) *y = __float2bfloat16_rn(v[0]);
        else *y = v[0];
    } else {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (sizeof(T) == 2) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                u[e] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                u[e] = __float_as_uint(v[e]);
            }
        }
        *reinterpret_cast<uint4*>(y) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

template <typename T, int N>
__global__ void __launch_bounds__(R_THREADS) expert_combine_kernel(const RParams p, int chunks) {
    const int64_t t = blockIdx.x / chunks;
    const int64_t c = ((int64_t)(blockIdx.x % chunks) * R_THREADS + threadIdx.x) * N;
    if (c >= p.d) return;
    const T* X = static_cast<const T*>(p.X);
    float acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
    for (int j = 0; j < p.top; ++j) {
        const int64_t at = place(p, t * p.top + j);
        if (at < 0) continue;
        const float w = p.w ? p.w[t * p.top + j] : 1.0f;
        float v[N];
        load_row<T, N>(X + at * p.ldx + c, v);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = fmaf(w, v[e], acc[e]);
    }
    store_row<T, N>(static_cast<T*>(p.Y) + t * p.ldy + c, acc);
}

// One CTA per token: dy is read once per slot from L1, ys once, dys written once.
template <typename T, int N>
__global__ void __launch_bounds__(R_THREADS) expert_combine_grad_kernel(const RParams p) {
    const T* X = static_cast<const T*>(p.X);
    T* Y = static_cast<T*>(p.Y);
    if (blockIdx.x >= p.tokens) {
        const int64_t n = gridDim.x - p.tokens;
        float zero[N] = {};
        for (int64_t r = live_rows(p) + (blockIdx.x - p.tokens); r < p.slots; r += n)
            for (int64_t c = threadIdx.x * N; c < p.d; c += R_THREADS * N) store_row<T, N>(Y + r * p.ldy + c, zero);
        return;
    }
    __shared__ float part[R_THREADS / 32];
    const int64_t t = blockIdx.x;
    const T* dy = static_cast<const T*>(p.dY) + t * p.lddy;
    for (int j = 0; j < p.top; ++j) {
        const int64_t at = place(p, t * p.top + j);   // the same for the whole CTA
        float dot = 0.0f;
        if (at >= 0) {
            const float w = p.w[t * p.top + j];
            for (int64_t c = threadIdx.x * N; c < p.d; c += R_THREADS * N) {
                float a[N], b[N];
                load_row<T, N>(dy + c, a);
                load_row<T, N>(X + at * p.ldx + c, b);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    dot = fmaf(a[e], b[e], dot);
                    a[e] *= w;
                }
                store_row<T, N>(Y + at * p.ldy + c, a);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float sum = 0.0f;
            for (int i = 0; i < R_THREADS / 32; ++i) sum += part[i];
            p.dw[t * p.top + j] = sum;
        }
        __syncthreads();
    }
}

bool bad_dtype(int t) { return t != GPTQ_F32 && t != GPTQ_BF16; }
bool vec16(const void* p, int64_t ld, int64_t esize) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * esize) % 16 == 0; }
constexpr int64_t kMaxSlots = (1ll << 31) - 4096;
bool bad_shape(int64_t tokens, int64_t top, int64_t d) {
    return tokens < 0 || top < 1 || top > 65535 || d < 0 || d > kMaxSlots || tokens > kMaxSlots / top;
}
// CTAs that clear the rows past the last live one (none is known on the host)
int tail_ctas(int64_t slots) { return (int)std::min<int64_t>(slots, 304); }

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" size_t gptq_expert_sort_workspace_bytes(int64_t tokens, int64_t top, int64_t experts) {
    if (tokens < 0 || top < 1 || experts < 1 || tokens > kMaxSlots / top || experts > S_MAX_EXPERTS) return 0;
    const int64_t ctas = ceil_div(tokens * top, sort_chunk(tokens * top));
    return ctas > 1 ? (size_t)(ctas * experts * 4) : 0;
}

extern "C" int gptq_expert_sort(const int32_t* ids, int64_t tokens, int64_t top, int64_t experts, int32_t* offsets,
                                int32_t* src, int32_t* pos, void* ws, size_t ws_bytes, void* stream) {
    if (bad_shape(tokens, top, 0) || experts < 1) return GPTQ_ERR_INVALID_ARG;
    if (experts > S_MAX_EXPERTS) return GPTQ_ERR_UNSUPPORTED;
    if (!offsets || (tokens > 0 && (!ids || !src || !pos))) return GPTQ_ERR_INVALID_ARG;
    const size_t need = gptq_expert_sort_workspace_bytes(tokens, top, experts);
    if (need > 0 && (!ws || ws_bytes < need)) return GPTQ_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    SParams p{ids, tokens * top, sort_chunk(tokens * top), (int)experts, offsets, src, pos, static_cast<int32_t*>(ws), st.word};
    const unsigned grid = (unsigned)std::max<int64_t>(1, ceil_div(p.slots, p.chunk));
    const size_t smem = sizeof(int32_t) * S_WARPS * experts;
    if (grid > 1) {
        GPTQ_LAUNCH(K_EXPERT_SORT, s, expert_count_kernel<<<grid, S_THREADS, smem, s>>>(p));
        GPTQ_LAUNCH_CHECK();
    }
    GPTQ_LAUNCH(K_EXPERT_SORT, s, expert_place_kernel<<<grid, S_THREADS, smem + sizeof(int32_t) * experts, s>>>(p));
    GPTQ_LAUNCH_CHECK();
    return st.finish(s);
}

extern "C" int gptq_expert_gather(const void* X, int dtype, int64_t tokens, int64_t d, int64_t ldx, const int32_t* pos,
                                  int64_t top, const int32_t* offsets, int64_t experts, void* Xs, int64_t lds, void* stream) {
    if (bad_shape(tokens, top, d) || bad_dtype(dtype) || experts < 1) return GPTQ_ERR_INVALID_ARG;
    if (tokens == 0 || d == 0) return GPTQ_OK;
    if (!X || !pos || !offsets || !Xs || ldx < d || lds < d) return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    const int64_t es = dtype == GPTQ_BF16 ? 2 : 4;
    const bool vec = vec16(X, ldx, es) && vec16(Xs, lds, es) && (d * es) % 16 == 0;
    const int64_t unit = vec ? 16 / es : 1, units = d / unit;
    RParams p{X, ldx / unit, nullptr, 0, Xs, lds / unit, tokens, tokens * top, (int)top, d, pos, offsets + experts, nullptr, nullptr, st.word};
    const int64_t chunks = ceil_div(units, R_THREADS), main_ctas = tokens * chunks;
    if (main_ctas > kMaxSlots) return GPTQ_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)(main_ctas + tail_ctas(p.slots));
    auto go = [&](auto kern) { GPTQ_LAUNCH(K_EXPERT_GATHER, s, kern<<<grid, R_THREADS, 0, s>>>(p, units, (int)chunks, main_ctas)); };
    if (vec) go(expert_gather_kernel<uint4>);
    else if (es == 2) go(expert_gather_kernel<uint16_t>);
    else go(expert_gather_kernel<uint32_t>);
    GPTQ_LAUNCH_CHECK();
    return st.finish(s);
}

extern "C" int gptq_expert_combine(const void* Ys, int dtype, int64_t tokens, int64_t d, int64_t ldys, const int32_t* pos,
                                   int64_t top, const float* weights, void* Y, int64_t ldy, void* stream) {
    if (bad_shape(tokens, top, d) || bad_dtype(dtype)) return GPTQ_ERR_INVALID_ARG;
    if (tokens == 0 || d == 0) return GPTQ_OK;
    if (!Ys || !pos || !Y || ldys < d || ldy < d) return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    const int64_t es = dtype == GPTQ_BF16 ? 2 : 4;
    const bool vec = vec16(Ys, ldys, es) && vec16(Y, ldy, es) && (d * es) % 16 == 0;
    RParams p{Ys, ldys, nullptr, 0, Y, ldy, tokens, tokens * top, (int)top, d, pos, nullptr, weights, nullptr, st.word};
    const int64_t chunks = ceil_div(d, R_THREADS * (vec ? 16 / es : 1));
    if (tokens * chunks > kMaxSlots) return GPTQ_ERR_UNSUPPORTED;
    auto go = [&](auto kern) { GPTQ_LAUNCH(K_EXPERT_COMBINE, s, kern<<<(unsigned)(tokens * chunks), R_THREADS, 0, s>>>(p, (int)chunks)); };
    if (dtype == GPTQ_BF16) vec ? go(expert_combine_kernel<__nv_bfloat16, 8>) : go(expert_combine_kernel<__nv_bfloat16, 1>);
    else vec ? go(expert_combine_kernel<float, 4>) : go(expert_combine_kernel<float, 1>);
    GPTQ_LAUNCH_CHECK();
    return st.finish(s);
}

extern "C" int gptq_expert_combine_grad(const void* dY, int64_t lddy, const void* Ys, int64_t ldys, int dtype, int64_t tokens,
                                        int64_t d, const int32_t* pos, int64_t top, const int32_t* offsets, int64_t experts,
                                        const float* weights, void* dYs, int64_t lddys, float* dW, void* stream) {
    if (bad_shape(tokens, top, d) || bad_dtype(dtype) || experts < 1) return GPTQ_ERR_INVALID_ARG;
    if (tokens == 0) return GPTQ_OK;
    if (!dY || !Ys || !pos || !offsets || !weights || !dYs || !dW || lddy < d || ldys < d || lddys < d) return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    const int64_t es = dtype == GPTQ_BF16 ? 2 : 4;
    const bool vec = vec16(dY, lddy, es) && vec16(Ys, ldys, es) && vec16(dYs, lddys, es) && (d * es) % 16 == 0;
    RParams p{Ys, ldys, dY, lddy, dYs, lddys, tokens, tokens * top, (int)top, d, pos, offsets + experts, weights, dW, st.word};
    const unsigned grid = (unsigned)(tokens + tail_ctas(p.slots));
    auto go = [&](auto kern) { GPTQ_LAUNCH(K_EXPERT_GRAD, s, kern<<<grid, R_THREADS, 0, s>>>(p)); };
    if (dtype == GPTQ_BF16) vec ? go(expert_combine_grad_kernel<__nv_bfloat16, 8>) : go(expert_combine_grad_kernel<__nv_bfloat16, 1>);
    else vec ? go(expert_combine_grad_kernel<float, 4>) : go(expert_combine_grad_kernel<float, 1>);
    GPTQ_LAUNCH_CHECK();
    return st.finish(s);
}

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
#include <initializer_list>
#include <type_traits>

#include "common.cuh"

namespace gptq {

namespace {

// ------------------------------------------------------------------------------------ sort
// Up to S_ALONE slots are sorted by one CTA of 32 warps in one launch; more by CTAs of 8 warps, which
// count their slots in a first launch and place them in a second. Either way a warp owns a
// contiguous share of the slots and counts equal experts among 32 slots at a time, so places are
// stable without atomics. Equal experts are found by one ballot per bit of the expert's number
// (match.any took several times as long). Bound by latency: 10 slots 2.4 us, 32768 slots and 8 experts
// 8 us in two launches, of which the second starts while the first runs; one CTA for all of them
// took 22.
constexpr int S_ALONE = 4096;
constexpr int S_CHUNK = 512;           // otherwise the least slots per CTA
constexpr int S_MAX_EXPERTS = 1024;    // one counter per warp and expert in shared memory
constexpr int S_MAX_CTAS = 152;        // every CTA reads every CTA's counts
constexpr int S_AHEAD = 8;             // loads of 32 slots in flight per warp

struct SParams {
    const int32_t* ids;
    int64_t slots, chunk;      // chunk: slots per CTA
    int experts;
    int32_t *offsets, *src, *pos;
    int32_t* counts;           // [cta][expert], when there is more than one CTA
    int* status;
};

// the experts of up to 32 S_AHEAD slots from i0 on, -1 where there is none
__device__ __forceinline__ void load_experts(const SParams& p, int64_t i0, int64_t end, int (&e)[S_AHEAD]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < S_AHEAD; ++u) e[u] = i0 + 32 * u + lane < end ? p.ids[i0 + 32 * u + lane] : -1;
#pragma unroll
    for (int u = 0; u < S_AHEAD; ++u) {
        if (e[u] >= p.experts) {
            set_status(p.status, GPTQ_ERR_INVALID_ARG);
            e[u] = -1;
        }
        e[u] = max(e[u], -1);
    }
}

// the lanes with the same expert (bits: of the largest expert's number)
__device__ __forceinline__ uint32_t same_expert(int e, int bits) {
    uint32_t same = __ballot_sync(0xffffffffu, e >= 0);
    for (int b = 0; b < bits; ++b) {
        const bool one = e >> b & 1;
        const uint32_t m = __ballot_sync(0xffffffffu, one);
        same &= one ? m : ~m;
    }
    return same;   // only looked at by lanes with an expert
}

// mine[e] += the slots of expert e in this warp's share
__device__ __forceinline__ void count_slots(const SParams& p, int64_t begin, int64_t end, int32_t* mine) {
    const int lane = threadIdx.x & 31, bits = 32 - __clz(p.experts - 1);
    for (int64_t i0 = begin; i0 < end; i0 += 32 * S_AHEAD) {
        int e[S_AHEAD];
        load_experts(p, i0, end, e);
#pragma unroll
        for (int u = 0; u < S_AHEAD; ++u) {
            if (i0 + 32 * u >= end) break;
            const uint32_t same = same_expert(e[u], bits);
            if (e[u] >= 0 && (same & ((1u << lane) - 1u)) == 0) mine[e[u]] += __popc(same);
            __syncwarp();
        }
    }
}

template <int WARPS>
__device__ __forceinline__ void warp_share(const SParams& p, int64_t* begin, int64_t* end) {
    // whole groups of 32 slots per warp
    const int64_t cta = (int64_t)blockIdx.x * p.chunk, last = min(cta + p.chunk, p.slots);
    const int64_t share = ((last - cta + 32 * WARPS - 1) / (32 * WARPS)) * 32;
    *begin = min(cta + (threadIdx.x >> 5) * share, last);
    *end = min(*begin + share, last);
}

template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS) expert_count_kernel(const SParams p) {
    extern __shared__ int32_t cnt[];   // [WARPS][experts]
    pdl_trigger();
    for (int i = threadIdx.x; i < WARPS * p.experts; i += 32 * WARPS) cnt[i] = 0;
    __syncthreads();
    int64_t b, e;
    warp_share<WARPS>(p, &b, &e);
    count_slots(p, b, e, cnt + (threadIdx.x >> 5) * p.experts);
    __syncthreads();
    for (int i = threadIdx.x; i < p.experts; i += 32 * WARPS) {
        int32_t n = 0;
        for (int w = 0; w < WARPS; ++w) n += cnt[w * p.experts + i];
        p.counts[(int64_t)blockIdx.x * p.experts + i] = n;
    }
}

// Places every slot. With one CTA the counts are its own; with more, each CTA sums the counts of
// all CTAs (totals, for the offsets) and of those before it.
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS) expert_place_kernel(const SParams p) {
    constexpr int THREADS = 32 * WARPS;
    extern __shared__ int32_t cnt[];       // [WARPS][experts]
    __shared__ int32_t warp_sum[WARPS], carry;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < WARPS * p.experts; i += THREADS) cnt[i] = 0;
    if (threadIdx.x == 0) carry = 0;
    __syncthreads();
    pdl_trigger();   // the gather's launch
    int64_t b, e;
    warp_share<WARPS>(p, &b, &e);
    count_slots(p, b, e, cnt + warp * p.experts);
    __syncthreads();
    pdl_wait();   // the counts of the other CTAs (everything before is this kernel's own input)
    // exclusive prefix over the experts, THREADS at a time; where there are fewer, several threads share
    // the CTAs' counts of one (with one thread each the sum over 64 CTAs took 4 us)
    int wide = 32;
    while (wide < p.experts && wide < THREADS) wide <<= 1;
    const int groups = THREADS / wide, mine_of = (int)threadIdx.x % wide, group = (int)threadIdx.x / wide;
    for (int e0 = 0; e0 < p.experts; e0 += THREADS) {
        const int x = e0 + threadIdx.x;
        int32_t all = 0, before = 0;
        if (gridDim.x > 1) {
            __shared__ int32_t sum_all[THREADS], sum_before[THREADS];
            if (e0 + mine_of < p.experts) {
#pragma unroll 4
                for (int c = group; c < (int)gridDim.x; c += groups) {
                    const int32_t n = p.counts[(int64_t)c * p.experts + e0 + mine_of];
                    all += n;
                    if (c < (int)blockIdx.x) before += n;
                }
            }
            sum_all[threadIdx.x] = all;
            sum_before[threadIdx.x] = before;
            __syncthreads();
            all = before = 0;
            if (x < p.experts && group == 0)
                for (int k = 0; k < groups; ++k) {
                    all += sum_all[k * wide + mine_of];
                    before += sum_before[k * wide + mine_of];
                }
        } else if (x < p.experts) {
            for (int w = 0; w < WARPS; ++w) all += cnt[w * p.experts + x];
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
            if (blockIdx.x == 0) p.offsets[x] = first;
            // where each warp's slots of this expert start
            int32_t at = first + before;
            for (int w = 0; w < WARPS; ++w) {
                const int32_t n = cnt[w * p.experts + x];
                cnt[w * p.experts + x] = at;
                at += n;
            }
        }
        __syncthreads();
        if (threadIdx.x == THREADS - 1) carry = first + all;
        __syncthreads();
    }
    const int32_t live = carry;
    if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[p.experts] = live;
    int32_t* mine = cnt + warp * p.experts;
    const int bits = 32 - __clz(p.experts - 1);
    for (int64_t i0 = b; i0 < e; i0 += 32 * S_AHEAD) {
        int x[S_AHEAD];
        load_experts(p, i0, e, x);
#pragma unroll
        for (int u = 0; u < S_AHEAD; ++u) {
            const int64_t i = i0 + 32 * u + lane;
            if (i0 + 32 * u >= e) break;
            const uint32_t same = same_expert(x[u], bits);
            const int rank = __popc(same & ((1u << lane) - 1u));
            int32_t at = -1;
            if (x[u] >= 0) at = mine[x[u]] + rank;
            __syncwarp();
            if (x[u] >= 0 && rank == 0) mine[x[u]] += __popc(same);
            __syncwarp();
            if (i < e) {
                p.pos[i] = at;
                if (at >= 0) p.src[at] = (int32_t)i;
            }
        }
    }
    for (int64_t i = live + (int64_t)blockIdx.x * THREADS + threadIdx.x; i < p.slots; i += (int64_t)gridDim.x * THREADS)
        p.src[i] = -1;
}

int64_t sort_chunk(int64_t slots) {
    if (slots <= S_ALONE) return S_ALONE;
    return ceil_div(std::max<int64_t>(S_CHUNK, ceil_div(slots, S_MAX_CTAS)), 256) * 256;
}

template <int WARPS>
cudaError_t launch_place(const SParams& p, unsigned grid, cudaStream_t s) {
    const size_t smem = sizeof(int32_t) * WARPS * p.experts;
    cudaError_t e = cudaSuccess;
    // 48 KB, static and dynamic together, is what a launch may have by default. The limit is the kernel's and not the
    // call's, so it is raised to what the most experts need: another thread's call sets the same. (8 warps
    // stay below 48 KB.)
    constexpr size_t kStatic = sizeof(int32_t) * (2 * 32 * WARPS + WARPS + 1) + 64, kMost = sizeof(int32_t) * WARPS * S_MAX_EXPERTS;
    static_assert(kStatic + kMost <= 227 * 1024, "an SM's shared memory");
    if (smem + kStatic > 48 * 1024)
        e = cudaFuncSetAttribute(expert_place_kernel<WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
    if (e != cudaSuccess) return e;
    if (grid > 1) GPTQ_LAUNCH(K_EXPERT_SORT, s, e = launch_pdl(expert_place_kernel<WARPS>, dim3(grid), dim3(32 * WARPS), smem, s, p));
    else GPTQ_LAUNCH(K_EXPERT_SORT, s, expert_place_kernel<WARPS><<<grid, 32 * WARPS, smem, s>>>(p));
    return e != cudaSuccess ? e : cudaGetLastError();
}

// ---------------------------------------------------------------------------- rows there and back
// Rows move in units of 16 bytes where pointers, strides and lengths allow, of 4 bytes or of one
// element otherwise; neighbouring threads take neighbouring units, and of the short ones several
// each, so that as many bytes are in flight (rows of 4095 bf16 took four times as long as rows of 4096
// with one element per thread). A CTA has as many threads as a row has work for, up to 256.
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

// Each row of x is read once and written `top` times, so the traffic is the least there is: 16384 x 2 x
// 4096 bf16, 403 MB, in 55 us (7.3 TB/s).
template <typename U, int UNITS>
__global__ void __launch_bounds__(R_THREADS) expert_gather_kernel(const RParams p, int64_t units, int chunks, int64_t main_ctas) {
    const U* X = static_cast<const U*>(p.X);
    U* Y = static_cast<U*>(p.Y);
    pdl_wait();
    if (blockIdx.x >= main_ctas) {   // the rows past the last live one
        const int64_t n = gridDim.x - main_ctas;
        const U zero = {};
        for (int64_t r = live_rows(p) + (blockIdx.x - main_ctas); r < p.slots; r += n)
            for (int64_t u = threadIdx.x; u < units; u += blockDim.x) Y[r * p.ldy + u] = zero;
        return;
    }
    const int64_t t = blockIdx.x / chunks;
    const int64_t u0 = (int64_t)(blockIdx.x % chunks) * (blockDim.x * UNITS) + threadIdx.x;
    U v[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
        if (u0 + i * blockDim.x < units) v[i] = X[t * p.ldx + u0 + i * blockDim.x];
    for (int j = 0; j < p.top; ++j) {
        const int64_t at = place(p, t * p.top + j);
        if (at < 0) continue;
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
            if (u0 + i * blockDim.x < units) Y[at * p.ldy + u0 + i * blockDim.x] = v[i];
    }
}

// a unit of N consecutive elements as fp32
template <typename T, int N>
__device__ __forceinline__ void load_row(const T* x, float (&v)[N]) {
    if constexpr (N == 1) {
        if constexpr (sizeof(T) == 2) v[0] = __bfloat162float(*x);
        else v[0] = *x;
    } else {
        uint32_t u[N * sizeof(T) / 4];
        if constexpr (N * sizeof(T) == 4) {
            u[0] = *reinterpret_cast<const uint32_t*>(x);
        } else {
            const uint4 w = *reinterpret_cast<const uint4*>(x);
            u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
        }
#pragma unroll
        for (int e = 0; e < (int)(N * sizeof(T) / 4); ++e) {
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
        uint32_t u[N * sizeof(T) / 4];
#pragma unroll
        for (int e = 0; e < (int)(N * sizeof(T) / 4); ++e) {
            if constexpr (sizeof(T) == 2) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                u[e] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                u[e] = __float_as_uint(v[e]);
            }
        }
        if constexpr (N * sizeof(T) == 4) *reinterpret_cast<uint32_t*>(y) = u[0];
        else *reinterpret_cast<uint4*>(y) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// The places of SLOTS of a token's slots from j0 on, 0 where there is none (a row that may be read, and
// is, so that all the rows' loads are in flight together), and which of them count.
template <int SLOTS>
__device__ __forceinline__ uint32_t places(const RParams& p, int64_t t, int j0, int64_t (&at)[SLOTS]) {
    uint32_t live = 0;
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
        const int64_t a = SLOTS == 1 || j0 + j < p.top ? place(p, t * p.top + j0 + j) : -1;
        live |= (a >= 0 ? 1u : 0u) << j;
        at[j] = max(a, (int64_t)0);
    }
    return live;
}

// A thread sums UNITS units of N columns of a token over its slots, SLOTS rows in flight. Bound by memory:
// 16384 x 2 x 4096 bf16, 403 MB, in 66 us (6.1 TB/s); with the rows one after another 76, with loads
// behind the test of their slot 128.
template <typename T, int N, int UNITS, int SLOTS>
__global__ void __launch_bounds__(R_THREADS) expert_combine_kernel(const RParams p, int chunks) {
    const int64_t t = blockIdx.x / chunks;
    const int64_t step = (int64_t)blockDim.x * N;
    const int64_t c = (int64_t)(blockIdx.x % chunks) * step * UNITS + threadIdx.x * N;
    if (c >= p.d) return;
    const T* X = static_cast<const T*>(p.X) + c;
    float acc[UNITS][N] = {};
    for (int j0 = 0; j0 < p.top; j0 += SLOTS) {
        int64_t at[SLOTS];
        float v[SLOTS][UNITS][N];
        const uint32_t live = places<SLOTS>(p, t, j0, at);
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
                if (UNITS == 1 || c + i * step < p.d) load_row<T, N>(X + at[j] * p.ldx + i * step, v[j][i]);
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const float w = p.w ? (live >> j & 1 ? p.w[t * p.top + j0 + j] : 0.0f) : 1.0f;
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
#pragma unroll
                for (int e = 0; e < N; ++e) acc[i][e] = live >> j & 1 ? fmaf(w, v[j][i][e], acc[i][e]) : acc[i][e];
        }
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
        if (UNITS == 1 || c + i * step < p.d) store_row<T, N>(static_cast<T*>(p.Y) + t * p.ldy + c + i * step, acc[i]);
}

// One CTA per token, SLOTS slots at a time: dy and the slots' rows are read once (dy again for each
// further group), the products of a group are summed across the CTA together. Bound by memory: 16384 x
// 2 x 4096 bf16, 671 MB, in 99 us (6.8 TB/s); slot by slot, with a sum across the CTA for each, 108.
template <typename T, int N, int UNITS, int SLOTS>
__global__ void __launch_bounds__(R_THREADS) expert_combine_grad_kernel(const RParams p) {
    const T* X = static_cast<const T*>(p.X);
    T* Y = static_cast<T*>(p.Y);
    const int64_t step = (int64_t)blockDim.x * N;
    if (blockIdx.x >= p.tokens) {
        const int64_t n = gridDim.x - p.tokens;
        float zero[N] = {};
        for (int64_t r = live_rows(p) + (blockIdx.x - p.tokens); r < p.slots; r += n)
            for (int64_t c = threadIdx.x * N; c < p.d; c += step) store_row<T, N>(Y + r * p.ldy + c, zero);
        return;
    }
    __shared__ float part[R_THREADS / 32][SLOTS];
    const int64_t t = blockIdx.x;
    const T* dy = static_cast<const T*>(p.dY) + t * p.lddy;
    for (int j0 = 0; j0 < p.top; j0 += SLOTS) {
        int64_t at[SLOTS];
        const uint32_t live = places<SLOTS>(p, t, j0, at);   // the same for the whole CTA
        float w[SLOTS], dot[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            w[j] = live >> j & 1 ? p.w[t * p.top + j0 + j] : 0.0f;
            dot[j] = 0.0f;
        }
        for (int64_t c = threadIdx.x * N; c < p.d; c += step * UNITS) {
            float a[UNITS][N], b[SLOTS][UNITS][N];
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
                if (UNITS == 1 || c + i * step < p.d) load_row<T, N>(dy + c + i * step, a[i]);
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
#pragma unroll
                for (int i = 0; i < UNITS; ++i)
                    if (UNITS == 1 || c + i * step < p.d) load_row<T, N>(X + at[j] * p.ldx + c + i * step, b[j][i]);
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
#pragma unroll
                for (int i = 0; i < UNITS; ++i) {
                    if (UNITS > 1 && c + i * step >= p.d) continue;
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        dot[j] = fmaf(a[i][e], b[j][i][e], dot[j]);
                        b[j][i][e] = a[i][e] * w[j];
                    }
                    if (live >> j & 1) store_row<T, N>(Y + at[j] * p.ldy + c + i * step, b[j][i]);
                }
        }
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < SLOTS && j0 + (int)threadIdx.x < p.top) {
            float sum = 0.0f;
            for (int i = 0; i < (int)blockDim.x / 32; ++i) sum += part[i][threadIdx.x];
            p.dw[t * p.top + j0 + threadIdx.x] = live >> threadIdx.x & 1 ? sum : 0.0f;
        }
        __syncthreads();
    }
}

// Calls f(T(), columns per unit, units per thread, slots per group), the last three as constants
template <typename F>
void with_row_types(int dtype, int unit_bytes, int64_t top, F f) {
    auto slots = [&](auto t, auto n, auto u) {
        if (top == 1) f(t, n, u, std::integral_constant<int, 1>());
        else if (top == 2) f(t, n, u, std::integral_constant<int, 2>());
        else f(t, n, u, std::integral_constant<int, 4>());
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 4> four;
    if (dtype == GPTQ_BF16) {
        if (unit_bytes == 16) slots(__nv_bfloat16(), std::integral_constant<int, 8>(), one);
        else if (unit_bytes == 4) slots(__nv_bfloat16(), std::integral_constant<int, 2>(), four);
        else slots(__nv_bfloat16(), one, four);
    } else {
        if (unit_bytes == 16) slots(float(), four, one);
        else slots(float(), one, four);
    }
}

// threads for rows of `units` units, several per thread
unsigned row_threads(int64_t units, int per) {
    const int64_t n = ceil_div(ceil_div(units, per), 32) * 32;
    return (unsigned)std::min<int64_t>(std::max<int64_t>(n, 32), R_THREADS);
}

bool bad_dtype(int t) { return t != GPTQ_F32 && t != GPTQ_BF16; }
// bytes of the units that all these rows of d elements can move in
struct Rows {
    const void* p;
    int64_t ld;
};
int unit_of(int64_t es, int64_t d, std::initializer_list<Rows> rows) {
    uint64_t all = (uint64_t)(d * es);
    for (const Rows& r : rows) all |= reinterpret_cast<uintptr_t>(r.p) | (uint64_t)(r.ld * es);
    return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : (int)es;
}
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
    if (need > 0 && reinterpret_cast<uintptr_t>(ws) % sizeof(int32_t) != 0) return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    SParams p{ids, tokens * top, sort_chunk(tokens * top), (int)experts, offsets, src, pos, static_cast<int32_t*>(ws), st.word};
    const unsigned grid = (unsigned)std::max<int64_t>(1, ceil_div(p.slots, p.chunk));
    if (grid > 1) {
        GPTQ_LAUNCH(K_EXPERT_SORT, s, expert_count_kernel<8><<<grid, 256, sizeof(int32_t) * 8 * experts, s>>>(p));
        GPTQ_LAUNCH_CHECK();
        GPTQ_CUDA_TRY(launch_place<8>(p, grid, s));
    } else if (p.slots <= 1024) {
        GPTQ_CUDA_TRY(launch_place<8>(p, grid, s));
    } else {
        GPTQ_CUDA_TRY(launch_place<32>(p, grid, s));
    }
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
    const int bytes = unit_of(es, d, {{X, ldx}, {Xs, lds}}), per = bytes == 16 ? 1 : bytes == 4 ? 4 : 8;
    const int64_t unit = bytes / es, units = d / unit;
    RParams p{X, ldx / unit, nullptr, 0, Xs, lds / unit, tokens, tokens * top, (int)top, d, pos, offsets + experts, nullptr, nullptr, st.word};
    const unsigned threads = row_threads(units, per);
    const int64_t chunks = ceil_div(units, threads * per), main_ctas = tokens * chunks;
    if (main_ctas > kMaxSlots) return GPTQ_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)(main_ctas + tail_ctas(p.slots));
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kern) {
        GPTQ_LAUNCH(K_EXPERT_GATHER, s, e = launch_pdl(kern, dim3(grid), dim3(threads), 0, s, p, units, (int)chunks, main_ctas));
    };
    if (bytes == 16) go(expert_gather_kernel<uint4, 1>);
    else if (bytes == 4) go(expert_gather_kernel<uint32_t, 4>);
    else go(expert_gather_kernel<uint16_t, 8>);
    GPTQ_CUDA_TRY(e);
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
    const int bytes = unit_of(es, d, {{Ys, ldys}, {Y, ldy}}), per = bytes == 16 ? 1 : 4;
    RParams p{Ys, ldys, nullptr, 0, Y, ldy, tokens, tokens * top, (int)top, d, pos, nullptr, weights, nullptr, st.word};
    const int64_t units = d / (bytes / es);
    const unsigned threads = row_threads(units, per);
    const int64_t chunks = ceil_div(units, threads * per);
    if (tokens * chunks > kMaxSlots) return GPTQ_ERR_UNSUPPORTED;
    with_row_types(dtype, bytes, top, [&](auto t, auto n, auto u, auto k) {
        auto kern = expert_combine_kernel<decltype(t), decltype(n)::value, decltype(u)::value, decltype(k)::value>;
        GPTQ_LAUNCH(K_EXPERT_COMBINE, s, kern<<<(unsigned)(tokens * chunks), threads, 0, s>>>(p, (int)chunks));
    });
    GPTQ_LAUNCH_CHECK();
    return st.finish(s);
}

extern "C" int gptq_expert_combine_grad(const void* dY, int64_t lddy, const void* Ys, int64_t ldys, int dtype, int64_t tokens,
                                        int64_t d, const int32_t* pos, int64_t top, const int32_t* offsets, int64_t experts,
                                        const float* weights, void* dYs, int64_t lddys, float* dW, void* stream) {
    if (bad_shape(tokens, top, d) || bad_dtype(dtype) || experts < 1) return GPTQ_ERR_INVALID_ARG;
    if (tokens == 0) return GPTQ_OK;
    if ((d > 0 && (!dY || !Ys || !dYs)) || !pos || !offsets || !weights || !dW || lddy < d || ldys < d || lddys < d)
        return GPTQ_ERR_INVALID_ARG;   // (rows of no columns are no memory; dW is 0)
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    const int64_t es = dtype == GPTQ_BF16 ? 2 : 4;
    const int bytes = unit_of(es, d, {{dY, lddy}, {Ys, ldys}, {dYs, lddys}});
    RParams p{Ys, ldys, dY, lddy, dYs, lddys, tokens, tokens * top, (int)top, d, pos, offsets + experts, weights, dW, st.word};
    const unsigned grid = (unsigned)(tokens + tail_ctas(p.slots)), threads = row_threads(d / (bytes / es), bytes == 16 ? 1 : 4);
    with_row_types(dtype, bytes, top, [&](auto t, auto n, auto u, auto k) {
        auto kern = expert_combine_grad_kernel<decltype(t), decltype(n)::value, decltype(u)::value, decltype(k)::value>;
        GPTQ_LAUNCH(K_EXPERT_GRAD, s, kern<<<grid, threads, 0, s>>>(p));
    });
    GPTQ_LAUNCH_CHECK();
    return st.finish(s);
}

// int8_matmul.cu — Y = X W^T for two matrices in the 8-bit integer form (int8.cuh), dense or with one
// weight per expert over rows sorted by expert:
//   Y[t][o] = act(sx[t] sw[e(t)][o] sum_k x[t][k] w[e(t)][o][k])
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "int8.cuh"
#include "pair.cuh"
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
    int ftiles;               // feature tiles
    int tokens_first;         // neighbouring tiles share their features, not their tokens
    int splits;               // SPLIT: shares of the columns, each a pair of its own
    int box, raw;             // SPLIT: rows of a token box, and stages of codes
    int relu, bf16_out, vec;  // vec: bf16 rows that 16-byte stores can take
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

// ------------------------------------------------------------------------ pairs of SMs, tcgen05
// There is no integer tensor instruction on sm_103a, but 8-bit integers are exact in fp16, their products and,
// below 2^24, the sums of them exact in fp32. So the codes stay 8 bits wide up to the SM and are
// expanded there to what tcgen05.mma kind::f16 multiplies. The weights are the M operand and are expanded into
// TMEM, the tokens the N operand and are expanded into shared memory, which spares the shared memory one of
// the two operands' writes and reads.
//
// Two CTAs on neighbouring SMs work on a tile of 256 features x up to 256 tokens: each brings and expands
// its own 128 features and half of the tokens, 128 columns at a time. Roles in each CTA (persistent, one per SM):
//   warp 0        producer: two TMA copies per stage, 128 x 128 codes of each operand (128-byte swizzle)
//   warp 1        in the even CTA: the MMAs (warps 2 and 3 help with the set-up)
//   warps 4..7    weights: shared memory -> fp16 -> TMEM, a row per lane
//   warps 8..15   tokens: shared memory -> fp16 -> shared memory (128-byte swizzle), a row per lane; two groups
//                 that take every other stage
//   warps 16..23  epilogue: TMEM -> registers -> Y; they take registers that the other warps give up
// TMEM: 256 columns of sums (tokens), then the expanded weights of W_SLOTS stages, 64 columns each.
//
// SPLIT: few tiles, so a cluster of up to 8 CTAs shares the columns of one tile, and its pairs' sums are added
// through each other's shared memory, each pair for its own part of the tokens. Such tiles are mostly narrow,
// bound by the weights and the time that one stage takes: more stages of codes are in flight, three groups of
// warps (4..15) expand the weights in turn, the tokens' warps (16..19) are as many groups as a stage's tokens
// leave free, and 4 warps (20..23) are the epilogue.
// Every mbarrier wait is bounded (GPTQ_ERR_TIMEOUT into the status word, then unwind: each CTA waits for its own
// copies, the even one for the MMAs, and all meet before any leaves).
constexpr int W_F = 128, W_PF = 2 * W_F;   // features per CTA and per tile
constexpr int W_T = 256;                   // most tokens per tile
constexpr int W_K = 128;                   // columns per stage
constexpr int W_RAW = 3, W_SLOTS = 3;      // stages of codes, and of expanded operands
constexpr int W_MOST_RAW = 8;              // the former where token boxes are small
constexpr int W_THREADS = 32 * 24;
constexpr int W_CODES = W_F * W_K;         // bytes of one operand's codes per stage
constexpr int W_WIDE = 2 * W_T / 2 * W_K;  // bytes of the expanded tokens per stage
constexpr uint32_t W_TMEM = 512, W_A0 = 256;
constexpr int W_TURN = 32 * 64;            // bytes of a warp's buffer: 32 tokens x 32 features of bf16
constexpr int W_RING = W_RAW * 2 * W_CODES + W_SLOTS * W_WIDE;
constexpr int W_BARS = 2 * W_MOST_RAW + 2 * W_SLOTS + 3;

struct WMaps {
    CUtensorMap w, x[3];   // tokens: boxes of 128, 64 and 32 rows
};

// Token tiles of rows [lo, hi), all of one width: a multiple of 32, so both CTAs have whole groups of 16
__device__ __forceinline__ int token_tiles(int lo, int hi) { return hi <= lo ? 0 : (hi - lo + W_T - 1) / W_T; }

struct WTile {
    int e, f0;        // expert, first feature
    int t0, n;        // first token, tokens (a multiple of 32, the last of which may be past hi)
    int hi;           // the end of the expert's tokens
};

// What finding a tile takes, in shared memory: token tiles before each expert, and each one's rows
struct WRows {
    int32_t* start;   // [experts + 1]
    int2* rows;       // [experts]
};

__device__ __forceinline__ WTile find_tile(const IParams& p, const WRows& w, uint32_t i) {
    WTile t;
    const uint32_t ttiles = (uint32_t)w.start[p.experts], by = p.tokens_first ? ttiles : (uint32_t)p.ftiles;
    const uint32_t major = i / by, minor = i - major * by;
    const int tt = (int)(p.tokens_first ? minor : major);
    t.f0 = (int)(p.tokens_first ? major : minor) * W_PF;
    int a = 0, b = p.experts;   // start[a] <= tt < start[b]
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (w.start[m] <= tt) a = m;
        else b = m;
    }
    t.e = a;
    const int first = w.start[a], tiles = w.start[a + 1] - first;
    const int2 r = w.rows[a];
    t.hi = r.y;
    const int width = ((int)((uint32_t)(r.y - r.x + tiles - 1) / (uint32_t)tiles) + 31) & ~31;
    t.t0 = r.x + (tt - first) * width;
    t.n = min(max(t.hi - t.t0 + 31, 32) & ~31, width);
    return t;
}

// four codes to four fp16 numbers: code + 128 in the low bits of 1024, less 1152
__device__ __forceinline__ void to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
    w ^= 0x80808080u;
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// a shared-memory address in another CTA of the cluster
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ void commit_to(uint32_t bar, uint32_t ctas) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)ctas)
        : "memory");
}

// D (+)= A B with A in TMEM, fp16, by both CTAs
__device__ __forceinline__ void umma_half(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::f16: [4,6) sums (1 = fp32) | [7,10), [10,13) operands (0 = fp16), both K-major |
// [17,23) N >> 3 | [24,29) M >> 4
__device__ __forceinline__ uint32_t half_idesc(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(W_PF >> 4) << 24); }

// 32 tokens of one feature to Y: the lanes of a warp hold consecutive features, so each token is one store of 64 or
// 128 consecutive bytes. sx: the tokens' scales
template <typename T>
__device__ __forceinline__ void store_tokens(T* y, int64_t ldy, const uint32_t (&v)[32], float sw, const float* sx, bool relu,
                                             int last) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        if (j < last) {
            const float x = scaled(__uint_as_float(v[j]), sw, sx[j]), z = relu ? relu_of(x) : x;
            if constexpr (sizeof(T) == 2) *y = __float2bfloat16_rn(z);
            else *y = z;
        }
        y += ldy;
    }
}

// half of tmem_ld_16x256b_x4
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// two sums times a feature's scale and their tokens' scales, as a pair of bf16
__device__ __forceinline__ uint32_t pair_bf16(uint32_t a, uint32_t b, float sw, float2 sx) {
    uint32_t r;
    asm("{\n\t.reg .b64 v, w, x;\n\t.reg .b32 lo, hi;\n\t"
        "mov.b64 v, {%1, %2};\n\tmov.b64 w, {%3, %3};\n\tmov.b64 x, {%4, %5};\n\t"
        "mul.rn.f32x2 v, v, w;\n\tmul.rn.f32x2 v, v, x;\n\t"
        "mov.b64 {lo, hi}, v;\n\tcvt.rn.bf16x2.f32 %0, hi, lo;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b), "r"(__float_as_uint(sw)), "r"(__float_as_uint(sx.x)), "r"(__float_as_uint(sx.y)));
    return r;
}
__device__ __forceinline__ uint32_t relu_bf16(uint32_t v) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0u));
    return r;
}

// 32 tokens x 32 features, packed for stmatrix (v[j][..]: tokens 8 j ..), to Y through the warp's 2 KB of shared
// memory: rows of 64 bytes, one per token, whose 16-byte pieces are permuted so that neither side has conflicts
__device__ __forceinline__ void turn_tokens(const IParams& p, const uint32_t (&v)[4][4], int tok, int hi, int f0, uint32_t buf) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int row = 8 * j + (lane & 7);
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                         buf + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4)),
                     "r"(v[j][0]), "r"(v[j][1]), "r"(v[j][2]), "r"(v[j][3])
                     : "memory");
    }
    __syncwarp();
    const int f = f0 + 8 * (lane & 3);
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.Y) + f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int row = 8 * j + (lane >> 2), r = tok + row;
        const uint4 w = lds128(buf + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
        if (f < p.N && r < hi) *reinterpret_cast<uint4*>(y + (int64_t)r * p.ldy) = w;
    }
    __syncwarp();
}

template <bool SPLIT>
__global__ void __launch_bounds__(W_THREADS, 1) int8_matmul_kernel(const __grid_constant__ WMaps m, const IParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + W_RING + 8 * W_TURN);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + W_BARS);
    float* token_scales = reinterpret_cast<float*>(tmem_slot + 2);              // [8][W_T / 2]
    WRows w;
    w.rows = reinterpret_cast<int2*>(token_scales + 4 * W_T);
    w.start = reinterpret_cast<int32_t*>(w.rows + p.experts);

    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = uniform(cluster_rank()), half = rank & 1u, even = rank & ~1u;
    const uint32_t sbase = smem_u32(smem), bar0 = smem_u32(bars);
    auto raw_full = [&](int s) { return bar0 + 8u * s; };                                      // copies landed
    auto raw_free = [&](int s) { return bar0 + 8u * (W_MOST_RAW + s); };                       // all have read them
    auto wide_full = [&](int s) { return bar0 + 8u * (2 * W_MOST_RAW + s); };                  // even CTA: both have expanded
    auto wide_free = [&](int s) { return bar0 + 8u * (2 * W_MOST_RAW + W_SLOTS + s); };        // the stage's MMAs are done
    const uint32_t tfull = bar0 + 8u * (2 * W_MOST_RAW + 2 * W_SLOTS), tfree = tfull + 8, drain_bar = tfull + 16;
    // warps that expand one stage's tokens, and the groups of them
    const int token_warps = SPLIT ? p.box / 32 : 4, token_groups = SPLIT ? 4 / token_warps : 2;
    // the expanded tokens first, then the stages of codes
    const int box_rows = SPLIT ? p.box : W_F, raws = SPLIT ? p.raw : W_RAW;
    const uint32_t wide_bytes = box_rows * 2 * W_K, raw_bytes = W_CODES + box_rows * W_K;
    const uint32_t rbase = sbase + W_SLOTS * wide_bytes;
    const int per_tile = SPLIT ? 2 * p.splits : 2;
    const uint32_t first = blockIdx.x / per_tile, step = gridDim.x / per_tile;
    // this pair's stages
    const int all = (p.K + W_K - 1) / W_K, share = (int)(rank >> 1);
    const int k0 = SPLIT ? all * share / p.splits : 0, k1 = SPLIT ? all * (share + 1) / p.splits : all;

    // (each in a warp of its own, side by side)
    if (warp == 2 && elect_one()) {
        for (int s = 0; s < raws; ++s) {
            mbar_init(raw_full(s), 1);
            mbar_init(raw_free(s), 4 + token_warps);
        }
        for (int s = 0; s < W_SLOTS; ++s) {
            mbar_init(wide_full(s), 2 * (4 + token_warps));
            mbar_init(wide_free(s), 1);
        }
        mbar_init(tfull, 1);
        mbar_init(tfree, 16);
        mbar_init(drain_bar, 1);
        fence_barrier_init();
    }
    if (warp == 3 && elect_one()) {
        tma_prefetch_desc(&m.w);
        tma_prefetch_desc(&m.x[0]);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(W_TMEM)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_wait();   // from here on memory that the kernel before writes or reads is touched
    if (warp == 0) {
        // token tiles before each expert
        int carry = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            int lo = 0, hi = 0;
            if (e0 + lane < p.experts) expert_rows(p, e0 + lane, &lo, &hi);
            const int n = token_tiles(lo, hi);
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (e0 + lane < p.experts) {
                w.start[e0 + lane] = carry + inc - n;
                w.rows[e0 + lane] = make_int2(lo, hi);
            }
            carry += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) w.start[p.experts] = carry;
    }
    tc_fence_before();
    __syncthreads();
    // all CTAs' barriers are ready before any signals another's (the producer signals only its own)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (warp != 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    const uint64_t limit = *static_cast<volatile unsigned long long*>(&g_pipeline_wait_limit_ns);
    bool ok = true;   // false: a wait gave up
    const uint32_t ntiles = uniform((uint32_t)w.start[p.experts] * (uint32_t)p.ftiles);

    // registers of 6 groups of 4 warps: the CTA starts with 6 x 80 a lane, and 40 + 3 x 64 + 2 x 120 is 472
    if (warp < 4) {
        if constexpr (!SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            // ------------------------------- producer -----------------------------------
            const bool leader = elect_one();
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_par = 0;
            for (uint32_t i = first; i < ntiles && ok; i += step) {
                const WTile t = find_tile(p, w, i);
                const int n = (int)uniform(t.n), e = (int)uniform(t.e);
                const int box = n > 128 ? 0 : n > 64 ? 1 : 2;   // (its rows are at most SPLIT's)
                const uint32_t bytes = W_CODES + (W_CODES >> box);
                const int wrow = e * p.N + (int)uniform(t.f0) + (int)half * W_F, xrow = (int)uniform(t.t0) + (int)half * (n >> 1);
                for (int k = k0; k < k1; ++k) {
                    ok = wait_all(raw_free(stage), phase ^ 1u, limit);
                    if (!ok) break;
                    if (leader) {
                        const uint32_t base = rbase + stage * raw_bytes, bar = raw_full(stage);
                        mbar_expect_tx(bar, bytes);
                        tma_load_2d(base, &m.w, bar, k * W_K, wrow);
                        tma_load_2d(base + W_CODES, &m.x[box], bar, k * W_K, xrow);
                    }
                    __syncwarp();
                    issued |= 1u << stage;
                    issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
                    if (++stage == raws) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (leader)
                for (int s = 0; s < raws; ++s)
                    if (issued & (1u << s)) drain(raw_full(s), (issued_par >> s) & 1u);
            __syncwarp();
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else if (warp == 1) {
            // --------------------------- MMA issuer (even CTA) --------------------------
            if (half == 0) {
                int slot = 0;
                uint32_t phase = 0, tile = 0;
                for (uint32_t i = first; i < ntiles && ok; i += step, ++tile) {
                    const WTile t = find_tile(p, w, i);
                    const uint32_t idesc = half_idesc((int)uniform(t.n));
                    ok = wait_all(tfree, (tile & 1u) ^ 1u, limit);
                    if (!ok) break;
                    tc_fence_after();
                    for (int k = k0; k < k1; ++k) {
                        ok = wait_all(wide_full(slot), phase, limit);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const int ksteps = (p.K - k * W_K + 15) / 16;
                            const uint32_t a = tmem + W_A0 + slot * (W_K / 2);
                            const uint64_t b = smem_desc(sbase + slot * wide_bytes, 16, 1024, kSwizzle128B);
    #pragma unroll
                            for (int j = 0; j < W_K / 16; ++j)
                                if (j < ksteps)
                                    umma_half(tmem, a + 8 * j, b + (j >> 2) * (wide_bytes / 2 / 16) + 2 * (j & 3), idesc, (k > k0 || j > 0) ? 1u : 0u);
                            commit_to(wide_free(slot), 3u << even);
                            if (k == k1 - 1) commit_to(tfull, 3u << even);
                        }
                        __syncwarp();
                        if (++slot == W_SLOTS) {
                            slot = 0;
                            phase ^= 1u;
                        }
                    }
                }
                if (elect_one()) {
                    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drain_bar) : "memory");
                    drain(drain_bar, 0);
                }
                __syncwarp();
            }
        }
    } else if (warp < (SPLIT ? 20 : 16)) {
        // -------------------------- expansion, a row per lane -----------------------
        if constexpr (!SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        const bool weights = warp < (SPLIT ? 16 : 8);
        const int member = warp - (weights ? 4 : SPLIT ? 16 : 8), size = weights ? 4 : token_warps;
        const int q = member % size, groups = weights ? (SPLIT ? 3 : 1) : token_groups;
        const int r = 32 * q + lane, x = r & 7;
        int stage = 0, slot = 0, turn = member / size;   // stages until this group's next one
        uint32_t rphase = 0, sphase = 0;
        for (uint32_t i = first; i < ntiles && ok; i += step) {
            const WTile t = find_tile(p, w, i);
            const bool live = weights || 64 * q < (int)uniform(t.n);
            for (int k = k0; k < k1; ++k) {
                if (turn == 0) {
                    ok = wait_all(raw_full(stage), rphase, limit);
                    if (!ok) break;
                    const uint32_t src = rbase + stage * raw_bytes + (weights ? 0 : W_CODES) + r * W_K;
                    const uint32_t dst = sbase + slot * wide_bytes + r * 128;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[32];
                        if (live) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const uint4 w = lds128(src + (((4 * h + c) ^ x) << 4));
                                to_half(w.x, v[8 * c], v[8 * c + 1]);
                                to_half(w.y, v[8 * c + 2], v[8 * c + 3]);
                                to_half(w.z, v[8 * c + 4], v[8 * c + 5]);
                                to_half(w.w, v[8 * c + 6], v[8 * c + 7]);
                            }
                        }
                        if (h == 0) {
                            ok = wait_all(wide_free(slot), sphase ^ 1u, limit);
                            if (!ok) break;
                            if (weights) tc_fence_after();
                        } else {
                            __syncwarp();
                            if (lane == 0) mbar_arrive(raw_free(stage));
                        }
                        if (weights) {
                            tmem_st_32x32b_x32(tmem + ((uint32_t)(32 * q) << 16) + W_A0 + slot * (W_K / 2) + 32 * h, v);
                        } else if (live) {
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                sts128(dst + h * (wide_bytes / 2) + ((c ^ x) << 4), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
                        }
                    }
                    if (!ok) break;
                    if (weights) {
                        tmem_st_wait();
                        tc_fence_before();
                    } else {
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    // (arrive_cluster's CTA scope: each SM's tensor core reads what its own CTA wrote, which the fence
                    // above has put before the arrival; .release.cluster held a warp up for 900 to 1500 cycles a stage)
                    if (lane == 0) arrive_cluster(in_cta(wide_full(slot), even));
                }
                turn = turn == 0 ? groups - 1 : turn - 1;
                if (++stage == raws) {
                    stage = 0;
                    rphase ^= 1u;
                }
                if (++slot == W_SLOTS) {
                    slot = 0;
                    sphase ^= 1u;
                }
            }
        }
    } else if constexpr (SPLIT) {
        // ---- the sums to this CTA's shared memory, [token][feature], which no copy or MMA uses any more
        if (first < ntiles) {   // (one tile per cluster)
            const WTile t = find_tile(p, w, first);
            ok = wait_all(tfull, 0, limit);
            tc_fence_after();
            if (ok) {
                const int q = warp & 3;
                for (int c = 0; c < t.n; c += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * q) << 16) + c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) reinterpret_cast<uint32_t*>(smem)[(c + j) * W_F + 32 * q + lane] = v[j];
                }
            }
        }
    } else {
        // ------------------------------- epilogue -----------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
        const int q = warp & 3;
        const int c0 = W_T / 2 * ((warp - 16) >> 2);   // its half of the columns
        const uint32_t sums = tmem + ((uint32_t)(32 * q) << 16) + c0;
        const uint32_t turn = sbase + W_RING + (warp - 16) * W_TURN;
        float* sx = token_scales + (warp - 16) * (W_T / 2);   // the scales of its tokens
        const bool relu = p.relu != 0;
        uint32_t tile = 0;
        for (uint32_t i = first; i < ntiles; i += step, ++tile) {
            const WTile t = find_tile(p, w, i);
            const int f0 = t.f0 + (int)half * W_F + 32 * q;
            const float* ws = p.ws + (int64_t)t.e * p.N;
            __syncwarp();
#pragma unroll
            for (int c = lane; c < W_T / 2; c += 32) sx[c] = t.t0 + c0 + c < t.hi ? p.xs[t.t0 + c0 + c] : 0.0f;
            __syncwarp();
            const float mine = ws[min(f0 + lane, p.N - 1)];
            // (an ordinary weight's scale first cannot overflow: below 2^96 times a sum below 2^31)
            const bool far = __any_sync(0xffffffffu, mine > 0x1p96f);
            ok = wait_all(tfull, tile & 1u, limit);
            if (!ok) break;
            tc_fence_after();
            if (p.vec && !far) {
                // packed before the buffer is free, stored after it
                uint32_t v[4][4][4];
                float sw[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) sw[g] = __shfl_sync(0xffffffffu, mine, 8 * g + (lane >> 2));
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c0 + 32 * c < t.n) {
#pragma unroll
                        for (int j = 0; j < 4; j += 2) {
                            uint32_t a[2][8];
                            tmem_ld_16x256b_x2(sums + 32 * c + 8 * j, a[0]);
                            tmem_ld_16x256b_x2(sums + (16u << 16) + 32 * c + 8 * j, a[1]);
                            tmem_ld_wait();
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const float2 s = *reinterpret_cast<const float2*>(sx + 32 * c + 8 * (j + u) + 2 * (lane & 3));
#pragma unroll
                                for (int g = 0; g < 4; ++g)
                                    v[c][j + u][g] = pair_bf16(a[g >> 1][4 * u + 2 * (g & 1)], a[g >> 1][4 * u + 2 * (g & 1) + 1], sw[g], s);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(in_cta(tfree, even));
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c0 + 32 * c < t.n) {
                        if (relu) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[c][j >> 2][j & 3] = relu_bf16(v[c][j >> 2][j & 3]);
                        }
                        turn_tokens(p, v[c], t.t0 + c0 + 32 * c, t.hi, f0, turn);
                    }
                }
            } else {
                const int f = f0 + lane;
                for (int c = 0; c < W_T / 2 && c0 + c < t.n; c += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(sums + c, v);
                    tmem_ld_wait();
                    const int tok = t.t0 + c0 + c;
                    const int64_t at = (int64_t)tok * p.ldy + f;
                    if (f >= p.N) continue;
                    if (p.bf16_out) store_tokens(static_cast<__nv_bfloat16*>(p.Y) + at, p.ldy, v, mine, sx + c, relu, t.hi - tok);
                    else store_tokens(static_cast<float*>(p.Y) + at, p.ldy, v, mine, sx + c, relu, t.hi - tok);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(in_cta(tfree, even));
            }
        }
    }

    if (!ok && lane == 0) set_status(p.status, GPTQ_ERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // no CTA leaves, or frees TMEM, while another may still use it
    if constexpr (SPLIT) {
        if (first < ntiles) {
            const WTile t = find_tile(p, w, first);
            const int a = t.n * share / p.splits, b = t.n * (share + 1) / p.splits;   // this pair's tokens
            const int f = t.f0 + (int)half * W_F + 4 * lane;   // four features per lane, a token per warp
            const uint32_t mine = sbase + 16 * lane;
            float sw[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) sw[g] = p.ws[(int64_t)t.e * p.N + min(f + g, p.N - 1)];
#pragma unroll 2
            for (int c = a + warp; c < min(b, t.hi - t.t0); c += W_THREADS / 32) {
                const float sx = p.xs[t.t0 + c];
                float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int j = 0; j < p.splits; ++j) {
                    const float4 u = ld_cluster(in_cta(mine + 4 * c * W_F, 2 * j + half));
                    s.x += u.x, s.y += u.y, s.z += u.z, s.w += u.w;
                }
                float v[4] = {scaled(s.x, sw[0], sx), scaled(s.y, sw[1], sx), scaled(s.z, sw[2], sx), scaled(s.w, sw[3], sx)};
                if (p.vec) {
                    if (f >= p.N) continue;
                    if (p.relu) {
#pragma unroll
                        for (int g = 0; g < 4; ++g) v[g] = relu_of(v[g]);
                    }
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.Y) + (int64_t)(t.t0 + c) * p.ldy + f) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                } else {
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        if (f + g < p.N) store_result(p, t.t0 + c, f + g, v[g]);
                }
            }
        }
        __syncthreads();
        cluster_sync();   // nor while another reads its sums
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(W_TMEM) : "memory");
    }
    if (p.offsets) zero_rest(p, blockIdx.x, gridDim.x);
}

bool code_map(CUtensorMap* m, const int8_t* codes, int64_t rows, int64_t cols, int box_rows) {
    auto enc = tma_encoder();
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)int8_pitch(cols)};
    cuuint32_t box[2] = {(cuuint32_t)W_K, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(codes), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool SPLIT>
cudaError_t configure(const IParams& p, unsigned ctas, cudaStream_t s, cudaLaunchConfig_t* cfg, cudaLaunchAttribute (&attr)[2]) {
    constexpr int kFixed = 1024 + W_RING + 8 * W_TURN + 8 * W_BARS + 8 + 16 * W_T;
    constexpr int kMost = kFixed + 12 * I_MAX_EXPERTS + 4;
    static_assert(kMost <= 227 * 1024, "an SM's shared memory");
    static_assert(W_T * W_F * 4 <= W_RING, "a split tile's sums take the place of the stages");
    *cfg = {};
    cfg->gridDim = dim3(ctas);
    cfg->blockDim = dim3(W_THREADS);
    cfg->dynamicSmemBytes = kFixed + 12 * p.experts + 4;
    cfg->stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * (SPLIT ? p.splits : 1);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = attr;
    cfg->numAttrs = 2;
    // the limit is the kernel's and not the call's: every thread's calls set it to the same number
    return cudaFuncSetAttribute(int8_matmul_kernel<SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
}

// How many clusters of 2 * splits CTAs the device holds at once (its GPCs are not all multiples of 8 SMs)
int clusters_at_once(int splits) {
    static std::atomic<int> known[16][2];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::atomic<int>* k = dev < 16 ? &known[dev][splits > 2] : nullptr;
    if (k && k->load(std::memory_order_relaxed)) return k->load(std::memory_order_relaxed);
    IParams p{};
    p.splits = splits;
    p.experts = I_MAX_EXPERTS;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (configure<true>(p, 2 * splits, nullptr, &cfg, attr) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, int8_matmul_kernel<true>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    if (k) k->store(n, std::memory_order_relaxed);
    return n;
}

template <bool SPLIT>
int launch_pairs(const WMaps& m, const IParams& p, int64_t most_tiles, cudaStream_t s) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    const unsigned ctas = SPLIT ? (unsigned)most_tiles * 2 * p.splits : 2 * (unsigned)std::min<int64_t>(most_tiles, device_sm_count() / 2);
    GPTQ_CUDA_TRY(configure<SPLIT>(p, ctas, s, &cfg, attr));
    cudaError_t e = cudaSuccess;
    GPTQ_LAUNCH(K_INT8_MM, s, e = cudaLaunchKernelEx(&cfg, int8_matmul_kernel<SPLIT>, m, p));
    GPTQ_CUDA_TRY(e);
    return GPTQ_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
constexpr int64_t kMaxDim = (1ll << 31) - 512;

bool few_rows_pay(int64_t T, int64_t N, int64_t K, int64_t experts) { return T <= 8 * experts; }

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
    // tile numbers have 31 bits (a Y beyond that is larger than the device)
    if ((ceil_div(T, W_T) + experts) * ceil_div(N, W_PF) > kMaxDim) return GPTQ_ERR_UNSUPPORTED;
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
    p.ftiles = (int)ceil_div(N, W_PF);
    p.tokens_first = experts * N > T ? 1 : 0;   // the larger operand is walked through once
    p.vec = p.bf16_out && N % 8 == 0 && ldy % 8 == 0 && aligned16(Y) ? 1 : 0;
    if (K == 0 || few_rows_pay(T, N, K, experts)) {
        cudaError_t e = cudaSuccess;
        const dim3 grid((unsigned)ceil_div(N, F_FEATURES), (unsigned)(experts + (offsets ? 1 : 0)));
        GPTQ_LAUNCH(K_INT8_MM, s, e = launch_pdl(int8_few_rows_kernel, grid, dim3(F_THREADS), 0, s, p));
        GPTQ_CUDA_TRY(e);
        return st.finish(s);
    }
    WMaps m;
    if (!code_map(&m.w, w_codes, experts * N, K, W_F)) return GPTQ_ERR_CUDA;
    for (int i = 0; i < 3; ++i)
        if (!code_map(&m.x[i], x_codes, T, K, W_F >> i)) return GPTQ_ERR_CUDA;
    // an expert's last tile may be partial
    const int64_t most = (ceil_div(T, W_T) + (offsets ? std::min(experts, T) : 0)) * p.ftiles;
    // few tiles: as many shares of the columns as the device holds at once, of four stages or more each
    p.splits = 1;
    for (int k = 4; k > 1 && p.splits == 1; k >>= 1)
        if (most * k <= device_sm_count() / 2 && ceil_div(K, W_K) >= 4 * k && most <= clusters_at_once(k)) p.splits = k;
    if (p.splits > 1) {
        const int64_t rows = offsets ? std::min<int64_t>(T, W_T) : ceil_div(T, ceil_div(T, W_T));   // of the widest tile
        p.box = rows <= 64 ? 32 : rows <= 128 ? 64 : 128;
        p.raw = std::min(W_MOST_RAW, (W_RING - W_SLOTS * p.box * 2 * W_K) / (W_CODES + p.box * W_K));
    }
    const int rc = p.splits > 1 ? launch_pairs<true>(m, p, most, s) : launch_pairs<false>(m, p, most, s);
    return rc != GPTQ_OK ? rc : st.finish(s);
}

namespace gptq {
// this file's copy of the pipeline-wait limit (the library's test hook sets every copy)
cudaError_t int8_set_wait_limit(unsigned long long ns) { return set_pipeline_wait_limit_this_unit(ns); }
}  // namespace gptq

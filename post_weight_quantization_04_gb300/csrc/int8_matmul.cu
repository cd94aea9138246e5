// int8_matmul.cu — Y = X W^T for two matrices in the 8-bit integer form (int8.cuh), dense or with one
// weight per expert over rows sorted by expert:
//   Y[t][o] = act(sx[t] sw[e(t)][o] sum_k x[t][k] w[e(t)][o][k])
// Few rows are the stream of the weights (mma.sync on codes expanded in registers), more are tcgen05 MMAs on codes expanded
// on their way to TMEM and shared memory. Sums are fp32: whole numbers, exact below 2^24.
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
// K products, each up to 2^14, sum to less than 2^31, which the packed epilogue relies on (weights' scales up to 2^96 times
// a sum stay within fp32). Sums are fp32 and rounded past 2^24, which takes more than 1024 products of the largest codes.
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
    int width;                // the widest tile: a multiple of 32 up to W_T
    int splits;               // SPLIT: shares of the columns, each a pair of its own
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
    const int64_t size = p.bf16_out ? 2 : 4;
    for (int r = cta; r < p.T - (last - first); r += ctas) {
        const int64_t row = r < first ? r : r + (last - first);
        char* y = static_cast<char*>(p.Y) + row * p.ldy * size;
        const int64_t bytes = p.N * size;
        if ((reinterpret_cast<uintptr_t>(y) & 15) == 0) {
            for (int64_t b = threadIdx.x * 16; b < (bytes & ~(int64_t)15); b += blockDim.x * 16)
                *reinterpret_cast<uint4*>(y + b) = make_uint4(0, 0, 0, 0);
            for (int64_t b = (bytes & ~(int64_t)15) + threadIdx.x * 2; b < bytes; b += blockDim.x * 2) *reinterpret_cast<uint16_t*>(y + b) = 0;
        } else {
            for (int64_t b = threadIdx.x * 2; b < bytes; b += blockDim.x * 2) *reinterpret_cast<uint16_t*>(y + b) = 0;
        }
    }
}

// four codes to four fp16 numbers: code + 128 in the low bits of 1024, less 1152
__device__ __forceinline__ void to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
    w ^= 0x80808080u;
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// ------------------------------------------------------------------------------- few rows
// With a handful of tokens the product is the stream of the weights, and what counts is to have all of it in
// flight at once. A CTA computes 16 features, its warps the columns in turn, 64 at a time: each thread loads 16 bytes
// of two features and of a token out of eight, expands them to fp16 in its registers and multiplies them with
// mma.sync (m16n8k16; any order of the columns will do if both operands have the same), 8 tokens at a time. No shared
// memory, barriers or TMEM lie between the loads and the products; the warps' sums are added at the end.
// While all CTAs run at once, what counts is one row's loads in flight: 8 warps with 8 steps each (4096 x 4096, one token: 5.7 us; 4
// steps 6.3). With more CTAs than that small ones that follow each other closely do better: 4 warps with 2 steps (8 experts of
// 14336 x 4096, 16 rows: 67 us, 7.0 TB/s; the others 81 and 90. 14336 x 4096, one token: 13.5 and 15.2).
constexpr int F_FEATURES = 16;

__device__ __forceinline__ void mma_half(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (Plain loads: this kernel starts while the one before may still be writing its operands, so they are not
// read-only for as long as it runs, which is what the read-only path asks for.)
// tokens t0 .. t0 + n - 1 (n <= 8 NT) of expert e times features f0 .. f0 + 15
// AHEAD: steps of 64 columns in flight
template <int NT, int WARPS, int AHEAD>
__device__ __forceinline__ void few_rows(const IParams& p, int e, int t0, int n, int f0, float* part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, col = 16 * (lane & 3);
    const int8_t* wc = p.wc + (int64_t)e * p.N * p.pitch + col;
    const int8_t* w0 = wc + min(f0 + g, p.N - 1) * p.pitch;
    const int8_t* w1 = wc + min(f0 + g + 8, p.N - 1) * p.pitch;
    const int8_t* x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j] = p.xc + (t0 + min(8 * j + g, n - 1)) * p.pitch + col;
    float acc[NT][4] = {};
    for (int64_t c0 = warp * 64; c0 < p.pitch; c0 += AHEAD * WARPS * 64) {
        uint4 a[AHEAD][2], b[AHEAD][NT];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int64_t c = c0 + u * WARPS * 64;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const bool in = c + col < p.pitch;
            a[u][0] = in ? *reinterpret_cast<const uint4*>(w0 + c) : zero;
            a[u][1] = in ? *reinterpret_cast<const uint4*>(w1 + c) : zero;
#pragma unroll
            for (int j = 0; j < NT; ++j) b[u][j] = in ? *reinterpret_cast<const uint4*>(x[j] + c) : zero;
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const uint32_t r0[4] = {a[u][0].x, a[u][0].y, a[u][0].z, a[u][0].w}, r1[4] = {a[u][1].x, a[u][1].y, a[u][1].z, a[u][1].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t lo0, hi0, lo1, hi1;
                to_half(r0[q], lo0, hi0);
                to_half(r1[q], lo1, hi1);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    uint32_t lo, hi;
                    to_half(q == 0 ? b[u][j].x : q == 1 ? b[u][j].y : q == 2 ? b[u][j].z : b[u][j].w, lo, hi);
                    mma_half(acc[j], lo0, lo1, hi0, hi1, lo, hi);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)   // feature g (+ 8), token 8 j + 2 (lane % 4) (+ 1)
            part[(warp * 8 * NT + 8 * j + 2 * (lane & 3) + (i & 1)) * F_FEATURES + g + 8 * (i >> 1)] = acc[j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < F_FEATURES * n; i += 32 * WARPS) {
        const int t = t0 + i / F_FEATURES, f = f0 + i % F_FEATURES;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < WARPS; ++k) v += part[k * 8 * NT * F_FEATURES + i];
        if (f < p.N) store_result(p, t, f, scaled(v, p.xs[t], p.ws[(int64_t)e * p.N + f]));
    }
    __syncthreads();
}

// MOST: groups of 8 tokens at a time; with fewer, more CTAs fit an SM. CTAS: of an SM, by registers
template <int MOST, int WARPS, int AHEAD, int CTAS>
__global__ void __launch_bounds__(32 * WARPS, CTAS) int8_few_rows_kernel(const IParams p) {
    __shared__ float part[WARPS][F_FEATURES * 8 * MOST];
    const int e = blockIdx.y, f0 = blockIdx.x * F_FEATURES;
    pdl_trigger();
    pdl_wait();
    if (e == p.experts) {   // (only with offsets)
        zero_rest(p, blockIdx.x, gridDim.x);
        return;
    }
    int lo, hi;
    expert_rows(p, e, &lo, &hi);
    for (int t = lo; t < hi; t += 8 * MOST) {
        const int n = min(hi - t, 8 * MOST);
        if (MOST >= 4 && n > 16) few_rows<MOST >= 4 ? 4 : 1, WARPS, AHEAD>(p, e, t, n, f0, part[0]);
        else if (MOST >= 2 && n > 8) few_rows<MOST >= 2 ? 2 : 1, WARPS, AHEAD>(p, e, t, n, f0, part[0]);
        else few_rows<1, WARPS, AHEAD>(p, e, t, n, f0, part[0]);
    }
}

// ------------------------------------------------------------------------ pairs of SMs, tcgen05
// tcgen05.mma has no integer kind on sm_103a, and mma.sync on 8-bit integers runs at a quarter of its rate on fp16. But 8-bit
// integers are exact in fp16, their products and, below 2^24, the sums of them exact in fp32. So the codes stay 8 bits wide up to the SM and are
// expanded there to what tcgen05.mma kind::f16 multiplies. The weights are the M operand and are expanded into
// TMEM, the tokens the N operand and are expanded into shared memory, which spares the shared memory one of
// the two operands' writes and reads.
//
// Two CTAs on neighbouring SMs work on a tile of 256 features x up to 256 tokens: each brings and expands
// its own 128 features and half of the tokens, 128 columns at a time. Roles in each CTA (persistent, one per SM):
//   warp 0        producer: two TMA copies per stage, 128 x 128 codes of each operand (128-byte swizzle)
//   warp 1        in the even CTA: the MMAs (warps 2 and 3 help with the set-up)
//   warps 4..11   weights: shared memory -> fp16 -> TMEM, half a row per lane
//   8 (BOX = 32: 4) warps  tokens: shared memory -> fp16 -> shared memory (128-byte swizzle), half or a quarter of a row per lane
//   8 warps       epilogue: TMEM -> registers -> Y; they take registers that the other warps give up
// All the warps that expand take part in every stage: groups that take stages in turn can be two phases of a barrier
// behind, which its parity does not tell from none.
// TMEM: 256 columns of sums (tokens), then the expanded weights of W_SLOTS stages, 64 columns each.
//
// BOX: the tokens that a CTA brings of a tile, 128, 64 or 32. Narrow tiles leave room for more stages of codes (w_raws), and what
// their tokens take is smaller: a stage of a tile of 64, 128, 256 tokens takes 680, 800, 1060 cycles. (The box was a variable
// once: 128 tokens then took 950, 256 of a split tile 1310.)
//
// SPLIT: few tiles, so a cluster of up to 4 pairs shares the columns of one tile, and its pairs' sums are added
// through each other's shared memory, each pair for its own part of the tokens, by all warps.
//
// What bounds it: with 256 tokens the MMAs, 128 cycles for 16 columns, so that a stage cannot take less than 1024; it takes 1030 to
// 1080. With fewer the expansion of the weights. 8192 x 8192 x 8192 545 us, 2.02 PFLOP/s, with the tensor pipe
// busy 89 % of the launch (a bf16 library product of that size takes 546 to 560); 16384 x 4096 x 14336 963 to
// 1040 us from one card to the next, by the clock that the power limit leaves. Small products are the launch, the first stage's way through all
// of it (3.5 us), 12 to 17 us for each round of 32 stages, and the last tile's stores (2.6 us).
// Taken back: expanding warps in groups that take stages in turn (no faster once all follow the barriers); two expanded
// stages and four of codes (10 % slower); codes let go before there is room for them (7 % slower); copies of later stages
// into L2 ahead (no faster); the arrivals at a stage's two barriers in one place (4 % slower).
// Every mbarrier wait is bounded (GPTQ_ERR_TIMEOUT into the status word, then unwind: each CTA waits for its own
// copies, the even one for the MMAs, and all meet before any leaves).
constexpr int W_F = 128, W_PF = 2 * W_F;   // features per CTA and per tile
constexpr int W_T = 256;                   // most tokens per tile
constexpr int W_K = 128;                   // columns per stage
constexpr int W_RAW = 3, W_SLOTS = 3;      // stages of codes, and of expanded operands
constexpr int W_MOST_RAW = 8;              // the former where token boxes are small
// warps that expand (8 + 8, or 8 + 4 where the tokens are 32 rows of four pieces), threads (whole groups of 4 warps: see the
// end), and below stages of codes
constexpr int w_expand(int box) { return box == 32 ? 12 : 16; }
constexpr int w_threads(int box, bool split) { return 32 * (w_expand(box) + (split ? 8 : 12)); }
constexpr int W_CODES = W_F * W_K;         // bytes of one operand's codes per stage
constexpr int W_WIDE = 2 * W_T / 2 * W_K;  // bytes of the expanded tokens per stage
constexpr uint32_t W_TMEM = 512, W_A0 = 256;
constexpr int W_TURN = 32 * 64;            // bytes of a warp's buffer: 32 tokens x 32 features of bf16
constexpr int W_RING = W_RAW * 2 * W_CODES + W_SLOTS * W_WIDE;
// A split tile's sums from its cluster's other pairs (three quarters of its tokens at most) have their own shared memory where
// there is room, which spares a meeting of the cluster (64 x 4096 x 4096 12.0 -> 11.1 us), and else the stages'. SPLIT has no
// use for the warps' buffers of the epilogue behind the stages.
constexpr int w_apart(int box, bool split) { return split && box < W_F ? 2 * box * 3 / 4 * W_F * 4 : 0; }
constexpr int w_room(bool split) { return W_RING + (split ? 8 * W_TURN : 0); }
constexpr int w_raws(int box, bool split) {
    return std::min(W_MOST_RAW, (w_room(split) - w_apart(box, split) - W_SLOTS * box * 2 * W_K) / (W_CODES + box * W_K));
}
constexpr int W_BARS = 2 * W_MOST_RAW + 2 * W_SLOTS + 3;

struct WMaps {
    CUtensorMap w, x[3];   // tokens: boxes of 128, 64 and 32 rows, those that the width of the tiles can need
};
__host__ __device__ __forceinline__ int first_box(int tokens) { return tokens > 128 ? 0 : tokens > 64 ? 1 : 2; }

// Token tiles of rows [lo, hi), all of one width: a multiple of 32, as an MMA of two CTAs wants it
__device__ __forceinline__ int token_tiles(int lo, int hi, int width) { return hi <= lo ? 0 : (hi - lo + width - 1) / width; }

struct WTile {
    int e, f0;        // expert, first feature
    int t0, n;        // first token, tokens (a multiple of 32, the last of which may be past hi)
    int hi;           // the end of its tokens, and of the expert's
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
    t.n = min((t.hi - t.t0 + 31) & ~31, width);
    t.hi = min(t.hi, t.t0 + t.n);
    return t;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void to_half8(const uint4& c, uint32_t* v) {
    to_half(c.x, v[0], v[1]);
    to_half(c.y, v[2], v[3]);
    to_half(c.z, v[4], v[5]);
    to_half(c.w, v[6], v[7]);
}

// N pieces of 32 columns of a row (x: its number modulo 8) of codes in the 128-byte swizzle, from piece `at` on
template <int N>
__device__ __forceinline__ void load_codes(uint32_t row, int at, int x, uint4 (&code)[2 * N]) {
#pragma unroll
    for (int c = 0; c < 2 * N; ++c) code[c] = lds128(row + (((2 * at + c) ^ x) << 4));
}

// the same pieces as fp16, in slabs of 64 columns
template <int N>
__device__ __forceinline__ void store_wide(uint32_t row, uint32_t slab, int at, int x, const uint4 (&code)[2 * N]) {
#pragma unroll
    for (int c = 0; c < 2 * N; ++c) {
        uint32_t v[8];
        to_half8(code[c], v);
        const int to = 4 * at + 2 * c;
        sts128(row + (to >> 3) * slab + (((to & 7) ^ x) << 4), v[0], v[1], v[2], v[3]);
        sts128(row + (to >> 3) * slab + (((to & 7) ^ x ^ 1) << 4), v[4], v[5], v[6], v[7]);
    }
}

// thread t writes lane (base + t), columns c..c+15
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
        "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// a shared-memory address in another CTA of the cluster
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
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

template <int BOX, bool SPLIT>
__global__ void __launch_bounds__(w_threads(BOX, SPLIT), 1) int8_matmul_kernel(const __grid_constant__ WMaps m, const IParams p) {
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
    // the expanded tokens first, then the stages of codes
    constexpr int raws = w_raws(BOX, SPLIT), epilogue = 4 + w_expand(BOX);   // (its first warp)
    constexpr uint32_t wide_bytes = BOX * 2 * W_K, raw_bytes = W_CODES + BOX * W_K;
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
            mbar_init(raw_free(s), w_expand(BOX));
        }
        for (int s = 0; s < W_SLOTS; ++s) {
            mbar_init(wide_full(s), 2 * w_expand(BOX));
            mbar_init(wide_free(s), 1);
        }
        mbar_init(tfull, 1);
        mbar_init(tfree, 16);
        mbar_init(drain_bar, 1);
        fence_barrier_init();
    }
    if (warp == 3 && elect_one()) {
        tma_prefetch_desc(&m.w);
        tma_prefetch_desc(&m.x[first_box(2 * BOX)]);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(W_TMEM)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_trigger();   // (the next kernel's CTAs find no room before this one's leave)
    pdl_wait();   // from here on memory that the kernel before writes or reads is touched
    if (warp == 0) {
        // token tiles before each expert
        int carry = 0, end = 0;   // the tiles, and the end of the rows, of the experts before
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            int lo = 0x7FFFFFFF, hi = lo;
            if (e0 + lane < p.experts) expert_rows(p, e0 + lane, &lo, &hi);
            // Offsets out of order (reported above): a row counts for the first expert that has it, so that there are no more
            // tiles than the host has counted. A split tile's cluster takes no second one: its MMAs would wait for the first
            // one's sums to be read until the wait gives up.
            const int up = __shfl_up_sync(0xffffffffu, hi, 1), before = lane ? up : end;
            if (__any_sync(0xffffffffu, lo < before)) {
                int most = before;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) most = max(most, __shfl_up_sync(0xffffffffu, most, o));
                lo = max(lo, most);
                hi = max(hi, lo);
            }
            end = __shfl_sync(0xffffffffu, hi, 31);
            const int n = token_tiles(lo, hi, p.width);
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

    // registers of 7 groups of 4 warps: the CTA starts with 7 x 72 a lane, and so is 40 + 4 x 56 + 2 x 120
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
                const int box = first_box(n);   // (its rows are at most BOX)
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
        } else if (SPLIT && warp >= 2) {
            // the scales, for the end
            if (first < ntiles) {
                const WTile t = find_tile(p, w, first);
                if (warp == 2)
                    for (int c = lane; c < t.n; c += 32) token_scales[c] = t.t0 + c < t.hi ? p.xs[t.t0 + c] : 0.0f;
                else
                    for (int c = lane; c < W_F; c += 32)
                        token_scales[W_T + c] = p.ws[(int64_t)t.e * p.N + min(t.f0 + (int)half * W_F + c, p.N - 1)];
            }
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
    } else if (warp < 4 + w_expand(BOX)) {
        // ------------- expansion: a row per lane, some of the stage's four pieces of 32 columns -------------
        if constexpr (!SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const bool weights = warp < 12;
        const int member = warp - (weights ? 4 : 12), row_warps = weights ? 4 : BOX / 32;
        const int q = member % row_warps, r = 32 * q + lane;
        // (fewer than 128 rows of tokens: one piece of them for each warp)
        const int pieces = row_warps == 4 ? 2 : 1, first_piece = member / row_warps * pieces;
        const uint32_t column = tmem + ((uint32_t)(32 * q) << 16) + W_A0 + 16 * first_piece;
        const uint32_t wide_remote = in_cta(wide_full(0), even);   // (mapa in the loop cost 5 %)
        int stage = 0, slot = 0;
        uint32_t rphase = 0, sphase = 0;
        for (uint32_t i = first; i < ntiles && ok; i += step) {
            const WTile t = find_tile(p, w, i);
            const bool live = 64 * q < (int)uniform(t.n);
            for (int k = k0; k < k1; ++k) {
                ok = wait_all(raw_full(stage), rphase, limit);
                if (!ok) break;
                const uint32_t src = rbase + stage * raw_bytes + (weights ? 0 : W_CODES) + r * W_K;
                const uint32_t dst = sbase + slot * wide_bytes + r * 128;
                auto freed = [&] { return ok = wait_all(wide_free(slot), sphase ^ 1u, limit); };
                // (only once what depends on the codes has been issued: the copy that follows this arrival has overtaken
                // loads whose values nothing had asked for yet)
                auto taken = [&] {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(raw_free(stage));
                };
                if (weights) {
                    uint4 code[4];
                    load_codes<2>(src, first_piece, r & 7, code);
                    if (!freed()) break;
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[16];
#pragma unroll
                        for (int c = 0; c < 2; ++c) to_half8(code[2 * h + c], &v[8 * c]);
                        tmem_st_32x32b_x16(column + slot * (W_K / 2) + 16 * h, v);
                    }
                    taken();
                    tmem_st_wait();
                    tc_fence_before();
                } else {
                    if constexpr (BOX < 128) {
                        uint4 code[2];
                        if (live) load_codes<1>(src, first_piece, r & 7, code);
                        if (!freed()) break;
                        if (live) store_wide<1>(dst, wide_bytes / 2, first_piece, r & 7, code);
                        taken();
                    } else {
                        uint4 code[4];
                        if (live) load_codes<2>(src, first_piece, r & 7, code);
                        if (!freed()) break;
                        if (live) store_wide<2>(dst, wide_bytes / 2, first_piece, r & 7, code);
                        taken();
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                // (arrive_cluster's CTA scope: each SM's tensor core reads what its own CTA wrote, which the fence
                // above has put before the arrival; .release.cluster held a warp up for 900 to 1500 cycles a stage)
                if (lane == 0) arrive_cluster(wide_remote + 8u * slot);
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
        if (first < ntiles) ok = wait_all(tfull, 0, limit);   // (one tile per cluster)
    } else {
        // ------------------------------- epilogue -----------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
        const int q = warp & 3;
        const int c0 = W_T / 2 * ((warp - epilogue) >> 2);   // its half of the columns
        const uint32_t sums = tmem + ((uint32_t)(32 * q) << 16) + c0;
        const uint32_t turn = sbase + W_RING + (warp - epilogue) * W_TURN;
        float* sx = token_scales + (warp - epilogue) * (W_T / 2);   // the scales of its tokens
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
                // packed before the buffer is free, stored after it; a last tile, that nobody waits for, as it is packed
                const bool final = i + step >= ntiles;
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
                                for (int g = 0; g < 4; ++g) {
                                    const uint32_t y = pair_bf16(a[g >> 1][4 * u + 2 * (g & 1)], a[g >> 1][4 * u + 2 * (g & 1) + 1], sw[g], s);
                                    v[c][j + u][g] = relu ? relu_bf16(y) : y;
                                }
                            }
                        }
                        if (final) turn_tokens(p, v[c], t.t0 + c0 + 32 * c, t.hi, f0, turn);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(in_cta(tfree, even));
                if (!final) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c0 + 32 * c < t.n) turn_tokens(p, v[c], t.t0 + c0 + 32 * c, t.hi, f0, turn);
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
    constexpr bool APART = w_apart(BOX, SPLIT) > 0;
    if (!APART) cluster_sync();   // no CTA leaves, or frees TMEM, while another may still use it
    if constexpr (SPLIT) {
        // No copy or MMA uses the memory that the sums go to (any more). Each pair sends the others their parts of its sums and
        // adds what it got to its own; all warps take part, each in its quarter of the lanes. ([source][token / 4][feature][4])
        tc_fence_after();
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const int feature = 32 * (warp & 3) + lane, mover = warp >> 2;
        const uint32_t sums = sbase + (APART ? w_room(SPLIT) - w_apart(BOX, SPLIT) : 0);
        const WTile t = first < ntiles ? find_tile(p, w, first) : WTile{0, 0, 0, 0, 0};
        // each pair's tokens, whole fours (n is a multiple of 32); the last ones may have fewer or none
        const int own = (t.n / 4 + p.splits - 1) / p.splits * 4, blocks = (own + 31) / 32;
        auto part_of = [&](int s) { return min(max(t.n - s * own, 0), own); };
        for (int b = mover; b < blocks * (p.splits - 1); b += w_threads(BOX, SPLIT) / 128) {
            const int other = b / blocks, to = other < share ? other : other + 1, c = b % blocks * 32;
            const int theirs = part_of(to);
            const uint32_t dst = in_cta(sums, 2 * to + half) + (uint32_t)((share < to ? share : share - 1) * own + c) * (W_F * 4) + feature * 16;
            uint32_t v[32];
            tmem_ld_32x32b_x32(lanes + to * own + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (c + 4 * u < theirs)
                    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + u * (W_F * 16)), "r"(v[4 * u]),
                                 "r"(v[4 * u + 1]), "r"(v[4 * u + 2]), "r"(v[4 * u + 3])
                                 : "memory");
        }
        cluster_sync();   // all have what they wait for, nobody's shared memory is touched any more, nor TMEM by another's MMAs
        const int mine = part_of(share);
        for (int b = mover; b < (mine + 31) / 32; b += w_threads(BOX, SPLIT) / 128) {
            const int c = 32 * b, tok = share * own + c;
            uint32_t v[32];
            tmem_ld_32x32b_x32(lanes + tok, v);
            tmem_ld_wait();
            for (int j = 0; j < p.splits - 1; ++j) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    if (c + 4 * u >= mine) break;
                    const uint4 a = lds128(sums + (uint32_t)(j * own + c + 4 * u) * (W_F * 4) + feature * 16);
                    v[4 * u] = __float_as_uint(__uint_as_float(v[4 * u]) + __uint_as_float(a.x));
                    v[4 * u + 1] = __float_as_uint(__uint_as_float(v[4 * u + 1]) + __uint_as_float(a.y));
                    v[4 * u + 2] = __float_as_uint(__uint_as_float(v[4 * u + 2]) + __uint_as_float(a.z));
                    v[4 * u + 3] = __float_as_uint(__uint_as_float(v[4 * u + 3]) + __uint_as_float(a.w));
                }
            }
            const int f = t.f0 + (int)half * W_F + feature, last = min(t.hi - t.t0, share * own + own) - tok;
            if (f < p.N) {
                const int64_t at = (int64_t)(t.t0 + tok) * p.ldy + f;
                const float sw = token_scales[W_T + feature];
                if (p.bf16_out) store_tokens(static_cast<__nv_bfloat16*>(p.Y) + at, p.ldy, v, sw, token_scales + tok, p.relu != 0, last);
                else store_tokens(static_cast<float*>(p.Y) + at, p.ldy, v, sw, token_scales + tok, p.relu != 0, last);
            }
        }
        tc_fence_before();
        __syncthreads();
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

template <int BOX, bool SPLIT>
cudaError_t configure(const IParams& p, unsigned ctas, cudaStream_t s, cudaLaunchConfig_t* cfg, cudaLaunchAttribute (&attr)[2]) {
    constexpr int kFixed = 1024 + W_RING + 8 * W_TURN + 8 * W_BARS + 8 + 16 * W_T;
    constexpr int kMost = kFixed + 12 * I_MAX_EXPERTS + 4;
    static_assert(kMost <= 227 * 1024, "an SM's shared memory");
    static_assert(W_T * W_F * 4 <= W_RING, "a split tile's sums take the place of the stages");
    *cfg = {};
    cfg->gridDim = dim3(ctas);
    cfg->blockDim = dim3(w_threads(BOX, SPLIT));
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
    return cudaFuncSetAttribute(int8_matmul_kernel<BOX, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
}

// How many clusters of 2 * splits CTAs the device holds at once (its GPCs are not all multiples of 8 SMs)
int clusters_at_once(int splits) {
    static std::atomic<int> known[16][5];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::atomic<int>* k = dev < 16 ? &known[dev][splits] : nullptr;
    if (k && k->load(std::memory_order_relaxed)) return k->load(std::memory_order_relaxed);
    IParams p{};
    p.splits = splits;
    p.experts = I_MAX_EXPERTS;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (configure<128, true>(p, 2 * splits, nullptr, &cfg, attr) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, int8_matmul_kernel<128, true>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    if (k) k->store(n, std::memory_order_relaxed);
    return n;
}

template <int BOX, bool SPLIT>
int launch_pairs(const WMaps& m, const IParams& p, int64_t most_tiles, cudaStream_t s) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    const unsigned ctas = SPLIT ? (unsigned)most_tiles * 2 * p.splits : 2 * (unsigned)std::min<int64_t>(most_tiles, device_sm_count() / 2);
    cudaError_t e = configure<BOX, SPLIT>(p, ctas, s, &cfg, attr);
    GPTQ_CUDA_TRY(e);
    GPTQ_LAUNCH(K_INT8_MM, s, e = cudaLaunchKernelEx(&cfg, int8_matmul_kernel<BOX, SPLIT>, m, p));
    GPTQ_CUDA_TRY(e);
    return GPTQ_OK;
}

struct Plan {
    int width, splits;
};
// The width of token tiles, and in how many shares the columns are split: what takes the fewest cycles by what was measured.
// In cycles: a stage takes 560 and 2 for each token of the width, a round of tiles 1700 more, a launch 5800 and 20 for each token;
// where the columns are split a launch and the sums' exchange take 8100 (256 tokens: 9500) and 28 (two shares) or 40 for each token. With experts
// their rows are not known here: the width is the one for evenly spread ones with room for half as many again or so, and an expert
// with more rows has several tiles. *most: the most tiles.
// Features x columns 4096 x 4096, us: 512 tokens as 256 x 2 shares 18.8, as 256 and 128 in whole 25.1 and 20.3; 256 tokens as 128 x 2
// 14.8, as 64 in whole 17.0, as 256 x 3 17.1; 64 tokens as 64 x 3 12.0, as 64 x 2 13.0. (These and the
// constants are from before narrow split tiles had memory apart for their sums: 64 x 3 takes 11.1 to 11.6 now, so the fixed part of split tiles
// up to 128 wide is counted 0.4 to 0.9 us too high.) 8 experts of 14336 x 4096, 200 rows in tiles
// of 64, 128, 256: 82, 85, 107; 320 rows 84, 86, 109; 500 rows 116, 92, 114; 700 rows 153, 96, 116; 1000 rows 171, 129, 120.
Plan plan_of(int64_t T, int64_t N, int64_t K, bool by_expert, int64_t experts, int64_t pairs, int64_t* most) {
    const int64_t ftiles = ceil_div(N, W_PF), stages = ceil_div(K, W_K);
    Plan best = {W_T, 1};
    int64_t least = -1;
    const int64_t fewest = ceil_div(T, W_T);
    for (int64_t tt = fewest;; ++tt) {
        const int width = by_expert ? (T <= 32 * experts ? 64 : T <= 96 * experts ? 128 : W_T) : (int)(ceil_div(ceil_div(T, tt), 32) * 32);
        const int64_t tiles = (ceil_div(T, width) + (by_expert ? std::min(experts, T) : 0)) * ftiles;
        for (int k = 1; k <= 4; ++k) {
            if (k > 1 && (tiles * k > pairs || stages < 2 * k || tiles > clusters_at_once(k))) break;
            const int64_t stage = 560 + 2 * width;
            const int64_t cycles = k > 1 ? ceil_div(stages, k) * stage + (width > 128 ? 9500 : 8100) + (k == 2 ? 28 : 40) * width
                                         : ceil_div(tiles, pairs) * (stages * stage + 1700) + 5800 + 20 * width;
            if (least < 0 || cycles < least) {
                least = cycles;
                best = {width, k};
                *most = tiles;
            }
        }
        // (in several rounds only somewhat narrower tiles pay, and in many rounds none)
        if (by_expert || width == 32 || (tiles > pairs && (tt > fewest + fewest / 2 || fewest > 64))) return best;
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
constexpr int64_t kMaxDim = (1ll << 31) - 512;

// Whether the kernel for few rows is the faster one. Measured (us, few rows / pairs; weights from memory, features x
// columns):
//                   1 token     16 tokens    32 tokens    64 tokens
//    4096 x 4096    5.7 / 11.0   7.1 / 11.4   9.0 / 11.1  15.2 / 11.1
//   14336 x 4096   13.7 / 18.0  18.6 / 18.0  25.8 / 18.1  43.5 / 18.9
//    4096 x 14336  14.5 / 21.2  17.7 / 21.3  25.2 / 21.4  44.6 / 22.1
//    1024 x 4096    4.2 /  8.1   5.7 /  9.2   7.0 /  8.7  13.4 /  8.7
//    4096 x 1024                                          6.9 /  8.2 (96 tokens 9.5 / 7.8)
//     512 x 512                                           4.2 /  5.6 (100 tokens 6.6 / 5.7)
// Experts, rows at random: 16 of 1024 x 4096, 32 rows 14.1 / 19.2, 64 rows 16.3 / 19.8, 96 rows 19.2 / 19.8, 128 rows 20.7 / 19.9;
// 8 of 14336 x 4096, 8 rows 51 / 62, 32 rows 78 / 80, 48 rows 82 / 80, 64 rows 98 / 80; 32 of 512 x 1024, 256 rows 7.6 / 10.5, 512 rows
// 15.6 / 10.4; 32 of 700 x 300, 100 rows 5.1 / 11.5, 400 rows 14.9 / 12.6
// The host does not know how the rows are spread: all on one expert they take that expert's weights in turns of 8 or 16 rows. At random / on
// one, by this rule: 16 of 1024 x 4096, 32 rows 12.5 / 15.7, 96 rows 17 / 44; 8 of 14336 x 4096, 16 rows 68 / 24, 48 rows 81 / 57;
// 32 of 512 x 1024, 192 rows 6.5 / 27; 256 of 1024 x 2048, 1536 rows 97 / 424
bool few_rows_pay(int64_t T, int64_t N, int64_t K, bool by_expert, int64_t experts) {
    if (by_expert) return T <= 6 * experts || (T <= 10 * experts && N * K <= 600000);
    return T <= 16 || (T <= 32 && N * K <= 24000000) || (T <= 64 && K <= 1024 && N * K <= 5000000);
}

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
    if (K == 0 || few_rows_pay(T, N, K, offsets != nullptr, experts)) {
        cudaError_t e = cudaSuccess;
        const dim3 grid((unsigned)ceil_div(N, F_FEATURES), (unsigned)(experts + (offsets ? 1 : 0)));
        auto go = [&](auto kern, int warps) { GPTQ_LAUNCH(K_INT8_MM, s, e = launch_pdl(kern, grid, dim3(32 * warps), 0, s, p)); };
        // (with experts the rows of each are not known here: mostly a share of them)
        const int64_t rows = offsets ? T / experts : T;
        const int64_t ctas = (int64_t)grid.x * experts, sms = device_sm_count();
        // (four steps ahead are 2048 columns of the CTA; 32 tokens, us with two, four, and four steps and all registers: 1024 x 4096 8.0, 7.2,
        // 7.0; 2048 x 4096 8.9, 8.4, 7.5; 4096 x 4096 9.5, 9.0, 13.6; 64 tokens 4096 x 1024 6.9, 8.8. 16 tokens, four steps and eight:
        // 2048 x 4096 6.5 and 6.1, 1024 x 2500 4.3 and 3.9)
        if (rows > 16 && p.pitch < 2048) go(int8_few_rows_kernel<4, 8, 2, 2>, 8);
        else if (rows > 16 && ctas > sms) go(int8_few_rows_kernel<4, 8, 4, 2>, 8);
        else if (rows > 16) go(int8_few_rows_kernel<4, 8, 4, 1>, 8);
        else if (rows > 8 && ctas <= sms && p.pitch > 2048) go(int8_few_rows_kernel<2, 8, 8, 1>, 8);
        else if (rows > 8) go(int8_few_rows_kernel<2, 8, 4, 2>, 8);
        else if (ctas <= 2 * sms) go(int8_few_rows_kernel<1, 8, 8, 2>, 8);
        else go(int8_few_rows_kernel<1, 4, 2, 8>, 4);
        GPTQ_CUDA_TRY(e);
        return st.finish(s);
    }
    int64_t most;
    const Plan plan = plan_of(T, N, K, offsets != nullptr, experts, device_sm_count() / 2, &most);
    p.width = plan.width;
    p.splits = plan.splits;
    WMaps m;
    if (!code_map(&m.w, w_codes, experts * N, K, W_F)) return GPTQ_ERR_CUDA;
    for (int i = first_box(p.width); i < 3; ++i)
        if (!code_map(&m.x[i], x_codes, T, K, W_F >> i)) return GPTQ_ERR_CUDA;
    const int rc = p.splits == 1 ? (p.width <= 64    ? launch_pairs<32, false>(m, p, most, s)
                                    : p.width <= 128 ? launch_pairs<64, false>(m, p, most, s)
                                                     : launch_pairs<128, false>(m, p, most, s))
                                 : (p.width <= 64    ? launch_pairs<32, true>(m, p, most, s)
                                    : p.width <= 128 ? launch_pairs<64, true>(m, p, most, s)
                                                     : launch_pairs<128, true>(m, p, most, s));
    return rc != GPTQ_OK ? rc : st.finish(s);
}

namespace gptq {
// this file's copy of the pipeline-wait limit (the library's test hook sets every copy)
cudaError_t int8_set_wait_limit(unsigned long long ns) { return set_pipeline_wait_limit_this_unit(ns); }
}  // namespace gptq

// fp4_matmul.cu — Y = X W^T for two matrices in the microscaled 4-bit form (fp4.cuh), dense or
// with one weight per expert over rows sorted by expert:
//   Y[t][o] = act(gx gw sum_b sx[t][b] sw[e(t)][o][b] sum_{k in b} x[t][k] w[e(t)][o][k])
//
// The tensor core multiplies this form itself (tcgen05.mma kind::mxf4 / kind::mxf4nvf4 with block
// scales, 64 columns per instruction, fp32 sums in TMEM). The weights are the M operand and the
// tokens the N operand, whose width is chosen per tile: an expert with few rows pays for few.
//
// Two CTAs on neighbouring SMs (a cluster) work on one tile of 256 features x up to 192 tokens with
// cta_group::2 MMAs: each holds its own 128 features, half of the tokens and all the tile's scales,
// so a stage brings 28 KB of codes into each SM where a 128 x 192 tile of its own would take 40.
// Roles in each CTA (persistent, one per SM):
//   warp 0       producer: per stage (256 columns) four TMA copies, the 128 x 128-byte box of weight
//                codes, that of token codes (128-byte swizzle), and the scale tiles of both
//   warp 1       in the even CTA: scale tiles shared memory -> TMEM (tcgen05.cp, both CTAs) and the
//                MMAs; in the odd CTA: tells the even one which stages have landed
//   warps 2..9   epilogue: TMEM -> registers -> Y. bf16 rows are turned in shared memory (stmatrix), so
//                that a token's features leave in 16-byte pieces; fp32, or a Y that is not aligned for
//                that, is stored straight from the registers, where a lane holds one feature
//
// TMEM: two buffers of sums, 192 columns (tokens) each, so one tile's sums are stored while the next
// tile's MMAs run, and two stages' scales in turn in the columns from 384. (Tiles of 256 tokens leave
// room for scales only if the two buffers overlap; waiting for the shared columns cost 1.2 us a tile.)
//
// The MMA warp's own loop takes about 200 cycles for each wait, whether or not it has to wait, so stages
// are filled and released one by one but waited for in pairs (8192 x 8192 x 8192: MX 151 -> 147 us, NV
// 184 -> 163; stages of twice the size instead left the copies too little room, 152 and 169).
//
// What bounds it: the tensor pipe, which needs 96 cycles for 64 columns of a 256 x 192 tile, 0.19 us a stage,
// and that is what a stage of MX takes while few pairs run (NV 0.21, with twice the scale copies in the
// same pipe); 0.21 and 0.24 when all of them do and the clock falls. Below 160 tokens a stage stays at
// 0.14 (NV 0.19). 8192 x 8192 x 8192: MX 147 us, 7.5 PFLOP/s, NV 163 us, 6.7. When run for long both
// meet the power limit (1.67 GHz at 1370 W: 16384 x 4096 x 14336 MX 283 us in short runs, 310 in long
// ones).
// Taken back: 256-token tiles with overlapping buffers, 128 and 64 tokens (slower at every size from 256
// tokens up), a cluster of 2 or 4 pairs sharing a tile's columns (slower but for K = 14336), the odd
// CTA's copies counted on the even one's barriers directly (no faster).
// Every mbarrier wait is bounded (GPTQ_ERR_TIMEOUT into the status word, then unwind: each CTA waits
// for its own copies, the even one for the MMAs, and both meet before either leaves).
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "fp4.cuh"
#include "tc_gemm.cuh"

namespace gptq {

namespace {

constexpr int M_F = 128;                 // features per CTA
constexpr int M_PF = 2 * M_F;            // features per tile
constexpr int M_T = 192;                 // most tokens per tile
constexpr int M_KB = 128;                // bytes of codes per row and stage (256 columns)
constexpr int M_TBOX = 32;               // tokens per TMA box where a CTA's half of a tile has at most this
constexpr int M_THREADS = 32 * 10;
constexpr uint32_t M_TMEM = 512, M_SF0 = 384;
constexpr int M_MAX_EXPERTS = 1024;
constexpr int M_TURN = 32 * 64;          // bytes of a warp's buffer: 32 tokens x 32 features of bf16

template <bool MX>
struct Stage {
    static constexpr int KA = MX ? 2 : 4;              // scale tiles along a stage's columns
    static constexpr int W = M_F * M_KB, X = M_T / 2 * M_KB;
    static constexpr int SW = KA * kFp4Tile, SX = 2 * KA * kFp4Tile;
    static constexpr int BYTES = W + X + SW + SX;      // a multiple of 1024
    static constexpr uint32_t SF_COLS = KA * 12;       // TMEM columns of one stage's scales
    static constexpr int N = 6;                        // stages: what fits in 227 KB; an even number
};

struct Maps {
    CUtensorMap w, x, xsmall;   // codes: 128-row boxes, and one of M_TBOX rows for narrow tiles
    CUtensorMap ws, xs;         // scales: tile bytes x tiles along the columns x row blocks
};

struct MParams {
    const uint8_t *xc, *xs, *wc, *ws;
    const float *xg, *wg;
    int T, N, K;
    int tiles_k;
    int row_blocks;            // 128-row blocks of one expert's weights
    int wg_stride;
    const int32_t* offsets;    // null: one expert, all rows
    int experts;
    int ftiles;                // feature tiles
    int tokens_first;          // neighbouring tiles share their features, not their tokens
    int relu, bf16_out, vec;   // vec: bf16 rows that 16-byte stores can take
    void* Y;
    int64_t ldy;
    int* status;
};

// rows [lo, hi) of expert e, made safe: within the rows of X
__device__ __forceinline__ void expert_rows(const MParams& p, int e, int* lo, int* hi) {
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

// rows that belong to no expert, before the first range and after the last one, are zero (ranges that
// were clamped are an error). One element at a time, with a division each, and by the pairs before their first
// tile, so it is dear where many rows are dropped: 8 experts of 4096 x 4096, 16384 rows to bf16, MX: 94 us with none
// dropped, 95 with 1 %, 131 with 30 % and 175 with 60 %, where the live rows alone take 69 and 46.
__device__ __forceinline__ void zero_rest(const MParams& p, int64_t i, int64_t step) {
    const int first = min(max(p.offsets[0], 0), p.T), last = max(min(p.offsets[p.experts], p.T), first);
    const int64_t n = (int64_t)(p.T - (last - first)) * p.N;
    for (; i < n; i += step) {
        const int64_t r = i / p.N, at = (r < first ? r : r + (last - first)) * p.ldy + i % p.N;
        if (p.bf16_out) static_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(0.0f);
        else static_cast<float*>(p.Y)[at] = 0.0f;
    }
}

// Token tiles of rows [lo, hi). They start on multiples of 64, where the tokens' scales may start in
// TMEM, so a tile of up to 192 tokens has its scales in two 128-row blocks.
__device__ __forceinline__ int token_tiles(int lo, int hi) {
    return hi <= lo ? 0 : (hi - (lo & ~63) + M_T - 1) / M_T;
}

struct Tile {
    int e, f0;        // expert, first feature
    int t0, n;        // first token (a multiple of 64), tokens (a multiple of 32)
    int lo, hi;       // the tokens that belong to the expert
};

// tile index -> tile; start[e] = token tiles before expert e
__device__ __forceinline__ Tile find_tile(const MParams& p, const int32_t* start, uint32_t i) {
    Tile t;
    const uint32_t ttiles = (uint32_t)start[p.experts];
    const int tt = (int)(p.tokens_first ? i % ttiles : i / (uint32_t)p.ftiles);
    t.f0 = (int)(p.tokens_first ? i / ttiles : i % (uint32_t)p.ftiles) * M_PF;
    int a = 0, b = p.experts;   // start[a] <= tt < start[b]
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (start[m] <= tt) a = m;
        else b = m;
    }
    t.e = a;
    if (p.offsets) {
        t.lo = min(max(p.offsets[a], 0), p.T);
        t.hi = min(max(p.offsets[a + 1], t.lo), p.T);
    } else {
        t.lo = 0;
        t.hi = p.T;
    }
    t.t0 = (t.lo & ~63) + (tt - start[a]) * M_T;
    t.n = min((t.hi - t.t0 + 31) & ~31, M_T);
    return t;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// One lane of a converged warp: unlike a test of the lane number, the branch on it leaves the values
// it uses warp-uniform, so the tensor instructions take their operands from uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// The bounded wait, by a whole converged warp. Only the time is looked at while it waits: what a wait
// that gave up has to record is done after the loops, because a global atomic (or the load of its
// limit) in them cost the warps that feed the tensor core more than the waiting itself
// (8192 x 8192 x 8192 MX: 225 us with mbar_wait, 155 us with this).
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, uint64_t limit) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (__any_sync(0xffffffffu, globaltimer_ns() - t0 >= limit)) return false;
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    }
}

// ------------------------------------ the pair of CTAs ------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// the even CTA's copy of a shared-memory address
__device__ __forceinline__ uint32_t in_even_cta(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

// What these arrivals order is TMEM and copies by TMA, neither written by this thread, so the default
// (CTA) scope of the release is enough; .release.cluster would wait for the thread's own earlier
// stores of Y to be acknowledged (8192 x 8192 x 8192 MX took 408 us with it and 269 without).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// arrive once on `bar` of both CTAs when the MMAs and scale copies issued before have completed
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// 32 rows x 16 bytes of each CTA's shared memory to four of its TMEM columns, in each quarter of the lanes
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(smem_desc(saddr, 0, 128, 0)) : "memory");
}

template <bool MX>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
    if (MX)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// Instruction descriptor of the block-scaled kinds: [4,6) B's scale byte | [7,10) A type (1 = e2m1) |
// [10,12) B type | [17,23) N >> 3 | [23] scale type (1 = e8m0, 0 = e4m3) | [24,29) M >> 4 |
// [29,31) A's scale byte
template <bool MX>
__device__ __forceinline__ uint32_t fp4_idesc(int n, uint32_t sf) {
    return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((MX ? 1u : 0u) << 23) |
           ((uint32_t)(M_PF >> 4) << 24) | (sf << 29);
}

// Waits for the phase of a barrier that counts copies or MMAs in flight, before the CTA leaves. They land
// within microseconds; the limit is for an unwinding pair, whose even CTA's stages may also be
// waiting for a word from the odd one that is not coming.
constexpr uint64_t M_DRAIN_NS = 20000000ull;
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < M_DRAIN_NS) {
    }
}

// The product of both tensor scales as g * back * back. back is 1 unless the product is subnormal or past
// fp32, where it would lose bits, or all of them, although the scales and the results are ordinary numbers
// (1e-22 * 1e-22 has 3 bits, while sums of codes and block scales reach 1e9).
struct TensorScale {
    float g, back;
};
__device__ __forceinline__ TensorScale tensor_scale(float a, float b) {
    const float m = fabsf(a * b);
    const float s = m < 0x1p-126f ? 0x1p32f : m > 0x1.fffffep127f ? 0x1p-64f : 1.0f;
    return {(a * s) * (b * s), 1.0f / s};
}

// sums times the tensor scale where that is not one number, which is left as 1
template <int N>
__device__ __forceinline__ void apply_unusual(uint32_t (&v)[N], const TensorScale& t) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * t.g * t.back * t.back);
}

// max(x, 0) that keeps a NaN
__device__ __forceinline__ float relu_of(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
    return y;
}

// 32 tokens of one feature to Y: the lanes of a warp hold consecutive features, so each token is
// one store of 64 or 128 consecutive bytes
template <typename T>
__device__ __forceinline__ void store_tokens(T* y, int64_t ldy, const uint32_t (&v)[32], float g, bool relu, int first, int last) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        if (j >= first && j < last) {
            const float x = __uint_as_float(v[j]) * g, z = relu ? relu_of(x) : x;
            if constexpr (sizeof(T) == 2) *y = __float2bfloat16_rn(z);
            else *y = z;
        }
        y += ldy;
    }
}

__device__ __forceinline__ void store_tokens(const MParams& p, const uint32_t (&v)[32], float g, const Tile& t, int tok, int f) {
    if (f >= p.N) return;
    const int first = max(t.lo - tok, 0), last = min(t.hi - tok, 32);
    const int64_t at = (int64_t)tok * p.ldy + f;
    if (p.bf16_out) store_tokens(static_cast<__nv_bfloat16*>(p.Y) + at, p.ldy, v, g, p.relu != 0, first, last);
    else store_tokens(static_cast<float*>(p.Y) + at, p.ldy, v, g, p.relu != 0, first, last);
}

// 16 lanes x 32 columns of TMEM: of each 8 columns thread i gets lane i / 4, columns 2 (i % 4) and the
// next, then the same of lane 8 + i / 4 (the layout that stmatrix takes)
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ uint32_t two_bf16(uint32_t a, uint32_t b, float g, bool relu) {
    float x = __uint_as_float(a) * g, y = __uint_as_float(b) * g;
    if (relu) {
        x = relu_of(x);
        y = relu_of(y);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 tokens x 32 features (v[h]: features 16 h ..) to Y through the warp's 2 KB of shared memory: rows
// of 64 bytes, one per token, whose 16-byte pieces are permuted so that neither side has conflicts
__device__ __forceinline__ void turn_tokens(const MParams& p, const uint32_t (&v)[2][16], float g, const Tile& t, int tok, int f0,
                                            uint32_t buf) {
    const int lane = threadIdx.x & 31;
    const bool relu = p.relu != 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int row = 8 * j + (lane & 7);
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                         buf + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4)),
                     "r"(two_bf16(v[0][4 * j], v[0][4 * j + 1], g, relu)), "r"(two_bf16(v[0][4 * j + 2], v[0][4 * j + 3], g, relu)),
                     "r"(two_bf16(v[1][4 * j], v[1][4 * j + 1], g, relu)), "r"(two_bf16(v[1][4 * j + 2], v[1][4 * j + 3], g, relu))
                     : "memory");
    }
    __syncwarp();
    const int f = f0 + 8 * (lane & 3);
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.Y) + f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int row = 8 * j + (lane >> 2), r = tok + row;
        uint4 w;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                     : "r"(buf + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4)));
        if (f < p.N && r >= t.lo && r < t.hi) *reinterpret_cast<uint4*>(y + (int64_t)r * p.ldy) = w;
    }
    __syncwarp();
}

template <bool MX>
__global__ void __launch_bounds__(M_THREADS, 1) fp4_matmul_kernel(const __grid_constant__ Maps m, const MParams p) {
    using S = Stage<MX>;
    constexpr int NS = S::N;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + NS * S::BYTES + 8 * M_TURN);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * NS + 5);
    int32_t* start = reinterpret_cast<int32_t*>(tmem_slot + 1);   // [experts + 1]

    // what steers a warp is made warp-uniform by a shuffle, so the branches and the operands of the
    // tensor instructions stay in uniform registers
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = uniform(cluster_rank());
    const uint32_t sbase = smem_u32(smem), bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * (s >> 1); };   // a pair of stages: copies landed (even CTA: the odd one's too)
    auto empty = [&](int s) { return bar0 + 8u * (NS + s); };           // the stage's MMAs are done
    auto tfull = [&](int b) { return bar0 + 8u * (2 * NS + b); };       // a tile's sums are done
    auto tfree = [&](int b) { return bar0 + 8u * (2 * NS + 2 + b); };   // even CTA: both have read a tile's sums
    const uint32_t drain_bar = bar0 + 8u * (2 * NS + 4);
    const int stages = (p.K + 4 * M_KB - 1) / (4 * M_KB) * 2;   // (a last one past the columns brings zeros)
    const uint32_t first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            if (!(s & 1)) mbar_init(full(s), rank == 0 ? 3 : 2);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tfree(b), 16);
        }
        mbar_init(drain_bar, 1);
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&m.w);
        tma_prefetch_desc(&m.x);
        tma_prefetch_desc(&m.ws);
        tma_prefetch_desc(&m.xs);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(M_TMEM)
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
            if (e0 + lane < p.experts) start[e0 + lane] = carry + inc - n;
            carry += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) start[p.experts] = carry;
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers are ready before either signals the other's
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    const uint64_t limit = *static_cast<volatile unsigned long long*>(&g_pipeline_wait_limit_ns);
    bool ok = true;   // false: a wait gave up
    const uint32_t ntiles = uniform((uint32_t)start[p.experts] * (uint32_t)p.ftiles);

    if (warp == 0) {
        // ------------------------------- producer -----------------------------------
        const bool leader = elect_one();
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_par = 0;
        for (uint32_t i = first; i < ntiles && ok; i += step) {
            const Tile t = find_tile(p, start, i);
            const int n = (int)uniform(t.n), t0 = (int)uniform(t.t0), e = (int)uniform(t.e);
            const int f = (int)uniform(t.f0) + (int)rank * M_F;
            const bool small = n <= 2 * M_TBOX;
            const CUtensorMap* tx = small ? &m.xsmall : &m.x;
            const uint32_t bytes = S::BYTES - (small ? (M_T / 2 - M_TBOX) * M_KB : 0);
            const int wrow = e * p.N + f, xrow = t0 + (int)rank * (n >> 1);
            // (features past the last one: their sums are not stored, so any scales will do)
            const int wblock = e * p.row_blocks + min(f >> 7, p.row_blocks - 1), xblock = t0 >> 7;
            for (int kt = 0; kt < stages; ++kt) {
                ok = wait_all(empty(stage), phase ^ 1u, limit);
                if (!ok) break;
                if (leader) {
                    const uint32_t base = sbase + stage * S::BYTES, bar = full(stage);
                    mbar_expect_tx(bar, bytes);
                    tma_load_2d(base, &m.w, bar, kt * M_KB, wrow);
                    tma_load_2d(base + S::W, tx, bar, kt * M_KB, xrow);
                    tma_load_3d(base + S::W + S::X, &m.ws, bar, 0, kt * S::KA, wblock);
                    tma_load_3d(base + S::W + S::X + S::SW, &m.xs, bar, 0, kt * S::KA, xblock);
                }
                __syncwarp();
                issued |= 1u << stage;
                issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
                if (++stage == NS) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (leader)
            for (int s = 0; s < NS; ++s)
                if (issued & (1u << s)) drain(full(s), (issued_par >> s) & 1u);
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        // ------------------------------- MMA issuer ---------------------------------
        int stage = 0;
        uint32_t phase = 0, tile = 0;
        for (uint32_t i = first; i < ntiles && ok; i += step, ++tile) {
            Tile t = find_tile(p, start, i);
            t.t0 = (int)uniform(t.t0);
            t.n = (int)uniform(t.n);
            const bool two = (t.t0 & 127) + t.n > 128;   // the tokens' scales are in two row blocks
            const uint32_t b = tile & 1u;
            ok = wait_all(tfree(b), ((tile >> 1) & 1u) ^ 1u, limit);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + b * (uint32_t)M_T;
            const uint32_t tcol = (uint32_t)(t.t0 & 127) >> 5;
            const uint32_t idesc = fp4_idesc<MX>(t.n, 0), idesc2 = fp4_idesc<MX>(t.n, 2);
            for (int kt = 0; kt < stages; kt += 2) {
                ok = wait_all(full(stage), phase, limit);
                if (!ok) break;
                tc_fence_after();
                // The scale copies need no wait of their own: the tensor pipe runs one thread's copies and MMAs
                // in the order they were issued, and with two slots in turn a whole stage's MMAs lie
                // between a slot's last reader and the copy that overwrites it. (Waiting for that
                // reader all the same cost 16 % at 8192 x 8192 x 8192, with the same results.)
                if (elect_one()) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t base = sbase + (stage + u) * S::BYTES;
                        const uint32_t sf = tmem + M_SF0 + u * S::SF_COLS;
                        const int ka = p.tiles_k - (kt + u) * S::KA;
                        const int ksteps = (p.K - (kt + u) * 2 * M_KB + 63) / 64;
#pragma unroll
                        for (int a = 0; a < S::KA; ++a) {
                            if (a < ka) {
                                copy_scales(sf + a * 4, base + S::W + S::X + a * kFp4Tile);
                                copy_scales(sf + S::KA * 4 + a * 8, base + S::W + S::X + S::SW + a * kFp4Tile);
                                if (two) copy_scales(sf + S::KA * 4 + a * 8 + 4, base + S::W + S::X + 2 * S::SW + a * kFp4Tile);
                            }
                        }
                        const uint64_t ad = smem_desc(base, 16, 1024, kSwizzle128B), bd = smem_desc(base + S::W, 16, 1024, kSwizzle128B);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (k < ksteps) {
                                const int a = MX ? k >> 1 : k;
                                umma_fp4<MX>(d, ad + 2 * k, bd + 2 * k, MX && (k & 1) ? idesc2 : idesc, sf + a * 4,
                                             sf + S::KA * 4 + a * 8 + tcol, (kt > 0 || u > 0 || k > 0) ? 1u : 0u);
                            }
                        }
                        commit_pair(empty(stage + u));
                    }
                    if (kt == stages - 2) commit_pair(tfull(b));
                }
                __syncwarp();
                if ((stage += 2) == NS) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (elect_one()) {
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drain_bar) : "memory");
            drain(drain_bar, 0);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------- odd CTA: passes on which stages have landed ------------
        const bool leader = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        for (uint32_t i = first; i < ntiles && ok; i += step) {
            for (int kt = 0; kt < stages; kt += 2) {
                ok = wait_all(full(stage), phase, limit);
                if (!ok) break;
                if (leader) arrive_cluster(in_even_cta(full(stage)));
                __syncwarp();
                if ((stage += 2) == NS) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else {
        // ------------------------------- epilogue -----------------------------------
        const int q = warp & 3;
        const int c0 = M_T / 2 * ((warp - 2) >> 2);   // its half of the columns
        const uint32_t lanes = (uint32_t)(32 * q) << 16;
        const uint32_t turn = sbase + NS * S::BYTES + (warp - 2) * M_TURN;
        if (p.offsets) zero_rest(p, (int64_t)blockIdx.x * 256 + threadIdx.x - 64, (int64_t)gridDim.x * 256);
        const float gx = MX ? 1.0f : *p.xg;
        uint32_t tile = 0;
        for (uint32_t i = first; i < ntiles; i += step, ++tile) {
            const Tile t = find_tile(p, start, i);
            const uint32_t b = tile & 1u;
            ok = wait_all(tfull(b), (tile >> 1) & 1u, limit);
            if (!ok) break;
            tc_fence_after();
            TensorScale g = {1.0f, 1.0f};
            if (!MX) g = tensor_scale(gx, p.wg[t.e * p.wg_stride]);
            const bool unusual = !MX && g.back != 1.0f;
            const int f0 = t.f0 + (int)rank * M_F + 32 * q;
            const uint32_t sums = tmem + lanes + b * (uint32_t)M_T + c0;
            // all of its columns into registers (those past the tile's tokens too: the buffer has them), so
            // the buffer is free before anything is stored
            if (p.vec) {
                uint32_t v[M_T / 64][2][16];
#pragma unroll
                for (int c = 0; c < M_T / 64; ++c) {
                    tmem_ld_16x256b_x4(sums + 32 * c, v[c][0]);
                    tmem_ld_16x256b_x4(sums + (16u << 16) + 32 * c, v[c][1]);
                }
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(in_even_cta(tfree(b)));
                if (unusual) {
#pragma unroll
                    for (int c = 0; c < M_T / 32; ++c) apply_unusual(v[c >> 1][c & 1], g);
                    g.g = 1.0f;
                }
#pragma unroll
                for (int c = 0; c < M_T / 64; ++c)
                    if (c0 + 32 * c < t.n) turn_tokens(p, v[c], g.g, t, t.t0 + c0 + 32 * c, f0, turn);
            } else {
                uint32_t v[M_T / 64][32];
#pragma unroll
                for (int c = 0; c < M_T / 64; ++c) tmem_ld_32x32b_x32(sums + 32 * c, v[c]);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(in_even_cta(tfree(b)));
                if (unusual) {
#pragma unroll
                    for (int c = 0; c < M_T / 64; ++c) apply_unusual(v[c], g);
                    g.g = 1.0f;
                }
#pragma unroll
                for (int c = 0; c < M_T / 64; ++c)
                    if (c0 + 32 * c < t.n) store_tokens(p, v[c], g.g, t, t.t0 + c0 + 32 * c, f0 + lane);
            }
        }
    }

    if (!ok && lane == 0) set_status(p.status, GPTQ_ERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // neither CTA leaves, or frees TMEM, while the other may still use it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(M_TMEM) : "memory");
    }
}

// ------------------------------------------------------------------------------- few rows
// With a handful of tokens the product is the stream of the weights, and what counts is to have all of
// it in flight at once. A CTA of 128 threads computes 8 features: a thread takes 32 columns (16 bytes of
// codes) of each feature and of up to 4 tokens, every 128th such piece. Codes become half2 (one
// conversion per byte), and the products of 16 columns are summed in half2: each is a multiple of
// 1/4 up to 36, so 8 of them per half stay below 512 in steps of 1/4, which 11 bits hold exactly. Those
// sums go to fp32 with both scales (whose product has at most 8 bits), and are added over the columns
// and, in a fixed order, over the CTA.
// The 8 features are two neighbours of each 32-row quarter of a scale tile, whose scales share sectors.
// One token x 4096 x 4096 MX: 5.6 us with its launch (9 MB; 4.3 where L2 has them); what bounds it there is
// latency, and with more weights the conversions (14336 x 4096: 11.8 us, 2.7 TB/s), where the other kernel takes over.
constexpr int F_THREADS = 128, F_FEATURES = 8, F_TOKENS = 4;

__device__ __forceinline__ void to_half2(const uint4& c, __half2 (&h)[16]) {
    const uint32_t u[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        h[i] = __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((u[i >> 2] >> (8 * (i & 3))) & 0xFFu), __NV_E2M1));
}

// the scales of 32 columns from a word of a scale tile: one (MX) or two (NV); c: index of the 32 columns
template <bool MX>
__device__ __forceinline__ float2 two_scales(uint32_t word, int c) {
    if (MX) {
        const float s = e8m0_value((word >> (8 * (c & 3))) & 0xFFu);
        return make_float2(s, s);
    }
    const uint32_t b = word >> (16 * (c & 1));
    return make_float2(e4m3_value(b & 0xFFu), e4m3_value((b >> 8) & 0xFFu));
}

// acc + v a b for a sum v of 32 products and two e8m0 scales. The product of the scales may be past fp32
// where v is 0 or v a b is not; v times the smaller scale is exact (at most 13 bits from 2^-129 up) and
// overflows only if v a b does. A NaN scale makes it NaN.
__device__ __forceinline__ float add_scaled(float v, float a, float b, float acc) {
    float lo, hi;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(lo) : "f"(a), "f"(b));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(hi) : "f"(a), "f"(b));
    return fmaf(v * lo, hi, acc);
}

// byte of the 16-byte row (4 quarters x 4 blocks) of scale tiles for row r and 32 columns c
template <bool MX>
__device__ __forceinline__ int64_t scale_row(int64_t r, int c, int tiles_k) {
    return ((r >> 7) * tiles_k + c / (MX ? 4 : 2)) * kFp4Tile + (r & 31) * 16;
}

// (Plain loads: this kernel starts while the one before may still be writing its operands, so they are not
// read-only for as long as it runs, which is what the read-only path asks for.)
// tokens t0 .. t0 + n - 1 (n <= NT) of expert e times features fb + (i & 1) + 32 (i >> 1), i < 8
template <bool MX, int NT>
__device__ __forceinline__ void few_rows(const MParams& p, int e, int t0, int n, int fb, float (*part)[F_FEATURES * F_TOKENS]) {
    const int64_t pitch = fp4_pitch(p.K);
    const uint8_t* wc = p.wc + (int64_t)e * p.N * pitch;
    const uint8_t* ws = p.ws + (int64_t)e * p.row_blocks * p.tiles_k * kFp4Tile;
    float acc[F_FEATURES][NT] = {};
    for (int c = threadIdx.x; c < (int)(pitch >> 4); c += F_THREADS) {
        uint4 w[F_FEATURES], x[NT], sw[2];
        uint32_t sx[NT];
#pragma unroll
        for (int i = 0; i < F_FEATURES; ++i) {
            const int f = min(fb + (i & 1) + 32 * (i >> 1), p.N - 1);
            w[i] = *(reinterpret_cast<const uint4*>(wc + f * pitch) + c);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) sw[i] = *reinterpret_cast<const uint4*>(ws + scale_row<MX>(fb + i, c, p.tiles_k));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = t0 + min(t, n - 1);
            x[t] = *(reinterpret_cast<const uint4*>(p.xc + r * pitch) + c);
            sx[t] = *(reinterpret_cast<const uint32_t*>(p.xs + scale_row<MX>(r, c, p.tiles_k)) + ((r >> 5) & 3));
        }
        __half2 xh[NT][16];
#pragma unroll
        for (int t = 0; t < NT; ++t) to_half2(x[t], xh[t]);
#pragma unroll
        for (int i = 0; i < F_FEATURES; ++i) {
            __half2 wh[16];
            to_half2(w[i], wh);
            const uint4& s4 = sw[i & 1];
            const float2 sc = two_scales<MX>(i < 2 ? s4.x : i < 4 ? s4.y : i < 6 ? s4.z : s4.w, c);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                __half2 h0 = __hmul2(wh[0], xh[t][0]), h1 = __hmul2(wh[8], xh[t][8]);
#pragma unroll
                for (int k = 1; k < 8; ++k) {
                    h0 = __hfma2(wh[k], xh[t][k], h0);
                    h1 = __hfma2(wh[8 + k], xh[t][8 + k], h1);
                }
                const float2 f0 = __half22float2(h0), f1 = __half22float2(h1), st = two_scales<MX>(sx[t], c);
                if (MX) acc[i][t] = add_scaled((f0.x + f0.y) + (f1.x + f1.y), sc.x, st.x, acc[i][t]);
                else acc[i][t] = fmaf(f1.x + f1.y, sc.y * st.y, fmaf(f0.x + f0.y, sc.x * st.x, acc[i][t]));
            }
        }
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < F_FEATURES; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float v = acc[i][t];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) part[warp][i * NT + t] = v;
        }
    __syncthreads();
    if (threadIdx.x < F_FEATURES * NT) {
        const int i = threadIdx.x / NT, t = threadIdx.x % NT, f = fb + (i & 1) + 32 * (i >> 1);
        float v = 0.0f;
        for (int k = 0; k < F_THREADS / 32; ++k) v += part[k][threadIdx.x];
        if (!MX) {
            const TensorScale g = tensor_scale(*p.xg, p.wg[e * p.wg_stride]);
            v = v * g.g * g.back * g.back;
        }
        if (p.relu) v = relu_of(v);
        if (f < p.N && t < n) {
            const int64_t at = (int64_t)(t0 + t) * p.ldy + f;
            if (p.bf16_out) static_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(v);
            else static_cast<float*>(p.Y)[at] = v;
        }
    }
    __syncthreads();
}

// MOST: the most tokens at a time; a kernel that cannot take four has the registers of one that is not
// made to, so more of its CTAs fit
template <bool MX, int MOST>
__global__ void __launch_bounds__(F_THREADS) fp4_few_rows_kernel(const MParams p) {
    __shared__ float part[F_THREADS / 32][F_FEATURES * F_TOKENS];
    const int e = blockIdx.y;
    pdl_wait();
    if (e == p.experts) {   // (only with offsets)
        zero_rest(p, (int64_t)blockIdx.x * F_THREADS + threadIdx.x, (int64_t)gridDim.x * F_THREADS);
        return;
    }
    int lo, hi;
    expert_rows(p, e, &lo, &hi);
    const int fb = (int)(blockIdx.x >> 4) * 128 + (int)(blockIdx.x & 15) * 2;
    for (int t = lo; t < hi;) {
        const int n = hi - t;
        if (MOST >= 4 && n >= 3) {
            few_rows<MX, 4>(p, e, t, min(n, 4), fb, part);
            t += 4;
        } else if (MOST >= 2 && n >= 2) {
            few_rows<MX, 2>(p, e, t, 2, fb, part);
            t += 2;
        } else {
            few_rows<MX, 1>(p, e, t, 1, fb, part);
            t += 1;
        }
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
constexpr int64_t kMaxDim = (1ll << 31) - 512;

// Whether the kernel for few rows is the faster one. Its time grows with the weights it reads and,
// token by token, expands and multiplies; the other one's with the columns alone while its tiles
// fit the device. Measured (us, few rows / pairs; weights from memory, features x columns; the bound was set on MX,
// dense, with the weights in L2):
//                        1 token      2 tokens     3 tokens     4 tokens
//   MX   4096 x 4096    5.6 / 8.0    6.6 / 8.1   11.0 / 8.0   11.0 / 8.1
//   NV   4096 x 4096    5.8 / 8.7    6.6 / 8.7   13.0 / 8.7   13.0 / 8.8
//   MX  14336 x 4096   11.8 / 9.8   14.5 / 9.8
//   NV  14336 x 4096   11.1 / 10.3  16.0 / 10.4
//   MX   1024 x 4096    2.6 / 6.5    3.2 / 6.5    5.3 / 6.5    5.3 / 6.5
//   NV   1024 x 4096    3.0 / 7.6    3.4 / 7.5    4.9 / 7.6    4.8 / 7.6
//   8 experts of 4096 x 4096, each row its own expert:
//   MX                  6.0 / 7.1    8.2 / 7.6   11.8 / 9.1   15.0 / 10.8
//   NV                  5.0 / 8.2    8.0 / 8.8   11.1 / 9.9   14.4 / 11.7
//   16 of 1024 x 4096: MX 3.1 / 7.1 to 6.3 / 8.2, NV 3.3 / 8.2 to 6.0 / 8.7 (all rows one expert's: 8.7 / 7.0 and 8.4 / 8.1)
// It takes the slower side where many columns meet one token (4096 x 14336: MX 12.8 / 15.6, NV 14.2 / 17.0, pairs
// taken), for 3 and 4 tokens on few columns (4096 x 1024: MX 8.7 / 4.9, NV 7.8 / 5.3, few rows taken), and for
// very many experts, whose CTAs start for nothing (128 of 768 x 2048: MX 9.5 / 6.7 and up, few rows taken).
bool few_rows_pay(int64_t T, int64_t N, int64_t K, int64_t experts) {
    return T <= 4 && (std::min(experts, T) + T) * N * K <= 60000000;
}

bool code_map(CUtensorMap* m, const uint8_t* codes, int64_t rows, int64_t pitch, int box_rows) {
    auto enc = tma_encoder();
    cuuint64_t dims[2] = {(cuuint64_t)pitch, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)pitch};
    cuuint32_t box[2] = {(cuuint32_t)M_KB, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// a scale tile is 128 32-bit elements; tiles past the columns or rows read as zero
bool scale_map(CUtensorMap* m, const uint8_t* scales, int64_t tiles_k, int64_t blocks, int ka, int box_blocks) {
    auto enc = tma_encoder();
    cuuint64_t dims[3] = {kFp4Tile / 4, (cuuint64_t)tiles_k, (cuuint64_t)blocks};
    cuuint64_t strides[2] = {kFp4Tile, (cuuint64_t)(tiles_k * kFp4Tile)};
    cuuint32_t box[3] = {kFp4Tile / 4, (cuuint32_t)ka, (cuuint32_t)box_blocks};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_INT32, 3, const_cast<uint8_t*>(scales), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool MX>
int launch_few(const MParams& p, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const dim3 grid((unsigned)(16 * p.row_blocks), (unsigned)(p.experts + (p.offsets ? 1 : 0)));
    // (with experts the rows of each are not known here: mostly one or two)
    auto go = [&](auto kern) { GPTQ_LAUNCH(K_FP4_MM, s, e = launch_pdl(kern, grid, dim3(F_THREADS), 0, s, p)); };
    if (p.T == 1) go(fp4_few_rows_kernel<MX, 1>);
    else if (p.T == 2 || p.offsets) go(fp4_few_rows_kernel<MX, 2>);
    else go(fp4_few_rows_kernel<MX, 4>);
    GPTQ_CUDA_TRY(e);
    return GPTQ_OK;
}

template <bool MX>
int launch(const Maps& m, const MParams& p, int64_t most_tiles, cudaStream_t s) {
    constexpr int kFixed = 1024 + Stage<MX>::N * Stage<MX>::BYTES + 8 * M_TURN + 8 * (2 * Stage<MX>::N + 5) + 8;
    constexpr int kMost = kFixed + 4 * (M_MAX_EXPERTS + 1);
    static_assert(kMost <= 227 * 1024, "an SM's shared memory");
    const int smem = kFixed + 4 * (p.experts + 1);
    // the limit is the kernel's and not the call's: every thread's calls set it to the same number
    GPTQ_CUDA_TRY(cudaFuncSetAttribute(fp4_matmul_kernel<MX>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(most_tiles, device_sm_count() / 2));
    cfg.blockDim = dim3(M_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaSuccess;
    GPTQ_LAUNCH(K_FP4_MM, s, e = cudaLaunchKernelEx(&cfg, fp4_matmul_kernel<MX>, m, p));
    GPTQ_CUDA_TRY(e);
    return GPTQ_OK;
}

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
    if (experts > M_MAX_EXPERTS || N > kMaxDim / experts) return GPTQ_ERR_UNSUPPORTED;
    // tile numbers have 31 bits (a Y beyond that is larger than the device)
    if ((ceil_div(T, M_T) + 2 * experts) * ceil_div(N, M_F) > kMaxDim) return GPTQ_ERR_UNSUPPORTED;
    if (T == 0 || N == 0) return GPTQ_OK;
    if (!Y || ldy < N || K < 1 || !x_codes || !x_scales || !w_codes || !w_scales || !aligned16(x_codes) || !aligned16(x_scales) ||
        !aligned16(w_codes) || !aligned16(w_scales) || (format == GPTQ_NVFP4 && (!x_g || !w_g)))
        return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t pitch = fp4_pitch(K), tiles_k = fp4_tiles(K, format), row_blocks = ceil_div(N, 128);
    const bool few = few_rows_pay(T, N, K, experts);
    const int ka = format == GPTQ_MXFP4 ? Stage<true>::KA : Stage<false>::KA;
    Maps m;
    if (!few && (!code_map(&m.w, w_codes, experts * N, pitch, M_F) || !code_map(&m.x, x_codes, T, pitch, M_T / 2) ||
        !code_map(&m.xsmall, x_codes, T, pitch, M_TBOX) || !scale_map(&m.ws, w_scales, tiles_k, experts * row_blocks, ka, 1) ||
        !scale_map(&m.xs, x_scales, tiles_k, ceil_div(T, 128), ka, 2)))
        return GPTQ_ERR_CUDA;
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    MParams p{};
    p.xc = x_codes;
    p.xs = x_scales;
    p.wc = w_codes;
    p.ws = w_scales;
    p.xg = x_g;
    p.wg = w_g;
    p.T = (int)T;
    p.N = (int)N;
    p.K = (int)K;
    p.tiles_k = (int)tiles_k;
    p.row_blocks = (int)row_blocks;
    p.wg_stride = (flags & GPTQ_FP4_EXPERT_G) ? 1 : 0;
    p.offsets = offsets;
    p.experts = (int)experts;
    p.ftiles = (int)ceil_div(N, M_PF);
    // The larger operand is walked through once, the smaller one read again from L2: 8 experts of
    // 14336 x 4096 with 8192 rows 166 us this way and 173 the other, 16384 x 4096 x 14336 281 and 302,
    // 1024 x 8192 x 14336 46 and 51
    p.tokens_first = experts * N > T ? 1 : 0;
    p.relu = (flags & GPTQ_DQ_RELU) ? 1 : 0;
    p.bf16_out = (flags & GPTQ_DQ_BF16_OUT) ? 1 : 0;
    p.vec = p.bf16_out && N % 8 == 0 && ldy % 8 == 0 && aligned16(Y) ? 1 : 0;
    p.Y = Y;
    p.ldy = ldy;
    p.status = st.word;
    if (few) {
        const int rc = format == GPTQ_MXFP4 ? launch_few<true>(p, s) : launch_few<false>(p, s);
        return rc != GPTQ_OK ? rc : st.finish(s);
    }
    // an expert's first tile may start up to 63 rows early and its last one be partial
    const int64_t most = (ceil_div(T, M_T) + (offsets ? 2 * std::min(experts, T) : 0)) * p.ftiles;
    const int rc = format == GPTQ_MXFP4 ? launch<true>(m, p, most, s) : launch<false>(m, p, most, s);
    return rc != GPTQ_OK ? rc : st.finish(s);
}

namespace gptq {
// this file's copy of the pipeline-wait limit (the library's test hook sets every copy)
cudaError_t fp4_set_wait_limit(unsigned long long ns) { return set_pipeline_wait_limit_this_unit(ns); }
}  // namespace gptq

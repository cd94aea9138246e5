// int8.cu — rows to 8-bit integers with a scale each, plain or behind a root-mean-square norm with the
// residual's addition, the inverse, and the norm's gradient.
//
//   quantise  a = max|x|, s = a / 127 (fp32), code = the whole number nearest to x / s (the fp32
//             quotient), ties to even; zeros where s = 0
//   norm      h = x + r rounded to x's type; rstd = 1 / sqrt(mean h^2 + eps); the same of
//             y = (h rstd) gain
//   gradient  with u = h rstd, v = dy gain: dx = dh + rstd (v - u mean(u v)), dgain = sum over rows of dy u
// Sums are fp32 in a fixed order.
#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "int8.cuh"

namespace gptq {

namespace {

// --------------------------------------------------------------------- sums over a row's threads
// A row has blockDim.x threads (whole warps); a CTA has blockDim.y rows at a time, more than one only where a
// warp takes a whole row. The sum is the same in all its threads. `part` [32]: one slot per warp, not the
// ones of the sum before.
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (blockDim.x == 32) return v;
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < warps) v += __shfl_xor_sync(0xffffffffu, v, o);
    return __shfl_sync(0xffffffffu, v, 0);
}

__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* part) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (blockDim.x == 32) return v;
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, part[lane < warps ? lane : 0]);
}

// a / 127, correctly rounded (see the quotient below); m: a's bits. NaN for what is not finite
__device__ __forceinline__ float scale_of(uint32_t m) {
    if (m >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    const float a = __uint_as_float(m);
    if (a < 0x1p-60f) return a / 127.0f;
    constexpr float inv = 1.0f / 127.0f;
    const float q = a * inv;
    return fmaf(fmaf(-q, 127.0f, a), inv, q);
}

// the larger of a magnitude and |v|, a NaN above all: as bits it is largest too
__device__ __forceinline__ float larger(float m, float v) { return max_nan(m, fabsf(v)); }
// the same of two pairs of bf16, as bits
__device__ __forceinline__ uint32_t larger_pair(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }

// ------------------------------------------------------------------------------------ units of a row
// A thread works on units of N = 16 / sizeof(T) neighbouring columns, unit j being columns N j .. N j + N - 1
// whatever the row's address. Memory is read and written in aligned 16-byte granules: a row that starts
// `o` elements into a granule has its unit j in granules j and j + 1, and the second one is the next unit's
// first. A warp's units are neighbours (its lane l has units 32 i + l past the warp's first one), so they come by
// shuffles but for the last one's, which its lane loads itself. Granules that are not the row's alone, at its ends, or
// not the warp's, are read and written element by element. All lanes of a warp take part. ANY = false: rows of whole
// granules.
template <typename T>
constexpr int kUnit = 16 / sizeof(T);

template <typename T>
__device__ __forceinline__ int row_start(const T* row) {   // elements
    return (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(T);
}

__device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }

template <typename T>
__device__ __forceinline__ uint4 load_granule(const T* row, int cols, int o, int g) {
    constexpr int N = kUnit<T>;
    const int c = g * N - o;   // its first column
    if (c >= 0 && c + N <= cols) return *reinterpret_cast<const uint4*>(row + c);
    uint32_t w[4] = {};
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (c + e >= 0 && c + e < cols) w[e * (int)sizeof(T) / 4] |= bits(row[c + e]) << (sizeof(T) == 2 ? 16 * (e & 1) : 0);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Calls f(whole words) with a constant for the words of a byte offset (0 .. 15) of bf16: the shift below then takes one
// permutation per word, and no selection. fp32 takes two selections per word instead and FOR_ALL words: the branches made the
// gradient's loads of four rows wait for one another (16384 x 4095 203 us so, 241 with them).
template <typename T, int FOR_ALL, typename F>
__device__ __forceinline__ void with_words(int bytes, F f) {
    if constexpr (sizeof(T) == 4) {
        f(std::integral_constant<int, FOR_ALL>());
    } else {
        switch (bytes >> 2) {
            case 0: f(std::integral_constant<int, 0>()); break;
            case 1: f(std::integral_constant<int, 1>()); break;
            case 2: f(std::integral_constant<int, 2>()); break;
            default: f(std::integral_constant<int, 3>()); break;
        }
    }
}

// the four words of w from `bytes` on, of which WORDS are whole words (bf16)
template <typename T, int WORDS>
__device__ __forceinline__ uint4 shifted(uint32_t (&w)[8], int bytes) {
    if constexpr (sizeof(T) == 4) {
        if (bytes & 8) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 2];
        }
        if (bytes & 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = w[i + 1];
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        const uint32_t selector = bytes & 2 ? 0x5432u : 0x3210u;
        const uint32_t* v = w + WORDS;
        return make_uint4(__byte_perm(v[0], v[1], selector), __byte_perm(v[1], v[2], selector), __byte_perm(v[2], v[3], selector),
                          __byte_perm(v[3], v[4], selector));
    }
}

// Granule j of a row, to be made unit j by to_words
template <typename T, bool ANY>
__device__ __forceinline__ uint4 load_raw(const T* row, int cols, int j) {
    if constexpr (ANY) return load_granule(row, cols, row_start(row), j);
    return j * kUnit<T> < cols ? *reinterpret_cast<const uint4*>(row + j * kUnit<T>) : make_uint4(0, 0, 0, 0);
}

// The warp's units from j on (this lane's first one; 32 apart) from the granules that the lanes have loaded, in place; zeros past the
// columns. (The last lane reads the next warp's first granule here, most likely from L1: before any barrier behind which that
// warp may write to it.)
template <typename T, bool ANY, int UNITS>
__device__ __forceinline__ void to_words(const T* row, int cols, int j, uint4 (&a)[UNITS]) {
    if constexpr (ANY) {
        const int o = row_start(row), lane = threadIdx.x & 31;
        if (o == 0) return;
        uint4 past = make_uint4(0, 0, 0, 0);   // what follows the warp's last granule
        if (lane == 31) past = load_granule(row, cols, o, j + 32 * (UNITS - 1) + 1);
        const int bytes = o * (int)sizeof(T);
        with_words<T, 2>(bytes, [&](auto words) {
            constexpr int W = decltype(words)::value;
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                // the next lane's granule behind this one's, and for the last lane the first lane's next
                uint32_t w[8] = {a[i].x, a[i].y, a[i].z, a[i].w};
                const uint4 after = i + 1 < UNITS ? a[i + 1 < UNITS ? i + 1 : i] : past;
                const uint32_t first[4] = {after.x, after.y, after.z, after.w};
#pragma unroll
                for (int k = 0; k <= W; ++k) {
                    w[4 + k] = __shfl_sync(0xffffffffu, i + 1 < UNITS && lane == 0 ? first[k] : w[k], (lane + 1) & 31);
                    if (i + 1 == UNITS && lane == 31) w[4 + k] = first[k];
                }
                a[i] = shifted<T, W>(w, bytes);
            }
        });
    }
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float (&v)[kUnit<T>]) {
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

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&v)[kUnit<T>]) {
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
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void put(float* p, const uint32_t (&w)[4], int e) { *p = __uint_as_float(w[e]); }
__device__ __forceinline__ void put(__nv_bfloat16* p, const uint32_t (&w)[4], int e) {
    *p = __ushort_as_bfloat16((unsigned short)(w[e >> 1] >> (16 * (e & 1))));
}

// writes the warp's units from j on (see to_words)
template <typename T, bool ANY, int UNITS>
__device__ __forceinline__ void store_units(T* row, int cols, int j, const uint4 (&p)[UNITS]) {
    constexpr int N = kUnit<T>;
    if constexpr (!ANY) {
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
            if ((j + 32 * i) * N < cols) *reinterpret_cast<uint4*>(row + (j + 32 * i) * N) = p[i];
    } else {
        const int o = row_start(row), lane = threadIdx.x & 31;
        // writes granule i, or those of its elements from `from` on that are the row's
        auto put_granule = [&](int i, const uint4& g, int from) {
            const int c = (j + 32 * i) * N - o;   // its first column
            if (from == 0 && c >= 0 && c + N <= cols) {
                *reinterpret_cast<uint4*>(row + c) = g;
            } else {
                const uint32_t w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (e >= from && c + e >= 0 && c + e < cols) put(row + c + e, w, e);
            }
        };
        if (o == 0) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i) put_granule(i, p[i], 0);
            return;
        }
        const int bytes = 16 - o * (int)sizeof(T);   // of the unit before that a granule does not have
        with_words<T, 1>(bytes, [&](auto words) {
            constexpr int W = decltype(words)::value;
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                // the unit before in front of this one: the lane before's, and for the first lane the last one's before
                const uint32_t own[4] = {p[i].x, p[i].y, p[i].z, p[i].w};
                const uint4 b = p[i > 0 ? i - 1 : 0];
                const uint32_t before[4] = {b.x, b.y, b.z, b.w};
                uint32_t w[8] = {};
#pragma unroll
                for (int k = W; k < 4; ++k) w[k] = __shfl_sync(0xffffffffu, lane == 31 ? before[k] : own[k], (lane + 31) & 31);
#pragma unroll
                for (int k = 0; k < 4; ++k) w[4 + k] = own[k];
                // (of its first granule the warp has only the elements from o on)
                put_granule(i, shifted<T, W>(w, bytes), i == 0 && lane == 0 ? o : 0);
            }
        });
        if (lane == 31) {   // and of the one after its last, the first o
            const uint4 l = p[UNITS - 1];
            const uint32_t w[4] = {l.x, l.y, l.z, l.w};
            const int c = (j + 32 * (UNITS - 1)) * N;
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (e >= N - o && c + e < cols) put(row + c + e, w, e);
        }
    }
}

// the gain of a unit's columns, zeros past them
template <int N, bool ANY>
__device__ __forceinline__ void load_gain(const float* gain, int cols, int c, float (&g)[N]) {
    if (!ANY || ((reinterpret_cast<uintptr_t>(gain) & 15) == 0 && c + N <= cols)) {
        if (c < cols) {
#pragma unroll
            for (int e = 0; e < N; e += 4) {
                const float4 v = *reinterpret_cast<const float4*>(gain + c + e);
                g[e] = v.x, g[e + 1] = v.y, g[e + 2] = v.z, g[e + 3] = v.w;
            }
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) g[e] = c + e < cols ? gain[c + e] : 0.0f;
}

// ------------------------------------------------------------------------------- the quotient
// code = rint(x / s), exactly as the fp32 quotient rounds: with the divisor's reciprocal correctly
// rounded, one residual step on the product x * (1 / s) rounds the quotient correctly (Markstein 1990)
// as long as nothing overflows or vanishes on the way, which a power of two sees to for scales far from
// 1. Adding 1.5 * 2^23 leaves the whole number, ties to even, in the low byte.
struct Step {
    float d, inv, f;   // the divisor, its reciprocal, and the power of two that both sides are brought near 1 by
    bool usual;        // the divisor is well inside fp32, so f is 1 and no quotient is past 127
};
__device__ __forceinline__ Step step_of(float s) {
    Step t;
    t.usual = s >= 0x1p-60f && s <= 0x1p60f;
    t.f = t.usual ? 1.0f : s < 1.0f ? 0x1p64f : 0x1p-64f;
    t.d = s * t.f;
    t.inv = s > 0.0f ? __frcp_rn(t.d) : 0.0f;   // (a NaN scale has codes of zero)
    return t;
}
__device__ __forceinline__ uint32_t code_of(float x, const Step& t) {   // in the low byte
    if (!t.usual) x *= t.f;
    float q = x * t.inv;
    q = fmaf(fmaf(-q, t.d, x), t.inv, q);
    // (a subnormal scale is rounded, up to half of it, so a quotient may be past 127)
    if (!t.usual) q = t.inv > 0.0f ? fminf(fmaxf(q, -127.0f), 127.0f) : 0.0f;
    return __float_as_uint(q + 12582912.0f);
}

// two fp32 operations at a time
struct Pair {
    uint64_t w;
    __device__ __forceinline__ Pair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit Pair(float a) : Pair(a, a) {}
    __device__ __forceinline__ void get(uint32_t& a, uint32_t& b) const { asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(w)); }
};
__device__ __forceinline__ Pair operator*(Pair a, const Pair& b) {
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a.w) : "l"(b.w));
    return a;
}
__device__ __forceinline__ Pair operator+(Pair a, const Pair& b) {
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a.w) : "l"(b.w));
    return a;
}
__device__ __forceinline__ Pair fma2(Pair a, const Pair& b, const Pair& c) {
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a.w) : "l"(b.w), "l"(c.w));
    return a;
}

template <int N>
__device__ __forceinline__ void store_codes(int8_t* y, const float (&v)[N], const Step& t) {
    uint32_t u[N], w[N / 4];
    if (t.usual) {
        const Pair inv(t.inv), minus(-t.d), one_half(12582912.0f);   // (1.5 * 2^23)
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const Pair x(v[e], v[e + 1]), q = x * inv;
            (fma2(fma2(q, minus, x), inv, q) + one_half).get(u[e], u[e + 1]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) u[e] = code_of(v[e], t);
    }
#pragma unroll
    for (int e = 0; e < N / 4; ++e)
        w[e] = __byte_perm(__byte_perm(u[4 * e], u[4 * e + 1], 0x0040), __byte_perm(u[4 * e + 2], u[4 * e + 3], 0x0040), 0x5410);
    if constexpr (N == 4) *reinterpret_cast<uint32_t*>(y) = w[0];
    else *reinterpret_cast<uint2*>(y) = make_uint2(w[0], w[1]);
}

// ----------------------------------------------------------------------------------- the rows
struct RowParams {
    const void* X;
    const void* R;           // norm: the residual, or null
    const float* gain;       // norm
    float eps;
    int64_t rows, cols, ldx, ldr;
    int64_t src_rows;        // quantise: rows of X
    const int32_t* index;    // quantise: row r is X row index[r] / per (negative: zeros); null: row r
    int64_t per;
    int8_t* codes;
    int64_t pitch;
    float* scales;
    void* H;                 // norm: x + r, where there is r
    int64_t ldh;
    float* rstd;
    int* status;
};

// 1 / sqrt(mean h^2 + eps) from the sum of squares; where the squares leave fp32's normal numbers the sum is
// taken again of scaled values (a row apart, so nothing is lost elsewhere). A mean below 2^-80 times 2^160 is the mean of less than
// 2^31 squares, so their sum is below 2^111, and what counts next to eps >= 2^-149 (2^11) stays normal. Squares past
// fp32 are below 2^256 times 2^-160, and 2^31 of them below 2^127.
template <typename F>
__device__ __forceinline__ float rstd_of(float sum, float inv_n, float eps, F again) {
    const float v = fmaf(sum, inv_n, eps);
    if (v >= 0x1p-80f && v <= 0x1.fffffep127f) return rsqrtf(v);
    const float f = v < 1.0f ? 0x1p80f : 0x1p-80f;
    return rsqrtf(again(f) * inv_n + eps * f * f) * f;
}

// the row of X that row r is, or -1
__device__ __forceinline__ int64_t source_row(const RowParams& p, int64_t r) {
    if (!p.index) return r;
    const int k = p.index[r];
    const int64_t sr = k < 0 ? -1 : k / p.per;
    if (sr < p.src_rows) return sr;
    set_status(p.status, GPTQ_ERR_INVALID_ARG);
    return -1;
}

// Rows in the registers of their threads, UNITS units each: a row is read once and everything written once. CTAs
// are persistent, and the next row's loads are under way while this one is reduced and written. Four units per thread, so
// that what every warp does for a row (its sums, scale and reciprocals) is shared by more columns.
// Bound by memory, and for bf16 nearly as much by instructions, the quantisation and the norm with a residual: 16384 x 4096
// bf16 34 us (6.0 TB/s) and 77 (6.1); fp32 51 (6.6) and 136 (6.4). The norm without a residual is not: bf16 53 (3.8), fp32 87 (3.9). For each row
// it reads the gain again (as many bytes as an fp32 row) and has two barriers, one after the other, as with a residual, but for less than
// half of the bytes. With two units per thread bf16 took 39 (quantisation) and 91 (norm with a residual), with a CTA for each row and no loads ahead 52 and 107. Rows at odd addresses pay for the shifting: 16384 x 4095
// bf16 44 and 128 us (column by column 109 and 278), fp32 65 and 165. MOST is 512 or, for longer rows of fp32, 1024 threads:
// the norm of 16384 x 4095 fp32 took 202 us within the 64 registers of the latter, the quantisation 74 instead of 65 with more.
template <typename T, int UNITS, bool NORM, bool ANY, int MOST>
__global__ void __launch_bounds__(NORM || sizeof(T) == 2 ? MOST : 1024, 1) int8_rows_kernel(const RowParams p) {
    constexpr int N = kUnit<T>;
    __shared__ float sum_part[2][32];
    __shared__ uint32_t max_part[2][32];
    pdl_trigger();   // the product's prologue may begin
    pdl_wait();
    // this lane's first unit, the others 32 apart
    const int j0 = (int)(threadIdx.x >> 5) * 32 * UNITS + (int)(threadIdx.x & 31), cols = (int)p.cols;
    const float inv_n = 1.0f / (float)cols;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    uint4 x[UNITS], res[UNITS];
    const T *row = nullptr, *rrow = nullptr;
    int n = 0;
    auto load = [&](int64_t r) {
        const int64_t sr = NORM ? r : source_row(p, r);
        n = sr < 0 ? 0 : cols;
        row = static_cast<const T*>(p.X) + (sr < 0 ? 0 : sr * p.ldx);
#pragma unroll
        for (int i = 0; i < UNITS; ++i) x[i] = load_raw<T, ANY>(row, n, j0 + 32 * i);
        if (NORM && p.R) {
            rrow = static_cast<const T*>(p.R) + r * p.ldr;
#pragma unroll
            for (int i = 0; i < UNITS; ++i) res[i] = load_raw<T, ANY>(rrow, n, j0 + 32 * i);
        }
    };
    int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (r < p.rows) load(r);
    int turn = 0;
    for (; r < p.rows; r += step, turn ^= 1) {
        float v[UNITS][N];
        to_words<T, ANY>(row, n, j0, x);
        if (NORM && p.R) to_words<T, ANY>(rrow, n, j0, res);
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            unpack<T>(x[i], v[i]);
            if (NORM && p.R) {
                float w[N];
                unpack<T>(res[i], w);
#pragma unroll
                for (int e = 0; e < N; ++e) v[i][e] += w[e];
                if constexpr (sizeof(T) == 2) unpack<T>(pack<T>(v[i]), v[i]);   // h as it is stored
            }
        }
        float top = 0.0f;   // the largest magnitude that is quantised
        if constexpr (!NORM && sizeof(T) == 2) {
            uint32_t two = 0;
#pragma unroll
            for (int i = 0; i < UNITS; ++i) two = larger_pair(larger_pair(larger_pair(larger_pair(two, x[i].x), x[i].y), x[i].z), x[i].w);
            top = __uint_as_float(max(two << 16, two & 0xFFFF0000u));
        }
        if (r + step < p.rows) load(r + step);
        if constexpr (NORM) {
            auto squares = [&](float f) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < UNITS; ++i)
#pragma unroll
                    for (int e = 0; e < N; ++e) s = fmaf(v[i][e] * f, v[i][e] * f, s);
                return s;
            };
            const float sum = row_sum(squares(1.0f), sum_part[turn]);
            const float rstd = rstd_of(sum, inv_n, p.eps, [&](float f) {
                if (blockDim.x > 32) __syncthreads();
                return row_sum(squares(f), sum_part[turn]);
            });
            if (threadIdx.x == 0) p.rstd[r] = rstd;
            if (p.R) {   // (H may be X or R: all of the row's threads have read it by now)
                T* h = static_cast<T*>(p.H) + r * p.ldh;
                uint4 w[UNITS];
#pragma unroll
                for (int i = 0; i < UNITS; ++i) w[i] = pack<T>(v[i]);
                store_units<T, ANY>(h, cols, j0, w);
            }
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                float g[N];
                load_gain<N, ANY>(p.gain, cols, (j0 + 32 * i) * N, g);
#pragma unroll
                for (int e = 0; e < N; ++e) v[i][e] = v[i][e] * rstd * g[e];
            }
        }
        if constexpr (NORM || sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
#pragma unroll
                for (int e = 0; e < N; ++e) top = larger(top, v[i][e]);
        }
        const uint32_t m = row_max(__float_as_uint(top), max_part[turn]);
        const bool bad = m >= 0x7F800000u;
        const float s = scale_of(m);
        if (threadIdx.x == 0) {
            p.scales[r] = s;
            if (bad) set_status(p.status, GPTQ_ERR_NONFINITE);
        }
        const Step t = step_of(s);
        int8_t* y = p.codes + r * p.pitch;
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
            if ((j0 + 32 * i) * N < (int)p.pitch) store_codes<N>(y + (j0 + 32 * i) * N, v[i], t);
    }
}

// The same for rows of any length: passes over the row, of which all but the first find it in L2, four units of a thread in
// flight at a time. (The norm's later passes read h, each thread what it wrote itself.) ANY: a warp's units take its columns in
// turn, element by element. 1024 x 40000 bf16 35 us, with single elements in flight 84; 4096 x 28672 81 (4.4 TB/s).
template <typename T, bool NORM, bool ANY>
__global__ void __launch_bounds__(1024) int8_long_rows_kernel(const RowParams p) {
    constexpr int N = kUnit<T>, UNITS = 4;
    __shared__ float sum_part[32];
    __shared__ uint32_t max_part[32];
    pdl_wait();
    const int64_t r = blockIdx.x, sr = NORM ? r : source_row(p, r);
    const T* x = static_cast<const T*>(p.X) + max(sr, (int64_t)0) * p.ldx;
    const uint32_t n = sr < 0 ? 0 : (uint32_t)p.cols, pitch = (uint32_t)p.pitch, units = pitch / N;
    // column e of unit j (some units past the row's end are asked for, whose columns may not have 31 bits)
    auto column = [](uint32_t j, int e) { return ANY ? (j & ~31u) * N + 32 * e + (j & 31) : j * N + e; };
    auto load = [&](const T* row, uint32_t j, float(&v)[N]) {
        if constexpr (ANY) {
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = column(j, e) < n ? load_one(row + column(j, e)) : 0.0f;
        } else {
            unpack<T>(j * N < n ? *reinterpret_cast<const uint4*>(row + j * N) : make_uint4(0, 0, 0, 0), v);
        }
    };
    // f(unit, its columns) for this thread's units of a row
    auto sweep = [&](const T* row, auto f) {
        for (uint32_t j0 = threadIdx.x; j0 < (ANY ? (units + 31) & ~31u : units); j0 += UNITS * 1024) {
            float v[UNITS][N];
#pragma unroll
            for (int u = 0; u < UNITS; ++u) load(row, j0 + 1024 * u, v[u]);
#pragma unroll
            for (int u = 0; u < UNITS; ++u) f(j0 + 1024 * u, v[u]);
        }
    };
    float rstd = 1.0f;
    if constexpr (NORM) {
        const T* res = p.R ? static_cast<const T*>(p.R) + r * p.ldr : nullptr;
        T* h = res ? static_cast<T*>(p.H) + r * p.ldh : nullptr;
        float s = 0.0f;
        sweep(x, [&](uint32_t j, float(&v)[N]) {
            if (res) {
                float d[N];
                load(res, j, d);
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] += d[e];
                const uint4 w = pack<T>(v);
                unpack<T>(w, v);   // h as it is stored
                if constexpr (ANY) {
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (column(j, e) < n) put(h + column(j, e), u, e);
                } else {
                    if (j * N < n) *reinterpret_cast<uint4*>(h + j * N) = w;
                }
            }
#pragma unroll
            for (int e = 0; e < N; ++e) s = fmaf(v[e], v[e], s);
        });
        if (res) x = h;
        const float sum = row_sum(s, sum_part);
        rstd = rstd_of(sum, 1.0f / (float)p.cols, p.eps, [&](float f) {
            __syncthreads();
            float q = 0.0f;
            sweep(x, [&](uint32_t, float(&v)[N]) {
#pragma unroll
                for (int e = 0; e < N; ++e) q = fmaf(v[e] * f, v[e] * f, q);
            });
            return row_sum(q, sum_part);
        });
        if (threadIdx.x == 0) p.rstd[r] = rstd;
    }
    auto scaled = [&](uint32_t j, float(&v)[N]) {   // the values that are quantised
        if constexpr (NORM) {
            float g[N];
            if constexpr (ANY) {
#pragma unroll
                for (int e = 0; e < N; ++e) g[e] = column(j, e) < n ? p.gain[column(j, e)] : 0.0f;
            } else {
                load_gain<N, false>(p.gain, (int)n, (int)min(j * N, n), g);
            }
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = v[e] * rstd * g[e];
        }
    };
    float top = 0.0f;
    sweep(x, [&](uint32_t j, float(&v)[N]) {
        scaled(j, v);
#pragma unroll
        for (int e = 0; e < N; ++e) top = larger(top, v[e]);
    });
    const uint32_t m = row_max(__float_as_uint(top), max_part);
    const bool bad = m >= 0x7F800000u;
    const float s = scale_of(m);
    if (threadIdx.x == 0) {
        p.scales[r] = s;
        if (bad) set_status(p.status, GPTQ_ERR_NONFINITE);
    }
    const Step t = step_of(s);
    int8_t* y = p.codes + r * p.pitch;
    sweep(x, [&](uint32_t j, float(&v)[N]) {
        scaled(j, v);
        if constexpr (ANY) {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (column(j, e) < pitch) y[column(j, e)] = (int8_t)code_of(v[e], t);
        } else {
            if (j < units) store_codes<N>(y + j * N, v, t);
        }
    });
}

// ------------------------------------------------------------------------------------ the inverse
struct BackParams {
    const int8_t* codes;
    const float* scales;
    int64_t rows, cols, pitch;
    void* Y;
    int64_t ldy;
};
constexpr int B_WARPS = 4;   // rows per CTA at a time

// A warp takes UNITS units per lane of a row. Bound by memory: 16384 x 4096 to bf16 31 us (6.5 TB/s), 16384 x 4095 36.
template <typename T, int UNITS, bool ANY>
__global__ void __launch_bounds__(32 * B_WARPS) int8_dequantize_kernel(const BackParams p) {
    constexpr int N = kUnit<T>;
    const int j0 = blockIdx.x * 32 * UNITS + threadIdx.x, cols = (int)p.cols;
    pdl_trigger();
    pdl_wait();
    for (int64_t r = (int64_t)blockIdx.y * B_WARPS + threadIdx.y; r < p.rows; r += (int64_t)gridDim.y * B_WARPS) {
        uint2 w[UNITS];
        uint4 out[UNITS];
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            const int8_t* src = p.codes + r * p.pitch + (j0 + 32 * i) * N;
            w[i] = make_uint2(0, 0);
            if ((j0 + 32 * i) * N < cols) {
                if constexpr (N == 8) w[i] = *reinterpret_cast<const uint2*>(src);
                else w[i].x = *reinterpret_cast<const uint32_t*>(src);
            }
        }
        const float s = p.scales[r];
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            float v[N];
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = (float)(int8_t)((e < 4 ? w[i].x : w[i].y) >> (8 * (e & 3))) * s;
            out[i] = pack<T>(v);
        }
        store_units<T, ANY>(static_cast<T*>(p.Y) + r * p.ldy, cols, j0, out);
    }
}

// ------------------------------------------------------------------------------ the norm's gradient
struct GradParams {
    const void *dY, *H, *dH;   // dH: the gradient that reaches h past the norm, or null
    const float *gain, *rstd;
    int64_t rows, cols, lddy, ldh, lddh;
    void* dX;
    int64_t lddx;
    float* part;               // [ctas][cols] sums of dy u over each CTA's rows
    int64_t per;               // rows per CTA
};

// the sum over the warps of one of a CTA's groups of threads, which has `warps` of them and a barrier of its own
__device__ __forceinline__ float group_sum(float v, float* part, int warps, int barrier) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;   // (threadIdx.x is the thread's number within its group)
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * warps) : "memory");
    v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A CTA takes a contiguous share of the rows, each of its blockDim.y groups of threads every so many of them, and a thread
// the same UNITS units of each: dgain's sums over the rows stay in its registers, and the groups' are added at the
// end. Rows are read once, the next one's loads under way (AHEAD) while this one is reduced and written. Wider rows leave no
// registers for that, and have the sums in shared memory (4096 x 14336 bf16 121 us, 3.9 TB/s, in registers 131; with loads ahead 147): there each
// row's loads start behind the last row's stores, which costs 1.4 to 1.75 times the time of the bytes.
// Narrower rows are bound by memory: 16384 x 4096 bf16 86 us (6.2 TB/s), fp32 163 (6.6), both with the sum over the CTAs (4 us). Without the
// loads ahead and with the gain read for every row it took 199. Rows at odd addresses: 16384 x 4095 bf16 183, fp32 203.
template <typename T, int UNITS, bool ANY, int MOST>
__global__ void __launch_bounds__(MOST, 1) int8_norm_grad_kernel(const GradParams p) {
    constexpr int N = kUnit<T>;
    constexpr bool AHEAD = UNITS <= 2;   // (and the gain and the sums stay in registers)
    constexpr bool LATE = MOST > 512;    // 64 registers: dH is read once the others are used (4096 x 16384 fp32 216 us, else 245)
    extern __shared__ float4 shared_sums[];   // AHEAD: [groups][columns] floats, where there are several groups; else [UNITS N / 4][threads]
    float* sums = reinterpret_cast<float*>(shared_sums);
    const int tid = threadIdx.x;
    __shared__ float part[2][32];
    pdl_trigger();
    pdl_wait();
    const int64_t first = (int64_t)blockIdx.x * p.per, last = min(first + p.per, p.rows);
    const int j0 = (int)(threadIdx.x >> 5) * 32 * UNITS + (int)(threadIdx.x & 31), step = blockDim.y, cols = (int)p.cols;
    const int warps = blockDim.x >> 5, group = threadIdx.y;
    const float inv_n = 1.0f / (float)cols;
    float gain[AHEAD ? UNITS : 1][N];
    if (AHEAD) {
#pragma unroll
        for (int i = 0; i < UNITS; ++i) load_gain<N, ANY>(p.gain, cols, (j0 + 32 * i) * N, gain[i]);
    }
    float acc[AHEAD ? UNITS : 1][N] = {};
    if (!AHEAD)
        for (int i = 0; i < UNITS * N / 4; ++i) shared_sums[i * blockDim.x + tid] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    uint4 dy[UNITS], h[UNITS], dh[UNITS];
    const T *ry = nullptr, *rh = nullptr, *rd = nullptr;
    float rstd = 0.0f;
    auto load = [&](int64_t r) {
        ry = static_cast<const T*>(p.dY) + r * p.lddy;
        rh = static_cast<const T*>(p.H) + r * p.ldh;
        rd = static_cast<const T*>(p.dH) + r * p.lddh;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            dy[i] = load_raw<T, ANY>(ry, cols, j0 + 32 * i);
            h[i] = load_raw<T, ANY>(rh, cols, j0 + 32 * i);
            if (!LATE && p.dH) dh[i] = load_raw<T, ANY>(rd, cols, j0 + 32 * i);
        }
        rstd = p.rstd[r];
    };
    int64_t r = first + group;
    if (AHEAD && r < last) load(r);
    int turn = 0;
    for (; r < last; r += step, turn ^= 1) {
        if (!AHEAD) load(r);
        // what is needed behind the barrier stays as the words it was read as: dX may be written over any input
        uint4 yw[UNITS], hw[UNITS], dw[UNITS];
        const float rs = rstd;
        to_words<T, ANY>(ry, cols, j0, dy);
        to_words<T, ANY>(rh, cols, j0, h);
        if (!LATE && p.dH) to_words<T, ANY>(rd, cols, j0, dh);
#pragma unroll
        for (int i = 0; i < UNITS; ++i) yw[i] = dy[i], hw[i] = h[i], dw[i] = dh[i];
        if (AHEAD && r + step < last) load(r + step);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            float u[N], v[N];
            float(&g)[N] = gain[AHEAD ? i : 0];
            if (!AHEAD) load_gain<N, ANY>(p.gain, cols, (j0 + 32 * i) * N, g);
            unpack<T>(hw[i], u);
            unpack<T>(yw[i], v);
            float(&a)[N] = acc[AHEAD ? i : 0];
            if (!AHEAD) {
#pragma unroll
                for (int e = 0; e < N; e += 4) {
                    const float4 w = shared_sums[(i * N / 4 + e / 4) * blockDim.x + tid];
                    a[e] = w.x, a[e + 1] = w.y, a[e + 2] = w.z, a[e + 3] = w.w;
                }
            }
#pragma unroll
            for (int e = 0; e < N; ++e) {
                u[e] *= rs;
                a[e] = fmaf(v[e], u[e], a[e]);
                dot = fmaf(u[e], v[e] * g[e], dot);
            }
            if (!AHEAD) {
#pragma unroll
                for (int e = 0; e < N; e += 4)
                    shared_sums[(i * N / 4 + e / 4) * blockDim.x + tid] = make_float4(a[e], a[e + 1], a[e + 2], a[e + 3]);
            }
        }
        if (LATE && p.dH) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i) dw[i] = load_raw<T, ANY>(rd, cols, j0 + 32 * i);
            to_words<T, ANY>(rd, cols, j0, dw);
        }
        const float k = group_sum(dot, part[turn] + group * warps, warps, 1 + group) * inv_n * rs;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            float u[N], v[N], d[N] = {};
            float(&g)[N] = gain[AHEAD ? i : 0];
            if (!AHEAD) load_gain<N, ANY>(p.gain, cols, (j0 + 32 * i) * N, g);
            unpack<T>(hw[i], u);
            unpack<T>(yw[i], v);
            if (p.dH) unpack<T>(dw[i], d);
#pragma unroll
            for (int e = 0; e < N; ++e) d[e] = fmaf(rs, fmaf(-u[e], k, v[e] * g[e]), d[e]);
            dw[i] = pack<T>(d);
        }
        store_units<T, ANY>(static_cast<T*>(p.dX) + r * p.lddx, cols, j0, dw);
    }
    float* out = p.part + blockIdx.x * p.cols;
    // each group leaves its sums in shared memory, and all add them up; rows at odd addresses are faster where the first group adds
    // the others' to its own (16384 x 4095 fp32 203 us, else 231; 16384 x 4096 bf16 90 so and 86)
    const int groups = blockDim.y;
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int c = (j0 + 32 * i) * N + e;
                if (AHEAD) {
                    if (c < cols) f(c, acc[i][e]);
                } else if (c < cols) {
                    f(c, sums[((i * N / 4 + e / 4) * blockDim.x + tid) * 4 + e % 4]);
                }
            }
    };
    if (AHEAD && groups > 1) {
        each([&](int c, float& v) { sums[group * cols + c] = v; });
        __syncthreads();
        if (ANY) {
            if (group > 0) return;
            each([&](int c, float& v) {
                for (int g = 1; g < groups; ++g) v += sums[g * cols + c];
            });
        } else {
            for (int c = group * blockDim.x + threadIdx.x; c < cols; c += groups * blockDim.x) {
                float s = 0.0f;
                for (int g = 0; g < groups; ++g) s += sums[g * cols + c];
                out[c] = s;
            }
            return;
        }
    }
    each([&](int c, float& v) { out[c] = v; });
}

// Rows of any length: the row's mean is taken in one pass over it, and its gradient in a second one, which finds
// the row in L2; a thread's share of dgain is added to the CTA's own row of `part` (each element by one
// thread, row after row).
template <typename T>
__global__ void __launch_bounds__(1024) int8_norm_grad_long_kernel(const GradParams p) {
    __shared__ float part[2][32];
    pdl_wait();
    const int64_t first = (int64_t)blockIdx.x * p.per, last = min(first + p.per, p.rows);
    const float inv_n = 1.0f / (float)p.cols;
    float* sums = p.part + blockIdx.x * p.cols;
    for (int64_t r = first; r < last; ++r) {
        const T* dy = static_cast<const T*>(p.dY) + r * p.lddy;
        const T* h = static_cast<const T*>(p.H) + r * p.ldh;
        const float rstd = p.rstd[r];
        float dot = 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) dot = fmaf(load_one(h + c) * rstd, load_one(dy + c) * p.gain[c], dot);
        dot = row_sum(dot, part[(r - first) & 1]) * inv_n;
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            const float u = load_one(h + c) * rstd, v = load_one(dy + c);
            const float d = p.dH ? load_one(static_cast<const T*>(p.dH) + r * p.lddh + c) : 0.0f;
            sums[c] = fmaf(v, u, r == first ? 0.0f : sums[c]);
            store_one(static_cast<T*>(p.dX) + r * p.lddx + c, fmaf(rstd, v * p.gain[c] - u * dot, d));
        }
    }
}

// out[c] = sum over the CTAs of part[cta][c], in a fixed order: 32 columns x 32 shares of the CTAs
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int ctas, int64_t cols, float* out) {
    __shared__ float sums[32][33];
    pdl_wait();
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 4
        for (int k = threadIdx.y; k < ctas; k += 32) s += part[k * cols + c];
    }
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = sums[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int64_t mine = (int64_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && mine < cols) out[mine] = s;
}

// ------------------------------------------------------------------------------------- host side
bool bad_dtype(int t) { return t != GPTQ_F32 && t != GPTQ_BF16; }
constexpr int64_t kMaxDim = (1ll << 31) - 4096;   // (a warp's last unit is up to 1024 columns past the row's end)
struct Rows {
    const void* p;
    int64_t ld;
};
// whether all these rows of `cols` elements are whole aligned granules of 16 bytes
bool whole_granules(int64_t es, int64_t cols, std::initializer_list<Rows> rows) {
    uint64_t all = (uint64_t)(cols * es);
    for (const Rows& r : rows)
        if (r.p) all |= reinterpret_cast<uintptr_t>(r.p) | (uint64_t)(r.ld * es);
    return all % 16 == 0;
}

template <int V>
using Const = std::integral_constant<int, V>;

// Calls f(T(), units per thread, whether rows start anywhere, the most threads) after setting the threads that a row of
// `units` units takes: one or two units per thread where a warp can take it so, FEW (2 or 4) with up to 512 threads, then 4.
// Only rows of fp32, whose units are half as many columns, fit the registers of 1024 threads. False: the row fits none.
template <typename T, int FEW, typename F>
bool with_units(bool any, int64_t units, unsigned* threads, F f) {
    auto go = [&](auto u, auto most) {
        const int64_t n = ceil_div(ceil_div(units, decltype(u)::value), 32) * 32;
        *threads = (unsigned)std::max<int64_t>(n, 32);
        any ? f(T(), u, Const<1>(), most) : f(T(), u, Const<0>(), most);
        return true;
    };
    if (units <= 32) return go(Const<1>(), Const<512>());
    if (units <= 64 || (FEW == 2 && units <= 2 * 512)) return go(Const<2>(), Const<512>());
    if (units <= 4 * 512) return go(Const<4>(), Const<512>());
    if constexpr (sizeof(T) == 4)
        if (units <= 4 * 1024) return go(Const<4>(), Const<1024>());
    return false;
}

// CTAs of a kernel that an SM holds at once, asked once for each number of threads
template <typename K>
int ctas_per_sm(K kern, unsigned threads, std::atomic<int> (&known)[33]) {
    std::atomic<int>& k = known[threads / 32];
    int n = k.load(std::memory_order_relaxed);
    if (n) return n;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, (int)threads, 0) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        return 1;
    }
    k.store(n, std::memory_order_relaxed);
    return n;
}

template <bool NORM>
int launch_rows(const RowParams& p, int dtype, bool any, int id, cudaStream_t s) {
    unsigned threads = 0;
    cudaError_t e = cudaSuccess;
    const int64_t units = p.pitch / (dtype == GPTQ_BF16 ? 8 : 4);
    auto go = [&](auto t, auto u, auto a, auto m) {
        auto kern = int8_rows_kernel<decltype(t), decltype(u)::value, NORM, decltype(a)::value != 0, decltype(m)::value>;
        static std::atomic<int> known[33];
        const unsigned rows = threads == 32 ? 8 : 1;   // a warp takes a whole row where it can
        const int64_t most = (int64_t)device_sm_count() * ctas_per_sm(kern, threads * rows, known);
        const unsigned ctas = (unsigned)std::min<int64_t>(ceil_div(p.rows, rows), most);
        GPTQ_LAUNCH(id, s, e = launch_pdl(kern, dim3(ctas), dim3(threads, rows), 0, s, p));
    };
    const bool fits = dtype == GPTQ_BF16 ? with_units<__nv_bfloat16, 4>(any, units, &threads, go)
                                         : with_units<float, 4>(any, units, &threads, go);
    if (!fits) {
        auto lengthy = [&](auto t, auto a) {
            auto kern = int8_long_rows_kernel<decltype(t), NORM, decltype(a)::value != 0>;
            GPTQ_LAUNCH(id, s, e = launch_pdl(kern, dim3((unsigned)p.rows), dim3(1024), 0, s, p));
        };
        if (dtype == GPTQ_BF16) any ? lengthy(__nv_bfloat16(), Const<1>()) : lengthy(__nv_bfloat16(), Const<0>());
        else any ? lengthy(float(), Const<1>()) : lengthy(float(), Const<0>());
    }
    GPTQ_CUDA_TRY(e);
    return GPTQ_OK;
}

// The most CTAs of the gradient, each with a row of partial sums
int64_t grad_ctas(int64_t rows) { return std::min<int64_t>(rows, 2 * kSMs); }

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" int64_t gptq_int8_pitch(int64_t cols) { return int8_pitch(cols); }

extern "C" int gptq_int8_quantize(const void* X, int dtype, int64_t src_rows, int64_t cols, int64_t ldx, const int32_t* index,
                                  int64_t per, int64_t rows, int8_t* codes, float* scales, void* stream) {
    if (src_rows < 0 || cols < 0 || rows < 0 || rows > kMaxDim || src_rows > kMaxDim || cols > kMaxDim || per < 1 || bad_dtype(dtype))
        return GPTQ_ERR_INVALID_ARG;
    if (rows == 0) return GPTQ_OK;   // (an empty index has no address)
    if ((!index && rows != src_rows) || !scales || (cols > 0 && ((src_rows > 0 && !X) || !codes || ldx < cols || reinterpret_cast<uintptr_t>(codes) % 16 != 0)))
        return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    RowParams p{};
    p.X = X;
    p.rows = rows;
    p.cols = cols;
    p.ldx = ldx;
    p.src_rows = src_rows;
    p.index = index;
    p.per = per;
    p.codes = codes;
    p.pitch = int8_pitch(cols);
    p.scales = scales;
    p.status = st.word;
    const int rc = launch_rows<false>(p, dtype, !whole_granules(dtype == GPTQ_BF16 ? 2 : 4, cols, {{X, ldx}}), K_INT8_QUANT, s);
    return rc != GPTQ_OK ? rc : st.finish(s);
}

extern "C" int gptq_int8_rms_norm(const void* X, int64_t ldx, const void* residual, int64_t ldr, int dtype, int64_t rows, int64_t cols,
                                  const float* gain, float eps, int8_t* codes, float* scales, void* H, int64_t ldh, float* rstd,
                                  void* stream) {
    if (rows < 0 || cols < 1 || rows > kMaxDim || cols > kMaxDim || bad_dtype(dtype) || !(eps > 0.0f) || eps > 3.0e38f)
        return GPTQ_ERR_INVALID_ARG;
    if (rows == 0) return GPTQ_OK;
    if (!X || !gain || !codes || !scales || !rstd || ldx < cols || reinterpret_cast<uintptr_t>(codes) % 16 != 0 ||
        (residual && (!H || ldr < cols || ldh < cols)))
        return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CallStatus st;
    GPTQ_CUDA_TRY(st.begin(s));
    RowParams p{};
    p.X = X;
    p.R = residual;
    p.gain = gain;
    p.eps = eps;
    p.rows = rows;
    p.cols = cols;
    p.ldx = ldx;
    p.ldr = ldr;
    p.codes = codes;
    p.pitch = int8_pitch(cols);
    p.scales = scales;
    p.H = H;
    p.ldh = ldh;
    p.rstd = rstd;
    p.status = st.word;
    const bool any =
        !whole_granules(dtype == GPTQ_BF16 ? 2 : 4, cols, {{X, ldx}, {residual, ldr}, {residual ? H : nullptr, ldh}, {gain, 0}});
    const int rc = launch_rows<true>(p, dtype, any, K_INT8_NORM, s);
    return rc != GPTQ_OK ? rc : st.finish(s);
}

extern "C" size_t gptq_int8_rms_norm_grad_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1 || rows > kMaxDim || cols > kMaxDim) return 0;
    return (size_t)(grad_ctas(rows) * cols * 4);
}

extern "C" int gptq_int8_rms_norm_grad(const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* dH, int64_t lddh, int dtype,
                                       int64_t rows, int64_t cols, const float* gain, const float* rstd, void* dX, int64_t lddx,
                                       float* dgain, void* ws, size_t ws_bytes, void* stream) {
    if (rows < 0 || cols < 1 || rows > kMaxDim || cols > kMaxDim || bad_dtype(dtype) || !dgain) return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        GPTQ_CUDA_TRY(cudaMemsetAsync(dgain, 0, (size_t)cols * 4, s));
        return GPTQ_OK;
    }
    if (!dY || !H || !gain || !rstd || !dX || lddy < cols || ldh < cols || lddx < cols || (dH && lddh < cols)) return GPTQ_ERR_INVALID_ARG;
    if (!ws || ws_bytes < gptq_int8_rms_norm_grad_workspace_bytes(rows, cols)) return GPTQ_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) % 4 != 0) return GPTQ_ERR_INVALID_ARG;
    const int64_t es = dtype == GPTQ_BF16 ? 2 : 4, units = ceil_div(cols, 16 / es);
    const bool any = !whole_granules(es, cols, {{dY, lddy}, {H, ldh}, {dH, lddh}, {dX, lddx}, {gain, 0}});
    GradParams p{dY, H, dH, gain, rstd, rows, cols, lddy, ldh, lddh, dX, lddx, static_cast<float*>(ws), 0};
    unsigned threads = 0, ctas = 0;
    cudaError_t e = cudaSuccess;
    auto share = [&](int64_t most) {   // each CTA's rows, and the CTAs
        p.per = ceil_div(rows, std::min(most, grad_ctas(rows)));
        ctas = (unsigned)ceil_div(rows, p.per);
    };
    auto go = [&](auto t, auto u, auto a, auto m) {
        auto kern = int8_norm_grad_kernel<decltype(t), decltype(u)::value, decltype(a)::value != 0, decltype(m)::value>;
        static std::atomic<int> known[33];
        // groups of threads up to 512, each with a barrier (15 of them besides the CTA's), none idle
        unsigned groups = std::max(1u, std::min(15u, 512 / threads));
        // (one row, or two at a time, are one CTA's, whose sums are dgain: 1 x 4096 bf16 3.6 us, with a launch to add them up 5.5)
        share(rows <= std::min(groups, 2u) ? 1 : (int64_t)device_sm_count() * ctas_per_sm(kern, threads * groups, known));
        if (ctas == 1) p.part = dgain;
        groups = (unsigned)std::min<int64_t>(groups, p.per);
        // (at most 512 threads of 16 columns, 32 KB; 4 units: up to 16384 columns, 64 KB)
        constexpr int kUnits = decltype(u)::value;
        const size_t smem = kUnits > 2 ? sizeof(float) * threads * kUnits * kUnit<decltype(t)> : groups > 1 ? sizeof(float) * groups * cols : 0;
        if (kUnits > 2 && (e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024)) != cudaSuccess) return;
        GPTQ_LAUNCH(K_INT8_GRAD, s, e = launch_pdl(kern, dim3(ctas), dim3(threads, groups), smem, s, p));
    };
    const bool fits = dtype == GPTQ_BF16 ? with_units<__nv_bfloat16, 2>(any, units, &threads, go)
                                         : with_units<float, 2>(any, units, &threads, go);
    if (!fits) {
        share(grad_ctas(rows));
        auto kern = dtype == GPTQ_BF16 ? int8_norm_grad_long_kernel<__nv_bfloat16> : int8_norm_grad_long_kernel<float>;
        GPTQ_LAUNCH(K_INT8_GRAD, s, e = launch_pdl(kern, dim3(ctas), dim3(1024), 0, s, p));
    }
    GPTQ_CUDA_TRY(e);
    if (p.part == dgain) return GPTQ_OK;
    GPTQ_LAUNCH(K_INT8_GRAD, s, e = launch_pdl(column_sum_kernel, dim3((unsigned)ceil_div(cols, 32)), dim3(32, 32), 0, s,
                                               (const float*)p.part, (int)ctas, cols, dgain));
    GPTQ_CUDA_TRY(e);
    return GPTQ_OK;
}

extern "C" int gptq_int8_dequantize(const int8_t* codes, const float* scales, int64_t rows, int64_t cols, void* Y, int dtype,
                                    int64_t ldy, void* stream) {
    if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim || bad_dtype(dtype)) return GPTQ_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return GPTQ_OK;
    if (!codes || !scales || !Y || ldy < cols || reinterpret_cast<uintptr_t>(codes) % 16 != 0) return GPTQ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const BackParams p{codes, scales, rows, cols, int8_pitch(cols), Y, ldy};
    const bool any = !whole_granules(dtype == GPTQ_BF16 ? 2 : 4, cols, {{Y, ldy}});
    const int64_t units = ceil_div(cols, dtype == GPTQ_BF16 ? 8 : 4);
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kern, int per) {
        const dim3 grid((unsigned)ceil_div(units, 32 * per), (unsigned)std::min<int64_t>(ceil_div(rows, B_WARPS), 65535));
        GPTQ_LAUNCH(K_INT8_DEQUANT, s, e = launch_pdl(kern, grid, dim3(32, B_WARPS), 0, s, p));
    };
    auto typed = [&](auto t) {
        using T = decltype(t);
        if (units <= 32) any ? go(int8_dequantize_kernel<T, 1, true>, 1) : go(int8_dequantize_kernel<T, 1, false>, 1);
        else any ? go(int8_dequantize_kernel<T, 4, true>, 4) : go(int8_dequantize_kernel<T, 4, false>, 4);
    };
    if (dtype == GPTQ_BF16) typed(__nv_bfloat16());
    else typed(float());
    GPTQ_CUDA_TRY(e);
    return GPTQ_OK;
}

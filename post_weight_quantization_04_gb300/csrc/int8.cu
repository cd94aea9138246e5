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
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "int8.cuh"

namespace gptq {

namespace {

// --------------------------------------------------------------------- sums over a row's threads
// A row has blockDim.x threads (whole warps); a CTA has blockDim.y rows, more than one only where a
// warp takes a whole row. The sum is the same in all its threads. `part` [32]: one slot per warp,
// another one each time it is used between two barriers.
template <typename V, typename Op>
__device__ __forceinline__ V row_reduce(V v, V* part, Op op) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (blockDim.x == 32) return v;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[(threadIdx.x & 31) < warps ? threadIdx.x & 31 : 0];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const V w = __shfl_down_sync(0xffffffffu, v, o);
        if ((int)(threadIdx.x & 31) + o < warps) v = op(v, w);
    }
    return __shfl_sync(0xffffffffu, v, 0);
}

struct Add {
    __device__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};

// the gain of N columns (16-byte aligned where N is 4 or 8)
template <int N>
__device__ __forceinline__ void load_gain(const float* p, float (&g)[N]) {
    if constexpr (N < 4) {
#pragma unroll
        for (int e = 0; e < N; ++e) g[e] = p[e];
    } else {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + e);
            g[e] = v.x, g[e + 1] = v.y, g[e + 2] = v.z, g[e + 3] = v.w;
        }
    }
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

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
    t.inv = s > 0.0f ? 1.0f / t.d : 0.0f;   // (a NaN scale has codes of zero)
    return t;
}
__device__ __forceinline__ uint32_t code_of(float x, const Step& t) {
    if (!t.usual) x *= t.f;
    float q = x * t.inv;
    q = fmaf(fmaf(-q, t.d, x), t.inv, q);
    // (a subnormal scale is rounded, up to half of it, so a quotient may be past 127)
    if (!t.usual) q = t.inv > 0.0f ? fminf(fmaxf(q, -127.0f), 127.0f) : 0.0f;
    return __float_as_uint(q + 12582912.0f) & 0xFFu;
}

template <int N>
__device__ __forceinline__ void store_codes(int8_t* y, const float (&v)[N], const Step& t) {
    uint32_t u[N];
#pragma unroll
    for (int e = 0; e < N; ++e) u[e] = code_of(v[e], t);
    if constexpr (N == 1) {
        *y = (int8_t)u[0];
    } else if constexpr (N == 2) {
        *reinterpret_cast<uint16_t*>(y) = (uint16_t)(u[0] | u[1] << 8);
    } else {
        uint32_t w[N / 4];
#pragma unroll
        for (int e = 0; e < N / 4; ++e)
            w[e] = __byte_perm(__byte_perm(u[4 * e], u[4 * e + 1], 0x0040), __byte_perm(u[4 * e + 2], u[4 * e + 3], 0x0040), 0x5410);
        if constexpr (N == 4) *reinterpret_cast<uint32_t*>(y) = w[0];
        else *reinterpret_cast<uint2*>(y) = make_uint2(w[0], w[1]);
    }
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
// taken again of scaled values (a row apart, so nothing is lost elsewhere)
template <typename F>
__device__ __forceinline__ float rstd_of(float sum, float n, float eps, F again) {
    const float v = sum / n + eps;
    if (v >= 0x1p-80f && v <= 0x1.fffffep127f) return rsqrtf(v);
    const float f = v < 1.0f ? 0x1p100f : 0x1p-80f;
    return rsqrtf(again(f) / n + eps * f * f) * f;
}

// One row in the registers of its threads, UNITS units of N columns each. The row is read once and
// everything written once.
template <typename T, int N, int UNITS, bool NORM>
__global__ void __launch_bounds__(1024) int8_rows_kernel(const RowParams p) {
    __shared__ float sum_part[32];
    __shared__ uint32_t max_part[32];
    const int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    pdl_trigger();   // the product's prologue may begin
    pdl_wait();
    if (r >= p.rows) return;   // (a whole warp, of a CTA without barriers)
    int64_t sr = r;
    if (!NORM && p.index) {
        const int k = p.index[r];
        sr = k < 0 ? -1 : k / p.per;
        if (sr >= p.src_rows) {
            sr = -1;
            set_status(p.status, GPTQ_ERR_INVALID_ARG);
        }
    }
    float v[UNITS][N];
    const T* x = static_cast<const T*>(p.X) + max(sr, (int64_t)0) * p.ldx;
    const int64_t n = sr < 0 ? 0 : p.cols;
    int64_t c = (int64_t)threadIdx.x * N;
    const int64_t step = (int64_t)blockDim.x * N;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        if (c + i * step < n) {
            load_unit<T, N>(x + c + i * step, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) v[i][e] = 0.0f;
        }
    }
    if constexpr (NORM) {
        if (p.R) {
            const T* res = static_cast<const T*>(p.R) + r * p.ldr;
            T* h = static_cast<T*>(p.H) + r * p.ldh;
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                if (c + i * step < n) {
                    float w[N];
                    load_unit<T, N>(res + c + i * step, w);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        v[i][e] += w[e];
                        if constexpr (sizeof(T) == 2) v[i][e] = __bfloat162float(__float2bfloat16_rn(v[i][e]));
                    }
                    store_unit<T, N>(h + c + i * step, v[i]);
                }
            }
        }
        auto squares = [&](float f) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
#pragma unroll
                for (int e = 0; e < N; ++e) s = fmaf(v[i][e] * f, v[i][e] * f, s);
            return s;
        };
        const float sum = row_reduce(squares(1.0f), sum_part, Add());
        const float rstd = rstd_of(sum, (float)p.cols, p.eps, [&](float f) {
            if (blockDim.x > 32) __syncthreads();
            return row_reduce(squares(f), sum_part, Add());
        });
        if (threadIdx.x == 0) p.rstd[r] = rstd;
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
            if (c + i * step < n) {
                float g[N];
                load_gain<N>(p.gain + c + i * step, g);
#pragma unroll
                for (int e = 0; e < N; ++e) v[i][e] = v[i][e] * rstd * g[e];
            }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) m = max(m, magnitude(v[i][e]));
    m = row_reduce(m, max_part, Max());
    const bool bad = m >= 0x7F800000u;
    const float s = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float(m) / 127.0f;
    if (threadIdx.x == 0) {
        p.scales[r] = s;
        if (bad) set_status(p.status, GPTQ_ERR_NONFINITE);
    }
    const Step t = step_of(s);
    int8_t* y = p.codes + r * p.pitch;
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
        if (c + i * step < p.cols) store_codes<N>(y + c + i * step, v[i], t);
    const int64_t pad = p.cols + threadIdx.x;
    if (pad < p.pitch) y[pad] = 0;
}

// The same for rows of any length: passes over the row, of which all but the first find it in L2. (The norm's
// later passes read h, each thread what it wrote itself.)
template <typename T, bool NORM>
__global__ void __launch_bounds__(1024) int8_long_rows_kernel(const RowParams p) {
    __shared__ float sum_part[32];
    __shared__ uint32_t max_part[32];
    pdl_wait();
    const int64_t r = blockIdx.x;
    int64_t sr = r;
    if (!NORM && p.index) {
        const int k = p.index[r];
        sr = k < 0 ? -1 : k / p.per;
        if (sr >= p.src_rows) {
            sr = -1;
            set_status(p.status, GPTQ_ERR_INVALID_ARG);
        }
    }
    const T* x = static_cast<const T*>(p.X) + max(sr, (int64_t)0) * p.ldx;
    const int64_t n = sr < 0 ? 0 : p.cols;
    float rstd = 1.0f;
    if constexpr (NORM) {
        const T* res = p.R ? static_cast<const T*>(p.R) + r * p.ldr : nullptr;
        T* h = res ? static_cast<T*>(p.H) + r * p.ldh : nullptr;
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < n; c += blockDim.x) {
            float a[1], b[1];
            load_unit<T, 1>(x + c, a);
            if (res) {
                load_unit<T, 1>(res + c, b);
                a[0] += b[0];
                if constexpr (sizeof(T) == 2) a[0] = __bfloat162float(__float2bfloat16_rn(a[0]));
                store_unit<T, 1>(h + c, a);
            }
            s = fmaf(a[0], a[0], s);
        }
        if (res) x = h;
        const float sum = row_reduce(s, sum_part, Add());
        rstd = rstd_of(sum, (float)p.cols, p.eps, [&](float f) {
            __syncthreads();
            float q = 0.0f;
            for (int64_t c = threadIdx.x; c < n; c += blockDim.x) {
                float a[1];
                load_unit<T, 1>(x + c, a);
                q = fmaf(a[0] * f, a[0] * f, q);
            }
            return row_reduce(q, sum_part, Add());
        });
        if (threadIdx.x == 0) p.rstd[r] = rstd;
    }
    auto value = [&](int64_t c, float (&a)[1]) {
        load_unit<T, 1>(x + c, a);
        if constexpr (NORM) a[0] = a[0] * rstd * p.gain[c];
    };
    uint32_t m = 0;
    for (int64_t c = threadIdx.x; c < n; c += blockDim.x) {
        float a[1];
        value(c, a);
        m = max(m, magnitude(a[0]));
    }
    m = row_reduce(m, max_part, Max());
    const bool bad = m >= 0x7F800000u;
    const float s = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float(m) / 127.0f;
    if (threadIdx.x == 0) {
        p.scales[r] = s;
        if (bad) set_status(p.status, GPTQ_ERR_NONFINITE);
    }
    const Step t = step_of(s);
    int8_t* y = p.codes + r * p.pitch;
    for (int64_t c = threadIdx.x; c < p.pitch; c += blockDim.x) {
        float a[1] = {0.0f};
        if (c < n) value(c, a);
        store_codes<1>(y + c, a, t);
    }
}

// ------------------------------------------------------------------------------------ the inverse
struct BackParams {
    const int8_t* codes;
    const float* scales;
    int64_t rows, cols, pitch;
    void* Y;
    int64_t ldy;
};
constexpr int B_THREADS = 128, B_ROWS = 4;   // rows in flight per thread

template <typename T, int N>
__global__ void __launch_bounds__(B_THREADS) int8_dequantize_kernel(const BackParams p) {
    const int64_t c = ((int64_t)blockIdx.x * B_THREADS + threadIdx.x) * N;
    if (c >= p.cols) return;
    pdl_wait();
    for (int64_t r0 = (int64_t)blockIdx.y * B_ROWS; r0 < p.rows; r0 += (int64_t)gridDim.y * B_ROWS) {
        uint32_t w[B_ROWS][N <= 4 ? 1 : 2];
        float s[B_ROWS];
#pragma unroll
        for (int i = 0; i < B_ROWS; ++i) {
            const int64_t r = min(r0 + i, p.rows - 1);
            const int8_t* src = p.codes + r * p.pitch + c;
            if constexpr (N == 8) {
                const uint2 u = *reinterpret_cast<const uint2*>(src);
                w[i][0] = u.x, w[i][1] = u.y;
            } else if constexpr (N == 4) {
                w[i][0] = *reinterpret_cast<const uint32_t*>(src);
            } else {
                w[i][0] = *reinterpret_cast<const uint8_t*>(src);
            }
            s[i] = p.scales[r];
        }
#pragma unroll
        for (int i = 0; i < B_ROWS; ++i) {
            if (r0 + i >= p.rows) break;
            float v[N];
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = (float)(int8_t)(w[i][e >> 2] >> (8 * (e & 3))) * s[i];
            store_unit<T, N>(static_cast<T*>(p.Y) + (r0 + i) * p.ldy + c, v);
        }
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

// A CTA takes a contiguous share of the rows, a thread the same UNITS units of N columns of each: dgain's
// sums over the rows stay in its registers. Rows are read once.
template <typename T, int N, int UNITS>
__global__ void __launch_bounds__(1024) int8_norm_grad_kernel(const GradParams p) {
    __shared__ float part[2][32];
    pdl_wait();
    const int64_t first = (int64_t)blockIdx.x * p.per, last = min(first + p.per, p.rows);
    const int64_t c = (int64_t)threadIdx.x * N, step = (int64_t)blockDim.x * N;
    float acc[UNITS][N] = {};
    const float inv_n = 1.0f / (float)p.cols;
    for (int64_t r = first; r < last; ++r) {
        const T* dy = static_cast<const T*>(p.dY) + r * p.lddy + c;
        const T* h = static_cast<const T*>(p.H) + r * p.ldh + c;
        const float rstd = p.rstd[r];
        float u[UNITS][N], v[UNITS][N], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            if (c + i * step < p.cols) {
                load_unit<T, N>(h + i * step, u[i]);
                load_unit<T, N>(dy + i * step, v[i]);
                float g[N];
                load_gain<N>(p.gain + c + i * step, g);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    u[i][e] *= rstd;
                    acc[i][e] = fmaf(v[i][e], u[i][e], acc[i][e]);
                    v[i][e] *= g[e];
                    dot = fmaf(u[i][e], v[i][e], dot);
                }
            }
        }
        dot = row_reduce(dot, part[(r - first) & 1], Add()) * inv_n;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            if (c + i * step < p.cols) {
                float d[N];
                if (p.dH) load_unit<T, N>(static_cast<const T*>(p.dH) + r * p.lddh + c + i * step, d);
#pragma unroll
                for (int e = 0; e < N; ++e) d[e] = fmaf(rstd, v[i][e] - u[i][e] * dot, p.dH ? d[e] : 0.0f);
                store_unit<T, N>(static_cast<T*>(p.dX) + r * p.lddx + c + i * step, d);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (c + i * step < p.cols) p.part[blockIdx.x * p.cols + c + i * step + e] = acc[i][e];
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
        float dot = 0.0f, u[1], v[1];
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            load_unit<T, 1>(h + c, u);
            load_unit<T, 1>(dy + c, v);
            dot = fmaf(u[0] * rstd, v[0] * p.gain[c], dot);
        }
        dot = row_reduce(dot, part[(r - first) & 1], Add()) * inv_n;
        for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
            float d[1] = {0.0f};
            load_unit<T, 1>(h + c, u);
            load_unit<T, 1>(dy + c, v);
            u[0] *= rstd;
            sums[c] = fmaf(v[0], u[0], r == first ? 0.0f : sums[c]);
            if (p.dH) load_unit<T, 1>(static_cast<const T*>(p.dH) + r * p.lddh + c, d);
            d[0] = fmaf(rstd, v[0] * p.gain[c] - u[0] * dot, d[0]);
            store_unit<T, 1>(static_cast<T*>(p.dX) + r * p.lddx + c, d);
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
constexpr int64_t kMaxDim = (1ll << 31) - 512;
struct Rows {
    const void* p;
    int64_t ld;
};
// bytes of the units that all these rows of `cols` elements can move in
int unit_of(int64_t es, int64_t cols, std::initializer_list<Rows> rows) {
    uint64_t all = (uint64_t)(cols * es);
    for (const Rows& r : rows)
        if (r.p) all |= reinterpret_cast<uintptr_t>(r.p) | (uint64_t)(r.ld * es);
    return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : (int)es;
}

template <int V>
using Const = std::integral_constant<int, V>;

// Calls f(T(), columns per unit, units per thread); a thread takes the units that the row's threads need it
// to. False: the row does not fit into the registers of a CTA.
template <typename F>
bool with_units(int dtype, int unit_bytes, int64_t cols, unsigned* threads, F f) {
    const int n = unit_bytes / (dtype == GPTQ_BF16 ? 2 : 4);
    const int64_t units = cols / n;
    auto go = [&](auto t, auto n, auto wide, auto most) {
        // `wide` units per thread while a row has few of them, `most` for the longest rows
        const int per = ceil_div(units, decltype(wide)::value) <= 512 ? decltype(wide)::value : decltype(most)::value;
        const int64_t need = ceil_div(ceil_div(units, per), 32) * 32;
        if (need > 1024) return false;
        *threads = (unsigned)std::max<int64_t>(need, 32);
        if (per == decltype(wide)::value) f(t, n, wide);
        else f(t, n, most);
        return true;
    };
    if (dtype == GPTQ_BF16) {
        if (unit_bytes == 16) return go(__nv_bfloat16(), Const<8>(), Const<2>(), Const<4>());
        if (unit_bytes == 4) return go(__nv_bfloat16(), Const<2>(), Const<4>(), Const<16>());
        return go(__nv_bfloat16(), Const<1>(), Const<8>(), Const<16>());
    }
    if (unit_bytes == 16) return go(float(), Const<4>(), Const<2>(), Const<8>());
    return go(float(), Const<1>(), Const<8>(), Const<16>());
}

template <bool NORM>
int launch_rows(const RowParams& p, int dtype, int unit_bytes, int id, cudaStream_t s) {
    unsigned threads = 0;
    cudaError_t e = cudaSuccess;
    const bool fits = with_units(dtype, unit_bytes, p.cols, &threads, [&](auto t, auto n, auto u) {
        auto kern = int8_rows_kernel<decltype(t), decltype(n)::value, decltype(u)::value, NORM>;
        const unsigned rows = threads == 32 ? 4 : 1;
        GPTQ_LAUNCH(id, s, e = launch_pdl(kern, dim3((unsigned)ceil_div(p.rows, rows)), dim3(threads, rows), 0, s, p));
    });
    if (!fits) {
        auto kern = dtype == GPTQ_BF16 ? int8_long_rows_kernel<__nv_bfloat16, NORM> : int8_long_rows_kernel<float, NORM>;
        GPTQ_LAUNCH(id, s, e = launch_pdl(kern, dim3((unsigned)p.rows), dim3(1024), 0, s, p));
    }
    GPTQ_CUDA_TRY(e);
    return GPTQ_OK;
}

// CTAs of the gradient, each with a row of partial sums
int64_t grad_ctas(int64_t rows) { return std::min<int64_t>(rows, 2 * kSMs); }

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" int64_t gptq_int8_pitch(int64_t cols) { return int8_pitch(cols); }

extern "C" int gptq_int8_quantize(const void* X, int dtype, int64_t src_rows, int64_t cols, int64_t ldx, const int32_t* index,
                                  int64_t per, int64_t rows, int8_t* codes, float* scales, void* stream) {
    if (src_rows < 0 || cols < 0 || rows < 0 || rows > kMaxDim || src_rows > kMaxDim || cols > kMaxDim || per < 1 || bad_dtype(dtype) ||
        (!index && rows != src_rows))
        return GPTQ_ERR_INVALID_ARG;
    if (rows == 0) return GPTQ_OK;
    if (!scales || (cols > 0 && ((src_rows > 0 && !X) || !codes || ldx < cols || reinterpret_cast<uintptr_t>(codes) % 16 != 0)))
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
    const int rc = launch_rows<false>(p, dtype, unit_of(dtype == GPTQ_BF16 ? 2 : 4, cols, {{X, ldx}}), K_INT8_QUANT, s);
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
    const int unit = unit_of(dtype == GPTQ_BF16 ? 2 : 4, cols, {{X, ldx}, {residual, ldr}, {residual ? H : nullptr, ldh}, {gain, 0}});
    const int rc = launch_rows<true>(p, dtype, unit, K_INT8_NORM, s);
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
    const int unit = unit_of(dtype == GPTQ_BF16 ? 2 : 4, cols, {{dY, lddy}, {H, ldh}, {dH, lddh}, {dX, lddx}, {gain, 0}});
    GradParams p{dY, H, dH, gain, rstd, rows, cols, lddy, ldh, lddh, dX, lddx, static_cast<float*>(ws), 0};
    p.per = ceil_div(rows, grad_ctas(rows));
    const unsigned ctas = (unsigned)ceil_div(rows, p.per);
    unsigned threads = 0;
    cudaError_t e = cudaSuccess;
    const bool fits = with_units(dtype, unit, cols, &threads, [&](auto t, auto n, auto u) {
        auto kern = int8_norm_grad_kernel<decltype(t), decltype(n)::value, decltype(u)::value>;
        GPTQ_LAUNCH(K_INT8_GRAD, s, e = launch_pdl(kern, dim3(ctas), dim3(threads), 0, s, p));
    });
    if (!fits) {
        auto kern = dtype == GPTQ_BF16 ? int8_norm_grad_long_kernel<__nv_bfloat16> : int8_norm_grad_long_kernel<float>;
        GPTQ_LAUNCH(K_INT8_GRAD, s, e = launch_pdl(kern, dim3(ctas), dim3(1024), 0, s, p));
    }
    GPTQ_CUDA_TRY(e);
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
    const bool vec = unit_of(dtype == GPTQ_BF16 ? 2 : 4, cols, {{Y, ldy}}) == 16;
    const int n = vec ? (dtype == GPTQ_BF16 ? 8 : 4) : 1;
    const dim3 grid((unsigned)ceil_div(ceil_div(cols, n), B_THREADS), (unsigned)std::min<int64_t>(ceil_div(rows, B_ROWS), 65535));
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kern) { GPTQ_LAUNCH(K_INT8_DEQUANT, s, e = launch_pdl(kern, grid, dim3(B_THREADS), 0, s, p)); };
    if (dtype == GPTQ_BF16) vec ? go(int8_dequantize_kernel<__nv_bfloat16, 8>) : go(int8_dequantize_kernel<__nv_bfloat16, 1>);
    else vec ? go(int8_dequantize_kernel<float, 4>) : go(int8_dequantize_kernel<float, 1>);
    GPTQ_CUDA_TRY(e);
    return GPTQ_OK;
}

// mx_rows.cu -- rows of microscaled values: quantization, reading back, the tiles of 4-bit
// weights, the root-mean-square norm with its output in blocks, and the sum over a token's experts.
// A thread takes eight values (16 or 32 bytes), four lanes a block.  The bounds are memory, for the norm also instructions:
// f32 weights of [11008, 4096] to 4 bits in 33 us cold (5.8 TB/s), into tiles 11 us (4.5 TB/s), the norm of 8191 bf16 rows of
// 4096 with residual 53 us in a captured graph (4.4 TB/s; 65 cold), the sum over 8 experts of 4095 tokens 46 us (6.4 TB/s).
#include <algorithm>

#include "mx.cuh"

namespace gq {
namespace {

// ---------------------------------------------------------------------------
// quantize, read back
// ---------------------------------------------------------------------------
constexpr int Q_THREADS = 256;

// Quotients of 31-bit numbers by a number known at launch: n * mul >> shift, with mul = ceil(2^shift / d) and shift = 31 +
// ceil(log2 d), for which the error stays below 1 / d.
struct Divisor {
    uint32_t mul;
    int shift;
    __device__ __forceinline__ uint32_t of(uint32_t n) const { return (uint32_t)((uint64_t)n * mul >> shift); }
};
Divisor divisor(uint32_t d) {
    int l = 0;
    while ((1u << l) < d) l++;
    return {(uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d), 31 + l};
}

// One group of 8 values per thread, U of them in flight; the K / 8 groups of a row are a multiple of four, so the four lanes of
// a block are in one row and all there.
template <typename T, bool E2M1>
__global__ void __launch_bounds__(Q_THREADS) quantize_mx_kernel(const T *__restrict__ x, int64_t ldx, uint8_t *__restrict__ codes,
                                                                uint8_t *__restrict__ scales, uint32_t groups, uint32_t per_row,
                                                                Divisor by_row, int S) {
    constexpr int U = sizeof(T) == 4 ? 2 : 4;
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t stride = gridDim.x * Q_THREADS;
    for (uint32_t first = blockIdx.x * Q_THREADS; first < groups; first += U * stride) {
        float v[U][8];
        uint32_t row[U], g[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t i = first + u * stride + threadIdx.x;
            row[u] = i < groups ? by_row.of(i) : 0;
            g[u] = i < groups ? i - row[u] * per_row : 0;
            load8(x + (int64_t)row[u] * ldx + g[u] * 8, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int b = mx_scale_byte(block_amax(v[u]), E2M1);
            const uint2 c = codes8<E2M1>(v[u], mx_inverse(b));
            if (first + u * stride + threadIdx.x >= groups) continue;
            const int64_t i = (int64_t)row[u] * per_row + g[u];
            if (E2M1)
                *reinterpret_cast<uint32_t *>(codes + i * 4) = c.x;
            else
                *reinterpret_cast<uint2 *>(codes + i * 8) = c;
            if ((g[u] & 3) == 0) scales[(int64_t)row[u] * S + (g[u] >> 2)] = (uint8_t)b;
            // the row's last block also writes the padding
            if (g[u] == per_row - 4)
                for (int j = per_row / 4; j < S; j++) scales[(int64_t)row[u] * S + j] = 0;
        }
    }
}

template <typename T, bool E2M1>
__global__ void __launch_bounds__(Q_THREADS) dequantize_mx_kernel(const uint8_t *__restrict__ codes,
                                                                  const uint8_t *__restrict__ scales, T *__restrict__ y,
                                                                  uint32_t groups, uint32_t per_row, Divisor by_row, int S) {
    constexpr int U = 4;
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t stride = gridDim.x * Q_THREADS;
    for (uint32_t first = blockIdx.x * Q_THREADS + threadIdx.x; first < groups; first += U * stride) {
        uint2 w[U];
        int b[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t i = first + u * stride < groups ? first + u * stride : first, row = by_row.of(i);
            w[u] = E2M1 ? make_uint2(__ldg(reinterpret_cast<const uint32_t *>(codes) + i), 0u) : __ldg(reinterpret_cast<const uint2 *>(codes) + i);
            b[u] = __ldg(scales + (int64_t)row * S + ((i - row * per_row) >> 2));
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (first + u * stride >= groups) break;
            const float p = mx_power(b[u]);
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                // two codes to two f16, exactly (NaN codes included)
                uint32_t h;
                const uint32_t c = E2M1 ? w[u].x >> (8 * j) & 0xFFu : (j < 2 ? w[u].x : w[u].y) >> (16 * (j & 1)) & 0xFFFFu;
                if (E2M1)
                    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h) : "r"(c));
                else
                    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
                v[2 * j] = half_lo(h) * p;
                v[2 * j + 1] = half_hi(h) * p;
            }
            store8(y + (int64_t)(first + u * stride) * 8, v);
        }
    }
}

// ---------------------------------------------------------------------------
// 4-bit weights into tiles
// ---------------------------------------------------------------------------
// One CTA per tile; a thread takes 16 bytes of codes (32 values, one scale) twice.  Of each eight codes, the
// first four go to bits 2 .. 5 of the four bytes, the others to bits 6 .. 9 from each byte on (around the end).
__device__ __forceinline__ uint32_t by_fours(uint32_t w) {
    uint32_t lo = w & 0xFFFFu, hi = w >> 16;      // codes 0 .. 3, 4 .. 7, one per nibble
    lo = (lo | lo << 8) & 0x00FF00FFu;
    lo = (lo | lo << 4) & 0x0F0F0F0Fu;
    hi = (hi | hi << 8) & 0x00FF00FFu;
    hi = (hi | hi << 4) & 0x0F0F0F0Fu;
    return lo << 2 | __funnelshift_l(hi, hi, 6);
}
__global__ void __launch_bounds__(256) repack_mxfp4_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                                           uint8_t *__restrict__ out, int64_t tiles, int64_t N, int64_t K,
                                                           int G, int KT, int S) {
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int t = (int)(tile % KT);
        const int64_t cg = tile / KT;
        const int g = (int)(cg % G);
        const int64_t c = cg / G;
        uint8_t *to = out + tile * MX_TILE_BYTES;
        for (int i = threadIdx.x; i < MX_TILE * 4; i += 256) {
            const int r = i >> 2, j = i & 3;
            const int64_t n = (int64_t)g * MX_TILE + r, k = (int64_t)t * MX_TILE + 32 * j;
            uint4 v = make_uint4(0, 0, 0, 0);
            uint8_t b = 0;
            if (n < N && k < K) {
                const int64_t row = c * N + n;
                v = *reinterpret_cast<const uint4 *>(codes + (row * K + k) / 2);
                b = scales[row * S + k / 32];
            }
            *reinterpret_cast<uint4 *>(to + j * 2048 + r * 16) = make_uint4(by_fours(v.x), by_fours(v.y), by_fours(v.z), by_fours(v.w));
            to[MX_TILE_CODES + (r & 31) * 16 + (r >> 5) * 4 + j] = b;
        }
    }
}

// ---------------------------------------------------------------------------
// the norm
// ---------------------------------------------------------------------------
// Two-term arithmetic: a value is hi + lo, |lo| at most half a unit of hi.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Two fast_two_sum(float a, float b) {   // |a| >= |b|
    const float s = a + b;
    return {s, b - (s - a)};
}
__device__ __forceinline__ Two two_prod(float a, float b) {
    const float p = a * b;
    return {p, fmaf(a, b, -p)};
}
__device__ __forceinline__ Two add(Two a, Two b) {
    Two s = two_sum(a.hi, b.hi);
    return fast_two_sum(s.hi, s.lo + (a.lo + b.lo));
}
__device__ __forceinline__ Two mul(Two a, Two b) {
    Two p = two_prod(a.hi, b.hi);
    return fast_two_sum(p.hi, p.lo + (a.hi * b.lo + a.lo * b.hi));
}

// hi + lo as an f32 rounded to odd: towards zero, and the last bit set if anything was cut off.
// A later rounding to fewer bits (a code of 4 significant bits, a comparison with a value of
// few bits) then decides as if it saw the exact sum.
__device__ __forceinline__ float to_odd(Two v) {
    if (v.lo == 0.0f || !(fabsf(v.lo) < INFINITY)) return v.hi;
    const uint32_t b = __float_as_uint(v.hi);
    return __uint_as_float((v.lo < 0.0f) == (v.hi < 0.0f) ? b | 1u : (b - 1u) | 1u);
}

// 1 / sqrt(a), a > 0: one step from the f32 value r.  With e = 1 - a r^2 (|e| < 2^-20),
// a^-1/2 = r (1 - e)^-1/2 = r (1 + e / 2 + 3 e^2 / 8 + ..), the next term below 2^-61.
__device__ __forceinline__ Two two_rsqrt(Two a) {
    const float r = rsqrtf(a.hi);
    const Two ar2 = mul(mul(a, Two{r, 0.0f}), Two{r, 0.0f});
    const float e = (1.0f - ar2.hi) - ar2.lo;
    return fast_two_sum(r, r * fmaf(0.375f * e, e, 0.5f * e));
}

struct NormParams {
    const void *x, *res;
    const float *w;
    void *h, *y, *codes;
    uint8_t *scales;
    int64_t ldx, ldr, ldh, M;
    double eps;
    float eps_hi, eps_lo;
    int K, S, y_bf16;
};

// Eight values as they lie in memory, and the sum of two such, rounded to the type: as it is stored, and widened.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; i++) v[i] = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; i++) reinterpret_cast<uint4 *>(p)[i] = v[i];
    }
    __device__ __forceinline__ void widen(float (&f)[8]) const { load8(reinterpret_cast<const T *>(v), f); }
    __device__ __forceinline__ void add(const Raw &o) {
        float a[8], b[8];
        widen(a);
        o.widen(b);
#pragma unroll
        for (int i = 0; i < 8; i++) a[i] += b[i];
        store8(reinterpret_cast<T *>(v), a);
    }
};

// The larger, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The norm of one row in 64 bits, by all of a CTA: for rows that leave the range in which f32 decides (below).  The squares
// of any f32 values, their sum and any product h w r are normal numbers of 64 bits.  h is read again, where this thread
// wrote it if it is kept.  This GPU has few 64-bit units: 20 us for a row of 4096.
template <typename T>
__device__ __noinline__ void norm_row64(const NormParams &p, int64_t row, double *part) {
    const int groups = p.K / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    auto load = [&](int g, float (&v)[8]) {
        Raw<T> h;
        if (p.h) {
            h.load(static_cast<const T *>(p.h) + row * p.ldh + g * 8);
        } else {
            h.load(static_cast<const T *>(p.x) + row * p.ldx + g * 8);
            if (p.res) {
                Raw<T> r;
                r.load(static_cast<const T *>(p.res) + row * p.ldr + g * 8);
                h.add(r);
            }
        }
        h.widen(v);
    };
    double sum = 0.0;
#pragma unroll 1
    for (int g = threadIdx.x; g < groups; g += blockDim.x) {
        float v[8];
        load(g, v);
#pragma unroll
        for (int i = 0; i < 8; i++) sum += (double)v[i] * (double)v[i];
    }
#pragma unroll 1
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (warps > 1) {
        if (lane == 0) part[warp] = sum;
        __syncthreads();
        sum = lane < warps ? part[lane] : 0.0;
#pragma unroll 1
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        __syncthreads();                                   // `part` is free
    }
    const double r = 1.0 / sqrt(sum / (double)p.K + p.eps);
#pragma unroll 1
    for (int g0 = 0; g0 < groups; g0 += blockDim.x) {
        const int g = g0 + threadIdx.x;
        const bool live = g < groups;
        float h[8], w[8];
        double v[8];
        double most = 0.0;                                 // infinity for blocks with a NaN, too
        load(live ? g : 0, h);
        if (p.w) load8(p.w + (live ? g * 8 : 0), w);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            v[i] = (p.w ? (double)h[i] * (double)w[i] : (double)h[i]) * r;
            const double a = fabs(v[i]);
            most = a < INFINITY ? fmax(most, a) : INFINITY;
        }
        most = fmax(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmax(most, __shfl_xor_sync(0xffffffffu, most, 2));
        if (!live) continue;
        if (p.y) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; i++) y[i] = (float)v[i];
            if (p.y_bf16)
                store8(static_cast<__nv_bfloat16 *>(p.y) + row * p.K + g * 8, y);
            else
                store8(static_cast<float *>(p.y) + row * p.K + g * 8, y);
        }
        if (!p.codes) continue;
        // as mx_scale_byte, and 2^(127 - b); what is scaled is cut to f32 with its last bit set if anything was cut off, so that
        // the code's rounding decides as if it saw all of it
        const int64_t bits = __double_as_longlong(most);
        const int e = (int)(bits >> 52);
        const int b = e == 2047 ? 255 : max(e - 1023 + 127 - 8 + ((bits & 0xFFFFFFFFFFFFF) > 0xC000000000000), 0);
        const double inverse = __longlong_as_double((int64_t)(b == 255 ? 0 : 1023 + 127 - b) << 52);
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const double x = v[i] * inverse;
            f[i] = __double2float_rz(x);
            if ((double)f[i] != x) f[i] = __uint_as_float(__float_as_uint(f[i]) | 1u);
        }
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.codes) + row * p.K + g * 8) = codes8<false>(f, b == 255 ? 0.0f : 1.0f);
        if ((g & 3) == 0) p.scales[row * p.S + (g >> 2)] = (uint8_t)b;
    }
}

// One CTA per row (in turn).  Thread t holds the groups of 8 values t, t + T, .. (C of them at most) from the load to the
// output, so that the row is read once.  The codes are those of the exact y, mostly without exact arithmetic.
// In f32, with positive terms only, the sum of squares is off by 17 roundings at most (4 additions in a thread, 3 levels
// there, 5 in the warp, 5 over the warps), which counts half in r, and a scaled value h w r 2^(127 - b) by 14 in
// all, less than 2^-20 of itself.  So if it gives the same code with 2^-20 more and with 2^-20 less (and so does the
// largest its scale), that is the code; if one value of the row does not (one row of 4096 in ten), the CTA forms the sum, r and
// the row's values again in two terms, from what it holds.
// That counts roundings, not what falls out of f32's range.  With r between 2^-60 and 2^30 the mean of squares is between 2^-60
// and 2^120: the sum is finite, and squares that fell below 2^-126 are off by 2^-150 each.  With a block's largest y between
// 2^-60 and 2^126 (2^-90 for one that f32 decides) its largest h w is finite and above 2^-90 (2^-120), and what its values and
// their second terms lose at 2^-150 is far below a code's step.  Rows with another r or another block are done in 64 bits,
// when the CTA is through with the others: a call within the loop would cost all rows registers (8191 rows 64 us, not 53).
// But blocks of zeros have their codes as they are, if a factor of each value is 0, and a row with a NaN is NaN.
// `later` has a bit for each of a CTA's turns, which some turns share past 2048 of them.
constexpr float R_MIN = 0x1p-60f, R_MAX = 0x1p30f, Y_MIN = 0x1p-60f, Y_MAX = 0x1p126f;
constexpr int LATER = 2048;
template <typename T, int C>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ __align__(8) Two part[32];
    __shared__ uint32_t later[LATER / 32];                 // which of the CTA's rows are left for the end, if any
    bool some_later = false;
    const int groups = p.K / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    // a row's loads are under way while the one before it is worked on
    Raw<T> rx[C], rr[C];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int g = threadIdx.x + c * blockDim.x;
            if (g >= groups) continue;
            rx[c].load(static_cast<const T *>(p.x) + row * p.ldx + g * 8);
            if (p.res) rr[c].load(static_cast<const T *>(p.res) + row * p.ldr + g * 8);
        }
    };
#pragma unroll
    for (int c = 0; c < C; c++) rx[c] = rr[c] = Raw<T>{};
    if (blockIdx.x < p.M) load(blockIdx.x);
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        Raw<T> h[C];
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int g = threadIdx.x + c * blockDim.x;
            if (p.res) rx[c].add(rr[c]);
            h[c] = rx[c];
            if (p.h && g < groups) h[c].store(static_cast<T *>(p.h) + row * p.ldh + g * 8);
        }
        if (row + gridDim.x < p.M) load(row + gridDim.x);
        float sq[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < C; c++) {
            float v[8];
            h[c].widen(v);
#pragma unroll
            for (int i = 0; i < 8; i++) sq[i] = fmaf(v[i], v[i], sq[i]);
        }
        float sum = ((sq[0] + sq[1]) + (sq[2] + sq[3])) + ((sq[4] + sq[5]) + (sq[6] + sq[7]));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (warps > 1) {
            if (lane == 0) part[warp].hi = sum;
            __syncthreads();
            sum = lane < warps ? part[lane].hi : 0.0f;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        }
        const float mean = sum / (float)p.K + p.eps_hi;
        float r;
        asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(mean));
        r = fmaf(0.5f * r, fmaf(-mean * r, r, 1.0f), r);          // to a unit
        bool wide = !(r > R_MIN && r < R_MAX), unsure = false;    // (true for NaN)
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int g = threadIdx.x + c * blockDim.x;
            // a warp's lanes leave together but at the row's end, where whole blocks of four lanes do
            const bool live = g < groups;
            if (!__any_sync(0xffffffffu, live)) continue;
            float w[8], v[8];
            h[c].widen(v);
            if (p.w) {
                load8(p.w + (live ? g * 8 : 0), w);
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] *= w[i];
            }
            if (p.y && live) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; i++) y[i] = v[i] * r;
                if (p.y_bf16)
                    store8(static_cast<__nv_bfloat16 *>(p.y) + row * p.K + g * 8, y);
                else
                    store8(static_cast<float *>(p.y) + row * p.K + g * 8, y);
            }
            float most = 0.0f;                             // NaN if any is: a weight may be, where r is not
#pragma unroll
            for (int i = 0; i < 8; i++) most = max_nan(most, fabsf(v[i]));
            if (!p.codes) {
                wide |= live && !(most * r > Y_MIN && most * r < Y_MAX);
                continue;
            }
            most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 2)) * r;
            const int b = mx_scale_byte(__float_as_uint(most * (1.0f + 0x1p-20f)), false);
            const float inv = fminf(mx_inverse(b) * r, 0x1p126f), less = inv * (1.0f - 0x1p-20f), more = inv * (1.0f + 0x1p-20f);
            uint32_t lo[4], differ = 0;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                lo[i] = e4m3x2(v[2 * i] * less, v[2 * i + 1] * less);
                differ |= lo[i] ^ e4m3x2(v[2 * i] * more, v[2 * i + 1] * more);
            }
            // (tiny, infinite and NaN blocks are not sure: there the f32 values are not that close)
            const bool sure = differ == 0 && mx_scale_byte(__float_as_uint(most * (1.0f - 0x1p-20f)), false) == b && b > 0 && b < 255 &&
                              inv < 0x1p100f && most > 0x1p-90f;
            if (live) {
                unsure |= !sure && most > 0.0f;
                wide |= !sure && !(most > Y_MIN && most < Y_MAX);
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.codes) + row * p.K + g * 8) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                if ((g & 3) == 0) p.scales[row * p.S + (g >> 2)] = (uint8_t)b;
            }
        }
        if (p.codes && threadIdx.x < p.S - p.K / 32) p.scales[row * p.S + p.K / 32 + threadIdx.x] = 0;
        // (the barrier also frees `part`)
        if (!(warps > 1 ? __syncthreads_or(unsure || wide) : __any_sync(0xffffffffu, unsure || wide))) continue;
        if (warps > 1 ? __syncthreads_or(wide) : __any_sync(0xffffffffu, wide)) {
            if (isnan(mean)) {                             // a NaN among h: the row is NaN, y is already
                if (p.codes)
                    for (int g = threadIdx.x; g < groups; g += blockDim.x) {
                        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.codes) + row * p.K + g * 8) = make_uint2(0u, 0u);
                        if ((g & 3) == 0) p.scales[row * p.S + (g >> 2)] = 255;
                    }
                continue;
            }
            // (blocks of zeros that are there because a factor of each is have their codes)
            wide = !(r > R_MIN && r < R_MAX);
#pragma unroll
            for (int c = 0; c < C; c++) {
                const int g = threadIdx.x + c * blockDim.x;
                float v[8], w[8], most = 0.0f;
                h[c].widen(v);
#pragma unroll
                for (int i = 0; i < 8; i++) w[i] = 1.0f;
                if (p.w) load8(p.w + (g < groups ? g * 8 : 0), w);
                bool zeros = true;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    zeros = zeros && v[i] * w[i] == 0.0f && (v[i] == 0.0f || w[i] == 0.0f);
                    most = max_nan(most, fabsf(v[i] * w[i]));
                }
                if (p.codes) {
                    most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 1));
                    most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 2));
                }
                wide |= g < groups && !zeros && !(most * r > Y_MIN && most * r < Y_MAX);
            }
            if (warps > 1 ? __syncthreads_or(wide) : __any_sync(0xffffffffu, wide)) {
                if (threadIdx.x == 0) {
                    if (!some_later)
                        for (int i = 0; i < LATER / 32; i++) later[i] = 0;
                    const int turn = (int)((row - blockIdx.x) / gridDim.x) % LATER;
                    later[turn >> 5] |= 1u << (turn & 31);
                }
                some_later = true;
                continue;
            }
            if (!(warps > 1 ? __syncthreads_or(unsure) : __any_sync(0xffffffffu, unsure))) continue;
        }
        Two total{0.0f, 0.0f};
#pragma unroll 1
        for (int i = 0; i < 8; i++) {
#pragma unroll
            for (int c = 0; c < C; c++) {
                float v[8], x = 0.0f;
                h[c].widen(v);
#pragma unroll
                for (int u = 0; u < 8; u++)
                    if (u == i) x = v[u];
                const Two square = two_prod(x, x), next = two_sum(total.hi, square.hi);
                total = {next.hi, total.lo + (next.lo + square.lo)};
            }
        }
        total = fast_two_sum(total.hi, total.lo);
#pragma unroll 1
        for (int d = 16; d > 0; d >>= 1)
            total = add(total, Two{__shfl_xor_sync(0xffffffffu, total.hi, d), __shfl_xor_sync(0xffffffffu, total.lo, d)});
        if (warps > 1) {
            if (lane == 0) part[warp] = total;
            __syncthreads();
            total = lane < warps ? part[lane] : Two{0.0f, 0.0f};
#pragma unroll 1
            for (int d = 16; d > 0; d >>= 1)
                total = add(total, Two{__shfl_xor_sync(0xffffffffu, total.hi, d), __shfl_xor_sync(0xffffffffu, total.lo, d)});
        }
        // mean = total / K: the quotient of the first terms, and what it leaves over
        const float k = (float)p.K, q = total.hi / k;
        const Two r2 = two_rsqrt(add(fast_two_sum(q, (fmaf(-q, k, total.hi) + total.lo) / k), Two{p.eps_hi, p.eps_lo}));
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int g = threadIdx.x + c * blockDim.x;
            const bool live = g < groups;
            if (!__any_sync(0xffffffffu, live)) continue;
            float v[8], w[8];
            h[c].widen(v);
#pragma unroll
            for (int i = 0; i < 8; i++) w[i] = 1.0f;
            if (p.w) load8(p.w + (live ? g * 8 : 0), w);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const Two hw = two_prod(v[i], w[i]);
                v[i] = hw.hi == 0.0f ? hw.hi : to_odd(mul(hw, r2));      // (a sum of terms would make +0 of -0)
            }
            const int b = mx_scale_byte(block_amax(v), false);
            const uint2 code = codes8<false>(v, mx_inverse(b));
            if (live) {
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.codes) + row * p.K + g * 8) = code;
                if ((g & 3) == 0) p.scales[row * p.S + (g >> 2)] = (uint8_t)b;
            }
        }
        if (warps > 1) __syncthreads();                    // `part` is free
    }
    if (!some_later) return;
    __syncthreads();
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, turn = (turn + 1) % LATER)
        if (later[turn >> 5] >> (turn & 31) & 1u) norm_row64<T>(p, row, reinterpret_cast<double *>(part));
}

// ---------------------------------------------------------------------------
// the sum over a token's experts
// ---------------------------------------------------------------------------
// Eight columns per thread.  Bound by the rows' bytes; four of them are under way at a time, so that one token's
// eight experts are two latencies, not eight.
template <typename TR, typename TO>
__global__ void __launch_bounds__(256) experts_combine_kernel(const float *__restrict__ y, int64_t R, const int32_t *__restrict__ pos,
                                                              const float *__restrict__ w, int k, const TR *res, int64_t ldr,
                                                              TO *out, int64_t ldo, uint32_t groups, uint32_t per_row, Divisor by_row) {
    constexpr int U = 4;
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t stride = gridDim.x * 256;
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < groups; i += stride) {
        const uint32_t t = by_row.of(i), g = i - t * per_row;
        const int32_t *const at = pos + (int64_t)t * k;
        const float *const by = w + (int64_t)t * k;
        float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (res) load8(res + t * ldr + g * 8, acc);
        for (int j = 0; j < k; j += U) {
            bool there[U];
            float a[U], v[U][8];
#pragma unroll
            for (int x = 0; x < U; x++) {
                const int64_t r = j + x < k ? at[j + x] : -1;
                there[x] = r >= 0 && r < R;
                a[x] = there[x] ? by[j + x] : 0.0f;
                if (there[x]) load8(y + (r * per_row + g) * 8, v[x]);
            }
#pragma unroll
            for (int x = 0; x < U; x++)
                if (there[x])
#pragma unroll
                    for (int u = 0; u < 8; u++) acc[u] = fmaf(a[x], v[x][u], acc[u]);
        }
        store8(out + t * ldo + g * 8, acc);
    }
}

// CTAs for `work` threads' worth of turns: as many as are resident at once, at most.
unsigned grid_for(int64_t work, int threads) {
    return (unsigned)std::min<int64_t>((work + threads - 1) / threads, (int64_t)sm_count() * (2048 / threads));
}

template <typename T, int C>
gq_status norm_launch(const NormParams &p, int threads, cudaStream_t s) {
    NormParams q = p;
    void *args[] = {&q};
    const int64_t fit = (int64_t)sm_count() * std::max(1, 1024 / threads);       // 64 registers
    return launch_pdl((const void *)rms_norm_kernel<T, C>, dim3((unsigned)std::min<int64_t>(p.M, fit)), dim3(threads), 0, s, args,
                      "norm launch");
}

// One group of 8 values per thread keeps a lone row's chain short (a row of 4096 2.8 us, by two 3.9); where rows abound
// (several for each SM) threads take two, for fewer and longer turns (8191 bf16 rows 53 us, by one 62; f32, more registers, 99
// and 96).  Rows of more than 16384 values need four.
template <typename T>
gq_status norm_width(const NormParams &p, cudaStream_t s) {
    const int groups = p.K / 8;
    int c = p.M >= 4LL * sm_count() && groups >= 64 ? 2 : 1;
    while ((groups + c - 1) / c > 1024) c *= 2;
    const int threads = ((groups + c - 1) / c + 31) / 32 * 32;
    if (c == 1) return norm_launch<T, 1>(p, threads, s);
    if (c == 2) return norm_launch<T, 2>(p, threads, s);
    return norm_launch<T, 4>(p, threads, s);
}

}  // namespace

gq_status launch_quantize_mx(const void *x, int64_t ldx, bool bf16, bool e2m1, void *codes, uint8_t *scales, int64_t M,
                             int64_t K, cudaStream_t s) {
    uint32_t per_row = (uint32_t)(K / 8);
    int S = (int)gq_mx_scale_cols(K);
    Divisor by_row = divisor(per_row);
    const int64_t most = std::max<int64_t>(1, ((1LL << 30) - 1) / per_row);      // rows of a launch: 31-bit numbers of groups
    const void *fn = bf16 ? (e2m1 ? (const void *)quantize_mx_kernel<__nv_bfloat16, true> : (const void *)quantize_mx_kernel<__nv_bfloat16, false>)
                          : (e2m1 ? (const void *)quantize_mx_kernel<float, true> : (const void *)quantize_mx_kernel<float, false>);
    for (int64_t m = 0; m < M; m += most) {
        uint32_t groups = (uint32_t)(std::min(most, M - m) * per_row);
        const uint8_t *from = static_cast<const uint8_t *>(x) + m * ldx * (bf16 ? 2 : 4);
        uint8_t *to = static_cast<uint8_t *>(codes) + m * K / (e2m1 ? 2 : 1), *to_scales = scales + m * S;
        void *args[] = {&from, &ldx, &to, &to_scales, &groups, &per_row, &by_row, &S};
        gq_status st = launch_pdl(fn, dim3(grid_for(groups, Q_THREADS)), dim3(Q_THREADS), 0, s, args, "mx quantize launch");
        if (st != GQ_OK) return st;
    }
    return GQ_OK;
}

gq_status launch_dequantize_mx(const void *codes, const uint8_t *scales, bool e2m1, void *y, bool bf16, int64_t M,
                               int64_t K, cudaStream_t s) {
    uint32_t per_row = (uint32_t)(K / 8);
    int S = (int)gq_mx_scale_cols(K);
    Divisor by_row = divisor(per_row);
    const int64_t most = std::max<int64_t>(1, ((1LL << 30) - 1) / per_row);
    const void *fn = bf16 ? (e2m1 ? (const void *)dequantize_mx_kernel<__nv_bfloat16, true> : (const void *)dequantize_mx_kernel<__nv_bfloat16, false>)
                          : (e2m1 ? (const void *)dequantize_mx_kernel<float, true> : (const void *)dequantize_mx_kernel<float, false>);
    for (int64_t m = 0; m < M; m += most) {
        uint32_t groups = (uint32_t)(std::min(most, M - m) * per_row);
        const uint8_t *from = static_cast<const uint8_t *>(codes) + m * K / (e2m1 ? 2 : 1), *from_scales = scales + m * S;
        uint8_t *to = static_cast<uint8_t *>(y) + m * K * (bf16 ? 2 : 4);
        void *args[] = {&from, &from_scales, &to, &groups, &per_row, &by_row, &S};
        gq_status st = launch_pdl(fn, dim3(grid_for(groups, Q_THREADS)), dim3(Q_THREADS), 0, s, args, "mx dequantize launch");
        if (st != GQ_OK) return st;
    }
    return GQ_OK;
}

gq_status launch_repack_mxfp4(const void *codes, const uint8_t *scales, void *rep, int64_t count, int64_t N, int64_t K,
                              cudaStream_t s) {
    int G = (int)((N + MX_TILE - 1) / MX_TILE), KT = (int)((K + MX_TILE - 1) / MX_TILE);
    int64_t tiles = count * G * KT;
    int S = (int)gq_mx_scale_cols(K);
    void *args[] = {&codes, &scales, &rep, &tiles, &N, &K, &G, &KT, &S};
    return launch_pdl((const void *)repack_mxfp4_kernel, dim3((unsigned)std::min<int64_t>(tiles, 1 << 20)), dim3(256), 0, s, args,
                      "mxfp4 repack launch");
}

gq_status launch_rms_norm_mx(const void *x, int64_t ldx, const void *res, int64_t ldr, bool bf16, const float *w,
                             double eps, void *h, int64_t ldh, void *y, bool y_bf16, void *codes, uint8_t *scales,
                             int64_t M, int64_t K, cudaStream_t s) {
    NormParams p{};
    p.x = x, p.res = res, p.w = w, p.h = h, p.y = y, p.codes = codes, p.scales = scales;
    p.ldx = ldx, p.ldr = ldr, p.ldh = ldh, p.M = M;
    p.eps = eps, p.eps_hi = (float)eps, p.eps_lo = (float)(eps - (double)p.eps_hi);
    p.K = (int)K, p.S = (int)gq_mx_scale_cols(K), p.y_bf16 = y_bf16;
    return bf16 ? norm_width<__nv_bfloat16>(p, s) : norm_width<float>(p, s);
}

gq_status launch_experts_combine(const float *y, int64_t R, const int32_t *pos, const float *w, int64_t k, const void *res,
                                 int64_t ldr, bool res_bf16, void *out, int64_t ldo, bool bf16, int64_t T, int64_t N,
                                 cudaStream_t s) {
    uint32_t per_row = (uint32_t)(N / 8);
    int kk = (int)k;
    Divisor by_row = divisor(per_row);
    const int64_t most = std::max<int64_t>(1, ((1LL << 30) - 1) / per_row);      // tokens of a launch, as above
    using B = __nv_bfloat16;
    const void *fn = res_bf16 ? (bf16 ? (const void *)experts_combine_kernel<B, B> : (const void *)experts_combine_kernel<B, float>)
                              : (bf16 ? (const void *)experts_combine_kernel<float, B> : (const void *)experts_combine_kernel<float, float>);
    for (int64_t m = 0; m < T; m += most) {
        uint32_t groups = (uint32_t)(std::min(most, T - m) * per_row);
        const int32_t *at = pos + m * k;
        const float *by = w + m * k;
        const uint8_t *from = res ? static_cast<const uint8_t *>(res) + m * ldr * (res_bf16 ? 2 : 4) : nullptr;
        uint8_t *to = static_cast<uint8_t *>(out) + m * ldo * (bf16 ? 2 : 4);
        void *args[] = {&y, &R, &at, &by, &kk, &from, &ldr, &to, &ldo, &groups, &per_row, &by_row};
        gq_status st = launch_pdl(fn, dim3(grid_for(groups, 256)), dim3(256), 0, s, args, "experts combine launch");
        if (st != GQ_OK) return st;
    }
    return GQ_OK;
}

}  // namespace gq

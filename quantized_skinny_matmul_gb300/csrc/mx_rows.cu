// mx_rows.cu -- rows of microscaled values: quantization, reading back, the tiles of 4-bit
// weights, the root-mean-square norm with its output in blocks, and the sum over a token's experts.
// All are bound by memory; a thread takes eight values (16 or 32 bytes), four lanes a block.
#include <algorithm>

#include "mx.cuh"

namespace gq {
namespace {

// ---------------------------------------------------------------------------
// quantize, read back
// ---------------------------------------------------------------------------
constexpr int Q_THREADS = 256;

// One group of 8 values per thread and turn; the K / 8 groups of a row are a multiple of four, so
// the four lanes of a block are in one row and all there.
template <typename T, bool E2M1>
__global__ void __launch_bounds__(Q_THREADS) quantize_mx_kernel(const T *__restrict__ x, int64_t ldx, uint8_t *__restrict__ codes,
                                                                uint8_t *__restrict__ scales, int64_t groups, int per_row,
                                                                int S) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t stride = (int64_t)gridDim.x * Q_THREADS;
    for (int64_t first = (int64_t)blockIdx.x * Q_THREADS; first < groups; first += stride) {
        const int64_t i = first + threadIdx.x;
        const bool live = i < groups;
        const int64_t row = live ? i / per_row : 0;
        const int g = live ? (int)(i - row * per_row) : 0;
        float v[8];
        load8(x + row * ldx + g * 8, v);
        const int b = mx_scale_byte(block_amax(v), E2M1);
        const uint2 c = codes8<E2M1>(v, mx_inverse(b));
        if (!live) continue;
        if (E2M1)
            *reinterpret_cast<uint32_t *>(codes + (row * per_row + g) * 4) = c.x;
        else
            *reinterpret_cast<uint2 *>(codes + (row * per_row + g) * 8) = c;
        if ((g & 3) == 0) scales[row * S + (g >> 2)] = (uint8_t)b;
        // the row's last block also writes the padding
        if (g == per_row - 4)
            for (int j = per_row / 4; j < S; j++) scales[row * S + j] = 0;
    }
}

template <typename T, bool E2M1>
__global__ void __launch_bounds__(Q_THREADS) dequantize_mx_kernel(const uint8_t *__restrict__ codes,
                                                                  const uint8_t *__restrict__ scales, T *__restrict__ y,
                                                                  int64_t groups, int per_row, int S) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t stride = (int64_t)gridDim.x * Q_THREADS;
    for (int64_t i = (int64_t)blockIdx.x * Q_THREADS + threadIdx.x; i < groups; i += stride) {
        const int64_t row = i / per_row;
        const int g = (int)(i - row * per_row);
        const float p = mx_power(scales[row * S + (g >> 2)]);
        float v[8];
        if (E2M1) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + i * 4);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                // sign, exponent and fraction in their places of an f16 are the value times 2^-14
                const uint32_t n = w >> (4 * j) & 15u;
                v[j] = __half2float(__ushort_as_half((unsigned short)((n & 8u) << 12 | (n & 7u) << 9))) * 16384.0f * p;
            }
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(codes + i * 8);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                // e4m3 likewise, times 2^-8; code 0x7F is a NaN
                const uint32_t n = (j < 4 ? w.x : w.y) >> (8 * (j & 3)) & 255u;
                v[j] = __half2float(__ushort_as_half((unsigned short)((n & 128u) << 8 | (n & 127u) << 7))) * 256.0f * p;
                if ((n & 127u) == 127u) v[j] = __uint_as_float(0x7FFFFFFFu);
            }
        }
        store8(y + i * 8, v);
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
    float eps_hi, eps_lo;
    int K, S, y_bf16;
};

// One CTA per row (in turn).  Thread t holds the groups of 8 values t, t + T, .. (C of them at most)
// from the load to the output, so that the row is read once.
template <typename T, int C>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormParams p) {
    __shared__ Two part[32];
    pdl_wait();
    pdl_launch_dependents();
    const int groups = p.K / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + row * p.ldx;
        const T *res = static_cast<const T *>(p.res) + row * p.ldr;
        float h[C][8];
        Two sum{0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int g = threadIdx.x + c * blockDim.x;
            if (g >= groups) continue;
            load8(x + g * 8, h[c]);
            if (p.res) {
                float r[8];
                load8(res + g * 8, r);
#pragma unroll
                for (int i = 0; i < 8; i++) h[c][i] = sizeof(T) == 4 ? h[c][i] + r[i] : __bfloat162float(__float2bfloat16_rn(h[c][i] + r[i]));
            }
            if (p.h) store8(static_cast<T *>(p.h) + row * p.ldh + g * 8, h[c]);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const Two sq = two_prod(h[c][i], h[c][i]);
                const Two s = two_sum(sum.hi, sq.hi);
                sum = {s.hi, sum.lo + (s.lo + sq.lo)};
            }
        }
        sum = fast_two_sum(sum.hi, sum.lo);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            sum = add(sum, Two{__shfl_xor_sync(0xffffffffu, sum.hi, d), __shfl_xor_sync(0xffffffffu, sum.lo, d)});
        if (warps > 1) {
            if (lane == 0) part[warp] = sum;
            __syncthreads();
            sum = lane < warps ? part[lane] : Two{0.0f, 0.0f};
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                sum = add(sum, Two{__shfl_xor_sync(0xffffffffu, sum.hi, d), __shfl_xor_sync(0xffffffffu, sum.lo, d)});
            __syncthreads();
        }
        // mean = sum / K: the quotient of the first terms, and what it leaves over
        const float k = (float)p.K, q = sum.hi / k;
        const Two mean = fast_two_sum(q, (fmaf(-q, k, sum.hi) + sum.lo) / k);
        const Two r = two_rsqrt(add(mean, Two{p.eps_hi, p.eps_lo}));
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int g = threadIdx.x + c * blockDim.x;
            // a warp's lanes leave together but at the row's end, where whole blocks of four lanes do
            const bool live = g < groups;
            if (!__any_sync(0xffffffffu, live)) continue;
            float w[8], odd[8], near[8];
            if (p.w && live) {
                load8(p.w + g * 8, w);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) w[i] = 1.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const Two y = mul(two_prod(live ? h[c][i] : 0.0f, w[i]), r);
                near[i] = y.hi;
                odd[i] = to_odd(y);
            }
            if (p.y && live) {
                if (p.y_bf16)
                    store8(static_cast<__nv_bfloat16 *>(p.y) + row * p.K + g * 8, near);
                else
                    store8(static_cast<float *>(p.y) + row * p.K + g * 8, near);
            }
            if (!p.codes) continue;
            const int b = mx_scale_byte(block_amax(odd), false);
            const uint2 code = codes8<false>(odd, mx_inverse(b));
            if (live) {
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.codes) + row * p.K + g * 8) = code;
                if ((g & 3) == 0) p.scales[row * p.S + (g >> 2)] = (uint8_t)b;
            }
        }
        if (p.codes && threadIdx.x < p.S - p.K / 32) p.scales[row * p.S + p.K / 32 + threadIdx.x] = 0;
    }
}

// ---------------------------------------------------------------------------
// the sum over a token's experts
// ---------------------------------------------------------------------------
template <typename TR, typename TO>
__global__ void __launch_bounds__(256) experts_combine_kernel(const float *__restrict__ y, int64_t R, const int32_t *__restrict__ pos,
                                                              const float *__restrict__ w, int k, const TR *res, int64_t ldr,
                                                              TO *out, int64_t ldo, int64_t groups, int per_row) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < groups; i += stride) {
        const int64_t t = i / per_row;
        const int g = (int)(i - t * per_row);
        float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (res) load8(res + t * ldr + g * 8, acc);
        for (int j = 0; j < k; j++) {
            const int64_t r = pos[t * k + j];
            if (r < 0 || r >= R) continue;
            const float a = w[t * k + j];
            float v[8];
            load8(y + (r * per_row + g) * 8, v);
#pragma unroll
            for (int u = 0; u < 8; u++) acc[u] = fmaf(a, v[u], acc[u]);
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
    const int64_t fit = (int64_t)sm_count() * std::max(1, 2048 / threads);
    return launch_pdl((const void *)rms_norm_kernel<T, C>, dim3((unsigned)std::min<int64_t>(p.M, fit)), dim3(threads), 0, s, args,
                      "norm launch");
}

// One group of 8 values per thread keeps a lone row's chain short; where rows abound (several for each
// SM) threads take up to four groups, for fewer and longer turns.
template <typename T>
gq_status norm_width(const NormParams &p, cudaStream_t s) {
    const int groups = p.K / 8;
    int c = p.M >= 4LL * sm_count() && groups >= 128 ? 4 : 1;
    while (c < 4 && (groups + c - 1) / c > 1024) c *= 2;
    const int threads = ((groups + c - 1) / c + 31) / 32 * 32;
    if (c == 1) return norm_launch<T, 1>(p, threads, s);
    if (c == 2) return norm_launch<T, 2>(p, threads, s);
    return norm_launch<T, 4>(p, threads, s);
}

}  // namespace

gq_status launch_quantize_mx(const void *x, int64_t ldx, bool bf16, bool e2m1, void *codes, uint8_t *scales, int64_t M,
                             int64_t K, cudaStream_t s) {
    int per_row = (int)(K / 8), S = (int)gq_mx_scale_cols(K);
    int64_t groups = M * per_row;
    void *args[] = {&x, &ldx, &codes, &scales, &groups, &per_row, &S};
    const void *fn = bf16 ? (e2m1 ? (const void *)quantize_mx_kernel<__nv_bfloat16, true> : (const void *)quantize_mx_kernel<__nv_bfloat16, false>)
                          : (e2m1 ? (const void *)quantize_mx_kernel<float, true> : (const void *)quantize_mx_kernel<float, false>);
    return launch_pdl(fn, dim3(grid_for(groups, Q_THREADS)), dim3(Q_THREADS), 0, s, args, "mx quantize launch");
}

gq_status launch_dequantize_mx(const void *codes, const uint8_t *scales, bool e2m1, void *y, bool bf16, int64_t M,
                               int64_t K, cudaStream_t s) {
    int per_row = (int)(K / 8), S = (int)gq_mx_scale_cols(K);
    int64_t groups = M * per_row;
    void *args[] = {&codes, &scales, &y, &groups, &per_row, &S};
    const void *fn = bf16 ? (e2m1 ? (const void *)dequantize_mx_kernel<__nv_bfloat16, true> : (const void *)dequantize_mx_kernel<__nv_bfloat16, false>)
                          : (e2m1 ? (const void *)dequantize_mx_kernel<float, true> : (const void *)dequantize_mx_kernel<float, false>);
    return launch_pdl(fn, dim3(grid_for(groups, Q_THREADS)), dim3(Q_THREADS), 0, s, args, "mx dequantize launch");
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
    p.eps_hi = (float)eps, p.eps_lo = (float)(eps - (double)p.eps_hi);
    p.K = (int)K, p.S = (int)gq_mx_scale_cols(K), p.y_bf16 = y_bf16;
    return bf16 ? norm_width<__nv_bfloat16>(p, s) : norm_width<float>(p, s);
}

gq_status launch_experts_combine(const float *y, int64_t R, const int32_t *pos, const float *w, int64_t k, const void *res,
                                 int64_t ldr, bool res_bf16, void *out, int64_t ldo, bool bf16, int64_t T, int64_t N,
                                 cudaStream_t s) {
    int per_row = (int)(N / 8), kk = (int)k;
    int64_t groups = T * per_row;
    void *args[] = {&y, &R, &pos, &w, &kk, &res, &ldr, &out, &ldo, &groups, &per_row};
    using B = __nv_bfloat16;
    const void *fn = res_bf16 ? (bf16 ? (const void *)experts_combine_kernel<B, B> : (const void *)experts_combine_kernel<B, float>)
                              : (bf16 ? (const void *)experts_combine_kernel<float, B> : (const void *)experts_combine_kernel<float, float>);
    return launch_pdl(fn, dim3(grid_for(groups, 256)), dim3(256), 0, s, args, "experts combine launch");
}

}  // namespace gq

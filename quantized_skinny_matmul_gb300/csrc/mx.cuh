// mx.cuh -- microscaled formats: what the kernels of rows, experts and products share.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gq_common.cuh"
#include "gq_internal.h"

namespace gq {

constexpr int MX_TILE = 128;                 // rows and columns of a tile of repacked 4-bit weights
constexpr int MX_TILE_CODES = MX_TILE * MX_TILE / 2;
constexpr int MX_TILE_SCALES = MX_TILE * MX_TILE / QK;
constexpr int MX_TILE_BYTES = MX_TILE_CODES + MX_TILE_SCALES;

// The scale byte of a block whose largest magnitude has these bits: amax = 1.f * 2^(e - 127), and
// the smallest power of two with amax <= top * power is 2^(e - 127 - 8) for top = 448 = 1.75 * 2^8 and
// 2^(e - 127 - 2) for top = 6 = 1.5 * 2^2, twice that if 1.f is above 1.75 (1.5).  Subnormal amax
// (e = 0) gives 0; infinities and NaN (e = 255) give 255.
__device__ __forceinline__ int mx_scale_byte(uint32_t amax_bits, bool e2m1) {
    const int e = (int)(amax_bits >> 23);
    const uint32_t f = amax_bits & 0x7FFFFFu;
    const int b = e2m1 ? e - 2 + (f > 0x400000u) : e - 8 + (f > 0x600000u);
    return e == 255 ? 255 : max(b, 0);
}
// 2^(127 - b): a normal number for every byte that mx_scale_byte gives (253 at most), 0 for 255.
__device__ __forceinline__ float mx_inverse(int b) { return b == 255 ? 0.0f : __uint_as_float((uint32_t)(254 - b) << 23); }
// 2^(b - 127); NaN for 255
__device__ __forceinline__ float mx_power(int b) {
    return __uint_as_float(b == 0 ? 0x400000u : b == 255 ? 0x7FFFFFFFu : (uint32_t)b << 23);
}

// Two codes of the nearest elements (ties to even); lo in the low byte (nibble).  |x| <= top here.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t, z;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tmov.b32 %0, {t, 0, 0, 0};\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r & 0xFFu;
}

// Eight values of a row, 16-byte aligned.
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The largest magnitude (as bits: NaN above infinity above the rest) of eight values and of the
// four lanes that hold a block.
__device__ __forceinline__ uint32_t block_amax(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// The codes of eight values: 8 bytes (e4m3) or 4 (e2m1, in the low word).
template <bool E2M1>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++)
        w[i] = inv == 0.0f ? 0u : E2M1 ? e2m1x2(v[2 * i] * inv, v[2 * i + 1] * inv) : e4m3x2(v[2 * i] * inv, v[2 * i + 1] * inv);
    if (E2M1) return make_uint2(w[0] | w[1] << 8 | w[2] << 16 | w[3] << 24, 0u);
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// launchers (arguments validated by the entry points)
gq_status launch_quantize_mx(const void *x, int64_t ldx, bool bf16, bool e2m1, void *codes, uint8_t *scales, int64_t M,
                             int64_t K, cudaStream_t s);
gq_status launch_dequantize_mx(const void *codes, const uint8_t *scales, bool e2m1, void *y, bool bf16, int64_t M,
                               int64_t K, cudaStream_t s);
gq_status launch_repack_mxfp4(const void *codes, const uint8_t *scales, void *rep, int64_t count, int64_t N, int64_t K,
                              cudaStream_t s);
gq_status launch_rms_norm_mx(const void *x, int64_t ldx, const void *res, int64_t ldr, bool bf16, const float *w,
                             double eps, void *h, int64_t ldh, void *y, bool y_bf16, void *codes, uint8_t *scales,
                             int64_t M, int64_t K, cudaStream_t s);
gq_status launch_experts_combine(const float *y, int64_t R, const int32_t *pos, const float *w, int64_t k, const void *res,
                                 int64_t ldr, bool res_bf16, void *out, int64_t ldo, bool bf16, int64_t T, int64_t N,
                                 cudaStream_t s);
gq_status launch_route(const gq_router &r, const void *logits, int64_t ldl, bool bf16, const int32_t *used, int32_t *ids,
                       float *weights, int32_t *offsets, int32_t *rows, int32_t *pos, int64_t T, cudaStream_t s);
// dst (codes == nullptr), or the gated unit's codes and scales (N is then F)
gq_status launch_mx_product(const void *rep, const gq_mx_rows &x, const gq_expert_rows *plan, void *dst, int64_t ldd,
                            bool bf16, void *codes, uint8_t *scales, int64_t N, int64_t K, cudaStream_t s);
// dst = rows of values (M <= MX_FEW_ROWS, quantized on the way by every CTA) . W^T.  Spares a launch: one row of [4096, 4096] 8.9 us
// against 9.9 by two kernels, of [11008, 4096] 11.6 against 12.3, and 9 against 12 us of the host's time; two rows the same, four rows of
// [11008, 4096] 15.2 against 12.3 (the two warps that quantize then fall behind the weights).
constexpr int64_t MX_FEW_ROWS = 2;
gq_status launch_mx_product_few(const void *rep, const void *values, int64_t ldv, bool values_bf16, void *dst, int64_t ldd, bool bf16,
                                int64_t M, int64_t N, int64_t K, cudaStream_t s);
// kv_pages.cu: a launch that may start before the grid in front has finished (its kernels wait for it)
gq_status launch_pdl(const void *fn, dim3 grid, dim3 block, size_t smem, cudaStream_t s, void **args, const char *what);

}  // namespace gq

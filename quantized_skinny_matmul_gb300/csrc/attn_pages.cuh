// attn_pages.cuh -- what the two attention kernels over the paged 8-bit KV cache share.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gq_common.cuh"
#include "gq_internal.h"
#include "kv_pages.cuh"

namespace gq {

constexpr float LOG2E = 1.4426950408889634f;

// A call, as the kernels take it.
struct AttnParams8 {
    PagesView c;
    const float *q;
    float *out;
    const int32_t *cu;
    const float *slopes;
    const int32_t *first, *prefix;
    float *parts;               // row kernel: [CTA][2][ROWS][D] sums, and [CTA][2][ROWS][2] maximum and denominator
    float *part_ml;
    int *counters;              // row kernel, per CTA: pieces of the item cut at its end that are done
    float *glse;                // [T * Hq][NG] log2 of the weight sums by group, or null (the slice's rows are there)
    float *lse;                 // [T * Hq] log2 of the denominators
    int row0, row1;             // the slice of packed rows that is worked out
    int64_t ldq, ldo, window;
    int T, max_n, Hq, G, NG, lgP, lgGroup;
    int rows_over;              // sequences with more query rows per KV head are the tile kernel's
    float scale, cap;
};

__device__ __forceinline__ uint4 sh_ld128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 sh_ld64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *map, int row, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tanh: the continued fraction x / (1 + x^2 / (3 + x^2 / (5 + ...))) cut after the fifth level for
// |x| <= 1 (off by 1e-7 relative at 1, less below), 1 - 2 / (e^2x + 1) beyond.
__device__ __forceinline__ float tanh_f32(float x) {
    const float u = x * x;
    const float small = x * fmaf(u, 105.0f + u, 945.0f) * __frcp_rn(fmaf(u, fmaf(15.0f, u, 420.0f), 945.0f));
    const float a = fabsf(x);
    if (a <= 1.0f) return small;
    const float t = 1.0f - 2.0f * __frcp_rn(ex2(2.0f * LOG2E * a) + 1.0f);
    return x < 0.0f ? -t : t;
}

// The two fp16 terms of two values.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// The four codes of a word as two exact fp16 pairs.
template <int KIND>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &p01, uint32_t &p23) {
    if constexpr (KIND == GQ_KV_I8) q8_to_f16x2(w, p01, p23);
    else e4m3x4_to_f16x2(w, p01, p23);
}
// A sequence's part of the step, as far as the slice goes: its rows there, as if those before
// had been held already (end is the whole step's).  One whose lengths are out of range keeps its
// rows, if cu itself is sound, and has no tokens (end = 0): its outputs are zero.
__device__ __forceinline__ SeqStep attn_step(const AttnParams8 &p, int b) {
    SeqStep s = seq_step(p.c, p.cu, b, p.T, p.max_n);
    if (s.bad) {
        const int t1 = p.cu[b + 1];
        const bool rows = s.t0 >= 0 && t1 > s.t0 && t1 <= p.T;   // (more than max_n too)
        s.n = rows ? t1 - s.t0 : 0;
        s.held = s.seen = 0;
    }
    const int off = max(0, p.row0 - s.t0);
    s.n = max(0, min(s.n - off, p.row1 - s.t0 - off));
    s.t0 += off;
    s.held += off;
    s.seen += off;
    return s;
}

// A call for the sequences with many query rows (attn_pages_tc.cu): those with more than
// `rows_over` rows per KV head.
size_t attn_pages_tc_workspace(const gq_kv_pages &c, int64_t rows, int64_t G);
gq_status launch_attn_pages_tc(const AttnParams8 &p, const gq_kv_pages &c, uint8_t *work, cudaStream_t s);

}  // namespace gq

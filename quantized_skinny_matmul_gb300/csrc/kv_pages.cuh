// kv_pages.cuh -- what the kernels of the paged 8-bit KV cache share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gq_common.cuh"
#include "gq_internal.h"

namespace gq {

// gq_kv_pages as the kernels take it.
struct PagesView {
    uint8_t *k, *v;
    float *ks, *vs;
    int32_t *table, *base;
    const int32_t *held, *seen;
    unsigned int *status;
    int B, Hkv, NB, P, pages;
};

gq_status pages_view(const gq_kv_pages &c, PagesView *v);
// A launch that may start before the grid in front has finished (its kernels wait for it).
gq_status launch_pdl(const void *fn, dim3 grid, dim3 block, size_t smem, cudaStream_t s, void **args, const char *what);

// One sequence's part of a step, checked: a sequence whose lengths are out of range has no
// new tokens (n = 0) and is reported by `bad`.  (seen >= held: the attention's choice of slots
// rests on no position being below its slot.)
struct SeqStep {
    int t0, n, held, seen;   // first packed row, new tokens, tokens held before, position of the first new one
    int end;                 // tokens held after
    bool bad;
};

__device__ __forceinline__ SeqStep seq_step(const PagesView &c, const int32_t *cu, int b, int T, int max_n) {
    SeqStep s;
    const int t1 = cu[b + 1];
    s.t0 = cu[b];
    s.held = c.held[b];
    s.seen = c.seen[b];
    const int64_t n = (int64_t)t1 - s.t0;
    s.bad = s.t0 < 0 || n < 0 || n > max_n || t1 > T || s.held < 0 || (int64_t)s.held + n > (int64_t)c.NB * c.P ||
            s.seen < s.held || (int64_t)s.seen + n > (1LL << 30);
    s.n = s.bad ? 0 : (int)n;
    s.end = s.bad ? 0 : s.held + s.n;
    return s;
}

// The four e4m3 codes of a word as two exact fp16 pairs: bytes (0, 1) and (2, 3).
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t &p01, uint32_t &p23) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(p01), "=r"(p23)
        : "r"(w));
}

}  // namespace gq

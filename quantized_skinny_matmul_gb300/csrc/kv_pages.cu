// kv_pages.cu -- the 8-bit KV cache in pages: append, read back, eviction.
//
// A page holds P tokens of one (sequence, KV head), D codes of 8 bits each, with one f32
// scale for its keys and one for its values (layouts and definitions: gq.h).  The three
// operators here move or choose pages; the attention over them is in attn_pages.cu.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "gq_common.cuh"
#include "gq_internal.h"
#include "kv_pages.cuh"

namespace gq {
namespace {

#define KV_TRY(expr)                  \
    do {                              \
        gq_status _st = (expr);       \
        if (_st != GQ_OK) return _st; \
    } while (0)

// ---------------------------------------------------------------------------
// Codes.  The code of a value x under the scale s is the 8-bit value nearest to the exact
// quotient x / s, ties to the even code.  The quotient is formed as x * r with r = 1 / s
// rounded (within 2^-22 relative of x / s); only a quotient that close to the border
// between two codes is decided exactly, from the sign of x - border * s: both products are
// within 2^-14 of each other there, so the fused multiply-add that subtracts them is exact.
// A held token's value is the product code * old scale, carried as p + pe (p rounded, pe
// its exact remainder); pe joins the sign.
// Scales below 2^-60 are first multiplied, with the values, by 2^64 (no underflow of r, pe).
// ---------------------------------------------------------------------------
struct Scale8 {
    float d, r, m;   // the scale times m, 1 / d (0 for a zero scale), m = 1 or 2^64
    bool small;      // m is not 1
};

__device__ __forceinline__ Scale8 scale8(float s) {
    Scale8 q;
    q.small = s < 0x1p-60f;
    q.m = q.small ? 0x1p64f : 1.0f;
    q.d = s * q.m;
    q.r = q.d == 0.0f ? 0.0f : 1.0f / q.d;
    return q;
}

// Is y too near a border between codes for its rounding to be trusted?  (y is off by at most
// 3 units in its last place: for INT8 at most 2^-15; for e4m3 of the 20 bits that the three
// mantissa bits leave.  Below 2^-6, where e4m3 steps are fixed, every value is looked at.)
template <int KIND>
__device__ __forceinline__ bool code_unsure(float y) {
    if constexpr (KIND == GQ_KV_I8) return !(fabsf(y - rintf(y)) < 0.5f - 0x1p-15f);
    const uint32_t b = __float_as_uint(y) & 0x7fffffffu;
    return b < 0x3C800000u || ((b - 0x7FFFCu) & 0xFFFFFu) < 8u;
}

// The 8-bit value (not the code) nearest to (a + ae) / d, given y near that quotient.
template <int KIND>
__device__ __forceinline__ float value_exact(float y, float a, float ae, float d) {
    const float ay = fabsf(y);
    float lo, step;   // the value at or below |y| and the distance to the next one
    bool odd;         // whether lo's code is odd (then a tie goes up)
    if (KIND == GQ_KV_I8) {
        lo = floorf(ay);
        step = 1.0f;
        odd = ((int)lo & 1) != 0;
    } else if (ay >= 0x1p-6f) {
        const uint32_t b = __float_as_uint(ay);
        lo = __uint_as_float(b & ~0xFFFFFu);
        step = __uint_as_float((b & 0x7F800000u) - (3u << 23));
        odd = ((b >> 20) & 1u) != 0;
    } else {
        const float k = floorf(ay * 512.0f);
        lo = k * 0x1p-9f;
        step = 0x1p-9f;
        odd = ((int)k & 1) != 0;
    }
    const float h = lo + 0.5f * step;
    // near the border x - h d is exact, so adding the remainder keeps the sign of the whole
    const bool neg = a < 0.0f;
    const float e = fmaf(-h, d, fabsf(a)) + (neg ? -ae : ae);
    const float v = (e > 0.0f || (e == 0.0f && odd)) ? lo + step : lo;
    return neg ? -v : v;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ int clamp127(float v) { return (int)fminf(fmaxf(v, -127.0f), 127.0f); }

// Four codes from four values v (+ remainders e, for held tokens), already times s.m: the nearest
// codes of the quotients, and, where some lane of the warp has one next to a border, the exact
// ones in their place (a few warps in a hundred; all 32 lanes call this).  Scales next to the
// smallest, where INT8 quotients may pass 127, always take the second way.
template <int KIND>
__device__ __forceinline__ uint32_t encode4(float4 v, float4 e, const Scale8 &s, bool live) {
    const float y[4] = {v.x * s.r, v.y * s.r, v.z * s.r, v.w * s.r};
    uint32_t code;
    bool unsure;
    if constexpr (KIND == GQ_KV_I8) {
        // the nearest integer in the low mantissa bits of y + 1.5 * 2^23
        uint32_t t[4];
        float off = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float z = y[i] + 12582912.0f;
            t[i] = __float_as_uint(z);
            off = fmaxf(off, fabsf(y[i] - (z - 12582912.0f)));
        }
        code = pack_bytes((int)t[0], (int)t[1], (int)t[2], (int)t[3]);
        unsure = !(off < 0.5f - 0x1p-15f) || s.small;
    } else {
        uint32_t least = 0x7fffffffu, near = 0xFFFFFu;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t b = __float_as_uint(y[i]) & 0x7fffffffu;
            least = min(least, b);
            near = min(near, (b - 0x7FFFCu) & 0xFFFFFu);
        }
        code = e4m3x4(y[0], y[1], y[2], y[3]);
        unsure = least < 0x3C800000u || near < 8u;
    }
    if (__any_sync(0xffffffffu, unsure && live)) {
        const float a[4] = {v.x, v.y, v.z, v.w}, ae[4] = {e.x, e.y, e.z, e.w};
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; i++) x[i] = code_unsure<KIND>(y[i]) ? value_exact<KIND>(y[i], a[i], ae[i], s.d) : y[i];
        if constexpr (KIND == GQ_KV_I8)
            code = pack_bytes(clamp127(rintf(x[0])), clamp127(rintf(x[1])), clamp127(rintf(x[2])), clamp127(rintf(x[3])));
        else
            code = e4m3x4(x[0], x[1], x[2], x[3]);
    }
    return s.r == 0.0f ? 0u : code;
}

// The values of four codes.
template <int KIND>
__device__ __forceinline__ float4 decode4(uint32_t w) {
    if constexpr (KIND == GQ_KV_I8) {
        return make_float4((float)(int8_t)(w & 0xff), (float)(int8_t)((w >> 8) & 0xff), (float)(int8_t)((w >> 16) & 0xff),
                           (float)(int8_t)(w >> 24));
    } else {
        uint32_t lo, hi;
        e4m3x4_to_f16x2(w, lo, hi);
        return make_float4(half_lo(lo), half_hi(lo), half_lo(hi), half_hi(hi));
    }
}

// ---------------------------------------------------------------------------
// Append.  One CTA per page that may get tokens, for keys or values (blockIdx.y): thread
// (row group, 4 columns) loads its share of the page's new rows at once into registers, the
// CTA takes their largest magnitude, and the codes go out from the registers: one pass over
// the input, bound by memory (5 bytes per value).  Held rows are only read when the page's
// scale grows.  Prompts of 8 x 2047 tokens x 32 heads, written and read back: 113 us, 77% of a
// copy's rate (158 with every code decided exactly and heads read one by one).
// ---------------------------------------------------------------------------
constexpr int AP_THREADS = 256;

struct AppendParams {
    PagesView c;
    const float *x[2];
    int64_t ld[2];
    const int32_t *cu;
    int T, max_n, blocks;   // blocks: pages a sequence's new tokens can touch
};

template <int KIND, int P, int D>
__global__ void __launch_bounds__(AP_THREADS) kv_pages_append_kernel(const AppendParams p) {
    constexpr int Q = D / 4, RP = AP_THREADS / Q, R = P / RP;   // columns of 4, rows per pass, rows per thread
    static_assert(P % RP == 0, "page rows");
    __shared__ float wmax[AP_THREADS / 32];
    const PagesView &c = p.c;
    pdl_launch_dependents();
    const int jb = blockIdx.x % p.blocks, bh = blockIdx.x / p.blocks, b = bh / c.Hkv, h = bh % c.Hkv;
    const int kv = blockIdx.y;
    pdl_wait();
    const SeqStep q = seq_step(c, p.cu, b, p.T, p.max_n);
    if (q.bad && threadIdx.x == 0 && jb == 0) atomicOr(c.status, STATUS_RANGE);
    if (q.n == 0) return;
    const int j = q.held / P + jb, s0 = j * P;   // page of the sequence, its first slot
    if (s0 >= q.held + q.n) return;
    const int fill = max(0, q.held - s0);        // held rows of the page
    const int end = min(P, q.held + q.n - s0);   // rows in use after the step
    const int page = c.table[(int64_t)bh * c.NB + j];
    if ((unsigned)page >= (unsigned)c.pages) {
        if (threadIdx.x == 0) atomicOr(c.status, STATUS_RANGE);
        return;
    }
    const int col = threadIdx.x % Q, r0 = threadIdx.x / Q;
    const float *x = p.x[kv] + (int64_t)h * D + 4 * col;
    const int64_t ld = p.ld[kv];
    const int trow = q.t0 + s0 - q.held;         // packed row of the page's row 0 (rows >= fill exist)
    float4 v[R];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < R; i++) {
        const int r = r0 + i * RP;
        v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r >= fill && r < end) v[i] = ldg_f4(x + (int64_t)(trow + r) * ld);
    }
#pragma unroll
    for (int i = 0; i < R; i++) amax = fmaxf(amax, absmax4(v[i]));
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = amax;
    float *scale = (kv ? c.vs : c.ks) + page;
    const float old = fill > 0 ? *scale : 0.0f;
    __syncthreads();   // every thread has read the old scale, too
    amax = wmax[0];
#pragma unroll
    for (int w = 1; w < AP_THREADS / 32; w++) amax = fmaxf(amax, wmax[w]);
    const float snew = fmaxf(old, amax / (KIND == GQ_KV_I8 ? 127.0f : 448.0f));
    const Scale8 s = scale8(snew);
    uint8_t *codes = (kv ? c.v : c.k) + ((int64_t)page * P) * D + 4 * col;
    const bool grow = fill > 0 && snew > old;
    const float om = old * s.m;
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < R; i++) {
        const int r = r0 + i * RP;
        uint32_t *at = reinterpret_cast<uint32_t *>(codes + r * D);
        const bool fresh = r >= fill && r < end;
        const float4 a = make_float4(v[i].x * s.m, v[i].y * s.m, v[i].z * s.m, v[i].w * s.m);
        const uint32_t code = encode4<KIND>(a, zero, s, fresh);
        if (fresh) *at = code;
    }
    if (grow)   // held tokens, coded again
        for (int i = 0; i < R; i++) {
            const int r = r0 + i * RP;
            uint32_t *at = reinterpret_cast<uint32_t *>(codes + r * D);
            const float4 k = decode4<KIND>(r < fill ? *at : 0u);
            const float4 a = make_float4(k.x * om, k.y * om, k.z * om, k.w * om);
            const float4 e = make_float4(fmaf(k.x, om, -a.x), fmaf(k.y, om, -a.y), fmaf(k.z, om, -a.z), fmaf(k.w, om, -a.w));
            const uint32_t code = encode4<KIND>(a, e, s, r < fill);
            if (r < fill) *at = code;
        }
    if (threadIdx.x == 0) {
        *scale = snew;
        if (kv == 0 && fill == 0) c.base[(int64_t)bh * c.NB + j] = q.seen + s0 - q.held;
    }
}

// ---------------------------------------------------------------------------
// Read back.  A warp takes RD_TOKENS tokens of one head, keys or values: their pages (two at most,
// as a page holds 16 tokens and more), then all their codes at once, then the f32 rows.  Bound by
// the f32 stores.
// ---------------------------------------------------------------------------
constexpr int RD_THREADS = 256, RD_TOKENS = 8;

struct ReadParams {
    PagesView c;
    float *out[2];
    const int32_t *start, *cu;
    int T, max_n, tiles, heads;   // tiles of tokens, groups of RD_THREADS / 32 heads
};

template <int KIND, int D>
__global__ void __launch_bounds__(RD_THREADS) kv_pages_read_kernel(const ReadParams p, int logP) {
    constexpr int Q = D / 4, PER = 32 / Q, N = RD_TOKENS / PER;   // columns of 4, tokens per access, accesses
    const PagesView &c = p.c;
    pdl_launch_dependents();
    const int hg = blockIdx.x % p.heads, tile = blockIdx.x / p.heads % p.tiles, b = blockIdx.x / p.heads / p.tiles;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = hg * (RD_THREADS / 32) + warp;
    float *out = p.out[blockIdx.y];
    pdl_wait();
    const int t0 = p.cu[b], t1 = p.cu[b + 1], s0 = p.start[b];
    const int64_t n = (int64_t)t1 - t0;
    if (t0 < 0 || n < 0 || n > p.max_n || t1 > p.T || s0 < 0 || s0 + n > ((int64_t)c.NB << logP)) {
        if (threadIdx.x == 0 && tile == 0) atomicOr(c.status, STATUS_RANGE);
        // rows of zeros, if cu itself is sound: this warp's head, the tiles' tokens in turn
        if (out && h < c.Hkv && t0 >= 0 && t1 <= p.T)
            for (int64_t i = tile; i < n; i += p.tiles)
                for (int x = lane; x < Q; x += 32)
                    reinterpret_cast<float4 *>(out + ((t0 + i) * c.Hkv + h) * D)[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        return;
    }
    const int i0 = tile * RD_TOKENS, ni = min(RD_TOKENS, (int)n - i0), slot = s0 + i0;
    if (ni <= 0 || !out || h >= c.Hkv) return;
    const uint8_t *pool = blockIdx.y ? c.v : c.k;
    const float *scale = blockIdx.y ? c.vs : c.ks;
    const int j0 = slot >> logP, j1 = (slot + ni - 1) >> logP;   // the pages of the first and of the last token
    const int32_t *row = c.table + ((int64_t)b * c.Hkv + h) * c.NB;
    int page[2] = {__ldg(row + j0), __ldg(row + j1)};
    float s[2];
#pragma unroll
    for (int e = 0; e < 2; e++) {
        const bool bad = (unsigned)page[e] >= (unsigned)c.pages;
        if (bad && lane == 0) atomicOr(c.status, STATUS_RANGE);
        if (bad) page[e] = -1;   // its tokens are zero
        s[e] = bad ? 0.0f : __ldg(scale + page[e]);
    }
    const int col = lane % Q, part = lane / Q;
    uint32_t w[N];
#pragma unroll
    for (int x = 0; x < N; x++) {
        const int i = x * PER + part, sl = slot + i, pg = sl >> logP == j0 ? page[0] : page[1];
        w[x] = 0u;
        if (i < ni && pg >= 0)
            w[x] = __ldg(reinterpret_cast<const uint32_t *>(pool + (((int64_t)pg << logP) + (sl & ((1 << logP) - 1))) * D) + col);
    }
#pragma unroll
    for (int x = 0; x < N; x++) {
        const int i = x * PER + part, sl = slot + i, e = sl >> logP == j0 ? 0 : 1;
        float4 f = decode4<KIND>(w[x]);
        f.x *= s[e];
        f.y *= s[e];
        f.z *= s[e];
        f.w *= s[e];
        if (i < ni)
            reinterpret_cast<float4 *>(out + ((int64_t)(t0 + i0 + i) * c.Hkv + h) * D)[col] = f;
    }
}

// ---------------------------------------------------------------------------
// Eviction.  One CTA per (sequence, KV head).  The row's weights become ordered integer keys in
// shared memory; the key of the last page that stays is found from the top, a byte a pass: counts
// of the byte's values among the keys that share the bytes before, which every warp then reads for
// itself (one barrier a pass; 16 passes of 2 bits by comparing, without counters in shared memory,
// cost 2.5 times the instructions).  Then each warp places its stretch of the row: a page's
// place among those that stay follows from how many before it are larger or must stay, and how
// many are equal.  Counts only: the result does not depend on timing.  All of the row is in
// shared memory before anything is written, so the outputs may be the inputs.  Bound by latency
// (few rows) or by instructions: 32 sequences x 32 heads x 2048 pages 22 us, 1.4 TB/s of the 24 bytes a
// page (keys counted from the row's least one, so that the first byte spreads: 22 as well).
// ---------------------------------------------------------------------------
constexpr int EV_MAX_WARPS = 32;

struct EvictParams {
    const int32_t *table, *base, *held;
    const float *w;
    int32_t *table_out, *base_out, *held_out;
    float *w_out;
    unsigned int *status;
    int Hkv, NB, P, budget, first, last;
    bool write_held;
};

__device__ __forceinline__ uint32_t order_key(float w) {   // larger weight, larger key; -0 like 0
    const uint32_t b = __float_as_uint(w + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int pages_in_use(int held, int P, int NB, bool &bad) {
    bad = held < 0 || (int64_t)held > (int64_t)NB * P;
    return bad ? 0 : (held + P - 1) / P;
}

__global__ void __launch_bounds__(EV_MAX_WARPS * 32) kv_pages_evict_kernel(const EvictParams p) {
    extern __shared__ uint32_t ev_smem[];
    __shared__ __align__(16) int hist[4][256];
    __shared__ int sure[EV_MAX_WARPS], ties[EV_MAX_WARPS];
    uint32_t *key = ev_smem;
    int32_t *tab = reinterpret_cast<int32_t *>(ev_smem + p.NB), *bas = tab + p.NB;
    const int bh = blockIdx.x, b = bh / p.Hkv, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int threads = blockDim.x, warps = threads >> 5;
    const int64_t row = (int64_t)bh * p.NB;
    pdl_launch_dependents();
    pdl_wait();
    const int held = p.held[b];
    bool bad;
    const int n = pages_in_use(held, p.P, p.NB, bad);
    if (bad && tid == 0) atomicOr(p.status, STATUS_RANGE);
    const bool evict = n > p.budget;
    if (tid == 0 && bh % p.Hkv == 0 && p.write_held) p.held_out[b] = evict ? held - (n - p.budget) * p.P : held;
    // the tail, and whole rows that lose nothing, are copied
    for (int i = (evict ? n : 0) + tid; i < p.NB; i += threads) {
        if (p.table_out != p.table) p.table_out[row + i] = p.table[row + i];
        if (p.base_out != p.base) p.base_out[row + i] = p.base[row + i];
        if (p.w_out != p.w) p.w_out[row + i] = p.w[row + i];
    }
    if (!evict) return;
    for (int i = tid; i < 4 * 256; i += threads) hist[i >> 8][i & 255] = 0;
#pragma unroll 4
    for (int i = tid; i < n; i += threads) {
        key[i] = order_key(p.w[row + i]);
        tab[i] = p.table[row + i];
        bas[i] = p.base[row + i];
    }
    __syncthreads();
    // ---- the want-th largest key among the middle pages
    const int m0 = p.first, m1 = n - p.last, want = p.budget - p.first - p.last;
    uint32_t cut = 0;
    if (want > 0) {
        int left = want;   // among the keys that share the bytes found so far
#pragma unroll 1
        for (int pass = 0; pass < 4; pass++) {
            const int shift = 24 - 8 * pass;
            for (int i = m0 + tid; i < m1; i += threads) {
                const uint32_t k = key[i];
                if (pass == 0 || (k ^ cut) >> (shift + 8) == 0) atomicAdd(&hist[pass][(k >> shift) & 255u], 1);
            }
            __syncthreads();
            // lane l has the counts of the bytes 255 - 8 l .. 248 - 8 l, from the top
            const int4 lo = *reinterpret_cast<const int4 *>(&hist[pass][248 - 8 * lane]);
            const int4 hi = *reinterpret_cast<const int4 *>(&hist[pass][252 - 8 * lane]);
            const int c[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
            int sum = 0;
#pragma unroll
            for (int i = 0; i < 8; i++) sum += c[i];
            int inc = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += t;
            }
            int above = inc - sum, digit = 0, rest = 0;
            const bool here = above < left && inc >= left;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                if (above < left && above + c[i] >= left) {
                    digit = 255 - 8 * lane - i;
                    rest = left - above;
                }
                above += c[i];
            }
            const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
            cut |= (uint32_t)__shfl_sync(0xffffffffu, digit, from) << shift;
            left = __shfl_sync(0xffffffffu, rest, from);
        }
    }
    // ---- places.  Warp w has the pages from w * span on.
    const int span = ((n + warps - 1) / warps + 31) & ~31, i0 = wid * span, i1 = min(n, i0 + span);
    auto kind = [&](int i) {   // 2: stays for sure, 1: equal to the cut, 0: dropped
        const uint32_t k = key[i];
        return i < m0 || i >= m1 ? 2 : want <= 0 ? 0 : k > cut ? 2 : k == cut ? 1 : 0;
    };
    int larger = 0, sures = 0, equal = 0;
    for (int i = i0 + lane; i < i1; i += 32) {
        const int k = kind(i);
        sures += k == 2;
        equal += k == 1;
    }
    sures = __reduce_add_sync(0xffffffffu, sures);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        sure[wid] = sures;
        ties[wid] = equal;
    }
    __syncthreads();
    const int s_all = __reduce_add_sync(0xffffffffu, lane < warps ? sure[lane] : 0);
    larger = __reduce_add_sync(0xffffffffu, lane < wid ? sure[lane] : 0);    // before this warp's stretch
    equal = __reduce_add_sync(0xffffffffu, lane < wid ? ties[lane] : 0);
    const int room = p.budget - s_all;   // of the equal ones, so many stay: the first
    for (int c0 = i0; c0 < i1; c0 += 32) {
        const int i = c0 + lane;
        const int k = i < i1 ? kind(i) : 0;
        const uint32_t ms = __ballot_sync(0xffffffffu, k == 2), mt = __ballot_sync(0xffffffffu, k == 1);
        const uint32_t below = (1u << lane) - 1u;
        const int eq = equal + __popc(mt & below), before = larger + __popc(ms & below) + min(eq, room);
        const bool keep = k == 2 || (k == 1 && eq < room);
        if (i < i1) {
            const int at = keep ? before : p.budget + (i - before);
            p.table_out[row + at] = tab[i];
            p.base_out[row + at] = bas[i];
            const uint32_t q = key[i], fb = q & 0x80000000u ? q & 0x7fffffffu : ~q;
            p.w_out[row + at] = keep ? __uint_as_float(fb) : 0.0f;
        }
        larger += __popc(ms);
        equal += __popc(mt);
    }
}

__global__ void kv_pages_held_kernel(const int32_t *held, int32_t *held_out, int B, int NB, int P, int budget) {
    pdl_wait();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= B) return;
    bool bad;
    const int h = held[b], n = pages_in_use(h, P, NB, bad);
    held_out[b] = n > budget ? h - (n - budget) * P : h;
}

template <int KIND, int P, int D>
gq_status append_launch(const AppendParams &p, int64_t grid, cudaStream_t s) {
    void *args[] = {(void *)&p};
    return launch_pdl((const void *)kv_pages_append_kernel<KIND, P, D>, dim3((unsigned)grid, 2), dim3(AP_THREADS), 0, s,
                      args, "paged append launch");
}

template <int KIND, int D>
gq_status append_page(const AppendParams &p, int P, int64_t grid, cudaStream_t s) {
    switch (P) {
        case 16: return append_launch<KIND, 16, D>(p, grid, s);
        case 32: return append_launch<KIND, 32, D>(p, grid, s);
        case 64: return append_launch<KIND, 64, D>(p, grid, s);
    }
    return append_launch<KIND, 128, D>(p, grid, s);
}

int log2_of(int64_t x) {
    int l = 0;
    while ((1LL << l) < x) l++;
    return l;
}

}  // namespace

gq_status launch_pdl(const void *fn, dim3 grid, dim3 block, size_t smem, cudaStream_t s, void **args, const char *what) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return check_cuda(cudaLaunchKernelExC(&cfg, fn, args), what);
}

gq_status pages_view(const gq_kv_pages &c, PagesView *v) {
    v->k = static_cast<uint8_t *>(c.k);
    v->v = static_cast<uint8_t *>(c.v);
    v->ks = c.ks;
    v->vs = c.vs;
    v->table = c.table;
    v->base = c.base;
    v->held = c.held;
    v->seen = c.seen;
    v->B = (int)c.B;
    v->Hkv = (int)c.Hkv;
    v->NB = (int)c.NB;
    v->P = (int)c.P;
    v->pages = (int)c.pages;
    v->status = device_status_word();
    return v->status ? GQ_OK : fail(GQ_ERR_CUDA, "device status word unavailable");
}

gq_status launch_kv_pages_append(const gq_kv_pages &c, const float *k, int64_t ldk, const float *v, int64_t ldv,
                                 const int32_t *cu, int64_t T, int64_t max_n, cudaStream_t s) {
    AppendParams p{};
    KV_TRY(pages_view(c, &p.c));
    p.x[0] = k;
    p.x[1] = v;
    p.ld[0] = ldk;
    p.ld[1] = ldv;
    p.cu = cu;
    p.T = (int)T;
    p.max_n = (int)max_n;
    p.blocks = (int)((max_n + c.P - 2) / c.P + 1);   // max_n tokens from the last row of a page on
    const int64_t grid = c.B * c.Hkv * p.blocks;
    if (grid > INT32_MAX) return fail(GQ_ERR_INVALID_ARG, "append grid too large");
    if (c.kind == GQ_KV_I8)
        return c.D == 64 ? append_page<GQ_KV_I8, 64>(p, (int)c.P, grid, s) : append_page<GQ_KV_I8, 128>(p, (int)c.P, grid, s);
    return c.D == 64 ? append_page<GQ_KV_E4M3, 64>(p, (int)c.P, grid, s)
                     : append_page<GQ_KV_E4M3, 128>(p, (int)c.P, grid, s);
}

gq_status launch_kv_pages_read(const gq_kv_pages &c, const int32_t *start, const int32_t *cu, int64_t T, int64_t max_n,
                               float *k, float *v, cudaStream_t s) {
    ReadParams p{};
    KV_TRY(pages_view(c, &p.c));
    p.out[0] = k;
    p.out[1] = v;
    p.start = start;
    p.cu = cu;
    p.T = (int)T;
    p.max_n = (int)max_n;
    p.tiles = (int)((max_n + RD_TOKENS - 1) / RD_TOKENS);
    p.heads = (int)((c.Hkv + RD_THREADS / 32 - 1) / (RD_THREADS / 32));
    const int64_t grid = c.B * p.tiles * p.heads;
    if (grid > INT32_MAX) return fail(GQ_ERR_INVALID_ARG, "read grid too large");
    int logP = log2_of(c.P);
    void *args[] = {(void *)&p, (void *)&logP};
    const void *fn = c.kind == GQ_KV_I8
                         ? (c.D == 64 ? (const void *)kv_pages_read_kernel<GQ_KV_I8, 64> : (const void *)kv_pages_read_kernel<GQ_KV_I8, 128>)
                         : (c.D == 64 ? (const void *)kv_pages_read_kernel<GQ_KV_E4M3, 64>
                                      : (const void *)kv_pages_read_kernel<GQ_KV_E4M3, 128>);
    return launch_pdl(fn, dim3((unsigned)grid, 2), dim3(RD_THREADS), 0, s, args, "paged read launch");
}

gq_status launch_kv_pages_evict(const gq_kv_pages &c, const float *w, int64_t budget, int64_t keep_first,
                                int64_t keep_last, int32_t *table_out, int32_t *base_out, float *w_out,
                                int32_t *held_out, cudaStream_t s) {
    EvictParams p{};
    p.table = c.table;
    p.base = c.base;
    p.held = c.held;
    p.w = w;
    p.table_out = table_out;
    p.base_out = base_out;
    p.held_out = held_out;
    p.w_out = w_out;
    p.status = device_status_word();
    if (!p.status) return fail(GQ_ERR_CUDA, "device status word unavailable");
    p.Hkv = (int)c.Hkv;
    p.NB = (int)c.NB;
    p.P = (int)c.P;
    p.budget = (int)std::min<int64_t>(budget, c.NB);   // a row never has more pages: nothing is dropped
    p.first = (int)keep_first;
    p.last = (int)keep_last;
    // the rows of one sequence all read held[b]: in place it is written by a launch of its own
    p.write_held = held_out != c.held;
    const size_t smem = (size_t)c.NB * 12;
    // eight pages a thread; many small CTAs hide each other's latency (2,048 pages: 24 KB, 8 CTAs an SM)
    const unsigned threads = (unsigned)std::min<int64_t>(EV_MAX_WARPS * 32, std::max<int64_t>(64, (c.NB / 8 + 31) / 32 * 32));
    static std::atomic<bool> smem_set[64];
    int dev = 0;
    KV_TRY(check_cuda(cudaGetDevice(&dev), "cudaGetDevice"));
    if (dev < 0 || dev >= 64) return fail(GQ_ERR_UNSUPPORTED_DEVICE, "device index %d", dev);
    if (!smem_set[dev].load(std::memory_order_acquire)) {
        KV_TRY(check_cuda(cudaFuncSetAttribute(kv_pages_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               16384 * 12),
                          "eviction shared-memory attribute"));
        smem_set[dev].store(true, std::memory_order_release);
    }
    void *args[] = {(void *)&p};
    KV_TRY(launch_pdl((const void *)kv_pages_evict_kernel, dim3((unsigned)(c.B * c.Hkv)), dim3(threads), smem, s, args,
                      "eviction launch"));
    if (!p.write_held) {
        const int32_t *held = c.held;
        int B = (int)c.B;
        void *hargs[] = {(void *)&held, (void *)&held_out, (void *)&B, (void *)&p.NB, (void *)&p.P, (void *)&p.budget};
        KV_TRY(launch_pdl((const void *)kv_pages_held_kernel, dim3((unsigned)((B + 255) / 256)), dim3(256), 0, s, hargs,
                          "eviction lengths launch"));
    }
    return GQ_OK;
}

}  // namespace gq

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
};

__device__ __forceinline__ Scale8 scale8(float s) {
    Scale8 q;
    q.m = s < 0x1p-60f ? 0x1p64f : 1.0f;
    q.d = s * q.m;
    q.r = q.d == 0.0f ? 0.0f : 1.0f / q.d;
    return q;
}

// Is y too near a border between codes for its rounding to be trusted?  (y is off by at most
// 2 units in its last place: for INT8 at most 2^-16; for e4m3 two steps of the 20 bits that
// the three mantissa bits leave, or 2^-20 of a step below 2^-6, where the step is fixed.)
template <int KIND>
__device__ __forceinline__ bool code_unsure(float y) {
    if constexpr (KIND == GQ_KV_I8) {
        return !(fabsf(y - rintf(y)) < 0.5f - 0x1p-15f);
    } else {
        const uint32_t b = __float_as_uint(y) & 0x7fffffffu;
        const float t = fabsf(y) * 512.0f;
        return b >= 0x3C800000u ? ((b & 0xFFFFFu) - 0x80000u + 4u) < 8u : !(fabsf(t - rintf(t)) < 0.5f - 0x1p-15f);
    }
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

// Four codes from four values v (+ remainders e, for held tokens), already times s.m.
template <int KIND>
__device__ __forceinline__ uint32_t encode4(float4 v, float4 e, const Scale8 &s) {
    float y[4] = {v.x * s.r, v.y * s.r, v.z * s.r, v.w * s.r};
    const float a[4] = {v.x, v.y, v.z, v.w}, ae[4] = {e.x, e.y, e.z, e.w};
    if (s.r == 0.0f) return 0u;
#pragma unroll
    for (int i = 0; i < 4; i++)
        if (code_unsure<KIND>(y[i])) y[i] = value_exact<KIND>(y[i], a[i], ae[i], s.d);
    if constexpr (KIND == GQ_KV_I8)
        return pack_bytes(clamp127(rintf(y[0])), clamp127(rintf(y[1])), clamp127(rintf(y[2])), clamp127(rintf(y[3])));
    else
        return e4m3x4(y[0], y[1], y[2], y[3]);
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
// scale grows.
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
        if (r < fill) {
            if (!grow) continue;
            const float4 k = decode4<KIND>(*at);
            const float4 a = make_float4(k.x * om, k.y * om, k.z * om, k.w * om);
            const float4 e = make_float4(fmaf(k.x, om, -a.x), fmaf(k.y, om, -a.y), fmaf(k.z, om, -a.z), fmaf(k.w, om, -a.w));
            *at = encode4<KIND>(a, e, s);
        } else if (r < end) {
            const float4 a = make_float4(v[i].x * s.m, v[i].y * s.m, v[i].z * s.m, v[i].w * s.m);
            *at = encode4<KIND>(a, zero, s);
        }
    }
    if (threadIdx.x == 0) {
        *scale = snew;
        if (kv == 0 && fill == 0) c.base[(int64_t)bh * c.NB + j] = q.seen + s0 - q.held;
    }
}

// ---------------------------------------------------------------------------
// Read back: a thread turns 4 codes into 4 f32; a CTA takes RD_TOKENS tokens of a sequence,
// all heads.  Bound by the f32 stores.
// ---------------------------------------------------------------------------
constexpr int RD_THREADS = 256, RD_TOKENS = 8;

struct ReadParams {
    PagesView c;
    float *out[2];
    const int32_t *start, *cu;
    int T, max_n, tiles;
};

template <int KIND>
__global__ void __launch_bounds__(RD_THREADS) kv_pages_read_kernel(const ReadParams p, int logP, int logQ) {
    const PagesView &c = p.c;
    pdl_launch_dependents();
    const int tile = blockIdx.x % p.tiles, b = blockIdx.x / p.tiles;
    pdl_wait();
    const int t0 = p.cu[b], n = p.cu[b + 1] - t0, s0 = p.start[b];
    const int64_t cap = (int64_t)c.NB << logP;
    if (t0 < 0 || n < 0 || n > p.max_n || (int64_t)t0 + n > p.T || s0 < 0 || (int64_t)s0 + n > cap) {
        if (threadIdx.x == 0 && tile == 0) atomicOr(c.status, STATUS_RANGE);
        return;
    }
    const int i0 = tile * RD_TOKENS, ni = min(RD_TOKENS, n - i0);
    if (ni <= 0) return;
    float *out = p.out[blockIdx.y];
    if (!out) return;
    const uint8_t *pool = blockIdx.y ? c.v : c.k;
    const float *scale = blockIdx.y ? c.vs : c.ks;
    const int D = 4 << logQ, per = c.Hkv << logQ;   // 4-value columns per token
    const int total = ni * per;
    bool bad = false;
#pragma unroll 4
    for (int x = threadIdx.x; x < total; x += RD_THREADS) {
        const int i = x / per, y = x - i * per, h = y >> logQ, col = y & ((1 << logQ) - 1);
        const int slot = s0 + i0 + i;
        const int page = __ldg(c.table + ((int64_t)b * c.Hkv + h) * c.NB + (slot >> logP));
        if ((unsigned)page >= (unsigned)c.pages) {
            bad = true;
            continue;
        }
        const float s = __ldg(scale + page);
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(
            pool + (((int64_t)page << logP) + (slot & ((1 << logP) - 1))) * D + 4 * col));
        float4 f = decode4<KIND>(w);
        f.x *= s;
        f.y *= s;
        f.z *= s;
        f.w *= s;
        *reinterpret_cast<float4 *>(out + ((int64_t)(t0 + i0 + i) * c.Hkv + h) * D + 4 * col) = f;
    }
    if (bad) atomicOr(c.status, STATUS_RANGE);
}

// ---------------------------------------------------------------------------
// Eviction.  One CTA per (sequence, KV head).  The row's weights become ordered integer
// keys in shared memory; a radix selection (four passes of 8 bits, counts in shared memory)
// finds the key of the last page that stays; then one pass over the row, in order, gives
// every page its place: the pages that stay first, the dropped ones behind them.  Integer
// counts only: the result does not depend on timing.  All of the row is in shared memory
// before anything is written, so the outputs may be the inputs.
// ---------------------------------------------------------------------------
constexpr int EV_THREADS = 512, EV_WARPS = EV_THREADS / 32;

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

__global__ void __launch_bounds__(EV_THREADS) kv_pages_evict_kernel(const EvictParams p) {
    extern __shared__ uint32_t ev_smem[];
    __shared__ int hist[256], warp_a[EV_WARPS], warp_b[EV_WARPS], pick[2];
    uint32_t *key = ev_smem;
    int32_t *tab = reinterpret_cast<int32_t *>(ev_smem + p.NB), *bas = tab + p.NB;
    const int bh = blockIdx.x, b = bh / p.Hkv, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
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
    for (int i = (evict ? n : 0) + tid; i < p.NB; i += EV_THREADS) {
        if (p.table_out != p.table) p.table_out[row + i] = p.table[row + i];
        if (p.base_out != p.base) p.base_out[row + i] = p.base[row + i];
        if (p.w_out != p.w) p.w_out[row + i] = p.w[row + i];
    }
    if (!evict) return;
    for (int i = tid; i < n; i += EV_THREADS) {
        key[i] = order_key(p.w[row + i]);
        tab[i] = p.table[row + i];
        bas[i] = p.base[row + i];
    }
    // the key of rank `want` among the middle pages, digit by digit from the top
    const int m0 = p.first, m1 = n - p.last;
    int want = p.budget - p.first - p.last;   // middle pages that stay; 0: none
    uint32_t prefix = 0;
    if (want > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += EV_THREADS) hist[i] = 0;
            __syncthreads();
            for (int i = m0 + tid; i < m1; i += EV_THREADS)
                if (shift == 24 || (key[i] >> (shift + 8)) == (prefix >> (shift + 8)))
                    atomicAdd(&hist[(key[i] >> shift) & 255], 1);
            __syncthreads();
            if (wid == 0) {   // counts from the top: lane l owns digits 255 - 8l .. 248 - 8l
                int c[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; i++) sum += c[i] = hist[255 - 8 * lane - i];
                int inc = sum;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int t = __shfl_up_sync(0xffffffffu, inc, d);
                    if (lane >= d) inc += t;
                }
                int above = inc - sum;
                if (above < want && inc >= want) {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        if (above < want && above + c[i] >= want) {
                            pick[0] = 255 - 8 * lane - i;
                            pick[1] = want - above;
                            break;
                        }
                        above += c[i];
                    }
                }
            }
            __syncthreads();
            prefix |= (uint32_t)pick[0] << shift;
            want = pick[1];   // of the pages that share this prefix, so many stay
        }
    } else {
        __syncthreads();
    }
    const bool some = p.budget > p.first + p.last;
    // places, in order: EV_THREADS pages at a time with running totals
    int ties = 0, kept = 0;   // equal keys seen, pages kept, before this chunk
    for (int i0 = 0; i0 < n; i0 += EV_THREADS) {
        const int i = i0 + tid;
        const bool in = i < n, mid = in && i >= m0 && i < m1;
        const uint32_t k = in ? key[i] : 0u;
        const bool tie = some && mid && k == prefix;
        const uint32_t tmask = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) warp_a[wid] = __popc(tmask);
        __syncthreads();
        int before = ties, all = 0;
        for (int w = 0; w < EV_WARPS; w++) {
            if (w < wid) before += warp_a[w];
            all += warp_a[w];
        }
        ties += all;
        before += __popc(tmask & ((1u << lane) - 1u));
        const bool keep = in && (!mid || (some && (k > prefix || (tie && before < want))));
        const uint32_t kmask = __ballot_sync(0xffffffffu, keep);
        if (lane == 0) warp_b[wid] = __popc(kmask);
        __syncthreads();
        int place = kept, total = 0;
        for (int w = 0; w < EV_WARPS; w++) {
            if (w < wid) place += warp_b[w];
            total += warp_b[w];
        }
        place += __popc(kmask & ((1u << lane) - 1u));   // pages kept before this one
        kept += total;
        if (in) {
            const int at = keep ? place : p.budget + (i - place);
            p.table_out[row + at] = tab[i];
            p.base_out[row + at] = bas[i];
            const uint32_t fb = k & 0x80000000u ? k & 0x7fffffffu : ~k;
            p.w_out[row + at] = keep ? __uint_as_float(fb) : 0.0f;
        }
        __syncthreads();   // warp_a is rewritten by the next chunk
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
    const int64_t grid = c.B * p.tiles;
    if (grid > INT32_MAX) return fail(GQ_ERR_INVALID_ARG, "read grid too large");
    int logP = log2_of(c.P), logQ = log2_of(c.D / 4);
    void *args[] = {(void *)&p, (void *)&logP, (void *)&logQ};
    return launch_pdl(c.kind == GQ_KV_I8 ? (const void *)kv_pages_read_kernel<GQ_KV_I8>
                                         : (const void *)kv_pages_read_kernel<GQ_KV_E4M3>,
                      dim3((unsigned)grid, 2), dim3(RD_THREADS), 0, s, args, "paged read launch");
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
    KV_TRY(launch_pdl((const void *)kv_pages_evict_kernel, dim3((unsigned)(c.B * c.Hkv)), dim3(EV_THREADS), smem, s, args,
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

// attn_pages.cu -- attention over the paged 8-bit KV cache, for few query rows per KV head.
//
// For a query at position p and the keys at positions x it sees (definition: gq.h),
//     z_x = f(scale * q . k_x, p, x),   out = sum_x softmax(z)_x v_x,
// with k_x = code * (the page's scale).  One pass over the cache with a running maximum and
// sum: a unit of 32 tokens gives scores z (base 2), the maximum m grows to m', the sums so
// far are scaled by 2^(m - m'), and the unit's 2^(z - m') join the denominator and, times
// the values, the output.
//
// Both products run as m16n8k16 fp16 MMAs with f32 accumulation at f32 accuracy: the codes
// widen to fp16 exactly and are the 16-row operand; a query row (scaled by a power of two) or a
// row of weights is carried as two fp16 terms, hi + lo, in two of the 8 columns.  So an MMA
// serves 4 query rows; items have up to 4 (one column tile) or up to 8 (two), and with one, half
// the accumulators of a layout with the query as the 16-row operand.  A lane's scores are those
// of its row (lane mod 4) for tokens g and g + 8 of 16 (g = lane / 4); the values' product takes
// tokens in the order (t, t + 8), (t + 4, t + 12) .., so that a weight pair moves to its place
// with one shuffle a term.  The order in which the MMAs take positions within a row (D) is
// chosen so that every lane reads its 16-byte chunks of codes as they lie in shared memory.
//
// Work is divided evenly, not by sequence: the (sequence, head, row tile) items' units are
// laid out in a line, every CTA takes an equal piece of it, and items cut at a piece's end
// are joined by the CTA that finishes last, in the order of the pieces (so the result does
// not depend on timing).  A producer warp streams the units' pages through a ring of
// shared-memory slots (tensor copies, 128-byte swizzle) and puts each unit's scales and
// positions beside them; seven consumer warps take the units in turn, each with its own
// running maximum and sums, joined at the end of the item.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn_pages.cuh"
#include "gq_common.cuh"
#include "gq_internal.h"

namespace gq {
namespace {

#define KV_TRY(expr)                  \
    do {                              \
        gq_status _st = (expr);       \
        if (_st != GQ_OK) return _st; \
    } while (0)

constexpr int UNIT = 32;                    // tokens per unit
// Consumer warps, and query rows of an item for 1 or 2 column tiles.  Two CTAs of 8 warps fill an
// SM's registers.  128 sequences x 32 heads on 2048 tokens, a row each: 303 us with the query as the
// 16-row operand, 274 with the codes there and slots of 32 tokens, 236 as it is (84% of a copy's
// rate; bound by memory).  Short ones are bound by the steps of an item (about 1 us each: the
// first slot, the query's fragments, the warps' sums joined, the pieces joined): 1 x 500 tokens of 32
// heads takes 13.5 us, 1 x 32768 of 8 heads 28.
constexpr int WARPS = 7;
__host__ __device__ constexpr int rows_of(int NN) { return 4 * NN; }
constexpr int ROWS_MOST = 8;
constexpr int ITEMS = 2;                    // items whose data is kept

// The ring's slots hold two units, 64 tokens' keys and values: the producer's time for a slot (a
// wait, a count of bytes, the copies) is what limits a CTA when slots are small.  They are filled in
// order and read by any warps.  A slot's next phase may be waited for only when the present one is
// over (a parity wait two phases ahead passes at once), and copies land in any order: so a warp
// first waits until the slot's last contents were given back.  That wait itself is never two phases
// ahead: a warp's units are W apart, which is at most W / 2 + 1 slots within an item (its first and
// last slot may hold one unit), and the slot before was filled when the one `slots` earlier was
// given back; and items end together.
__host__ __device__ constexpr int slots_of(int D, int NN) { return (NN == 1 ? 5 : 4) * (D == 128 ? 1 : 2); }
static_assert(slots_of(128, 2) >= WARPS / 2 + 1, "see above");
constexpr int MAX_SLOTS = 10;
// Places for units' data, taken 32 at a time (the last of an item may be few).  What the producer
// overwrites is done: either two items have begun since (ITEMS), or 32 units of one.
constexpr int METAS = 128;
static_assert(ITEMS == 2 && 16 >= MAX_SLOTS, "a unit's data stays until it is done");

// The tensor cores add to their f32 accumulators with truncation, one way: values of one sign that a warp
// sums over 9, 37, 146 and 585 units (a sequence of 2048 .. 131072 tokens in one CTA) came out 0.6, 4, 24
// and 110 e-6 of themselves too small.  So every FLUSH_UNITS units of a warp its sums are added to sums
// in shared memory, rounded to nearest, and begun anew: off by 0.5e-6 at every length (16 units: 1.2e-6).
// 64 sequences x 8 heads on 32768 tokens take 626 us with 4 rows a head and 781 with 8 (without: 623 and
// 757).  Where no warp can have more than FLUSH_FROM units of an item the kernel does without: the
// code alone costs 128 sequences on 2048 tokens 240 us for 235, and 1.2e-6 at most is left.
constexpr int FLUSH_UNITS = 8, FLUSH_FROM = 16;

struct UnitMeta {               // of a unit: scales and first positions of the two halves
    float ks[2], vs[2];
    int base[2];
    int live;                   // tokens of the unit that are held (0 .. 32)
    int lost;                   // bit i: half i has no usable page
};

// A stretch of an item's units that this CTA works on, put there by the producer.
struct ItemRec {
    int64_t item0;              // line position of the item's first unit
    int u0, u1, units;          // units of the stretch, units of the item
    int pre, start;             // its span
    int rows;                   // query rows
    int ti[ROWS_MOST], head[ROWS_MOST], qpos[ROWS_MOST];   // of each row: token, query head, position
    int first[ROWS_MOST], prefix[ROWS_MOST];
    float slope[ROWS_MOST];          // times log2 e
};

struct RowsSmem {
    uint64_t full[MAX_SLOTS], empty[MAX_SLOTS], item_full[ITEMS], item_empty[ITEMS];
    UnitMeta meta[METAS];       // of unit u of an item at (its first unit's place + u) mod METAS
    ItemRec item[ITEMS];
    float ml[WARPS][ROWS_MOST][2];    // maximum and denominator of each warp
    float2 sum_unit[WARPS][ROWS_MOST];   // of each warp's flushed sums: the maximum they are relative to, and vex as 2^vex
    int64_t start, total;       // line position of the sequence that the CTA starts in
    int start_b, last, failed;
    int64_t warp_sum[WARPS + 1];
};

template <int D, int NN>
struct RowsLayout {
    static constexpr int W = WARPS, ROWS = rows_of(NN);
    static constexpr int ring = 0;                                     // [slot]: keys, values of 64 tokens
    static constexpr int q = ring + slots_of(D, NN) * UNIT * D * 4;    // [ITEMS][ROWS][D] f32
    static constexpr int frag = q + ITEMS * ROWS * D * 4;              // the query's MMA fragments
    static constexpr int red = frag + D * 16 * NN;                     // [W][ROWS][D] f32
    static constexpr int ctl = red + W * ROWS * D * 4;
    static constexpr int total = ctl + (int)sizeof(RowsSmem);
    static_assert(2 * (total + 2048) <= 228 * 1024, "two CTAs per SM");
};

template <int N>
__device__ __forceinline__ void consumer_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

// Byte j of x and byte j of y as one exact fp16 pair, j = 0 .. 3.
template <int KIND>
__device__ __forceinline__ void widen_pairs(uint32_t x, uint32_t y, uint32_t (&o)[4]) {
    if constexpr (KIND == GQ_KV_I8) {
        x ^= 0x80808080u;
        y ^= 0x80808080u;
        const uint32_t i01 = __byte_perm(x, y, 0x5140), i23 = __byte_perm(x, y, 0x7362);
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
        uint32_t t[4] = {__byte_perm(i01, 0x64646464u, 0x4140), __byte_perm(i01, 0x64646464u, 0x4342),
                         __byte_perm(i23, 0x64646464u, 0x4140), __byte_perm(i23, 0x64646464u, 0x4342)};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            __half2 h = __hsub2(*reinterpret_cast<__half2 *>(&t[i]), off);
            o[i] = *reinterpret_cast<uint32_t *>(&h);
        }
    } else {
        e4m3x4_to_f16x2(__byte_perm(x, y, 0x5140), o[0], o[1]);
        e4m3x4_to_f16x2(__byte_perm(x, y, 0x7362), o[2], o[3]);
    }
}

// ---- the units of a sequence ------------------------------------------------------------
// Slots that some query of the step can see lie in [0, pre) and [start, n): key positions are
// at least their slot number and distinct, below seen + n, so the slots whose position is at
// least X number at most seen + new - X.
struct Span {
    int pre, start, units;   // units [0, pre) and [start, pre's end ..): `units` in all
};

__device__ __forceinline__ Span span_of(const AttnParams8 &p, const SeqStep &s) {
    Span r;
    const int n = s.end, end = (n + UNIT - 1) >> 5;
    int lo = 0, pre = 0, first = 0;
    if (s.n <= ROWS_MOST) {   // few tokens: look at each one's own range
        if (p.first) {
            first = 0x7fffffff;
            for (int i = 0; i < s.n; i++) first = min(first, p.first[s.t0 + i]);
        }
        if (p.prefix)
            for (int i = 0; i < s.n; i++) pre = max(pre, p.prefix[s.t0 + i]);
    } else if (p.prefix) {
        pre = n;
    }
    if (first > 0) lo = (int)max((int64_t)0, (int64_t)s.held - s.seen + first);
    if (p.window > 0) lo = (int)max((int64_t)lo, (int64_t)s.held - p.window + 1);
    // (whole slots of two units)
    r.start = (min(lo, n - 1) >> 6) * 2;
    r.pre = min(((min(max(pre, 0), n) + 2 * UNIT - 1) >> 6) * 2, r.start);
    r.units = r.pre + end - r.start;
    return r;
}

// Where a piece of work is: the item (sequence b, head h, row tile) and its sequence's data.
struct Cursor {
    int rows;                   // of an item
    int b, h, tile, tiles;
    SeqStep s;
    Span u;
};

__device__ __forceinline__ void load_seq(const AttnParams8 &p, Cursor &k) {
    k.s = attn_step(p, k.b);
    if (k.s.bad) {   // one unit that nobody sees
        k.u.pre = k.u.start = 0;
        k.u.units = 1;
    } else if (k.s.n > 0) {
        k.u = span_of(p, k.s);
    }
    k.tiles = k.s.n * p.G > p.rows_over ? 0 : (k.s.n * p.G + k.rows - 1) / k.rows;
}

__device__ __forceinline__ void next_item(const AttnParams8 &p, Cursor &k) {
    if (++k.tile < k.tiles) return;
    k.tile = 0;
    if (++k.h < p.c.Hkv) return;
    k.h = 0;
    do {
        if (++k.b >= p.c.B) return;
        load_seq(p, k);
    } while (k.tiles == 0);
}

// Joins the pieces of an item that several CTAs worked on, in their order, into its output rows:
// a warp per row, a lane per D / 32 columns.  The lanes first take 32 pieces' maxima and
// denominators each; then every piece's weight goes from its lane to all.
template <int D, int W, int ROWS>
__device__ __forceinline__ void join_pieces(const AttnParams8 &p, const ItemRec &it, int c0, int c1, int warp, int lane) {
    constexpr int V = D / 32;
    const int n = c1 - c0 + 1;
    for (int rr = warp; rr < it.rows; rr += W) {
        // the item begins in CTA c0 (its slot 1); it is the first item of the others (slot 0)
        auto piece = [&](int i) { return ((int64_t)(c0 + i) * 2 + (i == 0)) * ROWS + rr; };
        float mt = -INFINITY;
        for (int i = lane; i < n; i += 32) mt = fmaxf(mt, __ldcg(p.part_ml + piece(i) * 2));
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, d));
        float a[V], l = 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++) a[v] = 0.0f;
        for (int i0 = 0; i0 < n && mt != -INFINITY; i0 += 32) {
            float e = 0.0f, el = 0.0f;
            if (i0 + lane < n) {
                const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + piece(i0 + lane) * 2));
                e = ex2(ml.x - mt);
                el = e * ml.y;
            }
            const int m = min(32, n - i0);
#pragma unroll 8
            for (int i = 0; i < m; i++) {
                const float w = __shfl_sync(0xffffffffu, e, i);
                l += __shfl_sync(0xffffffffu, el, i);
                const float *src = p.parts + piece(i0 + i) * D + V * lane;
                if constexpr (V == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
                    a[0] = fmaf(w, x.x, a[0]);
                    a[1] = fmaf(w, x.y, a[1]);
                    a[2] = fmaf(w, x.z, a[2]);
                    a[3] = fmaf(w, x.w, a[3]);
                } else {
                    const float2 x = __ldcg(reinterpret_cast<const float2 *>(src));
                    a[0] = fmaf(w, x.x, a[0]);
                    a[1] = fmaf(w, x.y, a[1]);
                }
            }
        }
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        float *out = p.out + (int64_t)it.ti[rr] * p.ldo + (int64_t)it.head[rr] * D + V * lane;
        if constexpr (V == 4) *reinterpret_cast<float4 *>(out) = make_float4(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
        else *reinterpret_cast<float2 *>(out) = make_float2(a[0] * inv, a[1] * inv);
        if (p.lse && lane == 0) p.lse[(int64_t)it.ti[rr] * p.Hq + it.head[rr]] = l > 0.0f ? mt + log2f(l) : INFINITY;
    }
}

template <int KIND, int D, int NN, bool FLUSH>
__global__ void __launch_bounds__((WARPS + 1) * 32, 2)
    attn_pages_rows_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                           const AttnParams8 p) {
    using L = RowsLayout<D, NN>;
    constexpr int W = L::W, ROWS = L::ROWS, CONSUMERS = W * 32, THREADS = CONSUMERS + 32;
    constexpr int SLOTS = slots_of(D, NN), HALF = UNIT * D;  // bytes of a unit's keys
    constexpr int KS = D / 16;                               // MMA steps of a score
    constexpr int RUN = D / 4;                               // positions per lane of a score
    constexpr int MT = D / 16;                               // row tiles of the output
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);   // (an offset: the compiler keeps the address space)
    RowsSmem &sm = *reinterpret_cast<RowsSmem *>(smem + L::ctl);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagesView &c = p.c;

    pdl_launch_dependents();
    if (tid == 0) {
        for (int s = 0; s < SLOTS; s++) {
            mbar_init(smem_addr(sm.full + s), 1);
            mbar_init(smem_addr(sm.empty + s), 2);   // a slot's two units
        }
        for (int s = 0; s < ITEMS; s++) {
            mbar_init(smem_addr(sm.item_full + s), 1);
            mbar_init(smem_addr(sm.item_empty + s), W);
        }
        fence_barrier_init();
    }
    pdl_wait();

    // ---- this CTA's piece of the line of units
    {
        const int per = (c.B + THREADS - 1) / THREADS, b0 = tid * per, b1 = min(c.B, b0 + per);
        int64_t mine = 0;
        for (int b = b0; b < b1; b++) {
            Cursor k;
            k.rows = ROWS;
            k.b = b;
            load_seq(p, k);
            if (k.s.bad) atomicOr(c.status, STATUS_RANGE);
            if (k.tiles) mine += (int64_t)k.tiles * c.Hkv * k.u.units;
        }
        int64_t inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += t;
        }
        if (lane == 31) sm.warp_sum[warp] = inc;
        if (tid == 0) sm.failed = 0;
        __syncthreads();
        int64_t before = inc - mine, total = 0;
        for (int w = 0; w < THREADS / 32; w++) {
            if (w < warp) before += sm.warp_sum[w];
            total += sm.warp_sum[w];
        }
        const int64_t piece = max((int64_t)W, (total + gridDim.x - 1) / gridDim.x), lo = piece * blockIdx.x;
        if (lo >= before && lo < before + mine) {
            for (int b = b0; b < b1; b++) {
                Cursor k;
                k.rows = ROWS;
                k.b = b;
                load_seq(p, k);
                const int64_t u = k.tiles ? (int64_t)k.tiles * c.Hkv * k.u.units : 0;
                if (lo < before + u) {
                    sm.start_b = b;
                    sm.start = before;
                    break;
                }
                before += u;
            }
        }
        if (tid == 0) sm.total = total;
        __syncthreads();
    }
    const int64_t total = sm.total, piece = max((int64_t)W, (total + gridDim.x - 1) / gridDim.x);
    const int64_t lo = piece * blockIdx.x, hi = min(total, lo + piece);
    if (lo >= hi) return;

    // ---------------------------------------------------------------- producer
    if (warp == W) {
        Cursor k;
        k.rows = ROWS;
        k.b = sm.start_b;
        load_seq(p, k);
        int64_t item0;   // line position of the item's first unit
        {
            const int64_t i = (lo - sm.start) / k.u.units;
            k.tile = (int)(i % k.tiles);
            k.h = (int)(i / k.tiles);
            item0 = sm.start + i * k.u.units;
        }
        const uint64_t policy = l2_evict_first_policy();
        int count = 0, meta = 0, items = 0;   // slots filled, places for units' data, items
        bool ok = true;
        // Lane l < 8 copies group l mod 4 (16 tokens) of a slot, keys or values (l / 4); where a page holds
        // more, the first group's copy brings up to 64 tokens of it.
        const int per = min(c.P, 2 * UNIT), g = lane & 3;
        const uint32_t copy_bytes = (uint32_t)(per * D), my_dst = (uint32_t)((lane >> 2) * 2 * HALF + g * 16 * D);
        const bool copier = lane < 8 && g * 16 % per == 0;
        const CUtensorMap *my_map = lane < 4 ? &kmap : &vmap;
        for (int64_t at = lo; at < hi && ok;) {
            const int u0 = (int)(at - item0), u1 = (int)min((int64_t)k.u.units, hi - item0);
            const int64_t trow = ((int64_t)k.b * c.Hkv + k.h) * c.NB;
            const int n = k.s.end;
            // ---- the item: its rows (row r is token r / G, head r % G of the group) and queries
            {
                const int st = items % ITEMS, rows = min(ROWS, k.s.n * p.G - k.tile * ROWS);
                const int r = k.tile * ROWS + (lane < rows ? lane : 0), i = r / p.G;
                const int ti = k.s.t0 + i, head = k.h * p.G + r - i * p.G;
                const int first = p.first ? __ldg(p.first + ti) : 0, pre = p.prefix ? min(__ldg(p.prefix + ti), 1 << 30) : 0;
                const float slope = p.slopes ? __ldg(p.slopes + head) * LOG2E : 0.0f;
                if (items >= ITEMS)
                    ok = mbar_wait(smem_addr(sm.item_empty + st), (uint32_t)((items / ITEMS - 1) & 1), c.status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ItemRec &it = sm.item[st];
                if (lane < ROWS) {
                    it.ti[lane] = ti;
                    it.head[lane] = head;
                    it.qpos[lane] = k.s.seen + i;
                    it.first[lane] = first;
                    it.prefix[lane] = pre;
                    it.slope[lane] = slope;
                }
                if (lane == 0) {
                    it.item0 = item0;
                    it.u0 = u0;
                    it.u1 = u1;
                    it.units = k.u.units;
                    it.pre = k.u.pre;
                    it.start = k.u.start;
                    it.rows = rows;
                }
                __syncwarp();
                const uint32_t bar = smem_addr(sm.item_full + st);
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(rows * D * 4));
                __syncwarp();
                if (lane < rows)   // (a lane per row)
                    bulk_g2s(smem_addr(smem + L::q + (st * ROWS + lane) * D * 4), p.q + (int64_t)ti * p.ldq + (int64_t)head * D,
                             (uint32_t)(D * 4), bar);
                __syncwarp();
                items++;
            }
            for (int ub = u0 & ~1; ub < u1 && ok; ub += 32) {
                // each lane looks up one unit: its pages, their scales and positions
                const int u = ub + lane;
                const int slot = (u < k.u.pre ? u : k.u.start + u - k.u.pre) * UNIT;
                UnitMeta m;
                int row[2] = {-1, -1};   // pool rows (128 bytes) of the halves
                m.lost = 0;
                m.live = u >= u0 && u < u1 ? max(0, min(UNIT, n - slot)) : 0;
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    m.ks[i] = m.vs[i] = 0.0f;
                    m.base[i] = 0;
                    if (m.live > 16 * i) {
                        const int j = (slot + 16 * i) >> p.lgP, inpage = (slot + 16 * i) & (c.P - 1);
                        const int pg = __ldg(c.table + trow + j);
                        if ((unsigned)pg < (unsigned)c.pages) {
                            row[i] = (int)(((int64_t)pg * c.P + inpage) * D / 128);
                            m.ks[i] = __ldg(c.ks + pg);
                            m.vs[i] = __ldg(c.vs + pg);
                            m.base[i] = __ldg(c.base + trow + j) + inpage;
                        } else {
                            atomicOr(c.status, STATUS_RANGE);
                            m.base[i] = 0x7f000000;   // a position nobody sees
                            m.lost |= 1 << i;
                        }
                    }
                }
                const int todo = min(32, u1 - ub);
                if (lane < todo) sm.meta[(meta + lane) % METAS] = m;   // (what was there is done: METAS)
                meta += 32;
                __syncwarp();
                for (int i = 0; i < todo; i += 2) {   // units ub + i and the next one
                    // the group's row; where one copy brings all, from the first group that is there
                    const int from = i + (g >> 1);
                    const int ra = __shfl_sync(0xffffffffu, row[0], from), rb = __shfl_sync(0xffffffffu, row[1], from);
                    int r = g & 1 ? rb : ra;
                    if (per == 2 * UNIT) {
                        const uint32_t there = __ballot_sync(0xffffffffu, lane < 4 && r >= 0);
                        const int first = there ? __ffs(there) - 1 : 0;
                        r = __shfl_sync(0xffffffffu, r, first);
                        r = there ? r - first * 16 * D / 128 : -1;
                    }
                    const bool mine = copier && r >= 0;
                    const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * copy_bytes;
                    const int sl = count % SLOTS;
                    if (count >= SLOTS)
                        ok = mbar_wait(smem_addr(sm.empty + sl), (uint32_t)((count / SLOTS - 1) & 1), c.status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t bar = smem_addr(sm.full + sl);
                    if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                    __syncwarp();
                    if (mine) tma_rows(smem_addr(smem + L::ring) + (uint32_t)(sl * 4 * HALF) + my_dst, my_map, r, bar, policy);
                    __syncwarp();
                    count++;
                }
            }
            at = item0 + u1;
            if (u1 == k.u.units) {
                item0 += k.u.units;
                if (at < hi) next_item(p, k);
            }
        }
        // stay until every copy issued has landed: the CTA never ends with a copy in flight
        for (int i = max(0, count - SLOTS); i < count; i++)
            mbar_wait(smem_addr(sm.full + i % SLOTS), (uint32_t)((i / SLOTS) & 1), c.status);
        for (int i = max(0, items - ITEMS); i < items; i++)
            mbar_wait(smem_addr(sm.item_full + i % ITEMS), (uint32_t)((i / ITEMS) & 1), c.status);
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int g8 = lane >> 2, t = lane & 3;
    const uint32_t frag = smem_addr(smem + L::frag) + lane * 8;
    float *red = reinterpret_cast<float *>(smem + L::red);
    int count = 0, slots = 0, metas = 0;   // units, slots, places of units' data before the item
    bool failed = false;
    int64_t at = lo;
    // where this lane's chunks of key rows g8 and of value rows t lie in 16 tokens (D = 64: two rows a
    // 128-byte line)
    uint32_t koff[D / 64], voff;
#pragma unroll
    for (int hh = 0; hh < D / 64; hh++)
        koff[hh] = D == 128 ? g8 * 128 + (((2 * t + hh) ^ g8) << 4) : (g8 >> 1) * 128 + (((4 * (g8 & 1) + t) ^ (g8 >> 1)) << 4);
    voff = D == 128 ? t * 128 + ((g8 ^ t) << 4) : (t >> 1) * 128 + (((4 * (t & 1) + (g8 >> 1)) ^ (t >> 1)) << 4) + 8 * (g8 & 1);
    for (int items = 0; at < hi; items++) {
        const int st = items % ITEMS;
        const ItemRec &it = sm.item[st];
        failed = failed || !mbar_wait(smem_addr(sm.item_full + st), (uint32_t)((items / ITEMS) & 1), c.status);
        // ---- the query rows, scaled by powers of two into [2^14, 2^15), as MMA columns (row r: its hi
        // term column 2r, its lo term 2r + 1).  Lane (g8, t) makes column g8 of each tile, positions
        // RUN t ..; the warps share the work.
        const int nrows = failed ? 0 : it.rows;
        float f[NN];   // of row 4 nn + t: what turns a raw product into z (base 2), or into z / cap
#pragma unroll
        for (int nn = 0; nn < NN; nn++) {
            const int r = 4 * nn + (g8 >> 1);
            const bool there = r < nrows;
            const uint32_t qr = smem_addr(smem + L::q + (st * ROWS + r) * D * 4) + RUN * 4 * t;
            float am = 0.0f;
#pragma unroll
            for (int i = 0; i < KS; i++) {
                const uint4 v = there ? sh_ld128(qr + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
                am = fmaxf(am, absmax4(make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                                                   __uint_as_float(v.w))));
            }
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
            const int ex = min(max((int)((__float_as_uint(am) >> 23) & 255u) - 126, -100), 126);
            const float up = __uint_as_float((uint32_t)(15 - ex + 127) << 23);
            for (int i = warp; i < KS; i += W) {
                const uint4 v = there ? sh_ld128(qr + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
                uint32_t h0, l0, h1, l1;
                split2(__uint_as_float(v.x) * up, __uint_as_float(v.y) * up, h0, l0);
                split2(__uint_as_float(v.z) * up, __uint_as_float(v.w) * up, h1, l1);
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(frag + 256 * (i * NN + nn)), "r"(g8 & 1 ? l0 : h0),
                             "r"(g8 & 1 ? l1 : h1)
                             : "memory");
            }
            // the factor of row 4 nn + t comes from a lane that made its column
            const float fr = __uint_as_float((uint32_t)(ex - 15 + 127) << 23) * p.scale;
            f[nn] = __shfl_sync(0xffffffffu, p.cap > 0.0f ? fr / p.cap : fr * LOG2E, 8 * t);
        }
        // a wait that gave up ends the work of all the warps here
        if (failed) sm.failed = 1;
        consumer_sync<CONSUMERS>();
        if (*(volatile int *)&sm.failed) return;
        const int u0 = it.u0, u1 = it.u1;
        // rows 4 nn + t of this lane: what they see, x >= firstp and (x < pre or seelo <= x <= qpos)
        int qpos[NN], firstp[NN], pre[NN], seelo[NN], all_lo = 0, all_hi = 0x7fffffff;
        float slope[NN];
#pragma unroll
        for (int nn = 0; nn < NN; nn++) {
            const int r = 4 * nn + t;
            const bool real = r < nrows;
            qpos[nn] = real ? it.qpos[r] : 0;
            firstp[nn] = real ? it.first[r] : 0;
            pre[nn] = real ? it.prefix[r] : 0;
            slope[nn] = real ? it.slope[r] : 0.0f;
            seelo[nn] = p.window > 0 ? (int)max((int64_t)firstp[nn], (int64_t)qpos[nn] - p.window + 1) : firstp[nn];
            // a unit with all positions in [all_lo, all_hi] is seen whole by every row
            if (real) {
                all_lo = max(all_lo, seelo[nn]);
                all_hi = min(all_hi, qpos[nn]);
            }
        }
#pragma unroll
        for (int m = 1; m <= 2; m <<= 1) {
            all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, m));
            all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, m));
        }
        const float cap2 = p.cap * LOG2E;
        uint2 qb[NN == 1 ? KS : 1];   // the query's fragments: in registers where there is room
        if (NN == 1)
#pragma unroll
            for (int i = 0; i < KS; i++) qb[NN == 1 ? i : 0] = sh_ld64(frag + 256 * i);
        float o[MT][NN][4];
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int nn = 0; nn < NN; nn++) o[m][nn][0] = o[m][nn][1] = o[m][nn][2] = o[m][nn][3] = 0.0f;
        float mrow[NN], lrow[NN];
#pragma unroll
        for (int nn = 0; nn < NN; nn++) {
            mrow[nn] = -INFINITY;
            lrow[nn] = 0.0f;
        }
        int vex[NN];   // a row's sums are in units of 2^(vex - 14); the largest value scale it has seen is below 2^vex
#pragma unroll
        for (int nn = 0; nn < NN; nn++) vex[nn] = -100;

        // Flushed sums of the warp: lane (g8, t) holds positions D / 8 g8 .. of row 4 nn + t, at the place
        // where the item's end puts them (16-byte chunk y of row r lies at y ^ r).
        int done = 0;   // units of the item so far
        const uint32_t mine = smem_addr(red) + (uint32_t)((warp * ROWS + t) * D * 4);
        auto chunk = [&](int nn, int x) { return mine + (uint32_t)(4 * nn * D * 4) + (((D / 32 * g8 + x / 2) ^ (4 * nn + t)) << 4); };
        // what takes the flushed sums to the present units: 2^(their maximum - the present one) 2^(their vex - the present one)
        auto carry = [&](int nn) {
            const float2 was = sm.sum_unit[warp][4 * nn + t];
            const float a = was.x == mrow[nn] ? 1.0f : ex2(was.x - mrow[nn]);
            return a * was.y * __uint_as_float((uint32_t)(127 - vex[nn]) << 23);
        };

        // unit u of the item is unit count + u - u0 of this CTA; warp w takes every W-th
        for (int u = u0 + (warp + W - count % W) % W; u < u1; u += W) {
            if (FLUSH && done > 0 && done % FLUSH_UNITS == 0) {
#pragma unroll
                for (int nn = 0; nn < NN; nn++) {
                    const float a = done > FLUSH_UNITS ? carry(nn) : 0.0f;
#pragma unroll
                    for (int x = 0; x < MT; x += 2) {
                        const uint32_t at = chunk(nn, x);
                        const uint4 w = done > FLUSH_UNITS ? sh_ld128(at) : make_uint4(0u, 0u, 0u, 0u);
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                                     "f"(fmaf(__uint_as_float(w.x), a, o[x][nn][0] + o[x][nn][1])),
                                     "f"(fmaf(__uint_as_float(w.y), a, o[x][nn][2] + o[x][nn][3])),
                                     "f"(fmaf(__uint_as_float(w.z), a, o[x + 1][nn][0] + o[x + 1][nn][1])),
                                     "f"(fmaf(__uint_as_float(w.w), a, o[x + 1][nn][2] + o[x + 1][nn][3]))
                                     : "memory");
                        o[x][nn][0] = o[x][nn][1] = o[x][nn][2] = o[x][nn][3] = 0.0f;
                        o[x + 1][nn][0] = o[x + 1][nn][1] = o[x + 1][nn][2] = o[x + 1][nn][3] = 0.0f;
                    }
                }
                __syncwarp();   // (every lane has read the units)
                if (g8 == 0)
#pragma unroll
                    for (int nn = 0; nn < NN; nn++)
                        sm.sum_unit[warp][4 * nn + t] = make_float2(mrow[nn], __uint_as_float((uint32_t)(vex[nn] + 127) << 23));
                __syncwarp();
            }
            done++;
            const int i = slots + (u >> 1) - (u0 >> 1), sl = i % SLOTS, phase = i / SLOTS;
            if (failed) break;   // a wait gave up: no further ones
            bool got = phase == 0 || mbar_wait(smem_addr(sm.empty + sl), (uint32_t)((phase - 1) & 1), c.status);
            got = got && mbar_wait(smem_addr(sm.full + sl), (uint32_t)(phase & 1), c.status);
            failed = !__all_sync(0xffffffffu, got);
            if (failed) break;
            const uint32_t kb = smem_addr(smem + L::ring) + (uint32_t)(sl * 4 * HALF + (u & 1) * HALF), vb = kb + 2 * HALF;
            const UnitMeta &m = sm.meta[(metas + u - (u0 & ~1)) % METAS];
            const int live = m.live;
            // ---- scores of tokens 16 mt + g8 and + 8, rows 4 nn + t
            float s[2][NN][2];
#pragma unroll
            for (int mt = 0; mt < 2; mt++) {
                float acc[NN][4];
#pragma unroll
                for (int nn = 0; nn < NN; nn++) acc[nn][0] = acc[nn][1] = acc[nn][2] = acc[nn][3] = 0.0f;
#pragma unroll
                for (int hh = 0; hh < D / 64; hh++) {
                    const uint4 wa = sh_ld128(kb + koff[hh] + mt * 16 * D);
                    // (D = 64: eight rows on, the line's number changes by 4 and with it bit 6 of the chunk)
                    const uint4 wb = sh_ld128(kb + (D == 128 ? koff[hh] : koff[hh] ^ 64u) + mt * 16 * D + 8 * D);
                    const uint32_t av[4] = {wa.x, wa.y, wa.z, wa.w}, bv[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                    for (int x = 0; x < 4; x++) {
                        uint32_t a0, a1, a2, a3;
                        widen4<KIND>(av[x], a0, a2);
                        widen4<KIND>(bv[x], a1, a3);
#pragma unroll
                        for (int nn = 0; nn < NN; nn++) {
                            const uint2 q = NN == 1 ? qb[NN == 1 ? 4 * hh + x : 0] : sh_ld64(frag + 256 * ((4 * hh + x) * NN + nn));
                            mma_f16_16x8x16(acc[nn], a0, a1, a2, a3, q.x, q.y);
                        }
                    }
                }
#pragma unroll
                for (int nn = 0; nn < NN; nn++) {
                    const float fk = f[nn] * m.ks[mt];
                    s[mt][nn][0] = (acc[nn][0] + acc[nn][1]) * fk;
                    s[mt][nn][1] = (acc[nn][2] + acc[nn][3]) * fk;
                }
            }
            // ---- cap, bias, mask
            if (p.cap > 0.0f) {
#pragma unroll
                for (int mt = 0; mt < 2; mt++)
#pragma unroll
                    for (int nn = 0; nn < NN; nn++) {
                        s[mt][nn][0] = cap2 * tanh_f32(s[mt][nn][0]);
                        s[mt][nn][1] = cap2 * tanh_f32(s[mt][nn][1]);
                    }
            }
            if (p.slopes) {
#pragma unroll
                for (int mt = 0; mt < 2; mt++)
#pragma unroll
                    for (int nn = 0; nn < NN; nn++) {
                        const int d = qpos[nn] - (m.base[mt] + g8);
                        s[mt][nn][0] -= slope[nn] * (float)abs(d);
                        s[mt][nn][1] -= slope[nn] * (float)abs(d - 8);
                    }
            }
            const bool whole = live == UNIT && m.base[0] >= all_lo && m.base[1] >= all_lo && m.base[0] + 15 <= all_hi &&
                               m.base[1] + 15 <= all_hi;   // warp-uniform
            float vmax[NN];   // the larger value scale of the halves that the row sees some of
#pragma unroll
            for (int nn = 0; nn < NN; nn++) vmax[nn] = whole ? fmaxf(m.vs[0], m.vs[1]) : 0.0f;
            if (!whole) {
#pragma unroll
                for (int mt = 0; mt < 2; mt++)
#pragma unroll
                    for (int nn = 0; nn < NN; nn++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const int x = m.base[mt] + g8 + 8 * e;
                            const bool see = 16 * mt + g8 + 8 * e < live && x >= firstp[nn] &&
                                             (x < pre[nn] || (x >= seelo[nn] && x <= qpos[nn]));
                            s[mt][nn][e] = see ? s[mt][nn][e] : -INFINITY;
                        }
#pragma unroll
                for (int mt = 0; mt < 2; mt++)
#pragma unroll
                    for (int nn = 0; nn < NN; nn++) {   // x0 .. x1 - 1: the half's positions
                        const int x0 = m.base[mt], x1 = x0 + min(live - 16 * mt, 16);
                        const bool some = max(x0, seelo[nn]) < min(x1, qpos[nn] + 1) || max(x0, firstp[nn]) < min(x1, pre[nn]);
                        // (times a weight of 0, a masked half's scale only has to stay finite: 2^-112 of it counts)
                        vmax[nn] = fmaxf(vmax[nn], m.vs[mt] * (some ? 1.0f : 0x1p-112f));
                    }
            }
            // ---- the running maxima
            int ve[NN];
            float mnew[NN];
            bool grow = false;
#pragma unroll
            for (int nn = 0; nn < NN; nn++) {
                float mx = fmaxf(fmaxf(s[0][nn][0], s[0][nn][1]), fmaxf(s[1][nn][0], s[1][nn][1]));
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                mnew[nn] = fmaxf(mrow[nn], mx);
                ve[nn] = max(vex[nn], min(max((int)((__float_as_uint(vmax[nn]) >> 23) & 255u) - 126, -100), 126));
                grow = grow || mnew[nn] > mrow[nn] || ve[nn] != vex[nn];
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nn = 0; nn < NN; nn++) {
                    // 2^(vex - ve): exact, 0 when it would underflow
                    const int dv = vex[nn] - ve[nn];
                    const float ov = dv < -126 ? 0.0f : __uint_as_float((uint32_t)(dv + 127) << 23);
                    const float a = mnew[nn] > mrow[nn] ? ex2(mrow[nn] - mnew[nn]) : 1.0f;   // 0 while nothing was seen
                    lrow[nn] *= a;
                    const float av = a * ov;
#pragma unroll
                    for (int y = 0; y < MT; y++) {
                        o[y][nn][0] *= av;
                        o[y][nn][1] *= av;
                        o[y][nn][2] *= av;
                        o[y][nn][3] *= av;
                    }
                    mrow[nn] = mnew[nn];
                    vex[nn] = ve[nn];
                }
            }
            // ---- weights; times value scales, in units of 2^(vex - 14), as two fp16 terms, moved to the
            // lanes that multiply them: column g8 is row g8 / 2's hi (even) or lo term
            uint32_t pb[2][NN][2];
#pragma unroll
            for (int nn = 0; nn < NN; nn++) {
                const float vu = __uint_as_float((uint32_t)(14 - vex[nn] + 127) << 23);
                const float msafe = mrow[nn] == -INFINITY ? 0.0f : mrow[nn];
                float gsum[2];
#pragma unroll
                for (int mt = 0; mt < 2; mt++) {
                    const float p0 = ex2(s[mt][nn][0] - msafe), p1 = ex2(s[mt][nn][1] - msafe), vv = m.vs[mt] * vu;
                    gsum[mt] = p0 + p1;
                    uint32_t hi, lo;
                    split2(p0 * vv, p1 * vv, hi, lo);
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int from = (t + 4 * e) * 4 + (g8 >> 1);
                        const uint32_t h = __shfl_sync(0xffffffffu, hi, from), l = __shfl_sync(0xffffffffu, lo, from);
                        pb[mt][nn][e] = g8 & 1 ? l : h;
                    }
                }
                lrow[nn] += gsum[0] + gsum[1];
                if (p.glse) {   // log2 of the weight sums by group of min(P, 32) tokens
#pragma unroll
                    for (int mt = 0; mt < 2; mt++)
#pragma unroll
                        for (int d = 4; d <= 16; d <<= 1) gsum[mt] += __shfl_xor_sync(0xffffffffu, gsum[mt], d);
                    const int r = 4 * nn + t;
                    if (g8 == 0 && r < nrows) {
                        const int slot = (u < it.pre ? u : it.start + u - it.pre) * UNIT;
                        float *gl = p.glse + ((int64_t)it.ti[r] * p.Hq + it.head[r]) * p.NG + (slot >> p.lgGroup);
                        if (p.lgGroup == 4) {
                            gl[0] = __log2f(gsum[0]) + msafe;
                            if (live > 16) gl[1] = __log2f(gsum[1]) + msafe;
                        } else {
                            gl[0] = __log2f(gsum[0] + gsum[1]) + msafe;
                        }
                    }
                }
            }
            // ---- values: k the 16 tokens of a step in the order (t, t + 8), (t + 4, t + 12); row g8 of
            // tile x is the 2x-th position of chunk g8, row g8 + 8 the next one
#pragma unroll
            for (int mt = 0; mt < 2; mt++) {
                uint32_t w[4][D / 32];   // this lane's chunk of tokens t, t + 8, t + 4, t + 12
#pragma unroll
                for (int x = 0; x < 4; x++) {
                    const int up = 8 * (x & 1) + 4 * (x >> 1), tok = 16 * mt + t + up;
                    if constexpr (D == 128) {   // (four rows on: the chunk's bit 2 changes, eight: nothing)
                        const uint4 q4 = sh_ld128(vb + (x >> 1 ? voff ^ 64u : voff) + (16 * mt + up) * 128);
                        w[x][0] = q4.x;
                        w[x][1] = q4.y;
                        w[x][2] = q4.z;
                        w[x][3] = q4.w;
                    } else {   // (four rows on: two lines, the chunk's bit 1 changes; eight: its bit 2)
                        const uint2 q2 = sh_ld64(vb + (voff ^ (x >> 1 ? 32u : 0u) ^ (x & 1 ? 64u : 0u)) + (16 * mt + up) * 64);
                        w[x][0] = q2.x;
                        w[x][1] = q2.y;
                    }
                    // slots past the last token may hold any bytes, NaN codes among them
                    if (KIND == GQ_KV_E4M3 && !whole && (tok >= live || ((m.lost >> mt) & 1)))
#pragma unroll
                        for (int y = 0; y < D / 32; y++) w[x][y] = 0u;
                }
#pragma unroll
                for (int y = 0; y < D / 32; y++) {
                    uint32_t b0[4], b1[4];   // positions 4y .. 4y + 3 of tokens (t, t + 8) and (t + 4, t + 12)
                    widen_pairs<KIND>(w[0][y], w[1][y], b0);
                    widen_pairs<KIND>(w[2][y], w[3][y], b1);
#pragma unroll
                    for (int x = 0; x < 2; x++)
#pragma unroll
                        for (int nn = 0; nn < NN; nn++)
                            mma_f16_16x8x16(o[2 * y + x][nn], b0[2 * x], b0[2 * x + 1], b1[2 * x], b1[2 * x + 1], pb[mt][nn][0],
                                            pb[mt][nn][1]);
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_addr(sm.empty + sl));
                // a slot's only unit gives both halves back
                if ((u == u0 && (u & 1)) || (u == u1 - 1 && !(u & 1))) mbar_arrive(smem_addr(sm.empty + sl));
            }
            __syncwarp();
        }
        count += u1 - u0;
        slots += ((u1 - 1) >> 1) - (u0 >> 1) + 1;
        metas += (u1 - (u0 & ~1) + 31) & ~31;

        // ---- join the warps: sums in units of 2^0, relative to the warp's own maximum
#pragma unroll
        for (int nn = 0; nn < NN; nn++) {
            const float vscale = __uint_as_float((uint32_t)(vex[nn] - 14 + 127) << 23);
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) lrow[nn] += __shfl_xor_sync(0xffffffffu, lrow[nn], d);
            const int r = 4 * nn + t;
            if (g8 == 0) {
                sm.ml[warp][r][0] = mrow[nn];
                sm.ml[warp][r][1] = lrow[nn];
            }
            const bool add = FLUSH && done > FLUSH_UNITS;
            const float a = add ? carry(nn) : 0.0f;
#pragma unroll
            for (int x = 0; x < MT; x += 2) {
                const uint32_t at = chunk(nn, x);
                const uint4 w = add ? sh_ld128(at) : make_uint4(0u, 0u, 0u, 0u);
                asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                             "f"(fmaf(__uint_as_float(w.x), a, o[x][nn][0] + o[x][nn][1]) * vscale),
                             "f"(fmaf(__uint_as_float(w.y), a, o[x][nn][2] + o[x][nn][3]) * vscale),
                             "f"(fmaf(__uint_as_float(w.z), a, o[x + 1][nn][0] + o[x + 1][nn][1]) * vscale),
                             "f"(fmaf(__uint_as_float(w.w), a, o[x + 1][nn][2] + o[x + 1][nn][3]) * vscale)
                             : "memory");
            }
        }
        consumer_sync<CONSUMERS>();
        const int rows = nrows;
        const bool cut0 = u0 > 0, cut1 = u1 < it.units;   // the item began before, goes on after this CTA
        const int piece_slot = blockIdx.x * 2 + (cut0 ? 0 : 1);
        for (int x = tid; x < rows * (D / 4); x += CONSUMERS) {
            const int rr = x / (D / 4), d4 = x % (D / 4);
            float mt = -INFINITY, l = 0.0f;
#pragma unroll
            for (int w = 0; w < W; w++) mt = fmaxf(mt, sm.ml[w][rr][0]);
            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < W; w++) {
                const float mw = sm.ml[w][rr][0], e = mw == -INFINITY ? 0.0f : ex2(mw - mt);
                l += sm.ml[w][rr][1] * e;
                const float4 v = *reinterpret_cast<const float4 *>(red + (w * ROWS + rr) * D + 4 * (d4 ^ rr));
                a.x = fmaf(v.x, e, a.x);
                a.y = fmaf(v.y, e, a.y);
                a.z = fmaf(v.z, e, a.z);
                a.w = fmaf(v.w, e, a.w);
            }
            if (!cut0 && !cut1) {
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                reinterpret_cast<float4 *>(p.out + (int64_t)it.ti[rr] * p.ldo + (int64_t)it.head[rr] * D)[d4] =
                    make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
                if (p.lse && d4 == 0) p.lse[(int64_t)it.ti[rr] * p.Hq + it.head[rr]] = l > 0.0f ? mt + log2f(l) : INFINITY;
            } else {
                reinterpret_cast<float4 *>(p.parts + ((int64_t)piece_slot * ROWS + rr) * D)[d4] = a;
                if (d4 == 0) {
                    p.part_ml[((int64_t)piece_slot * ROWS + rr) * 2] = mt;
                    p.part_ml[((int64_t)piece_slot * ROWS + rr) * 2 + 1] = l;
                }
            }
        }
        if (cut0 || cut1) {
            // the pieces of this item: CTAs c0 .. c1; the one that finishes last joins them in order
            const int64_t item0 = it.item0;
            const int c0 = (int)(item0 / piece), c1 = (int)((item0 + it.units - 1) / piece);
            __threadfence();
            consumer_sync<CONSUMERS>();
            if (tid == 0) {
                const int done = atomicAdd(p.counters + c0, 1);
                sm.last = done == c1 - c0;
                if (done == c1 - c0) p.counters[c0] = 0;   // left at zero for the next launch
            }
            consumer_sync<CONSUMERS>();
            if (sm.last) {
                __threadfence();
                join_pieces<D, W, ROWS>(p, it, c0, c1, warp, lane);
            }
        }
        at = it.item0 + u1;
        consumer_sync<CONSUMERS>();   // the item's data, the warps' sums and the fragments are free
        if (lane == 0) mbar_arrive(smem_addr(sm.item_empty + st));
        __syncwarp();
    }
}

// ---------------------------------------------------------------------------
// The weight that each page gathered: decay * in + sum over the step's query rows of
// 2^(log2 of the page's weight sum - log2 of the row's denominator).  A cluster of CL CTAs takes 32
// groups of tokens of one (sequence, head), a lane per group; its CTAs' WW warps share the tokens
// and are added in order.  The sums of groups that a row cannot see were never written: they are
// passed over.  Bound by the latency of the loads, so many rows want many warps, unless the items
// fill the GPU by themselves, and registers for two CTAs of 16 warps an SM (4 sequences of up to 1000
// tokens x 2 heads of 8 KV heads, 64 items: 68 us the whole step, 86 with 96 registers a thread; when it
// was 74, a CTA an item took 101).  8 x 8 tokens x 8 heads on 4096 (512 items): 91 us with 4 warps an
// item, 170 with 8 x 16.
// ---------------------------------------------------------------------------
template <int WW, int CL>
__global__ void __launch_bounds__(WW * 32, WW == 16 ? 2 : 12) __cluster_dims__(CL, 1, 1)
    attn_pages_weights_kernel(const AttnParams8 p, const float *w_in, float *w_out, float decay) {
    __shared__ float part[WW][32];
    const PagesView &c = p.c;
    pdl_launch_dependents();
    const int per = p.lgP - p.lgGroup;   // log2 of the groups of a page
    const int tiles = (((c.NB << per) + 31) / 32), item = blockIdx.x / CL, rank = blockIdx.x % CL;
    const int bh = item / tiles, b = bh / c.Hkv, h = bh % c.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = (item % tiles) * 32 + lane, j = g >> per;
    const int size = 1 << p.lgGroup;
    pdl_wait();
    const SeqStep s = attn_step(p, b);
    const int end = s.end, slot = g << p.lgGroup;
    const int64_t at = (int64_t)bh * c.NB + j;
    const bool used = slot < end;        // (a page is in use if its first group is)
    // an entry that is no page: seen by nobody, and its sums may never have been written
    const bool there = used && (unsigned)c.table[at] < (unsigned)c.pages;
    float sum = 0.0f;
    if (__any_sync(0xffffffffu, there)) {
        const int x0 = there ? c.base[at] + (slot & (c.P - 1)) : 0x7f000000, x1 = there ? x0 + size - 1 : 0x7f000000;
        const float *gl = p.glse + (there ? g : 0);
        // (loads of rows and groups that were never written are within the buffer, and passed over)
        auto row = [&](int i, int y) {
            const int64_t r = (int64_t)(s.t0 + i) * p.Hq + h * p.G + y;
            const int qpos = s.seen + i;
            const float v = __ldcg(gl + r * p.NG), l = __ldcg(p.lse + r);
            const int first = p.first ? __ldg(p.first + s.t0 + i) : 0, pre = p.prefix ? min(__ldg(p.prefix + s.t0 + i), 1 << 30) : 0;
            const int lo = p.window > 0 ? (int)max((int64_t)first, (int64_t)qpos - p.window + 1) : first;
            const bool see = there && ((x1 >= lo && x0 <= qpos && lo <= qpos) || (x0 < pre && x1 >= first && first < pre));
            sum += see ? ex2(v - l) : 0.0f;
        };
        if (WW == 4) {      // few rows
            for (int x = warp; x < s.n * p.G; x += WW) row(x / p.G, x % p.G);
        } else {
            for (int y = 0; y < p.G; y++)
#pragma unroll 4
                for (int i = rank * WW + warp; i < s.n; i += WW * CL) row(i, y);
        }
    }
    part[warp][lane] = sum;
    __syncthreads();
    float total = 0.0f;
    if (warp == 0) {
        total = part[0][lane];
        for (int w = 1; w < WW; w++) total += part[w][lane];
    }
    if (CL > 1) {
        if (warp == 0) part[0][lane] = total;
        cluster_sync();
        if (warp == 0 && rank == 0) {
            float other[CL];
#pragma unroll
            for (int r = 1; r < CL; r++) other[r] = ld_shared_cluster_f32(map_shared_rank(&part[0][lane], r));
#pragma unroll
            for (int r = 1; r < CL; r++) total += other[r];
        }
        cluster_sync();   // (shared memory stays until it is read)
    }
    if (warp == 0 && rank == 0) {
        for (int d = 1; d < 1 << per; d <<= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
        if (j < c.NB && (g & ((1 << per) - 1)) == 0) w_out[at] = used ? (w_in ? decay * w_in[at] : 0.0f) + total : 0.0f;
    }
}

// Page weights: up to WROWS_FEW rows of a KV head are left to 4 warps; more to 16, and to 16 of each of
// WCTAS CTAs where all of them fit the GPU at once.
constexpr int WROWS_FEW = 64, WCTAS = 8;

int log2_of(int64_t x) {
    int l = 0;
    while ((1LL << l) < x) l++;
    return l;
}

// Which kernel: a tile of the tensor-memory kernel holds 128 query rows of one KV head, as many as
// there are; the row kernel's time grows with them.  Sequences with at most ROWS_MAX rows take it.
// 16 sequences x 8 heads on 2048 tokens: 32 rows 72 us against 82 in tiles, 64 rows 126 against 82;
// 3 x 8 heads on 10000: 48 rows 83 against 77, 64 rows 103 against 78; 8 heads on 4096: 64 rows 33
// against 42.
constexpr int ROWS_MAX = 40;

// Bytes of the row and group sums that a call keeps at most, but for a single row's.
constexpr int64_t SUMS_MOST = 512ll << 20;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int KIND, int D, int NN>
gq_status launch_rows(AttnParams8 p, const gq_kv_pages &c, const float *w_in, float *w_out, float decay, cudaStream_t s) {
    constexpr size_t smem = RowsLayout<D, NN>::total + 1024;
    constexpr int ROWS = rows_of(NN), THREADS = (WARPS + 1) * 32;
    const void *kernels[2] = {(const void *)attn_pages_rows_kernel<KIND, D, NN, false>,
                              (const void *)attn_pages_rows_kernel<KIND, D, NN, true>};
    static std::atomic<bool> smem_set[64];
    int dev = 0;
    KV_TRY(check_cuda(cudaGetDevice(&dev), "cudaGetDevice"));
    if (dev < 0 || dev >= 64) return fail(GQ_ERR_UNSUPPORTED_DEVICE, "device index %d", dev);
    if (!smem_set[dev].load(std::memory_order_acquire)) {
        for (const void *kernel : kernels)
            KV_TRY(check_cuda(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem),
                              "paged attention shared-memory attribute"));
        smem_set[dev].store(true, std::memory_order_release);
    }
    const int grid = 2 * sm_count();
    const size_t parts = (size_t)grid * 2 * ROWS * D * 4, mls = (size_t)grid * 2 * ROWS * 8;
    const int64_t T = p.row1 - p.row0, max_n = std::min<int64_t>(p.max_n, T);   // of the slice
    const size_t lse = w_out ? ((size_t)T * p.Hq * 4 + 255) / 256 * 256 : 0;
    const size_t glse = w_out ? ((size_t)T * p.Hq * p.NG * 4 + 255) / 256 * 256 : 0;
    const bool tiles = max_n * p.G > ROWS_MAX;
    // Some sequence may still be small; with equal lengths, or one sequence, none should be (one that is,
    // in a step of fewer rows than T, is left to the tiles with the others)
    const bool rows = !tiles || (c.B > 1 && T < c.B * max_n);
    const size_t plan = tiles ? attn_pages_tc_workspace(c, T, p.G) : 0;
    Workspace ws{};
    KV_TRY(get_workspace(s, (size_t)grid * sizeof(int), parts + mls + lse + glse + plan, &ws));
    p.counters = reinterpret_cast<int *>(ws.counters);
    p.parts = reinterpret_cast<float *>(ws.data);
    p.part_ml = reinterpret_cast<float *>(ws.data + parts);
    if (w_out) {   // (the kernels index them by packed rows: from where row 0 would be)
        const size_t before = (size_t)p.row0 * p.Hq * 4;
        p.lse = reinterpret_cast<float *>(reinterpret_cast<uintptr_t>(ws.data + parts + mls) - before);
        p.glse = reinterpret_cast<float *>(reinterpret_cast<uintptr_t>(ws.data + parts + mls + lse) - before * p.NG);
    }
    p.rows_over = !tiles ? INT32_MAX : rows ? ROWS_MAX : 0;
    if (tiles) KV_TRY(launch_attn_pages_tc(p, c, ws.data + parts + mls + lse + glse, s));
    if (rows) {
        alignas(64) CUtensorMap kmap, vmap;
        const int64_t pool_rows = c.pages * c.P * c.D / 128;
        const int box = (int)(std::min<int64_t>(c.P, 2 * UNIT) * D / 128);
        KV_TRY(byte_rows_map(&kmap, c.k, pool_rows, box));
        KV_TRY(byte_rows_map(&vmap, c.v, pool_rows, box));
        void *args[] = {(void *)&kmap, (void *)&vmap, (void *)&p};
        // the units of an item that a CTA can have: the item's, and the CTA's piece of the line
        const int64_t units = ceil_div(c.NB * c.P, UNIT);
        const int64_t items = c.B * c.Hkv * ceil_div(std::min<int64_t>(max_n * p.G, ROWS_MAX), ROWS);
        const int64_t most = std::min(units, std::max<int64_t>(WARPS, ceil_div(items * units, grid)));
        KV_TRY(launch_pdl(kernels[most > FLUSH_FROM * WARPS], dim3((unsigned)grid), dim3(THREADS), smem, s, args,
                          "paged attention launch"));
    }
    if (w_out) {
        const int64_t items = c.B * c.Hkv * ((p.NG + 31) / 32);
        void *wargs[] = {(void *)&p, (void *)&w_in, (void *)&w_out, (void *)&decay};
        const bool few = max_n * p.G <= WROWS_FEW, spread = !few && items * WCTAS <= 4 * sm_count();
        const void *weigh = few      ? (const void *)attn_pages_weights_kernel<4, 1>
                            : spread ? (const void *)attn_pages_weights_kernel<16, WCTAS>
                                     : (const void *)attn_pages_weights_kernel<16, 1>;
        KV_TRY(launch_pdl(weigh, dim3((unsigned)(spread ? WCTAS * items : items)), dim3(few ? 128 : 512), 0, s, wargs,
                          "paged attention weights launch"));
    }
    return GQ_OK;
}

gq_status launch_slice(const AttnParams8 &p, const gq_kv_pages &c, const float *w_in, float *w_out, float decay,
                       cudaStream_t s) {
    // items of up to 4 rows, where a sequence's rows of a KV head are no more, else of up to 8: 32
    // sequences x 8 heads x 4 rows on 2048 tokens take 33 us with one column tile, 41 with two
    const bool few = (int64_t)std::min(p.max_n, p.row1 - p.row0) * p.G <= 4;
    if (c.kind == GQ_KV_I8) {
        if (c.D == 64)
            return few ? launch_rows<GQ_KV_I8, 64, 1>(p, c, w_in, w_out, decay, s)
                       : launch_rows<GQ_KV_I8, 64, 2>(p, c, w_in, w_out, decay, s);
        return few ? launch_rows<GQ_KV_I8, 128, 1>(p, c, w_in, w_out, decay, s)
                   : launch_rows<GQ_KV_I8, 128, 2>(p, c, w_in, w_out, decay, s);
    }
    if (c.D == 64)
        return few ? launch_rows<GQ_KV_E4M3, 64, 1>(p, c, w_in, w_out, decay, s)
                   : launch_rows<GQ_KV_E4M3, 64, 2>(p, c, w_in, w_out, decay, s);
    return few ? launch_rows<GQ_KV_E4M3, 128, 1>(p, c, w_in, w_out, decay, s)
               : launch_rows<GQ_KV_E4M3, 128, 2>(p, c, w_in, w_out, decay, s);
}

}  // namespace

gq_status launch_attn_pages(const gq_kv_pages &c, const gq_attn_scores &sc, const float *q, int64_t ldq,
                            const int32_t *cu, int64_t T, int64_t max_n, int64_t Hq, float *out, int64_t ldo,
                            const float *w_in, float *w_out, float decay, cudaStream_t s) {
    AttnParams8 p{};
    KV_TRY(pages_view(c, &p.c));
    p.q = q;
    p.out = out;
    p.cu = cu;
    p.slopes = sc.slopes;
    p.first = sc.first;
    p.prefix = sc.prefix;
    p.ldq = ldq;
    p.ldo = ldo;
    p.window = sc.window;
    p.T = (int)T;
    p.max_n = (int)max_n;
    p.Hq = (int)Hq;
    p.G = (int)(Hq / c.Hkv);
    p.lgP = log2_of(c.P);
    p.lgGroup = std::min(p.lgP, 5);
    p.NG = (int)((c.NB * c.P) >> p.lgGroup);
    p.scale = sc.scale;
    p.cap = sc.cap;
    // The page weights need the sums of every row and group until the step is worked out, as much as the cache
    // has room for: steps for which that is more than SUMS_MOST are worked out in slices of rows.
    const int64_t row_bytes = Hq * p.NG * 4;
    const int64_t slice = w_out ? std::max<int64_t>(1, SUMS_MOST / row_bytes) : T;
    for (int64_t row0 = 0; row0 < T; row0 += slice) {
        p.row0 = (int)row0;
        p.row1 = (int)std::min(T, row0 + slice);
        // (a later slice adds to what the ones before gathered)
        KV_TRY(row0 == 0 ? launch_slice(p, c, w_in, w_out, decay, s) : launch_slice(p, c, w_out, w_out, 1.0f, s));
    }
    return GQ_OK;
}

}  // namespace gq

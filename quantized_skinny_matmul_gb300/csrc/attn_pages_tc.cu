// attn_pages_tc.cu -- attention over the paged 8-bit KV cache for many query rows per KV head
// (prompts and prompt chunks), on the 5th-generation tensor cores.
//
// The mathematics is attn_pages.cu's: a running maximum and sum over the cache, codes widened
// to fp16 exactly, queries and softmax weights carried as two fp16 terms.  Per 128 query rows
// and 128 tokens that is four 128 x 128 x D products: S = Qhi K + Qlo K, then
// O += Phi V + Plo V: the bound is the tensor pipe at twice the arithmetic of the formula.
//
// One CTA per SM holds two tiles of 128 rows (row r = token r / G, head r % G of one KV head):
//   warps 0-3, 4-7   softmax of tile 0 and tile 1, a thread per row: the scores come from
//                    tensor memory, the weights' two terms go back in their place (the A
//                    operand of the second product); also the query's conversion and the
//                    output.  The output stays in tensor memory; it is rescaled only when a
//                    row's maximum has grown by more than 2^6 (the weights have that room);
//   warps 8-11       widen the codes of a block of 128 tokens from the raw copies into the
//                    128-byte-swizzled operands (K by rows for the first product; the same
//                    layout of V is the token-major B operand of the second);
//   warp 12          chooses items and blocks, looks up pages, scales and positions, and
//                    streams the raw codes in (tensor copies);
//   warp 13          issues the MMAs: for block j and tile t, P_t(j) V(j), then Q_t K(j + 1),
//                    so that the softmax of one tile runs beside the products of the other.
// Tensor memory: S of both tiles (2 x 128 columns), O of both (2 x D).
// Items (sequence, head, pair of tiles) are taken from a list that a small kernel lays out, in
// turn, longest first within a sequence; which CTA takes which does not change any result.
//
// A prompt of 4096 tokens x 32 heads (8 KV heads, D = 128): 285 us, 482 TFLOP/s of the formula's
// operations, 964 of those issued (51% of a library product's rate; 281 us before a row's unit of
// values was its own, and in the comparisons below).  A block of both tiles takes
// about 7,000 cycles, 4,100 of them products: per tile, 4,000 from scores to weights, then 2,600 for
// the second half of its P V and the next Q K, which share the operands' memory with the widening;
// an item's change takes about 25,000 more (14,000 of them the queries' loads).  Two threads a row
// halve neither: twice the fixed work in half the registers (312 us when this was 288).
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

constexpr int BR = 128;                     // query rows of a tile
constexpr int BT = 128;                     // tokens of a block
constexpr int GROUPS = BT / 16;             // scales and positions come by 16 tokens
constexpr int METAS = 4;                    // blocks whose data is kept
// The tensor cores add to their f32 accumulators with truncation: after N products an output is
// off by about N 2^-26 of itself, one way.  Every FLUSH blocks (16 products each) a tile's O is
// added to a running sum in memory, rounded to nearest, and begun anew.  A row over 4,500 tokens is
// off by 8e-6 without it, by 2.5e-6 every 8 blocks, 1.4e-6 every 4 and 0.9e-6 every 2 (elementary
// operations in f32: 1.2e-6); a prompt of 4096 takes 266, 281 and 308 us with 8, 4 and 2 (a tile's
// sums go out at 32 bytes a cycle: 2,000 cycles).
constexpr int FLUSH = 4;
constexpr int THREADS = 512;
// Registers per thread of the four warpgroups: they add up to the 4 x 128 of the launch.  (A prompt
// of 4096 takes 281 us; 283 with 152 and 104, 286 with 136 and 120.)
constexpr int REGS_SOFTMAX = 144, REGS_REST = 112;
static_assert(2 * REGS_SOFTMAX + 2 * REGS_REST <= 4 * 65536 / THREADS, "register split");

enum : int { F_TILE0 = 1, F_TILE1 = 2, F_FIRST = 4, F_LAST = 8, F_EXIT = 16 };

struct BlockMeta {
    int flags;
    int b, h, pair;             // the item
    int place;                  // of its share's outputs; -1: it has all keys
    SeqStep s;
    int slot, live;             // first slot of the block, tokens of it that are held
    int lost;                   // bit i: group i has no usable page
    float ks[GROUPS], vs[GROUPS];
    int base[GROUPS];           // position of the group's first token
};

enum : int {
    META_FULL = 0, META_EMPTY = META_FULL + METAS,
    RAWK_FULL = META_EMPTY + METAS, RAWK_EMPTY, RAWV_FULL, RAWV_EMPTY,
    K_FULL, V_FULL, V_EMPTY,   // (K is free once the scores of the block's last tile are there)
    Q_FULL, S_FULL = Q_FULL + 2, P_FULL = S_FULL + 2, O_FULL = P_FULL + 4,   // P: [half][tile]; a half's phases pass one by one
    TILE_SYNC = O_FULL + 2, ALL_DONE = TILE_SYNC + 2, NUM_BARS
};

struct TileSmem {
    uint64_t bars[NUM_BARS];
    BlockMeta meta[METAS];
    uint32_t tmem;
};

template <int D>
struct TileLayout {
    static constexpr int ATOM = BR * 128;                  // 128 rows x 64 halves: 16 KB
    static constexpr int OPERAND = BR * D * 2;             // a tile of 128 x D halves
    static constexpr int RAW = BT * D;
    static constexpr int q = 0;                            // [tile][hi, lo]
    static constexpr int k = q + 4 * OPERAND;
    static constexpr int v = k + OPERAND;
    static constexpr int rawk = v + OPERAND;
    static constexpr int rawv = rawk + RAW;
    static constexpr int ctl = rawv + RAW;
    static constexpr int total = ctl + (int)sizeof(TileSmem);
    static_assert(total + 1024 <= 227 * 1024, "shared memory");
};

constexpr uint32_t TM_S = 0, TM_O = 256;    // tensor-memory columns: S of tile t at 128 t, O at 256 + 128 t

struct PlanView {
    int4 *list;                 // (sequence, pair of tiles, share, shares)
    float *parts;               // [place][2 BR][D]: a share's outputs; null: nothing is shared
    float *part_lse;            // [place][2 BR]: log2 of its denominators (infinity: nothing seen)
    int places, room;           // room: entries that the list holds
    int *count, *next;          // entries, items taken
    float *sums;                // [CTA][2][D / 4][BR][4]: the tiles' flushed output sums
};

// ---- tcgen05 ---------------------------------------------------------------------------
// Shared-memory matrix descriptors of 128-byte-swizzled operands.  Both operands lie as atoms
// of 64 halves x rows (128 bytes a row, 8-row groups 1024 bytes apart).  Read by rows (K-major)
// a K step of 16 is 32 bytes inside the atom; read token-major (V: N the positions, K the
// tokens) the atoms are the leading offset and the 8-token groups the stride.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t leading) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(leading >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool b_mn_major) {
    return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of this warp's lanes.  tm_wait ties the registers to the wait: nothing reads them before.
__device__ __forceinline__ void tm_ld32(uint32_t a, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(a));
}
__device__ __forceinline__ void tm_wait(float *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                   "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                   "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                   "+f"(v[30]), "+f"(v[31])::"memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t a, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(a));
}
__device__ __forceinline__ void tm_wait16(float *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])::"memory");
}
__device__ __forceinline__ void tm_st32(uint32_t a, const float *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(a),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
        "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
        "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
        : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(a),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void red_add4(float4 *at, float a, float b, float c, float d) {
    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(at), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Two f32 at a time.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Waits of one role: after one gave up, the role waits no more and leaves.
struct Waiter {
    unsigned int *status;
    uint64_t *bars;
    bool failed;
    __device__ __forceinline__ bool operator()(int bar, int phase) {
        if (!failed && !mbar_wait(smem_addr(bars + bar), (uint32_t)(phase & 1), status)) failed = true;
        return !failed;
    }
    // the same for a whole warp, so that its lanes agree
    __device__ __forceinline__ bool warp(int bar, int phase) {
        (*this)(bar, phase);
        failed = __any_sync(0xffffffffu, failed);
        return !failed;
    }
    __device__ __forceinline__ void arrive(int bar) { mbar_arrive(smem_addr(bars + bar)); }
};

// The bits lo .. hi of 16 (none where hi < lo).
__device__ __forceinline__ uint32_t bits16(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 15);
    return hi < lo ? 0u : (2u << hi) - (1u << lo);
}

__device__ __forceinline__ int exponent_of(float x) {   // x < 2^e, clamped to [-100, 126]
    return min(max((int)((__float_as_uint(x) >> 23) & 255u) - 126, -100), 126);
}
__device__ __forceinline__ float pow2i(int e) {         // 2^e, 0 below 2^-126
    return e < -126 ? 0.0f : __uint_as_float((uint32_t)(e + 127) << 23);
}

// ---- the list of items --------------------------------------------------------------------
// Where the items leave most SMs idle, the keys of long ones are shared out, as far as all shares
// run at once and none has under SHARE_BLOCKS blocks; attn_pages_join_kernel joins them.  64 rows of
// one head on 32768 tokens, 64 shares: 61 us (16 shares: 107); 8 heads on 4096: 42 us (3 blocks: 43).
constexpr int SHARE_BLOCKS = 4, MOST_SHARES = 64;

__global__ void __launch_bounds__(256) attn_pages_plan_kernel(const AttnParams8 p, const PlanView plan) {
    __shared__ int sums[8];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the CTA's sum of x, and of those of the threads before
    auto scan = [&](int x, int &before) {
        int inc = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += t;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = inc;
        __syncthreads();
        int all = 0;
        before = inc - x;
        for (int w = 0; w < 8; w++) {
            if (w < warp) before += sums[w];
            all += sums[w];
        }
        return all;
    };
    int64_t at = 0, total = 0;
    int most = 1;
    for (int phase = 0; phase < 2; phase++) {   // count the pairs, then write the list
        for (int b0 = 0; b0 < p.c.B; b0 += 256) {
            const int b = b0 + tid;
            int pairs = 0, splits = 1, before;
            if (b < p.c.B) {
                const SeqStep s = attn_step(p, b);
                if (s.bad && phase == 0) atomicOr(p.c.status, STATUS_RANGE);
                if (s.n * p.G > p.rows_over) pairs = (s.n * p.G + 2 * BR - 1) / (2 * BR);
                int keys = s.end;
                if (p.window > 0) keys = (int)min((int64_t)keys, p.window + 2 * BR / p.G);
                splits = max(1, min(most, keys / (SHARE_BLOCKS * BT)));
            }
            const int all = scan(phase ? pairs * splits : pairs, before);
            if (phase)
                for (int i = 0; i < pairs * splits && at + before + i < plan.room; i++)
                    plan.list[at + before + i] = make_int4(b, pairs - 1 - i / splits, i % splits, splits);
            if (phase) at += all;
            else total += all;
        }
        // Sequences whose rows are their own have no more pairs than the list holds.  A cu that decreases
        // can name rows again and again: the pairs beyond are left out.
        if (phase == 0 && total > plan.room && tid == 0) atomicOr(p.c.status, STATUS_RANGE);
        if (phase == 0 && plan.parts && total > 0)
            most = (int)max((int64_t)1, min((int64_t)MOST_SHARES, plan.places / (total * p.c.Hkv)));
    }
    if (tid == 0) {
        *plan.count = (int)min(at, (int64_t)plan.room);
        *plan.next = 0;
    }
}

// ---- warp 12: items, blocks, raw copies ---------------------------------------------------
struct Item {
    int b, h, pair, z, splits, place;
    SeqStep s;
};

template <int KIND, int D>
__device__ __forceinline__ void lead_role(const AttnParams8 &p, const PlanView &plan, const CUtensorMap &kmap,
                                          const CUtensorMap &vmap, uint8_t *smem, TileSmem &sm, Waiter &wait, int lane) {
    using L = TileLayout<D>;
    const PagesView &c = p.c;
    const int items = *plan.count * c.Hkv;   // below 2^31: checked on the host
    const uint32_t rawk = smem_addr(smem + L::rawk), rawv = smem_addr(smem + L::rawv);
    const uint64_t policy = l2_evict_first_policy();
    const int per = c.P / 16;                // groups per page
    int nmeta = 0, nk = 0, nraw = 0;   // blocks published, copies of keys and of values issued

    // (the values of a block's groups are in the eight lanes from 8 q on)
    auto publish = [&](const Item &x, int flags, int slot, int live, int lost, int q, float ks, float vs, int base) {
        const int st = nmeta % METAS;
        if (nmeta >= METAS && !wait.warp(META_EMPTY + st, nmeta / METAS - 1)) return;
        BlockMeta &d = sm.meta[st];
        if (lane >> 3 == q) {
            d.ks[lane & 7] = ks;
            d.vs[lane & 7] = vs;
            d.base[lane & 7] = base;
        }
        if (lane == 0) {
            d.flags = flags;
            d.b = x.b;
            d.h = x.h;
            d.pair = x.pair;
            d.place = x.place;
            d.s = x.s;
            d.slot = slot;
            d.live = live;
            d.lost = lost;
        }
        __syncwarp();
        if (lane == 0) wait.arrive(META_FULL + st);
        nmeta++;
    };

    while (!wait.failed) {
        int item = 0;
        if (lane == 0) item = atomicAdd(plan.next, 1);
        item = __shfl_sync(0xffffffffu, item, 0);
        Item x{0, 0, 0, 0, 1, -1, {0, 0, 0, 0, 0, false}};
        if (item >= items) {
            publish(x, F_EXIT, 0, 0, 0, 0, 0.0f, 0.0f, 0);
            break;
        }
        const int4 e = __ldcg(plan.list + item / c.Hkv);
        x.b = e.x;
        x.h = item % c.Hkv;
        x.pair = e.y;
        x.z = e.z;
        x.splits = e.w;
        x.place = x.splits > 1 ? item : -1;
        x.s = attn_step(p, x.b);
        // the queries, on their way to L2 while the item before is finished (a prompt of 4096: 281 us,
        // 285 without; the CTA's first ones are needed at once)
        for (int i = nmeta == 0 ? x.s.n : x.pair * 2 * BR / p.G + lane; i < x.s.n && i * p.G < (x.pair + 1) * 2 * BR; i += 32)
            bulk_prefetch_l2(p.q + (int64_t)(x.s.t0 + i) * p.ldq + (int64_t)x.h * p.G * D, (uint32_t)(p.G * D * 4));
        const int end = x.s.end;             // slots in use (0 for an unusable sequence)
        // what the rows of each tile can see: positions lo .. hi, and those below pre
        int lo[2] = {0, 0}, hi[2] = {-1, -1}, pre[2] = {0, 0}, lomin = 0x7fffffff, premax = 0, imax = 0;
#pragma unroll
        for (int t = 0; t < 2; t++) {
            const int r0 = (x.pair * 2 + t) * BR, r1 = min(x.s.n * p.G, r0 + BR);
            if (r0 >= r1) continue;
            const int i0 = r0 / p.G, i1 = (r1 - 1) / p.G;
            int l = 0x7fffffff, q = 0;
            for (int i = i0 + lane; i <= i1; i += 32) {
                int f = p.first ? __ldg(p.first + x.s.t0 + i) : 0;
                if (p.window > 0) f = (int)max((int64_t)f, (int64_t)x.s.seen + i - p.window + 1);
                l = min(l, f);
                if (p.prefix) q = max(q, min(__ldg(p.prefix + x.s.t0 + i), 1 << 30));
            }
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) {
                l = min(l, __shfl_xor_sync(0xffffffffu, l, d));
                q = max(q, __shfl_xor_sync(0xffffffffu, q, d));
            }
            lo[t] = max(l, 0);
            hi[t] = x.s.seen + i1;
            pre[t] = q;
            lomin = min(lomin, lo[t]);
            premax = max(premax, q);
            imax = max(imax, i1);
        }
        // blocks [0, bp) and [b0, b1).  Positions are at least their slot, and distinct below
        // seen + n: a position of at least X is in a slot of at least held - seen + X.
        int b0 = 0, b1 = 0, bp = 0;
        if (end > 0) {
            const int top = max(x.s.held + imax + 1, min(end, premax));
            const int low = (int)min((int64_t)(end - 1), max((int64_t)0, (int64_t)x.s.held - x.s.seen + lomin));
            b1 = (top + BT - 1) / BT;
            b0 = min(low / BT, b1);
            bp = min((min(end, premax) + BT - 1) / BT, b0);
        }
        const int all = bp + b1 - b0, ib = (int)((int64_t)all * x.z / x.splits);   // this share's first block
        const int blocks = (int)((int64_t)all * (x.z + 1) / x.splits) - ib;
        const int64_t trow = ((int64_t)x.b * c.Hkv + x.h) * c.NB;
        // Blocks are looked up four at a time, a lane per group of 16 tokens; the pages of the next four,
        // and then their scales, are under way while these are worked on (one by one, these dependent
        // loads were what a block took longest).
        struct Look {
            int page, base, live;   // page -1: none, -2: not usable
            float ks, vs;
        };
        auto slot_of = [&](int i) { return (ib + i < bp ? ib + i : b0 + ib + i - bp) * BT; };
        auto pages = [&](int i0, Look &l) {
            const int i = i0 + (lane >> 3), at = slot_of(i) + 16 * (lane & 7);
            l.page = -1;
            l.base = 0x7f000000;   // a position nobody sees
            l.live = i < blocks ? min(BT, end - slot_of(i)) : 0;
            if (16 * (lane & 7) < l.live) {
                l.page = __ldg(c.table + trow + (at >> p.lgP));
                l.base = __ldg(c.base + trow + (at >> p.lgP)) + (at & (c.P - 1));
            }
        };
        auto scales = [&](Look &l) {
            l.ks = l.vs = 0.0f;
            if (l.page == -1) return;
            if ((unsigned)l.page >= (unsigned)c.pages) {
                atomicOr(c.status, STATUS_RANGE);
                l.page = -2;
                l.base = 0x7f000000;
            } else {
                l.ks = __ldg(c.ks + l.page);
                l.vs = __ldg(c.vs + l.page);
            }
        };
        Look now{-1, 0, 0, 0.0f, 0.0f}, next = now, later = now;
        // A block that some row sees is sent once the next one is known, so that the last can say
        // so.  w...: the one that waits, its groups' values in the lanes from 8 wq on.
        int wflags = 0, wslot = 0, wlive = 0, wlost = 0, wq = 0;
        Look w = now;
        bool first = true;
        for (int i = -8; i <= blocks && !wait.failed; i++) {
            const bool done = i == blocks;
            const int q = i & 3;
            if (q == 0) {
                now = next;
                next = later;
                scales(next);
                pages(i + 8, later);
            }
            if (i < 0) {
                i += 3;
                continue;
            }
            int active = 0, lost = 0;
            if (!done) {
                lost = (int)(__ballot_sync(0xffffffffu, now.page == -2) >> (8 * q)) & 255;
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    const bool see = now.page >= 0 && hi[t] >= 0 &&
                                     ((now.base + 15 >= lo[t] && now.base <= hi[t]) || now.base < pre[t]);
                    if ((__ballot_sync(0xffffffffu, see) >> (8 * q)) & 255u) active |= F_TILE0 << t;
                }
                if (!active) continue;
            }
            if (wflags || done) {   // (with no block at all: one that says only that the item is over)
                publish(x, wflags | (first ? F_FIRST : 0) | (done ? F_LAST : 0), wslot, wlive, wlost, wq, w.ks, w.vs, w.base);
                first = false;
                if (wflags && !wait.failed) {
                    const bool mine = lane >> 3 == wq && w.page >= 0 && (lane & 7) % per == 0;
                    const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, mine)) * c.P * D);
                    const int row = (int)((int64_t)w.page * c.P * D / 128);
                    const uint32_t to = (uint32_t)((lane & 7) * 16 * D);
                    if (nraw > 0 && !wait.warp(RAWK_EMPTY, nraw - 1)) break;
                    if (lane == 0) mbar_arrive_expect_tx(smem_addr(sm.bars + RAWK_FULL), bytes);
                    __syncwarp();
                    if (mine) tma_rows(rawk + to, &kmap, row, smem_addr(sm.bars + RAWK_FULL), policy);
                    nk++;
                    if (nraw > 0 && !wait.warp(RAWV_EMPTY, nraw - 1)) break;
                    if (lane == 0) mbar_arrive_expect_tx(smem_addr(sm.bars + RAWV_FULL), bytes);
                    __syncwarp();
                    if (mine) tma_rows(rawv + to, &vmap, row, smem_addr(sm.bars + RAWV_FULL), policy);
                    nraw++;
                }
            }
            wflags = active;
            wslot = slot_of(i);
            wlive = min(BT, end - wslot);
            wlost = lost;
            wq = q;
            w = now;
        }
    }
    // stay until every copy issued has landed
    if (nk > 0) mbar_wait(smem_addr(sm.bars + RAWK_FULL), (uint32_t)((nk - 1) & 1), c.status);
    if (nraw > 0) mbar_wait(smem_addr(sm.bars + RAWV_FULL), (uint32_t)((nraw - 1) & 1), c.status);
}

// ---- warp 13: the products ------------------------------------------------------------------
// One thread.  Few MMAs can be queued, so what it does between two groups of them is time that the
// tensor pipe stands still: no votes, and the waits that may be over early come early.
template <int D>
__device__ __forceinline__ void mma_role(uint8_t *smem, TileSmem &sm, Waiter &wait, uint32_t tmem) {
    using L = TileLayout<D>;
    constexpr uint32_t idq = idesc_f16(BR, BT, false), idp = idesc_f16(BR, D, true);
    const uint64_t qd0 = desc_sw128(smem_addr(smem + L::q), 16), kd = desc_sw128(smem_addr(smem + L::k), 16);
    const uint64_t vd = desc_sw128(smem_addr(smem + L::v), L::ATOM);
    // blocks, products with V, items; of tile 0 in the low half of a word and tile 1 in the high half:
    // weights multiplied, and those of the item
    int nk = 0, nv = 0, nitem = 0;
    uint32_t np = 0, no = 0;
    int prev = 0, fresh_q = 0;    // tiles whose weights wait for V; queries not yet waited for

    auto commit = [&](int bar) { mma_commit(smem_addr(sm.bars + bar)); };
    for (int i = 0;; i++) {
        const int st = i % METAS;
        if (!wait(META_FULL + st, i / METAS)) return;
        const int flags = sm.meta[st].flags;
        wait.arrive(META_EMPTY + st);
        if (flags & F_EXIT) return;
        if (flags & F_FIRST) {
            nitem++;
            no = 0;
            fresh_q = F_TILE0 | F_TILE1;
        }
        // A pass: for each tile P V of the block before, then Q K of this one.  After an item's last
        // block one more, for its P V.  (One copy of the code.)
        const int passes = flags & F_LAST ? 2 : 1;
#pragma unroll 1
        for (int pass = 0; pass < passes; pass++) {
            const int now = pass == 0 ? flags & (F_TILE0 | F_TILE1) : 0;
            if (prev && !wait(V_FULL, nv)) return;
            bool have_k = false;
#pragma unroll 1
            for (int t = 0; t < 2; t++) {
                const uint32_t one = 1u << (16 * t);
                if ((prev >> t) & 1) {
                    // the item's first product, and the first after a flush, overwrites O_t
                    const uint32_t s = tmem + TM_S + 128 * t, o = tmem + TM_O + 128 * t;
                    const int ph = (int)(np >> (16 * t)) & 0xffff;
                    uint32_t keep = (no >> (16 * t)) % FLUSH ? 1u : 0u;   // (FLUSH divides 2^16)
#pragma unroll 1
                    for (int half = 0; half < 2; half++) {   // 64 tokens' weights at a time, as they come
                        if (!wait(P_FULL + 2 * half + t, ph)) return;
                        tc_after();
#pragma unroll
                        for (int term = 0; term < 2; term++)
#pragma unroll
                            for (int kk = 0; kk < 4; kk++) {
                                mma_ts(o, s + 64 * half + 32 * (kk >> 1) + 16 * term + 8 * (kk & 1),
                                       vd + (uint64_t)((8192 * half + 2048 * kk) >> 4), idp, term || kk ? 1u : keep);
                            }
                        keep = 1u;
                    }
                    np = t ? np + one : (np & 0xffff0000u) | ((np + 1) & 0xffffu);
                    no = t ? no + one : (no & 0xffff0000u) | ((no + 1) & 0xffffu);
                    if (t == 1 || !(prev & F_TILE1)) commit(V_EMPTY);
                }
                if (pass == 1) {
                    // a tile that saw nothing too: its queries are waited for, and its next ones come
                    // only after O_FULL (else they come phases ahead of this wait)
                    if (((fresh_q >> t) & 1) && !wait(Q_FULL + t, nitem - 1)) return;
                    commit(O_FULL + t);
                }
                if ((now >> t) & 1) {
                    if (!have_k && !wait(K_FULL, nk)) return;
                    have_k = true;
                    if (((fresh_q >> t) & 1) && !wait(Q_FULL + t, nitem - 1)) return;
                    fresh_q &= ~(1 << t);
                    tc_after();
                    uint64_t qd = qd0 + (uint64_t)((2 * t + 1) * L::OPERAND >> 4);
                    // the small terms first: less is lost to truncation
#pragma unroll
                    for (int term = 1; term >= 0; term--) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; kk++) {
                            const uint64_t step = (uint64_t)(((kk >> 2) * L::ATOM + (kk & 3) * 32) >> 4);
                            mma_ss(tmem + TM_S + 128 * t, qd + step, kd + step, idq, term == 0 || kk ? 1u : 0u);
                        }
                        qd -= (uint64_t)(L::OPERAND >> 4);
                    }
                    commit(S_FULL + t);
                }
            }
            if (prev) nv++;
            if (now) nk++;
            prev = now;
        }
    }
}

// ---- warps 8-11: codes to operands, a thread per token ----------------------------------------
template <int KIND, int D>
__device__ __forceinline__ void widen_tile(uint32_t raw, uint32_t op, int tok, bool dead) {
    using L = TileLayout<D>;
#pragma unroll 1
    for (int ch = 0; ch < D / 16; ch++) {
        uint32_t a;
        if (D == 128) a = raw + tok * 128 + ((ch ^ (tok & 7)) << 4);
        else a = raw + (tok >> 1) * 128 + (((4 * (tok & 1) + ch) ^ ((tok >> 1) & 7)) << 4);
        uint4 w = sh_ld128(a);
        if (dead) w = make_uint4(0u, 0u, 0u, 0u);
        uint32_t o[8];
        widen4<KIND>(w.x, o[0], o[1]);
        widen4<KIND>(w.y, o[2], o[3]);
        widen4<KIND>(w.z, o[4], o[5]);
        widen4<KIND>(w.w, o[6], o[7]);
        const uint32_t dst = op + (ch >> 2) * L::ATOM + tok * 128;
#pragma unroll
        for (int x = 0; x < 2; x++)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + ((((ch & 3) * 2 + x) ^ (tok & 7)) << 4)),
                         "r"(o[4 * x]), "r"(o[4 * x + 1]), "r"(o[4 * x + 2]), "r"(o[4 * x + 3])
                         : "memory");
    }
}

template <int KIND, int D>
__device__ __forceinline__ void widen_role(uint8_t *smem, TileSmem &sm, Waiter &wait, int tok, int lane) {
    using L = TileLayout<D>;
    int n = 0, ns0 = 0, ns1 = 0, last = 0;   // blocks, scores of each tile, the last tile of the block before
    for (int i = 0;; i++) {
        const int st = i % METAS;
        if (!wait.warp(META_FULL + st, i / METAS)) return;
        const BlockMeta &m = sm.meta[st];
        const int flags = m.flags;
        // slots past the last token, and lost pages, may hold any bytes (NaN codes among them)
        const bool dead = tok >= m.live || ((m.lost >> (tok >> 4)) & 1);
        __syncwarp();
        if (lane == 0) wait.arrive(META_EMPTY + st);
        if (flags & F_EXIT) return;
        if (!(flags & (F_TILE0 | F_TILE1))) continue;
#pragma unroll 1
        for (int kv = 0; kv < 2; kv++) {
            wait.warp(kv ? RAWV_FULL : RAWK_FULL, n);
            if (n > 0) {
                if (kv) wait.warp(V_EMPTY, n - 1);
                else wait.warp(S_FULL + last, (last ? ns1 : ns0) - 1);
            }
            if (wait.failed) return;
            widen_tile<KIND, D>(smem_addr(smem + (kv ? L::rawv : L::rawk)), smem_addr(smem + (kv ? L::v : L::k)), tok, dead);
            fence_proxy_async_shared();   // the MMAs (async proxy) read what these threads wrote
            __syncwarp();
            if (lane == 0) {
                wait.arrive(kv ? V_FULL : K_FULL);
                wait.arrive(kv ? RAWV_EMPTY : RAWK_EMPTY);
            }
        }
        n++;
        ns0 += flags & F_TILE0 ? 1 : 0;
        ns1 += flags & F_TILE1 ? 1 : 0;
        last = flags & F_TILE1 ? 1 : 0;
    }
}

// ---- warps 0-7: softmax, a thread per row ------------------------------------------------------
template <int D>
__device__ __forceinline__ void softmax_role(const AttnParams8 &p, uint8_t *smem, TileSmem &sm, Waiter &wait, uint32_t tmem,
                                             const PlanView &plan, int t, int row, int lane) {
    using L = TileLayout<D>;
    const uint32_t lanes = (uint32_t)(row & ~31) << 16;   // this warp's tensor-memory lanes
    const uint32_t ts = tmem + lanes + TM_S + 128 * t, to = tmem + lanes + TM_O + 128 * t;
    const float cap2 = p.cap * LOG2E;
    int ns = 0, no = 0;
    // the row
    bool real = false;
    int ti = 0, head = 0, qpos = 0, seelo = 0, firstp = 0, pre = 0, all_lo = 0, all_hi = 0, vex = 0;
    float f = 0.0f, slope = 0.0f, mrow = -INFINITY, lrow = 0.0f;
    // the running sum of flushed parts: this thread's float4s, D / 4 of them, BR apart; in units of
    // 2^gex, relative to gmax
    float4 *sum = reinterpret_cast<float4 *>(plan.sums) + ((size_t)blockIdx.x * 2 + t) * (D / 4) * BR + row;
    int blocks = 0, gex = 0;       // blocks of the item so far
    float gmax = -INFINITY;
    // the four warps of the tile, with a bounded wait
    int nsync = 0;
    auto sync_tile = [&]() {
        __syncwarp();
        if (lane == 0) wait.arrive(TILE_SYNC + t);
        return wait.warp(TILE_SYNC + t, nsync++);
    };
    // what takes the running sum to the present units
    auto carry = [&]() { return blocks <= FLUSH ? 0.0f : (gmax == mrow ? 1.0f : ex2(gmax - mrow)) * pow2i(gex - vex); };

    for (int i = 0;; i++) {
        const int st = i % METAS;
        if (!wait.warp(META_FULL + st, i / METAS)) return;
        const BlockMeta &m = sm.meta[st];
        const int flags = m.flags;
        if (flags & F_EXIT) return;
        if (flags & F_FIRST) {
            const SeqStep s = m.s;
            const int r = (m.pair * 2 + t) * BR + row;
            real = r < s.n * p.G;
            ti = s.t0 + (real ? r / p.G : 0);
            head = m.h * p.G + (real ? r % p.G : 0);
            qpos = s.seen + ti - s.t0;
            // (positions are in [0, 2^30): within these limits no difference to one wraps)
            firstp = p.first ? max(__ldg(p.first + ti), 0) : 0;
            pre = p.prefix ? min(max(__ldg(p.prefix + ti), 0), 1 << 30) : 0;
            slope = p.slopes ? __ldg(p.slopes + head) * LOG2E : 0.0f;
            seelo = p.window > 0 ? (int)max((int64_t)firstp, (int64_t)qpos - p.window + 1) : firstp;
            all_lo = real ? seelo : 0;
            all_hi = real ? qpos : 0x7fffffff;
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) {
                all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, d));
                all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, d));
            }
            mrow = -INFINITY;
            lrow = 0.0f;
            blocks = 0;
            // The query rows of this warp, each scaled by a power of two into [2^14, 2^15), as two fp16
            // terms.  A row is read by D / 4 lanes together (whole lines: a lane per row costs 32 L1
            // accesses an instruction), and the row's thread is told its power.
            constexpr int LPR = D / 4, RPI = 32 / LPR, BATCH = 8;
            const int64_t mine = real ? (int64_t)ti * p.ldq + (int64_t)head * D : -1;
            const int part = lane / LPR, col = lane % LPR;
            const uint32_t qs = smem_addr(smem + L::q) + 2 * t * L::OPERAND + (col >> 4) * L::ATOM + (col & 1) * 8;
            int ex = 0;
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += BATCH * RPI) {
                float4 v[BATCH];
#pragma unroll
                for (int x = 0; x < BATCH; x++) {
                    const int64_t at = __shfl_sync(0xffffffffu, mine, r0 + x * RPI + part);
                    v[x] = at >= 0 ? __ldg(reinterpret_cast<const float4 *>(p.q + at) + col) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
                // the maxima of BATCH rows over LPR lanes: each exchange halves the rows a lane holds
                float am[BATCH];
#pragma unroll
                for (int x = 0; x < BATCH; x++) am[x] = absmax4(v[x]);
#pragma unroll
                for (int h = BATCH / 2, d = LPR / 2; d >= 1; d >>= 1, h >>= 1) {
                    if (h >= 1) {
                        const bool up = (col & d) != 0;
#pragma unroll
                        for (int x = 0; x < BATCH / 2; x++)
                            if (x < h) {
                                const float send = up ? am[x] : am[x + h], keep = up ? am[x + h] : am[x];
                                am[x] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, d));
                            }
                    } else {
                        am[0] = fmaxf(am[0], __shfl_xor_sync(0xffffffffu, am[0], d));
                    }
                }
                // lane (part, col) holds row x = col / (LPR / BATCH) of its part
                const int e0 = exponent_of(am[0]);
#pragma unroll
                for (int x = 0; x < BATCH; x++) {
                    const int e = __shfl_sync(0xffffffffu, e0, part * LPR + x * (LPR / BATCH));
                    const int rr = r0 + x * RPI + part, R = (row & ~31) + rr;
                    const float up = p.scale < 0.0f ? -pow2i(15 - e) : pow2i(15 - e);   // f is not negative
                    uint32_t h0, h1, l0, l1;
                    split2(v[x].x * up, v[x].y * up, h0, l0);
                    split2(v[x].z * up, v[x].w * up, h1, l1);
                    const uint32_t at = qs + R * 128 + ((((col & 15) >> 1) ^ (R & 7)) << 4);
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(h0), "r"(h1) : "memory");
                    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + L::OPERAND), "r"(l0), "r"(l1) : "memory");
                }
                // the row's own thread: row lane = r0 + x RPI + y is held by part y, row x
                const int x = (lane - r0) / RPI, y = (lane - r0) % RPI;
                const int ey = __shfl_sync(0xffffffffu, e0, (y * LPR + x * (LPR / BATCH)) & 31);
                if (lane >= r0 && lane < r0 + BATCH * RPI) ex = ey;
            }
            f = pow2i(ex - 15) * fabsf(p.scale);
            f = p.cap > 0.0f ? f / p.cap : f * LOG2E;
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) wait.arrive(Q_FULL + t);
        }
        if (flags & (F_TILE0 << t)) {
            const int live = m.live;
            bool whole = live == BT;   // every row sees every token (warp-uniform)
            float vmax = 0.0f;         // the largest value scale of the groups that the row sees some of
#pragma unroll
            for (int g = 0; g < GROUPS; g++) {
                whole = whole && m.base[g] >= all_lo && m.base[g] + 15 <= all_hi;
                vmax = fmaxf(vmax, m.vs[g]);
            }
            if (!whole) vmax = 0.0f;
            const bool simple = whole && p.cap == 0.0f && !p.slopes;
            if (!wait.warp(S_FULL + t, ns++)) return;
            tc_after();
            // ---- the block's maximum.  Where more than the scales is to be applied, the finished
            // scores go back to tensor memory, so that it is done once.
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (simple) {   // f is not negative: a group's largest raw score is its largest score
#pragma unroll 1
                for (int x = 0; x < BT; x += 32) {
                    float s0[16], s1[16];
                    tm_ld16(ts + x, s0);
                    tm_ld16(ts + x + 16, s1);
                    tm_wait16(s0);
                    tm_wait16(s1);
                    float a0 = s0[0], a1 = s1[0];
#pragma unroll
                    for (int e = 1; e < 15; e += 2) {
                        a0 = max3(a0, s0[e], s0[e + 1]);
                        a1 = max3(a1, s1[e], s1[e + 1]);
                    }
                    a0 = fmaxf(a0, s0[15]);
                    a1 = fmaxf(a1, s1[15]);
                    mx[0] = fmaxf(mx[0], a0 * (f * m.ks[x / 16]));
                    mx[1] = fmaxf(mx[1], a1 * (f * m.ks[x / 16 + 1]));
                }
            } else {
#pragma unroll 1
                for (int g = 0; g < GROUPS; g++) {
                    float s[16];
                    tm_ld16(ts + 16 * g, s);
                    tm_wait16(s);
                    const float fk = f * m.ks[g];
                    const int base = m.base[g];
#pragma unroll
                    for (int e = 0; e < 16; e++) s[e] *= fk;
                    if (p.cap > 0.0f) {
#pragma unroll
                        for (int e = 0; e < 16; e++) s[e] = cap2 * tanh_f32(s[e]);
                    }
                    if (p.slopes) {
#pragma unroll
                        for (int e = 0; e < 16; e++) s[e] -= slope * (float)abs(qpos - (base + e));
                    }
                    if (!whole) {   // bit e: the group's token e is there and seen
                        const uint32_t see = (bits16(seelo - base, qpos - base) | bits16(firstp - base, pre - 1 - base)) &
                                             bits16(0, live - 16 * g - 1);
#pragma unroll
                        for (int e = 0; e < 16; e++)
                            if (!(see & (1u << e))) s[e] = -INFINITY;
                        // (times a weight of 0, a masked group's scale only has to stay finite: 2^-112 of it counts)
                        vmax = fmaxf(vmax, m.vs[g] * (see ? 1.0f : 0x1p-112f));
                    }
#pragma unroll
                    for (int e = 0; e < 16; e++) mx[e & 3] = fmaxf(mx[e & 3], s[e]);
                    uint32_t u[16];
#pragma unroll
                    for (int e = 0; e < 16; e++) u[e] = __float_as_uint(s[e]);
                    tm_st16(ts + 16 * g, u);
                }
                tm_wait_st();
            }
            const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            // The sums are relative to mrow, which may lag behind the maximum by 6 (the weights then
            // reach 2^6), and O to 2^(vex - 8), where a value scale may reach 2^(vex + 1): weights times
            // scales stay below 2^15.  fp16 ends at 2^-25: a weight times its scale is carried to 2^-33
            // of the largest of both among the tokens that the row sees (vex is the row's own: the scales
            // of masked groups would push small values below that; the whole block's, for all rows alike,
            // took 282 us where this takes 284).  (A lag of 4 would carry it to 2^-35, but rescales O too
            // often: a prompt of 4096 takes 311 us instead of 281; one of 8 saves nothing.)
            const int ve = exponent_of(vmax);
            const bool grow = mb > mrow + 6.0f || (mrow == -INFINITY && mb != -INFINITY);
            // (this block's scores come after the products of the block before: O is complete up to it)
            if (blocks > 0 && blocks % FLUSH == 0) {
                const float cs = carry();
                // the sum is in the same units as O (nearly always): added without being read
                const bool add = blocks > FLUSH && __all_sync(0xffffffffu, cs == 1.0f);
#pragma unroll 1
                for (int x = 0; x < D; x += 32) {
                    float o[32];
                    tm_ld32(to + x, o);
                    tm_wait(o);
#pragma unroll
                    for (int y = 0; y < 32; y += 4) {
                        float4 *at = sum + (x + y) / 4 * BR;
                        if (add) {
                            red_add4(at, o[y], o[y + 1], o[y + 2], o[y + 3]);
                            continue;
                        }
                        float4 g = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (blocks > FLUSH) g = __ldcg(at);
                        __stcg(at, make_float4(fmaf(g.x, cs, o[y]), fmaf(g.y, cs, o[y + 1]), fmaf(g.z, cs, o[y + 2]),
                                               fmaf(g.w, cs, o[y + 3])));
                    }
                }
                gmax = mrow;
                gex = vex;
            }
            const bool have_o = blocks % FLUSH != 0;
            const int vnew = blocks == 0 || ve > vex + 1 ? ve : vex;
            if (__any_sync(0xffffffffu, grow || vnew != vex)) {
                const float mnew = grow ? mb : mrow;
                const float a = mnew == mrow ? 1.0f : ex2(mrow - mnew);
                lrow *= a;
                if (have_o) {
                    const float ao = a * pow2i(vex - vnew);
#pragma unroll 1
                    for (int x = 0; x < D; x += 32) {
                        float o[32];
                        tm_ld32(to + x, o);
                        tm_wait(o);
#pragma unroll
                        for (int y = 0; y < 32; y++) o[y] *= ao;
                        tm_st32(to + x, o);
                    }
                }
                mrow = mnew;
                vex = vnew;
            }
            blocks++;
            // ---- the weights: 32 tokens at a time, their two terms in the columns of their scores
            // (columns 0 .. 15 of each 32 the first term, 16 .. 31 the second)
            const float msafe = mrow == -INFINITY ? 0.0f : mrow, vu = pow2i(8 - vex);
            float *gl = nullptr;
            if (p.glse) gl = p.glse + ((int64_t)ti * p.Hq + head) * p.NG + (m.slot >> p.lgGroup);
            const uint64_t nm = pack2(-msafe, -msafe);
            const uint64_t minus = pack2(-1.0f, -1.0f);
            float cur[32];
            tm_ld32(ts, cur);
            tm_wait(cur);
            // 32 tokens at a time, while the next 32 are on their way.  (One copy of this code: the five
            // roles' loops together have to fit the instruction caches; unrolled, waiting for instructions
            // was a third of the stalls.)
#pragma unroll 1
            for (int x = 0; x < BT; x += 32) {
                uint64_t z[16];
                float vv[2], sum[2];
#pragma unroll
                for (int g = 0; g < 2; g++) {
                    vv[g] = m.vs[x / 16 + g] * vu;
                    const float fk = simple ? f * m.ks[x / 16 + g] : 1.0f;
                    const uint64_t fk2 = pack2(fk, fk);
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        z[8 * g + e] = fma2(pack2(cur[16 * g + 2 * e], cur[16 * g + 2 * e + 1]), fk2, nm);
                }
                if (x + 32 < BT) tm_ld32(ts + x + 32, cur);
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int g = 0; g < 2; g++) {
                    const uint64_t vv2 = pack2(vv[g], vv[g]);
                    uint64_t q = 0ull;
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        float p0, p1;
                        unpack2(z[8 * g + e / 2], p0, p1);
                        const uint64_t w = pack2(ex2(p0), ex2(p1));
                        q = add2(q, w);
                        // the first term: the leading 11 bits; the second: the rest, exact in f32
                        const uint64_t y = mul2(w, vv2);
                        unpack2(y, p0, p1);
                        p0 = __uint_as_float(__float_as_uint(p0) & 0xFFFFE000u);
                        p1 = __uint_as_float(__float_as_uint(p1) & 0xFFFFE000u);
                        hi[8 * g + e / 2] = half2_of(p0, p1);
                        unpack2(fma2(pack2(p0, p1), minus, y), p0, p1);
                        lo[8 * g + e / 2] = half2_of(p0, p1);
                    }
                    float q0, q1;
                    unpack2(q, q0, q1);
                    sum[g] = q0 + q1;
                }
                lrow += sum[0] + sum[1];
                if (gl && real && x < live) {
                    if (p.lgGroup == 4) {
                        gl[x / 16] = __log2f(sum[0]) + msafe;
                        if (x + 16 < live) gl[x / 16 + 1] = __log2f(sum[1]) + msafe;
                    } else {
                        gl[x / 32] = __log2f(sum[0] + sum[1]) + msafe;
                    }
                }
                tm_st16(ts + x, hi);
                tm_st16(ts + x + 16, lo);
                if (x & 32) {   // half of the weights are there: their product may begin
                    tm_wait_st();
                    tc_before();
                    __syncwarp();
                    if (lane == 0) wait.arrive(P_FULL + (x >> 6) * 2 + t);
                }
                if (x + 32 < BT) tm_wait(cur);
            }
        }
        if (flags & F_LAST) {
            const float l = lrow;
            const float inv = l > 0.0f ? pow2i(vex - 8) / l : 0.0f;
            const float cs = carry() * inv;
            if (!wait.warp(O_FULL + t, no++)) return;
            tc_after();
            // out by way of the query's memory (every product that read it is done): a row is stored
            // by D / 4 lanes together.  Each warp has a quarter of it: 32 rows of D f32, 16-byte
            // chunk x of row r at chunk x ^ (r mod 8).
            constexpr int LPR = D / 4, RPI = 32 / LPR;
            const uint32_t stage = smem_addr(smem + L::q) + 2 * t * L::OPERAND + (row >> 5) * (L::OPERAND / 2);
            if (!sync_tile()) return;   // the four warps' products: all of them are done
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                float o[32];
                if (blocks > 0) {
                    tm_ld32(to + x, o);
                    tm_wait(o);
                }
#pragma unroll
                for (int y = 0; y < 32; y += 4) {
                    float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f), g = r;
                    if (blocks > FLUSH) g = __ldcg(sum + (x + y) / 4 * BR);
                    if (l > 0.0f)
                        r = make_float4(fmaf(g.x, cs, o[y] * inv), fmaf(g.y, cs, o[y + 1] * inv),
                                        fmaf(g.z, cs, o[y + 2] * inv), fmaf(g.w, cs, o[y + 3] * inv));
                    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * D * 4 + ((((x + y) / 4) ^ (lane & 7)) << 4)),
                                 "f"(r.x), "f"(r.y), "f"(r.z), "f"(r.w)
                                 : "memory");
                }
            }
            __syncwarp();
            const int64_t to_part = ((int64_t)m.place * 2 + t) * BR + row;
            const int64_t mine = !real ? -1 : m.place >= 0 ? to_part * D : (int64_t)ti * p.ldo + (int64_t)head * D;
            float *out = m.place >= 0 ? plan.parts : p.out, *lse = m.place >= 0 ? plan.part_lse + to_part : p.lse + (int64_t)ti * p.Hq + head;
            const int part = lane / LPR, col = lane % LPR;
#pragma unroll 8
            for (int r0 = 0; r0 < 32; r0 += RPI) {
                const int rr = r0 + part;
                const int64_t at = __shfl_sync(0xffffffffu, mine, rr);
                const uint4 v = sh_ld128(stage + rr * D * 4 + ((col ^ (rr & 7)) << 4));
                if (at >= 0) *(reinterpret_cast<uint4 *>(out + at) + col) = v;
            }
            if (!sync_tile()) return;   // the next item's queries go into the same memory
            if (real && (p.lse || m.place >= 0)) *lse = l > 0.0f ? mrow + log2f(l) : INFINITY;
            tc_before();   // O is overwritten only after these loads (the next item's P_FULL)
        }
        __syncwarp();
        if (lane == 0) wait.arrive(META_EMPTY + st);
    }
}

// ---- the kernel ------------------------------------------------------------------------------
template <int KIND, int D>
__global__ void __launch_bounds__(THREADS, 1)
    attn_pages_tile_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                           const AttnParams8 p, const PlanView plan) {
    using L = TileLayout<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);   // (an offset: the compiler keeps the address space)
    TileSmem &sm = *reinterpret_cast<TileSmem *>(smem + L::ctl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PagesView &c = p.c;
    Waiter wait{c.status, sm.bars, false};

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        auto init = [&](int bar, int n) { mbar_init(smem_addr(sm.bars + bar), (uint32_t)n); };
        for (int i = 0; i < METAS; i++) {
            init(META_FULL + i, 1);
            init(META_EMPTY + i, 13);      // 8 softmax warps, 4 widening warps, the MMA warp
        }
        init(RAWK_FULL, 1);
        init(RAWV_FULL, 1);
        init(RAWK_EMPTY, 4);
        init(RAWV_EMPTY, 4);
        init(K_FULL, 4);
        init(V_FULL, 4);
        init(V_EMPTY, 1);
        for (int t = 0; t < 2; t++) {
            init(Q_FULL + t, 4);
            init(S_FULL + t, 1);
            init(P_FULL + t, 4);
            init(P_FULL + 2 + t, 4);
            init(O_FULL + t, 1);
            init(TILE_SYNC + t, 4);
        }
        init(ALL_DONE, 1);
        fence_barrier_init();
    }
    if (warp == 13) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = sm.tmem;
    pdl_wait();

    if (warp >= 12) {
        regs_dec<REGS_REST>();
        if (warp == 12) lead_role<KIND, D>(p, plan, kmap, vmap, smem, sm, wait, lane);
        if (warp == 13) {
            if (lane == 0) {
                mma_role<D>(smem, sm, wait, tmem);
                // the products issued have completed before shared and tensor memory are given up
                mma_commit(smem_addr(sm.bars + ALL_DONE));
                mbar_wait(smem_addr(sm.bars + ALL_DONE), 0u, c.status);
            }
            __syncwarp();
        }
    } else if (warp >= 8) {
        regs_dec<REGS_REST>();
        widen_role<KIND, D>(smem, sm, wait, threadIdx.x - 256, lane);
    } else {
        regs_inc<REGS_SOFTMAX>();
        softmax_role<D>(p, smem, sm, wait, tmem, plan, warp >> 2, threadIdx.x & 127, lane);
    }
    __syncthreads();
    if (warp == 13) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

// ---- shares of an item joined -------------------------------------------------------------------
// A row of D / 4 lanes at a time: the shares' outputs by their denominators, in order.
constexpr int JOIN_ROWS = 16;

template <int D>
__global__ void __launch_bounds__(256) attn_pages_join_kernel(const AttnParams8 p, const PlanView plan) {
    pdl_launch_dependents();
    pdl_wait();
    const int Hkv = (int)p.c.Hkv, place = blockIdx.y;
    if (place / Hkv >= __ldcg(plan.count)) return;
    const int4 e = __ldcg(plan.list + place / Hkv);
    const int splits = e.w;
    if (splits == 1 || e.z > 0) return;   // (the first share's blocks join)
    const SeqStep s = attn_step(p, e.x);
    constexpr int LPR = D / 4, RPI = 256 / LPR;
    const int col = threadIdx.x % LPR;
#pragma unroll
    for (int r0 = 0; r0 < JOIN_ROWS; r0 += RPI) {
        const int row = blockIdx.x * JOIN_ROWS + r0 + threadIdx.x / LPR, r = e.y * 2 * BR + row;
        if (r >= s.n * p.G) return;
        float lse = -INFINITY, sum = 0.0f;
        auto part = [&](int z) { return (int64_t)(place + z * Hkv) * 2 * BR + row; };
#pragma unroll 8
        for (int z = 0; z < splits; z++) {
            const float x = __ldcg(plan.part_lse + part(z));
            if (x != INFINITY) lse = fmaxf(lse, x);
        }
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int z = 0; z < splits; z++) {   // (a share that saw nothing has zeros)
            const float x = __ldcg(plan.part_lse + part(z));
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(plan.parts + part(z) * D) + col);
            const float w = x == INFINITY ? 0.0f : ex2(x - lse);
            sum += w;
            o.x = fmaf(w, v.x, o.x);
            o.y = fmaf(w, v.y, o.y);
            o.z = fmaf(w, v.z, o.z);
            o.w = fmaf(w, v.w, o.w);
        }
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        const int ti = s.t0 + r / p.G;
        const int64_t head = (int64_t)(place % Hkv) * p.G + r % p.G;
        reinterpret_cast<float4 *>(p.out + ti * p.ldo + head * D)[col] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (p.lse && col == 0) p.lse[(int64_t)ti * p.Hq + head] = sum > 0.0f ? lse + log2f(sum) : INFINITY;
    }
}

template <int KIND, int D>
gq_status launch_tiles(const AttnParams8 &p, const gq_kv_pages &c, const PlanView &plan, int64_t items, cudaStream_t s) {
    auto kernel = attn_pages_tile_kernel<KIND, D>;
    constexpr int smem = TileLayout<D>::total + 1024;
    static std::atomic<bool> smem_set[64];
    int dev = 0;
    KV_TRY(check_cuda(cudaGetDevice(&dev), "cudaGetDevice"));
    if (dev < 0 || dev >= 64) return fail(GQ_ERR_UNSUPPORTED_DEVICE, "device index %d", dev);
    if (!smem_set[dev].load(std::memory_order_acquire)) {
        KV_TRY(check_cuda(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                          "paged attention shared-memory attribute"));
        smem_set[dev].store(true, std::memory_order_release);
    }
    alignas(64) CUtensorMap kmap, vmap;
    const int64_t rows = c.pages * c.P * c.D / 128;
    const int box = (int)(c.P * D / 128);
    KV_TRY(byte_rows_map(&kmap, c.k, rows, box));
    KV_TRY(byte_rows_map(&vmap, c.v, rows, box));
    void *args[] = {(void *)&kmap, (void *)&vmap, (void *)&p, (void *)&plan};
    return launch_pdl((const void *)kernel, dim3((unsigned)std::min<int64_t>(items, sm_count())), dim3(THREADS), smem, s,
                      args, "paged attention (tiles) launch");
}

// At most so many pairs of tiles: the rows of all sequences, and a last pair of each.
int64_t most_pairs(const gq_kv_pages &c, int64_t rows, int64_t G) { return rows * G / (2 * BR) + std::min(c.B, rows) + 1; }

}  // namespace

// Whether the rows, if all are in tiles, may leave half of the SMs idle: places for shares' outputs.
static int share_places(const gq_kv_pages &c, int64_t rows, int64_t G) {
    return rows * G / (2 * BR) * c.Hkv * 2 > sm_count() ? 0 : sm_count();
}

static size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

size_t attn_pages_tc_workspace(const gq_kv_pages &c, int64_t rows, int64_t G) {
    const size_t places = (size_t)share_places(c, rows, G);
    return 256 + round_up(((size_t)most_pairs(c, rows, G) + places) * sizeof(int4)) +
           (size_t)sm_count() * 2 * c.D * BR * 4 + places * 2 * BR * (c.D + 1) * 4;
}

gq_status launch_attn_pages_tc(const AttnParams8 &p, const gq_kv_pages &c, uint8_t *work, cudaStream_t s) {
    PlanView plan{};
    const int64_t rows = p.row1 - p.row0;
    plan.places = share_places(c, rows, p.G);
    const int64_t entries = most_pairs(c, rows, p.G) + plan.places;
    plan.room = (int)std::min<int64_t>(entries, INT32_MAX);
    plan.count = reinterpret_cast<int *>(work);
    plan.next = plan.count + 1;
    plan.list = reinterpret_cast<int4 *>(work + 256);
    plan.sums = reinterpret_cast<float *>(work + 256 + round_up((size_t)entries * sizeof(int4)));
    plan.parts = plan.places ? plan.sums + (size_t)sm_count() * 2 * c.D * BR : nullptr;
    plan.part_lse = plan.places ? plan.parts + (size_t)plan.places * 2 * BR * c.D : nullptr;
    if (entries * c.Hkv > INT32_MAX) return fail(GQ_ERR_INVALID_ARG, "attention grid too large");
    void *args[] = {(void *)&p, (void *)&plan};
    KV_TRY(launch_pdl((const void *)attn_pages_plan_kernel, dim3(1), dim3(256), 0, s, args, "paged attention plan launch"));
    const int64_t items = entries * c.Hkv;
    gq_status st;
    if (c.kind == GQ_KV_I8)
        st = c.D == 64 ? launch_tiles<GQ_KV_I8, 64>(p, c, plan, items, s) : launch_tiles<GQ_KV_I8, 128>(p, c, plan, items, s);
    else
        st = c.D == 64 ? launch_tiles<GQ_KV_E4M3, 64>(p, c, plan, items, s)
                       : launch_tiles<GQ_KV_E4M3, 128>(p, c, plan, items, s);
    if (st != GQ_OK || !plan.places) return st;
    return launch_pdl(c.D == 64 ? (const void *)attn_pages_join_kernel<64> : (const void *)attn_pages_join_kernel<128>,
                      dim3(2 * BR / JOIN_ROWS, (unsigned)plan.places), dim3(256), 0, s, args, "paged attention join launch");
}

}  // namespace gq

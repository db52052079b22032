// mx_gemm.cu -- products of e4m3 blocks with 4-bit (e2m1) block weights on tcgen05, for one matrix
// or for the matrices of many experts, and the gated unit silu(gate) * up with its output in blocks.
//
// dst^T = W . X^T: a tile is 128 weight rows (the MMA's M, tensor-memory lanes) by up to BN rows of
// activations (its N, tensor-memory columns; an MMA is as wide as its tile's rows need, in steps of
// 16).  kind::mxf8f6f4 multiplies the codes and each block of 32 by its two powers of two.  What bounds a
// full tile is shared memory's 128 bytes a cycle, so the weights go through it once, packed, and reach the
// MMAs in tensor memory:
//   warp 0     one thread copies, some stages of 128 columns ahead: the weights' tile (packed codes, scales) by a
//              bulk copy, the activations' codes by a tensor copy, of four rows at a time where a plan names
//              them (16-row tiles; for larger ones that would be too many copies for a thread, and a kernel in front
//              brings the rows into the plan's order);
//   warps 2, 3     copy the activations' scales (of one or two rows of values: quantize them);
//   warps 12 .. 19  two teams, for every other stage each (a stage is mostly latency).  A weight row per thread:
//              64 bytes of packed codes become 128 bytes, a code in bits 2 .. 5 of each (the form of 4-bit operands
//              in tensor memory), and go there, and so do the scales of both operands.  The tiles hold the codes so
//              that three instructions place eight of them;
//   warp 1     one thread issues 4 MMAs a stage (8 for the gated unit, whose gate and up tiles share the
//              activations).  The thread is elected, not picked by its lane: the compiler then keeps the
//              descriptors in uniform registers (measured: 39 cycles per MMA of 16 columns, not 80);
//   warps 4 .. 11  take the sums over: the tensor cores' accumulators cut off what does not fit 24 bits, so
//              every 8 to 16 stages they are added, rounded, to f32 registers, while the next stages go
//              to another set of accumulators; then they store the tile.
// CTAs take tiles in turn (persistent), those of one expert's weight rows next to each other.  With few
// tiles a cluster of 2 or 4 CTAs shares a tile's columns; the first adds the others' sums in order.
//
// Measured, products of blocks in a captured graph, weights from memory: 2047 rows by [4096, 11008] 75 us, 2.5 PFLOP/s (81
// under ncu: 13 TB/s from L2, as each CTA fetches its own operands, which bounds the large tiles; the tensor pipe is busy for
// 48 %); 61 tokens on 8 of 64 experts of [2816, 2048] 50 us, 4.0 TB/s from memory (a stage's latencies); a row by
// [4096, 4096] 8.5 us.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>

#include "mx.cuh"

namespace gq {
namespace {

constexpr int THREADS = 640;
constexpr int EPI_WARPS = 8;
constexpr int SPREAD_WARPS = 4;              // of a team, 32 weight rows each
constexpr int SCALE_WARPS = 2;
constexpr int MAX_E = 1024;
constexpr int MAX_STAGES = 16, MAX_SLOTS = 8, MAX_SETS = 4;
constexpr int FEW_REGS = 56, MANY_REGS = 152;   // per thread, of 96 at launch: 3 x 56 + 2 x 152 < 5 x 96

// BN: rows of activations per tile.  GATED: two weight tiles (gate, up) per stage.
template <int BN, bool GATED>
struct Cfg {
    static constexpr int NA = GATED ? 2 : 1;
    static constexpr int ST = BN <= 16 ? (GATED ? 8 : 16) : BN <= 64 ? (GATED ? 6 : 10) : 6;   // stages in shared memory
    static constexpr int PARTS = BN > 64 ? 2 : 1;           // tensor copies of a tile's activations, BN / PARTS rows each
    static constexpr int BOX = BN / PARTS;
    static constexpr int CW = BN <= 16 ? 8 : 16;            // columns per read of tensor memory
    static constexpr int CHUNKS = BN / CW;
    static constexpr int MINE = (CHUNKS + 1) / 2;           // chunks of a warpgroup
    static constexpr bool BIG = NA * MINE * CW >= 64;       // more sums per thread than an even share of registers holds
    static constexpr bool GATHERS = BN <= 16;
    static constexpr bool QUANTIZES = BN <= 16 && !GATED;   // takes rows of f32 or bf16 too
    static constexpr int MAX_SPLIT = BN <= 16 ? 4 : 1;      // (for 64 rows two: 17 rows 9.7 us against 10.1, 65 rows 10.9 against 10.6)
    // Tensor memory: sets of accumulators, then slots of a stage's weights and scales.  The gated unit's large
    // tile has one set only; its accumulators are taken over every 16 stages (2048 columns; what is cut
    // off meanwhile, 2^-24 of the sums 64 times at most, is far below its output's 2^-4), gate before up, so
    // that the next gate MMAs wait for half of it.
    static constexpr int ACC = NA * BN;
    static constexpr int SETS = GATED ? (BN <= 16 ? 4 : BN <= 64 ? 2 : 1) : (BN <= 64 ? 4 : 2);
    // Stages per take-over of the accumulators.  An MMA cuts off what is below a unit of its sum, a take-over rounds: sums of
    // one sign over 8192 columns came out within 2.1e-7 (3e-8 low on average), in f32 FMAs within 2.2e-7.  For the plain
    // product's large tile 12 (96 us for 2047 rows; 97 by 8, 101 by 4: the further the MMAs run ahead, the more of a
    // tile's output they hide).
    static constexpr int FLUSH = SETS == 1 ? 16 : BN > 64 ? 12 : 8;
    static constexpr int NR = (BN + 31) / 32;               // scales of activation rows: columns, words of a lane
    static constexpr int SFB = NR <= 1 ? 4 : NR <= 4 ? 4 : 8;
    static constexpr int SLOT = NA * 36 + SFB;              // 32 columns of codes and 4 of scales per weight tile
    static constexpr int NS = BN <= 16 ? (GATED ? 4 : 8) : BN <= 64 ? (GATED ? 3 : 6) : 3;
    static constexpr int SLOTS = SETS * ACC;                // their first column
    static constexpr int COLS_USED = SLOTS + NS * SLOT;
    static constexpr int COLS = COLS_USED <= 256 ? 256 : 512;
    static_assert(COLS_USED <= 512, "tensor memory");
    static_assert(BOX % 8 == 0 && BN % 16 == 0, "tile rows");
    static_assert(ST % 2 == 0 && NS < ST && NS <= MAX_SLOTS && ST <= MAX_STAGES && SETS <= MAX_SETS, "barriers");
    // shared memory from a 1024-aligned base
    static constexpr int B_STAGE = BN * 128;
    static constexpr int b = 0;
    static constexpr int w = b + ST * B_STAGE;
    static constexpr int part = w + ST * NA * MX_TILE_BYTES;
    static constexpr int PART_BYTES = NA * BN * MX_TILE * 4;
    static constexpr int SB_STAGE = NR * 32 * 4;            // a stage's scales of the activation rows
    static constexpr int sb = part + (MAX_SPLIT - 1) * PART_BYTES;
    static constexpr int starts = sb + ST * SB_STAGE;
    static constexpr int bars = starts + 3 * (MAX_E + 4) * 4;
    static constexpr int total = bars + 768;
    static_assert(total + 1024 <= 227 * 1024, "shared memory");
};

enum : int {
    RAW = 0,                     // a stage's copies have landed
    EMPTY = RAW + MAX_STAGES,    // its MMAs are done
    FULL = EMPTY + MAX_STAGES,   // a slot's weights and scales are in tensor memory
    ACC_FULL = FULL + MAX_SLOTS,
    ACC_EMPTY = ACC_FULL + MAX_SETS,         // gate and up apart
    SCALES = ACC_EMPTY + 2 * MAX_SETS,   // a stage's scales of activations have landed
    PART_FULL = SCALES + MAX_STAGES,
    PART_EMPTY,
    NUM_BARS
};
static_assert(NUM_BARS * 8 + 8 <= 768, "barrier area");

struct MxParams {
    const uint8_t *w;              // tiles
    const uint8_t *x_scales;
    const int32_t *offsets, *rows;
    void *dst;
    uint8_t *codes, *scales;       // gated: the output's
    unsigned int *status;
    int lo, hi, base;              // rows of the plan that this launch does; which of them is row 0 of x
    int64_t ldd, x_rows;
    int N, K, KT, G, S, So;        // S, So: scale bytes per row of x and of the gated output
    int E, R, split, bf16;
    const void *values;            // rows to quantize (no plan, at most MX_FEW_ROWS), instead of x's codes and scales
    int64_t ldv;
    int values_bf16;
};

// ---------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------
// K-major operand, 128-byte swizzle, 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
// kind::mxf8f6f4: A e2m1 (5), B e4m3 (0), both K-major, scales ue8m0, f32 sums; the scale bytes'
// places (0 .. 3) go to bits 4 and 29
__device__ __forceinline__ uint32_t mx_idesc(int n) {
    return 5u << 7 | (uint32_t)(n >> 3) << 17 | 1u << 23 | (uint32_t)(MX_TILE >> 4) << 24;
}
// A, D and the scales in tensor memory; the descriptor of B in two halves (the low one holds the address)
__device__ __forceinline__ void mma_mx(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %7, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], [%1], b, %4, [%5], [%6], p;\n\t}"
        ::"r"(d), "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// one 32-bit column per value, this warp's 32 lanes
template <int W>
__device__ __forceinline__ void write_tmem(uint32_t taddr, const uint32_t (&r)[W]) {
    if constexpr (W == 1)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r[0]) : "memory");
    else if constexpr (W == 2)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(r[0]), "r"(r[1]) : "memory");
    else if constexpr (W == 16)
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
                taddr),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
            "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
            : "memory");
    else if constexpr (W == 4)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                     : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                     "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
}
// Eight codes as the tiles hold them (0 .. 3 in bits 2 .. 5 of the bytes, 4 .. 7 in bits 6 .. 9 from each byte on, the
// last around the word's end), each into bits 2 .. 5 of a byte.
__device__ __forceinline__ void spread8(uint32_t w, uint32_t &lo, uint32_t &hi) {
    lo = w & 0x3C3C3C3Cu;
    hi = __funnelshift_r(w, w, 4) & 0x3C3C3C3Cu;
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void copy_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
// four rows of 128 bytes
__device__ __forceinline__ void copy_rows4(uint32_t dst, const CUtensorMap *map, int c0, int4 r, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
        : "memory");
}
// one lane of the warp
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// 4 bytes, zeros unless `there`
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
// this thread's copies so far will arrive there (once) when they are done
__device__ __forceinline__ void arrive_copied(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
// Whether a phase is over, without waiting.  Asked ahead of time: an answer takes over a hundred cycles.
__device__ __forceinline__ bool ready(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// A place in the ring of stages and the parity of its turn.
template <int ST>
struct Ring {
    int st = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void next() {
        if (++st == ST) st = 0, turn ^= 1;
    }
};
// A role's registers (all warps of a warpgroup take the same step).
template <bool BIG, bool MANY>
__device__ __forceinline__ void set_registers() {
    if constexpr (BIG && MANY) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(MANY_REGS));
    if constexpr (BIG && !MANY) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FEW_REGS));
}
// W columns of this warp's 32 lanes; the values are there after tcgen05.wait::ld
template <int W>
__device__ __forceinline__ void read_acc(uint32_t taddr, uint32_t (&r)[W]) {
    if constexpr (W == 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr));
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
}
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
// a value read from tensor memory, not used before the wait in front of this
__device__ __forceinline__ float keep(uint32_t r) {
    asm volatile("" : "+r"(r));
    return __uint_as_float(r);
}

__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// as mbar_wait, and what other CTAs of the cluster wrote before they arrived is seen
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, unsigned int *status) {
    for (uint32_t i = 0; i < WAIT_LIMIT; i++) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return true;
    }
    flag_timeout(status);
    return false;
}

// x / (1 + exp(-x)), within (1.25 |x| + 10) 2^-24 of itself: the exponential's argument is a rounded product with a rounded
// log2(e), off by 1.22 |x| 2^-24 in e's exponent, the fast exponential by 2^-22 and the reciprocal by 2^-23.  Both
// flush denormals: of the exponential that leaves 1 + 0, and the reciprocal is taken of a quarter of the sum, so that
// it has none.  From -88.73 down the exponential is infinite and this 0, where x exp(x) is 2.6e-37 or less.
__device__ __forceinline__ float swish(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e, 0.25f, 0.25f)));
    return x * (0.25f * r);
}

// Where tiles lie, in shared memory: starts[e] tiles of BN rows (for one group of weight rows) come before
// expert e, whose rows are first[e] .. last[e] - 1.
struct Where {
    int32_t *starts, *first, *last;
};
// Tile `i` of the launch: expert e, weight rows 128 g .., activation rows r0 .. r0 + n - 1.
struct Tile {
    int e, g, r0, n;
};
template <int BN>
__device__ __forceinline__ Tile tile_at(const MxParams &p, const Where &w, int i) {
    int lo = 0, hi = p.E;                                  // starts[e] * G <= i < starts[e + 1] * G
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (w.starts[mid] * p.G <= i)
            lo = mid;
        else
            hi = mid;
    }
    const int nt = w.starts[lo + 1] - w.starts[lo], local = i - w.starts[lo] * p.G;
    Tile t;
    t.e = lo;
    t.g = local / nt;
    t.r0 = w.first[lo] + (local - t.g * nt) * BN;
    t.n = min(BN, w.last[lo] - t.r0);
    return t;
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int BN, bool GATED>
__global__ void __launch_bounds__(THREADS, 1)
    mx_product_kernel(const __grid_constant__ CUtensorMap map_x, const MxParams p) {
    using C = Cfg<BN, GATED>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::bars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + NUM_BARS);
    Where where;
    where.starts = reinterpret_cast<int32_t *>(smem + C::starts);
    where.first = where.starts + MAX_E + 4;
    where.last = where.first + MAX_E + 4;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int split = p.split, rank = (int)blockIdx.x % split, cluster = (int)blockIdx.x / split, clusters = (int)gridDim.x / split;
    auto bar = [&](int i) { return smem_addr(bars + i); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::ST; i++) {
            mbar_init(bar(RAW + i), 1);
            mbar_init(bar(EMPTY + i), 1);
            mbar_init(bar(SCALES + i), SCALE_WARPS * 32);
        }
        for (int i = 0; i < C::NS; i++) mbar_init(bar(FULL + i), SPREAD_WARPS);
        for (int i = 0; i < C::SETS; i++) mbar_init(bar(ACC_FULL + i), 1);
        for (int i = 0; i < C::SETS * C::NA; i++) mbar_init(bar(ACC_EMPTY + i), EPI_WARPS);
        mbar_init(bar(PART_FULL), (split - 1) * EPI_WARPS + (split == 1));
        mbar_init(bar(PART_EMPTY), EPI_WARPS);
    }
    fence_barrier_init();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)), "r"(C::COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) {
        // tiles of BN rows in front of each expert; ranges are disjoint, so that the host's count of tiles bounds them
        int before = 0, end = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int tiles = 0, r0 = 0, r1 = 0, most = 0;
            if (e < p.E) {
                r0 = p.offsets ? p.offsets[e] : 0, r1 = p.offsets ? p.offsets[e + 1] : p.R;
                if (r0 >= 0 && r1 >= r0 && r1 <= p.R) most = r1;
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, most, d);
                if (lane >= d) most = max(most, u);
            }
            int front = __shfl_up_sync(0xffffffffu, most, 1);      // the largest end of the experts in front
            front = lane ? max(front, end) : end;
            end = max(end, __shfl_sync(0xffffffffu, most, 31));
            if (e < p.E) {
                if (r0 < front || r1 < r0 || r1 > p.R) {
                    atomicOr(p.status, STATUS_RANGE);
                    r0 = r1 = 0;
                }
                r0 = max(r0, p.lo);
                r1 = min(r1, p.hi);
                where.first[e] = r0;
                where.last[e] = r1;
                if (r1 > r0) tiles = (r1 - r0 + BN - 1) / BN;
            }
            int s = tiles;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, s, d);
                if (lane >= d) s += u;
            }
            if (e < p.E) where.starts[e] = before + s - tiles;
            before += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) where.starts[p.E] = before;
    }
    fence_before();
    __syncthreads();
    if (split > 1) cluster_sync();            // every CTA's barriers are there before others arrive on them
    fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const int tiles = where.starts[p.E] * p.G;
    const int kt0 = (int)((int64_t)p.KT * rank / split), nk = (int)((int64_t)p.KT * (rank + 1) / split) - kt0;
    bool failed = false;
    if (warp == 0) {
        // ------------------------------------------------------------------ copies
        set_registers<C::BIG, false>();
        if (elect()) {
            Ring<C::ST> ring;
            int filled = 0;
            for (int i = cluster; i < tiles && !failed; i += clusters) {
                const Tile t = tile_at<BN>(p, where, i);
                GQ_DCHECK(t.e < p.E && t.g < p.G && t.n > 0 && t.r0 >= p.lo && t.r0 + t.n <= p.hi, p.status);
                const uint8_t *w = p.w + (((int64_t)t.e * C::NA * p.G + t.g) * p.KT + kt0) * MX_TILE_BYTES;
                const int64_t up = (int64_t)p.G * p.KT * MX_TILE_BYTES;    // from the gate's tile to the up matrix's
                const int parts = t.n > C::BOX ? C::PARTS : 1;
                const bool quantizes = C::QUANTIZES && p.values;
                const uint32_t bytes = (uint32_t)(C::NA * MX_TILE_BYTES + (quantizes ? 0 : parts * C::BOX * 128));
                int4 from[4];                              // gathered rows; past the tile and outside x: zeros
                if (C::GATHERS && p.rows)
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        int r[4];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            r[j] = u * 4 + j < t.n ? __ldg(p.rows + t.r0 + u * 4 + j) : (int)p.x_rows;
                            if (r[j] < 0 || r[j] > p.x_rows) r[j] = (int)p.x_rows;
                        }
                        from[u] = make_int4(r[0], r[1], r[2], r[3]);
                    }
                for (int k = 0; k < nk; k++, w += MX_TILE_BYTES, ring.next()) {
                    if (filled == C::ST) {
                        if (!mbar_wait(bar(EMPTY + ring.st), ring.turn ^ 1, p.status)) {
                            failed = true;
                            break;
                        }
                    } else {
                        filled++;
                    }
                    const uint32_t raw = bar(RAW + ring.st);
                    mbar_arrive_expect_tx(raw, bytes);
#pragma unroll
                    for (int a = 0; a < C::NA; a++)
                        bulk_g2s(smem_addr(smem + C::w) + (uint32_t)((ring.st * C::NA + a) * MX_TILE_BYTES), w + a * up, MX_TILE_BYTES, raw);
                    if (quantizes) continue;
                    if (C::GATHERS && p.rows) {
#pragma unroll
                        for (int u = 0; u < 4; u++)
                            copy_rows4(smem_addr(smem + C::b) + (uint32_t)(ring.st * C::B_STAGE + u * 512), &map_x, (kt0 + k) * MX_TILE, from[u], raw);
                        continue;
                    }
#pragma unroll
                    for (int u = 0; u < C::PARTS; u++)
                        if (u < parts)
                            copy_2d(smem_addr(smem + C::b) + (uint32_t)(ring.st * C::B_STAGE + u * C::BOX * 128), &map_x, (kt0 + k) * MX_TILE,
                                    t.r0 - p.base + u * C::BOX, raw);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMAs
        set_registers<C::BIG, false>();
        if (elect()) {
            Ring<C::ST> ring;
            Ring<C::NS> slot;
            Ring<C::SETS> set;
            const uint32_t full = bar(FULL), empty = bar(EMPTY), slots = tmem + (uint32_t)C::SLOTS;
            const uint64_t bdesc = operand_desc(smem_addr(smem + C::b));
            const uint32_t b_lo = (uint32_t)bdesc, b_hi = (uint32_t)(bdesc >> 32);
            int chunks = 0;
            bool full_ready = false;
            for (int i = cluster; i < tiles && !failed; i += clusters) {
                const Tile t = tile_at<BN>(p, where, i);
                uint32_t idesc[4];                         // of the scale bytes' four places
#pragma unroll
                for (int kk = 0; kk < 4; kk++) idesc[kk] = mx_idesc((t.n + 15) & ~15) + (uint32_t)kk * ((1u << 4) | (1u << 29));
                int in_chunk = 0;
                for (int k = 0; k < nk; k++) {
                    // (whoever arrived there had waited for the stage's copies)
                    if (!full_ready && !mbar_wait(full + slot.st * 8, slot.turn, p.status)) failed = true;
                    const uint32_t sl = slots + (uint32_t)(slot.st * C::SLOT), acc = tmem + (uint32_t)(set.st * C::ACC);
                    const uint32_t bd = b_lo + (uint32_t)(ring.st * (C::B_STAGE >> 4));
#pragma unroll
                    for (int a = 0; a < C::NA; a++) {
                        if (in_chunk == 0 && chunks == C::SETS && !failed &&
                            !mbar_wait(bar(ACC_EMPTY + set.st * C::NA + a), set.turn ^ 1, p.status))
                            failed = true;
                        if (failed) break;
                        fence_after();
#pragma unroll
                        for (int kk = 0; kk < 4; kk++)     // 32 columns: 8 of tensor memory, 32 bytes of the activations, the next scale byte
                            mma_mx(acc + a * BN, sl + (uint32_t)(a * 32 + kk * 8), bd + kk * 2, b_hi, idesc[kk], sl + (uint32_t)(C::NA * 32 + a * 4),
                                   sl + (uint32_t)(C::NA * 36), in_chunk > 0 || kk > 0);
                    }
                    if (failed) break;
                    commit(empty + ring.st * 8);
                    ring.next();
                    slot.next();
                    full_ready = ready(full + slot.st * 8, slot.turn);
                    if (++in_chunk == C::FLUSH || k == nk - 1) {
                        commit(bar(ACC_FULL + set.st));
                        set.next();
                        in_chunk = 0;
                        if (chunks < C::SETS) chunks++;
                    }
                }
            }
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------------ the activations' scales
        set_registers<C::BIG, false>();
        const int x = (warp - 2) * 32 + lane;
        constexpr int SROWS = (C::NR * 32 + 63) / 64;      // thread x copies the scales of the tile's rows x, x + 64, ..
        int scale_row[SROWS], filled = 0;
        Ring<C::ST> ring;
        bool free = false;
        auto row = [&](const Tile &t, int c) {             // the tile's row c in x, or -1
            int r = -1;
            if (c < t.n) {
                r = p.rows ? __ldg(p.rows + t.r0 + c) : t.r0 - p.base + c;
                if (r < 0 || r >= p.x_rows) atomicOr(p.status, STATUS_RANGE), r = -1;
            }
            return r;
        };
        // One or two rows that are not quantized yet: these threads write the codes too, those of 8 stages at a time (a quarter
        // of a block each, four times), the next ones' values under way.  Rows past them hold anything: their columns of the sums
        // are not stored.
        auto quantize = [&](const auto *values) {
            constexpr int many = 8;
            const int r = (x >> 4) & 1, block = (x >> 2) & 3;      // row, block of the stage (u * 2 + x / 32)
            for (int i = cluster; i < tiles && !failed; i += clusters) {
                const Tile t = tile_at<BN>(p, where, i);
                float v[4][8];
                auto load = [&](int k) {
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const int stage = k + u * 2 + (x >> 5), col = (kt0 + stage) * MX_TILE + block * QK + (x & 3) * 8;
#pragma unroll
                        for (int c = 0; c < 8; c++) v[u][c] = 0.0f;
                        if (stage < nk && r < t.n && col < p.K) load8(values + (t.r0 + r) * p.ldv + col, v[u]);
                    }
                };
                load(0);
                for (int k = 0; k < nk; k += many) {
                    uint2 code[4];
                    int byte[4];
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        byte[u] = mx_scale_byte(block_amax(v[u]), false);
                        code[u] = codes8<false>(v[u], mx_inverse(byte[u]));
                    }
                    const int stages = min(many, nk - k);
                    if (k + many < nk) load(k + many);
                    Ring<C::ST> at = ring;
                    for (int j = 0; j < stages; j++, at.next()) {
                        if (filled < C::ST)
                            filled++;
                        else if (!failed && !mbar_wait(bar(EMPTY + at.st), at.turn ^ 1, p.status))
                            failed = true;
                    }
                    failed = __any_sync(0xffffffffu, failed);
                    if (failed) break;
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const int j = u * 2 + (x >> 5), st = ring.st + j < C::ST ? ring.st + j : ring.st + j - C::ST;
                        if (j >= stages) continue;
                        // (16 bytes' place in a row of 128: swizzled by the row)
                        uint8_t *const to = smem + C::b + st * C::B_STAGE + r * 128 + ((block * 2 + ((x & 3) >> 1)) ^ r) * 16;
                        *reinterpret_cast<uint2 *>(to + (x & 1) * 8) = code[u];
                        if ((x & 3) == 0) smem[C::sb + st * C::SB_STAGE + r * 4 + block] = (uint8_t)byte[u];
                    }
                    fence_proxy_async_shared();            // (the MMAs read the codes)
                    for (int j = 0; j < stages; j++, ring.next()) mbar_arrive(bar(SCALES + ring.st));
                }
            }
        };
        if (C::QUANTIZES && p.values) {
            if (p.values_bf16)
                quantize(static_cast<const __nv_bfloat16 *>(p.values));
            else
                quantize(static_cast<const float *>(p.values));
        } else {
            for (int i = cluster; i < tiles && !failed; i += clusters) {
                const Tile t = tile_at<BN>(p, where, i);
#pragma unroll
                for (int j = 0; j < SROWS; j++) scale_row[j] = row(t, j * 64 + x);
                for (int k = 0; k < nk; k++) {
                    const int kt = kt0 + k;
                    if (filled == C::ST) {
                        if (!free && !mbar_wait(bar(EMPTY + ring.st), ring.turn ^ 1, p.status)) failed = true;
                        failed = __any_sync(0xffffffffu, failed);
                        if (failed) break;
                    } else {
                        filled++;
                    }
                    GQ_DCHECK(kt >= 0 && kt < p.KT && kt * 4 < p.S, p.status);
                    const uint32_t scales = smem_addr(smem + C::sb) + (uint32_t)(ring.st * C::SB_STAGE + x * 4);
#pragma unroll
                    for (int j = 0; j < SROWS; j++)
                        if (j * 64 + x < C::NR * 32)
                            copy4(scales + j * 256, p.x_scales + (scale_row[j] >= 0 ? (int64_t)scale_row[j] * p.S + kt * 4 : 0), scale_row[j] >= 0);
                    arrive_copied(bar(SCALES + ring.st));
                    ring.next();
                    free = filled == C::ST && ready(bar(EMPTY + ring.st), ring.turn ^ 1);
                }
            }
        }
        copy_wait();                                    // (nothing of this CTA's shared memory is under way at its end)
    } else if (warp >= 12) {
        // ------------------------------------------------------------------ weights and scales into tensor memory
        set_registers<C::BIG, false>();
        const int q = warp & 3, team = (warp - 12) >> 2;   // tensor-memory lanes, weight rows 32 q ..; every other stage
        constexpr int WB = C::NR == 3 ? 4 : C::NR > 4 ? 8 : C::NR;
        const int steps = cluster < tiles ? (tiles - cluster + clusters - 1) / clusters * nk : 0;
        const int blocks = p.K / QK - kt0 * 4;             // scale bytes of this CTA's columns
        const uint32_t raw0 = smem_addr(smem + C::w) + (uint32_t)((q * 32 + lane) * 16), sb0 = smem_addr(smem + C::sb) + (uint32_t)(lane * 4);
        const uint32_t raw_bar = bar(RAW), scales_bar = bar(SCALES), empty = bar(EMPTY), full = bar(FULL);
        const uint32_t sl0 = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)C::SLOTS;
        Ring<C::ST> ring, freed;                           // this stage; the one whose MMAs read the slot last
        Ring<C::NS> slot;
        int k = 0;
        if (team) {
            ring.next();
            slot.next();
            if (++k == nk) k = 0;
        }
        // The stage NS before this one; for the first ones there is none.
        auto to_freed = [&](int step) {
            const int f = step - C::NS;
            freed.st = f % C::ST, freed.turn = (uint32_t)(f / C::ST) & 1;
        };
        bool raw_ready = false, scales_ready = false, slot_ready = true;
        for (int step = team; step < steps; step += 2) {
            if (!raw_ready && !mbar_wait(raw_bar + ring.st * 8, ring.turn, p.status)) failed = true;
            if (!scales_ready && !failed && !mbar_wait(scales_bar + ring.st * 8, ring.turn, p.status)) failed = true;
            if (!slot_ready && !failed && !mbar_wait(empty + freed.st * 8, freed.turn, p.status)) failed = true;
            failed = __any_sync(0xffffffffu, failed);
            if (failed) break;
            fence_after();
            const uint32_t raw = raw0 + (uint32_t)(ring.st * C::NA * MX_TILE_BYTES), sl = sl0 + (uint32_t)(slot.st * C::SLOT);
            // every warp takes the scales of all activation rows (row 32 j + lane): each quarter of tensor memory's lanes
            // holds a copy
            uint32_t sfb[WB];
#pragma unroll
            for (int j = 0; j < WB; j++) sfb[j] = j < C::NR ? lds32(sb0 + (uint32_t)(ring.st * C::SB_STAGE + j * 128)) : 0u;
            uint4 v[4], sfa[C::NA];
#pragma unroll
            for (int a = 0; a < C::NA; a++) {
                sfa[a] = lds128(raw + a * MX_TILE_BYTES + MX_TILE_CODES - q * 512);
#pragma unroll
                for (int j = 0; j < 4; j++) v[j] = lds128(raw + a * MX_TILE_BYTES + j * 2048);
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    uint32_t c[16];
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        spread8(v[j + h].x, c[8 * h], c[8 * h + 1]);
                        spread8(v[j + h].y, c[8 * h + 2], c[8 * h + 3]);
                        spread8(v[j + h].z, c[8 * h + 4], c[8 * h + 5]);
                        spread8(v[j + h].w, c[8 * h + 6], c[8 * h + 7]);
                    }
                    write_tmem<16>(sl + (uint32_t)(a * 32 + j * 8), c);
                }
                const uint32_t s4[4] = {sfa[a].x, sfa[a].y, sfa[a].z, sfa[a].w};
                write_tmem<4>(sl + (uint32_t)(C::NA * 32 + a * 4), s4);
            }
            // bytes past the row's end belong to columns of zeros, but must not be NaN
            const int left = blocks - k * 4;
            if (left < 4)
#pragma unroll
                for (int j = 0; j < C::NR; j++) sfb[j] &= (1u << (8 * left)) - 1u;
            write_tmem<WB>(sl + (uint32_t)(C::NA * 36), sfb);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(full + slot.st * 8);
            ring.next();
            ring.next();
            slot.next();
            slot.next();
            if (++k == nk) k = 0;
            if (++k == nk) k = 0;
            if (step + 2 < steps) {
                // (this team's stage before that one in the ring is done with: ST is even)
                raw_ready = ready(raw_bar + ring.st * 8, ring.turn);
                scales_ready = ready(scales_bar + ring.st * 8, ring.turn);
                if (step + 2 >= C::NS) {
                    to_freed(step + 2);
                    slot_ready = ready(empty + freed.st * 8, freed.turn);
                }
            }
        }
    } else {
        // ------------------------------------------------------------------ sums, output
        set_registers<C::BIG, true>();
        const int q = warp & 3, half = (warp - 4) >> 2;    // tensor-memory lanes 32 q .., column chunks half, half + 2, ..
        int turn = 0;
        Ring<C::SETS> set;
        for (int i = cluster; i < tiles && !failed; i += clusters, turn++) {
            const Tile t = tile_at<BN>(p, where, i);
            GQ_DCHECK(t.n <= BN && t.r0 >= 0 && t.r0 + t.n <= p.R && t.g * MX_TILE < p.N, p.status);
            const int cols = (t.n + C::CW - 1) / C::CW;    // chunks in use
            float acc[C::NA][C::MINE][C::CW];
#pragma unroll
            for (int a = 0; a < C::NA; a++)
#pragma unroll
                for (int j = 0; j < C::MINE; j++)
#pragma unroll
                    for (int c = 0; c < C::CW; c++) acc[a][j][c] = 0.0f;
            for (int k = 0; k < nk; k += C::FLUSH, set.next()) {
                if (!mbar_wait(bar(ACC_FULL + set.st), set.turn, p.status)) failed = true;
                failed = __any_sync(0xffffffffu, failed);
                if (failed) break;
                fence_after();
#pragma unroll
                for (int a = 0; a < C::NA; a++) {
                    const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(set.st * C::ACC + a * BN + half * C::CW);
                    // two reads of tensor memory under way at a time (where registers allow it)
                    constexpr int X = C::NA * C::MINE * C::CW > 96 ? 1 : 2;
#pragma unroll
                    for (int j = 0; j < C::MINE; j += X) {
                        uint32_t v[X][C::CW];
#pragma unroll
                        for (int x = 0; x < X; x++)
                            if (j + x < C::MINE && 2 * (j + x) + half < cols) read_acc<C::CW>(at + (uint32_t)(2 * (j + x) * C::CW), v[x]);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                        for (int x = 0; x < X; x++)
                            if (j + x < C::MINE && 2 * (j + x) + half < cols)
#pragma unroll
                                for (int c = 0; c < C::CW; c++) acc[a][j + x < C::MINE ? j + x : 0][c] += keep(v[x][c]);
                    }
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(ACC_EMPTY + set.st * C::NA + a));
                }
            }
            if (failed) break;
            if (C::MAX_SPLIT > 1 && split > 1) {
                // the others' sums, column by column, 128 weight rows each
                const int lrow = 32 * q + lane;
                if (rank > 0) {
                    if (turn > 0 && !wait_cluster(bar(PART_EMPTY), (uint32_t)((turn - 1) & 1), p.status)) failed = true;
                    failed = __any_sync(0xffffffffu, failed);
                    if (failed) break;
                    const uint32_t to = map_shared_rank_addr(smem_addr(smem + C::part + (rank - 1) * C::PART_BYTES), 0);
#pragma unroll
                    for (int a = 0; a < C::NA; a++)
#pragma unroll
                        for (int j = 0; j < C::MINE; j++)
                            if (2 * j + half < cols)
#pragma unroll
                                for (int c = 0; c < C::CW; c++) {
                                    const uint32_t at = to + (uint32_t)(((a * BN + (2 * j + half) * C::CW + c) * MX_TILE + lrow) * 4);
                                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(acc[a][j][c]) : "memory");
                                }
                    asm volatile("fence.acq_rel.cluster;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) arrive_remote(map_shared_rank_addr(bar(PART_FULL), 0));
                    continue;
                }
                if (!wait_cluster(bar(PART_FULL), (uint32_t)(turn & 1), p.status)) failed = true;
                failed = __any_sync(0xffffffffu, failed);
                if (failed) break;
                for (int z = 0; z < split - 1; z++) {
                    const float *from = reinterpret_cast<const float *>(smem + C::part + z * C::PART_BYTES);
#pragma unroll
                    for (int a = 0; a < C::NA; a++)
#pragma unroll
                        for (int j = 0; j < C::MINE; j++)
                            if (2 * j + half < cols)
#pragma unroll
                                for (int c = 0; c < C::CW; c++)
                                    acc[a][j][c] += from[(a * BN + (2 * j + half) * C::CW + c) * MX_TILE + lrow];
                }
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    for (int z = 1; z < split; z++) arrive_remote(map_shared_rank_addr(bar(PART_EMPTY), (uint32_t)z));
            }
            const int n = t.g * MX_TILE + 32 * q + lane;
            // Chunk by chunk, the sums moved up by one chunk each time: what the loop's body works on is always chunk 0.
            // (All chunks written out are more code than the instruction caches hold, and every tile fetches it
            // again: 32760 rows of the gated unit and back 537 us in all, so 427.)
            auto next_chunk = [&] {
#pragma unroll
                for (int a = 0; a < C::NA; a++)
#pragma unroll
                    for (int j = 0; j + 1 < C::MINE; j++)
#pragma unroll
                        for (int c = 0; c < C::CW; c++) acc[a][j][c] = acc[a][j + 1][c];
            };
            if constexpr (!GATED) {
                auto store = [&](auto *dst) {
                    const int64_t ldd = p.ldd;
                    dst += (int64_t)(t.r0 + half * C::CW) * ldd + n;
#pragma unroll 1
                    for (int col = half * C::CW; col < t.n; col += 2 * C::CW, dst += C::CW * ldd) {
                        if (n < p.N) {
                            if (col + C::CW <= t.n) {
#pragma unroll
                                for (int c = 0; c < C::CW; c++, dst += ldd) put(dst, acc[0][0][c]);
                            } else {
#pragma unroll
                                for (int c = 0; c < C::CW; c++, dst += ldd)
                                    if (col + c < t.n) put(dst, acc[0][0][c]);
                            }
                        }
                        next_chunk();
                    }
                };
                if (p.bf16)
                    store(static_cast<__nv_bfloat16 *>(p.dst));
                else
                    store(static_cast<float *>(p.dst));
            } else {
                // a warp's 32 lanes are one block of 32 output values of each column's row; N is a
                // multiple of 32, so the block is there as a whole or not at all
                const int block = t.g * 4 + q, last = p.N / QK - 1;
                if (block <= last) {
                    // lane l writes four codes of column l % 4, and lane l < 4 its scale
                    const int64_t first = t.r0 + half * C::CW + (lane & 3);
                    uint8_t *codes = p.codes + first * p.N + block * 32 + (lane & ~3);
                    uint8_t *scales = p.scales + first * p.So + block;
#pragma unroll 1
                    for (int col = half * C::CW; col < t.n; col += 2 * C::CW) {
                        float(&v)[C::CW] = acc[0][0];
                        uint32_t top[C::CW], most = 0;
#pragma unroll
                        for (int c = 0; c < C::CW; c++) v[c] = swish(v[c]) * acc[1][0][c];
#pragma unroll
                        for (int c = 0; c < C::CW; c++) {
                            top[c] = __reduce_max_sync(0xffffffffu, __float_as_uint(v[c]) & 0x7FFFFFFFu);
                            most = max(most, top[c]);
                        }
#pragma unroll
                        for (int c = 0; c < C::CW; c += 4) {
                            // the largest magnitude, rounded up to 7/4 times a power of two where above it: its exponent, less
                            // 8, is the scale byte (mx_scale_byte), and 262 less that of the scale's inverse
                            uint32_t e[4];
#pragma unroll
                            for (int x = 0; x < 4; x++) {
                                e[x] = max((top[c + x] + 0x1FFFFFu) >> 23, 8u);
                                v[c + x] *= __uint_as_float((262u - e[x]) << 23);
                            }
                            uint32_t word = e4m3x2(v[c], v[c + 1]) | e4m3x2(v[c + 2], v[c + 3]) << 16;
                            uint32_t byte = (lane & 2 ? (lane & 1 ? e[3] : e[2]) : (lane & 1 ? e[1] : e[0])) - 8;
                            if (most >= 0x7F800000u) {     // blocks with an infinity or a NaN
#pragma unroll
                                for (int x = 0; x < 4; x++)
                                    if (top[c + x] >= 0x7F800000u) {
                                        word &= ~(0xFFu << (8 * x));
                                        if ((lane & 3) == x) byte = 255;
                                    }
                            }
                            // four lanes turn their 4 x 4 codes: lane l & 3 then has column l & 3's four
                            uint32_t other = __shfl_xor_sync(0xffffffffu, word, 1);
                            word = __byte_perm(word, other, lane & 1 ? 0x3715 : 0x6240);
                            other = __shfl_xor_sync(0xffffffffu, word, 2);
                            word = __byte_perm(word, other, lane & 2 ? 0x3276 : 0x5410);
                            if (col + c + (lane & 3) < t.n) {
                                *reinterpret_cast<uint32_t *>(codes) = word;
                                if (lane < 4) *scales = (uint8_t)byte;
                            }
                            codes += 4 * (int64_t)p.N;
                            scales += 4 * (int64_t)p.So;
                        }
                        codes += C::CW * (int64_t)p.N;
                        scales += C::CW * (int64_t)p.So;
                        next_chunk();
                    }
                }
                // the scales' padding, by the warps of the rows' last block
                if (block == last && last + 1 + lane < p.So)
#pragma unroll 1
                    for (int col = half; col < t.n; col += 2) p.scales[(int64_t)(t.r0 + col) * p.So + last + 1 + lane] = 0;
            }
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (split > 1) cluster_sync();            // no CTA leaves while another may still reach its memory
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::COLS) : "memory");
    }
}

// Rows lo .. hi - 1 of the plan, as far as experts have them, brought into its order: codes and scales, 16 bytes a thread and
// turn.  A row whose index is out of range becomes zeros.  19 us for 32760 rows of 2048; four-row copies by the product's one
// copying thread keep up with tiles of 16 rows only.  What experts have is from the first begin to the largest end of the
// ranges that are in [0, R], as the product sees them (one that overlaps an earlier range it refuses, but such a row does no
// harm here): with offsets that go back at the end, offsets[E] is not the largest.
__global__ void __launch_bounds__(256) gather_rows_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                                          const int32_t *__restrict__ rows, const int32_t *__restrict__ offsets,
                                                          uint8_t *__restrict__ to_codes, uint8_t *__restrict__ to_scales, int lo, int hi,
                                                          int E, int R, int64_t x_rows, int K, int S, unsigned int *status) {
    __shared__ int range[2];                               // R - first begin, largest end
    if (threadIdx.x < 2) range[threadIdx.x] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    int from_end = 0, last = 0;
    for (int e = threadIdx.x; e < E; e += 256) {
        const int r0 = __ldg(offsets + e), r1 = __ldg(offsets + e + 1);
        if (r0 >= 0 && r1 > r0 && r1 <= R) from_end = max(from_end, R - r0), last = max(last, r1);
    }
    from_end = (int)__reduce_max_sync(0xffffffffu, (uint32_t)from_end);
    last = (int)__reduce_max_sync(0xffffffffu, (uint32_t)last);
    if ((threadIdx.x & 31) == 0 && last > 0) atomicMax(&range[0], from_end), atomicMax(&range[1], last);
    __syncthreads();
    const int begin = max(lo, R - range[0]), end = min(hi, range[1]), pieces = K / 16, all = pieces + S / 16;
    // a warp takes rows in turn
    const int lane = threadIdx.x & 31, warps = gridDim.x * 8;
    for (int r = begin + (int)(blockIdx.x * 8 + (threadIdx.x >> 5)); r < end; r += warps) {
        GQ_DCHECK(r >= lo && r < hi, status);
        const int from = __ldg(rows + r);
        const bool there = from >= 0 && from < x_rows;
        if (!there && lane == 0) atomicOr(status, STATUS_RANGE);
        const uint4 *c = reinterpret_cast<const uint4 *>(codes + (int64_t)(there ? from : 0) * K);
        const uint4 *b = reinterpret_cast<const uint4 *>(scales + (int64_t)(there ? from : 0) * S);
        uint4 *tc = reinterpret_cast<uint4 *>(to_codes + (int64_t)(r - lo) * K), *tb = reinterpret_cast<uint4 *>(to_scales + (int64_t)(r - lo) * S);
#pragma unroll 4
        for (int i = lane; i < all; i += 32) {
            const uint4 v = there ? __ldg(i < pieces ? c + i : b + (i - pieces)) : make_uint4(0u, 0u, 0u, 0u);
            *(i < pieces ? tc + i : tb + (i - pieces)) = v;
        }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int64_t GATHER_BYTES = 512LL << 20;   // of rows brought into order at a time

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

// rows of K bytes; boxes of 128 bytes x box_rows rows, 128-byte swizzle, zeros outside
gq_status encode(CUtensorMap *map, const void *base, int64_t rows, int64_t K, int box_rows) {
    std::call_once(g_encode_once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    if (!g_encode) return fail(GQ_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)K};
    const cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1u, 1u};
    const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(GQ_ERR_CUDA, "cuTensorMapEncodeTiled (mx rows) failed (%d)", (int)r);
    return GQ_OK;
}

constexpr int MAX_DEV = 64;

template <int BN, bool GATED>
gq_status launch(MxParams p, const gq_mx_rows &x, int64_t most_tiles, cudaStream_t s) {
    using C = Cfg<BN, GATED>;
    static std::atomic<bool> allowed[MAX_DEV];
    auto kernel = mx_product_kernel<BN, GATED>;
    int dev = 0;
    gq_status st = check_cuda(cudaGetDevice(&dev), "cudaGetDevice");
    if (st != GQ_OK) return st;
    if (dev < 0 || dev >= MAX_DEV || !allowed[dev].load(std::memory_order_acquire)) {
        st = check_cuda(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::total + 1024), "mx shared-memory attribute");
        if (st != GQ_OK) return st;
        if (dev >= 0 && dev < MAX_DEV) allowed[dev].store(true, std::memory_order_release);
    }
    CUtensorMap mx;
    if (p.values) {
        mx = {};                                           // (nothing is copied by it)
    } else {
        st = encode(&mx, x.codes, x.rows, p.K, p.rows ? 1 : C::BOX);
        if (st != GQ_OK) return st;
    }

    // K shared out where the tiles leave SMs idle, two stages a CTA at least ([4096, 4096], a row: 8.5 us by four, 9.1 by
    // two, 9.8 by one)
    const int sms = sm_count();
    int split = 1;
    while (split < C::MAX_SPLIT && most_tiles * 2 * split <= sms && p.KT / (2 * split) >= 2) split *= 2;
    p.split = split;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::total + 1024;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    const int64_t clusters = std::max<int64_t>(1, std::min<int64_t>(most_tiles, sms / split));
    cfg.gridDim = dim3((unsigned)(clusters * split));
    return check_cuda(cudaLaunchKernelEx(&cfg, kernel, mx, p), "mx product launch");
}

// What a product's operands do not decide.
gq_status product_params(MxParams *p, const void *rep, int64_t N, int64_t K, int64_t x_rows) {
    *p = MxParams{};
    p->status = device_status_word();
    if (!p->status) return fail(GQ_ERR_CUDA, "device status word unavailable");
    p->N = (int)N, p->K = (int)K, p->x_rows = x_rows;
    p->G = (int)((N + MX_TILE - 1) / MX_TILE), p->KT = (int)((K + MX_TILE - 1) / MX_TILE);
    p->S = (int)gq_mx_scale_cols(K);
    p->w = static_cast<const uint8_t *>(rep);
    return GQ_OK;
}

}  // namespace

gq_status launch_mx_product_few(const void *rep, const void *values, int64_t ldv, bool values_bf16, void *dst, int64_t ldd, bool bf16,
                                int64_t M, int64_t N, int64_t K, cudaStream_t s) {
    MxParams p;
    const gq_status st = product_params(&p, rep, N, K, M);
    if (st != GQ_OK) return st;
    p.E = 1, p.R = p.hi = (int)M;
    p.values = values, p.ldv = ldv, p.values_bf16 = values_bf16;
    p.dst = dst, p.ldd = ldd, p.bf16 = bf16;
    return launch<16, false>(p, gq_mx_rows{M, nullptr, nullptr}, p.G, s);
}

gq_status launch_mx_product(const void *rep, const gq_mx_rows &x, const gq_expert_rows *plan, void *dst, int64_t ldd,
                            bool bf16, void *codes, uint8_t *scales, int64_t N, int64_t K, cudaStream_t s) {
    MxParams p;
    gq_status st = product_params(&p, rep, N, K, x.rows);
    if (st != GQ_OK) return st;
    const bool gated = codes != nullptr;
    p.E = plan ? (int)plan->E : 1;
    p.R = plan ? (int)plan->R : (int)x.rows;
    p.offsets = plan ? plan->offsets : nullptr;
    p.rows = plan ? plan->rows : nullptr;
    p.bf16 = bf16, p.ldd = ldd, p.So = gated ? (int)gq_mx_scale_cols(N) : 0;
    p.dst = dst, p.codes = static_cast<uint8_t *>(codes), p.scales = scales, p.x_scales = x.scales;
    p.hi = p.R;

    // Rows per tile by the rows that an expert has on average (of the experts that can have any).  Its rows vary about
    // that, so with a plan a tile is taken for means up to seven eighths of it: 32 experts of [2816, 2048], us:
    //   mean    8 rows 24.4; 10: 24.6, by tiles of 64 28.4; 14: 28.8, 28.0 (gated 21.0, 25.9); 16: 33.1, 29.1 (26.0, 26.3)
    //   mean    40: 30.6, by larger tiles 35.9; 48: 31.4, 36.9 (29.0, 30.5); 56: 35.0, 36.9 (29.1, 29.9); 64: 42.4, 37.6 (34.6, 30.6)
    // And tiles of 64 rows where all of them run at once ([4096, 4096]: 65 rows 10.6 us against 12.3, 256 rows 10.8 against 14.9).
    // One row by tiles of 16 8.5 us, of 64 9.9.
    const int64_t some = std::min<int64_t>(p.E, p.R), mean = (p.R + some - 1) / some;
    auto most = [&](int bn) { return ((plan ? some : 0) + (p.R + bn - 1) / bn) * p.G; };
    if (most(16) >= (1LL << 31)) return fail(GQ_ERR_INVALID_ARG, "R=%lld rows of N=%lld are too many", (long long)p.R, (long long)N);
    const bool few = mean <= (plan ? 14 : 16), medium = mean <= (plan ? 56 : 64) || most(64) <= sm_count();
    auto run = [&](const gq_mx_rows &rows) {
        if (gated) {
            if (few) return launch<16, true>(p, rows, most(16), s);
            if (medium) return launch<64, true>(p, rows, most(64), s);
            return launch<128, true>(p, rows, most(128), s);
        }
        if (few) return launch<16, false>(p, rows, most(16), s);
        if (medium) return launch<64, false>(p, rows, most(64), s);
        return launch<176, false>(p, rows, most(176), s);
    };
    if (!p.rows || few) return run(x);
    // the rows in the plan's order, as many at a time as the workspace's share holds; the kernel sees them as rows lo .. of an
    // array that begins lo rows earlier
    const int64_t row_bytes = K + p.S, some_rows = std::min<int64_t>(p.R, std::max<int64_t>(1, GATHER_BYTES / row_bytes));
    Workspace ws;
    st = get_workspace(s, 0, (size_t)(some_rows * row_bytes), &ws);
    if (st != GQ_OK) return st;
    const int32_t *from = p.rows, *offsets = p.offsets;
    uint8_t *codes_to = ws.data, *scales_to = ws.data + some_rows * K;
    p.rows = nullptr;
    for (int64_t lo = 0; lo < p.R; lo += some_rows) {
        int l = (int)lo, h = (int)std::min<int64_t>(p.R, lo + some_rows), E = p.E, R = p.R, k = (int)K, S = p.S;
        int64_t x_rows = x.rows;
        const void *xc = x.codes;
        const uint8_t *xs = x.scales;
        unsigned int *status = p.status;
        void *args[] = {&xc, &xs, &from, &offsets, &codes_to, &scales_to, &l, &h, &E, &R, &x_rows, &k, &S, &status};
        st = launch_pdl((const void *)gather_rows_kernel, dim3((unsigned)std::min<int64_t>((h - l + 7) / 8, 8LL * sm_count())), dim3(256), 0, s,
                        args, "gather rows launch");
        if (st != GQ_OK) return st;
        p.lo = l, p.hi = h, p.base = l;
        p.x_scales = scales_to;
        p.x_rows = h - l;
        st = run(gq_mx_rows{h - l, codes_to, scales_to});
        if (st != GQ_OK) return st;
    }
    return GQ_OK;
}

}  // namespace gq

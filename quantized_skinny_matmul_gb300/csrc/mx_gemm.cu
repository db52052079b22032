// mx_gemm.cu -- products of e4m3 blocks with 4-bit (e2m1) block weights on tcgen05, for one matrix
// or for the matrices of many experts, and the gated unit silu(gate) * up with its output in blocks.
//
// dst^T = W . X^T: a tile is 128 weight rows (the MMA's M, tensor-memory lanes) by up to BN rows of
// activations (its N, tensor-memory columns; an MMA is as wide as its tile's rows need, in steps of
// 16).  kind::mxf8f6f4 multiplies the codes and each block of 32 by its two powers of two.  What bounds a
// full tile is shared memory's 128 bytes a cycle, so the weights go through it once, packed, and reach the
// MMAs in tensor memory:
//   warp 0     one thread copies, some stages of 128 columns ahead: the weights' tile (packed codes, scales) by a
//              bulk copy, the activations' codes by a tensor copy;
//   warps 2, 3     instead of the latter, where a plan names the rows: 16-byte asynchronous copies;
//   warps 12 .. 15  a weight row per thread: 64 bytes of packed codes become 128 bytes, a code in bits 2 .. 5 of
//              each (the form of 4-bit operands in tensor memory), and go there, and so do the scales of both
//              operands.  The tiles hold the codes so that three instructions place eight of them;
//   warp 1     one thread issues 4 MMAs a stage (8 for the gated unit, whose gate and up tiles share the
//              activations).  The thread is elected, not picked by its lane: the compiler then keeps the
//              descriptors in uniform registers (measured: 39 cycles per MMA of 16 columns, not 80);
//   warps 4 .. 11  take the sums over: the tensor cores' accumulators cut off what does not fit 24 bits, so
//              every few stages they are added, rounded, to f32 registers, while the next stages go
//              to another set of accumulators; then they store the tile.
// CTAs take tiles in turn (persistent), those of one expert's weight rows next to each other.  With few
// tiles a cluster of 2 or 4 CTAs shares a tile's columns; the first adds the others' sums in order.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>

#include "mx.cuh"

namespace gq {
namespace {

constexpr int THREADS = 512;
constexpr int EPI_WARPS = 8;
constexpr int SPREAD_WARPS = 4;              // 32 weight rows each
constexpr int GATHER_WARPS = 2;
constexpr int MAX_E = 1024;
constexpr int MAX_STAGES = 16, MAX_SLOTS = 8, MAX_SETS = 4;
constexpr int FEW_REGS = 88, MANY_REGS = 168;   // per thread, of 128 at launch: 2 x 88 + 2 x 168 = 4 x 128

// BN: rows of activations per tile.  GATED: two weight tiles (gate, up) per stage.
template <int BN, bool GATED>
struct Cfg {
    static constexpr int NA = GATED ? 2 : 1;
    static constexpr bool BIG = BN > 64;                    // more sums per thread than an even share of registers holds
    static constexpr int ST = BN <= 16 ? (GATED ? 8 : 16) : BN <= 64 ? (GATED ? 7 : 10) : 6;   // stages in shared memory
    static constexpr int PARTS = BN > 64 ? 2 : 1;           // tensor copies of a tile's activations, BN / PARTS rows each
    static constexpr int BOX = BN / PARTS;
    static constexpr int CW = BN <= 16 ? 8 : 16;            // columns per read of tensor memory
    static constexpr int CHUNKS = BN / CW;
    static constexpr int MINE = (CHUNKS + 1) / 2;           // chunks of a warpgroup
    static constexpr int MAX_SPLIT = BN <= 16 ? 4 : 1;
    // Tensor memory: sets of accumulators, then slots of a stage's weights and scales.  The gated unit's large
    // tile has one set only; its accumulators are taken over every 16 stages (2048 columns; what is cut
    // off meanwhile, 2^-24 of the sums 64 times at most, is far below its output's 2^-4), gate before up, so
    // that the next gate MMAs wait for half of it.
    static constexpr int ACC = NA * BN;
    static constexpr int SETS = GATED ? (BN <= 16 ? 4 : BN <= 64 ? 2 : 1) : (BN <= 64 ? 4 : 2);
    static constexpr int FLUSH = SETS == 1 ? 16 : 4;        // stages per take-over of the accumulators
    static constexpr int NR = (BN + 31) / 32;               // scales of activation rows: columns, words of a lane
    static constexpr int SFB = NR <= 1 ? 4 : NR <= 4 ? 4 : 8;
    static constexpr int SLOT = NA * 36 + SFB;              // 32 columns of codes and 4 of scales per weight tile
    static constexpr int NS = BN <= 16 ? (GATED ? 4 : 8) : BN <= 64 ? (GATED ? 3 : 6) : 3;
    static constexpr int SLOTS = SETS * ACC;                // their first column
    static constexpr int COLS_USED = SLOTS + NS * SLOT;
    static constexpr int COLS = COLS_USED <= 256 ? 256 : 512;
    static_assert(COLS_USED <= 512, "tensor memory");
    static_assert(BOX % 8 == 0 && BN % 16 == 0, "tile rows");
    static_assert(NS < ST && NS <= MAX_SLOTS && ST <= MAX_STAGES && SETS <= MAX_SETS, "barriers");
    // shared memory from a 1024-aligned base
    static constexpr int B_STAGE = BN * 128;
    static constexpr int b = 0;
    static constexpr int w = b + ST * B_STAGE;
    static constexpr int part = w + ST * NA * MX_TILE_BYTES;
    static constexpr int PART_BYTES = NA * BN * MX_TILE * 4;
    static constexpr int starts = part + (MAX_SPLIT - 1) * PART_BYTES;
    static constexpr int bars = starts + 3 * (MAX_E + 4) * 4;
    static constexpr int total = bars + 640;
    static_assert(total + 1024 <= 227 * 1024, "shared memory");
};

enum : int {
    RAW = 0,                     // a stage's copies have landed
    GATHERED = RAW + MAX_STAGES, // and so have its gathered rows
    EMPTY = GATHERED + MAX_STAGES,   // its MMAs are done
    FULL = EMPTY + MAX_STAGES,   // a slot's weights and scales are in tensor memory
    ACC_FULL = FULL + MAX_SLOTS,
    ACC_EMPTY = ACC_FULL + MAX_SETS,         // gate and up apart
    PART_FULL = ACC_EMPTY + 2 * MAX_SETS,
    PART_EMPTY,
    NUM_BARS
};
static_assert(NUM_BARS * 8 + 8 <= 640, "barrier area");

struct MxParams {
    const uint8_t *w;              // tiles
    const uint8_t *x_scales;
    const int32_t *offsets, *rows;
    void *dst;
    uint8_t *codes, *scales;       // gated: the output's
    unsigned int *status;
    const uint8_t *x_codes;        // for gathered rows
    int64_t ldd, x_rows;
    int N, K, KT, G, S, So;        // S, So: scale bytes per row of x and of the gated output
    int E, R, split, bf16;
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
// one lane of the warp
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// 16 bytes, zeros unless `there`
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
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

// x / (1 + exp(-x)); the exponential and the reciprocal are the fast ones, off by a few units of f32.
__device__ __forceinline__ float swish(float x) {
    float e, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return x * r;
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
            mbar_init(bar(GATHERED + i), GATHER_WARPS);
            mbar_init(bar(EMPTY + i), 1);
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
        // tiles of BN rows in front of each expert
        int before = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int tiles = 0;
            if (e < p.E) {
                const int r0 = p.offsets ? p.offsets[e] : 0, r1 = p.offsets ? p.offsets[e + 1] : p.R;
                where.first[e] = r0;
                where.last[e] = r1;
                if (r0 < 0 || r1 < r0 || r1 > p.R) {
                    atomicOr(p.status, STATUS_RANGE);
                } else {
                    tiles = (r1 - r0 + BN - 1) / BN;
                }
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
                const uint8_t *w = p.w + (((int64_t)t.e * C::NA * p.G + t.g) * p.KT + kt0) * MX_TILE_BYTES;
                const int64_t up = (int64_t)p.G * p.KT * MX_TILE_BYTES;    // from the gate's tile to the up matrix's
                const int parts = p.rows ? 0 : t.n > C::BOX ? C::PARTS : 1;
                const uint32_t bytes = (uint32_t)(C::NA * MX_TILE_BYTES + parts * C::BOX * 128);
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
#pragma unroll
                    for (int u = 0; u < C::PARTS; u++)
                        if (u < parts)
                            copy_2d(smem_addr(smem + C::b) + (uint32_t)(ring.st * C::B_STAGE + u * C::BOX * 128), &map_x, (kt0 + k) * MX_TILE,
                                    t.r0 + u * C::BOX, raw);
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
            for (int i = cluster; i < tiles && !failed; i += clusters) {
                const Tile t = tile_at<BN>(p, where, i);
                uint32_t idesc[4];                         // of the scale bytes' four places
#pragma unroll
                for (int kk = 0; kk < 4; kk++) idesc[kk] = mx_idesc((t.n + 15) & ~15) + (uint32_t)kk * ((1u << 4) | (1u << 29));
                int in_chunk = 0;
                for (int k = 0; k < nk; k++) {
                    // (whoever arrived there had waited for the stage's copies)
                    if (!mbar_wait(full + slot.st * 8, slot.turn, p.status)) failed = true;
                    if (p.rows && !failed && !mbar_wait(bar(GATHERED + ring.st), ring.turn, p.status)) failed = true;
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
        // ------------------------------------------------------------------ gathered rows
        set_registers<C::BIG, false>();
        if (p.rows) {
            // Thread x copies 16 bytes, piece x % 8, of the tile's rows x / 8, x / 8 + 8, ..; two stages are under
            // way before the first is waited for.
            constexpr int ROWS = BN / 8, AHEAD = 2;
            const int x = (warp - 2) * 32 + lane;
            int from[ROWS], filled = 0;
            Ring<C::ST> ring, done;
            int under_way = 0;
            auto finish = [&] {
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(GATHERED + done.st));
                done.next();
                under_way--;
            };
            for (int i = cluster; i < tiles && !failed; i += clusters) {
                const Tile t = tile_at<BN>(p, where, i);
#pragma unroll
                for (int j = 0; j < ROWS; j++) {
                    const int c = j * 8 + (x >> 3);
                    const int r = c < t.n ? __ldg(p.rows + t.r0 + c) : -1;
                    from[j] = r >= 0 && r < p.x_rows ? r : -1;
                }
                for (int k = 0; k < nk; k++, ring.next()) {
                    if (filled == C::ST) {
                        if (!mbar_wait(bar(EMPTY + ring.st), ring.turn ^ 1, p.status)) failed = true;
                        failed = __any_sync(0xffffffffu, failed);
                        if (failed) break;
                    } else {
                        filled++;
                    }
                    const int col = (kt0 + k) * MX_TILE + (x & 7) * 16;
                    const uint32_t to = smem_addr(smem + C::b) + (uint32_t)(ring.st * C::B_STAGE + (x >> 3) * 128 + (((x & 7) ^ (x >> 3)) << 4));
#pragma unroll
                    for (int j = 0; j < ROWS; j++)
                        if (j * 8 < t.n) {
                            const bool there = from[j] >= 0 && col < p.K;
                            copy16(to + j * 1024, p.x_codes + (there ? (int64_t)from[j] * p.K + col : 0), there);
                        }
                    copy_group();
                    if (++under_way > AHEAD) {
                        copy_wait<AHEAD>();
                        finish();
                    }
                }
            }
            if (!failed) {
                copy_wait<0>();
                while (under_way > 0) finish();
            }
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------------ weights and scales into tensor memory
        set_registers<C::BIG, false>();
        const int q = warp - 12;                           // tensor-memory lanes, weight rows 32 q ..
        // The scales of activation row 32 j + lane of the tile, loaded a stage ahead (rows that are not there: those of
        // row 0, put out by a mask).  Every warp brings all of them: each quarter of the lanes holds a copy.
        const uint32_t *from[C::NR];
        uint32_t next[C::NR], there = 0, there_now;
        constexpr int WB = C::NR == 3 ? 4 : C::NR > 4 ? 8 : C::NR;
        auto rows_of = [&](int i) {
            const Tile t = tile_at<BN>(p, where, i);
            there = 0;
#pragma unroll
            for (int j = 0; j < C::NR; j++) {
                const int c = j * 32 + lane;
                int r = -1;
                if (c < t.n) {
                    r = p.rows ? __ldg(p.rows + t.r0 + c) : t.r0 + c;
                    if (r < 0 || r >= p.x_rows) atomicOr(p.status, STATUS_RANGE), r = -1;
                }
                there |= (r >= 0 ? 1u : 0u) << j;
                from[j] = reinterpret_cast<const uint32_t *>(p.x_scales + (r >= 0 ? (int64_t)r * p.S : 0)) + kt0;
            }
        };
        auto load = [&] {
#pragma unroll
            for (int j = 0; j < C::NR; j++) next[j] = __ldg(from[j]++);
        };
        if (cluster < tiles) {
            rows_of(cluster);
            load();
        }
        Ring<C::ST> ring, freed;                           // this stage; the one whose MMAs read the slot last
        Ring<C::NS> slot;
        const uint32_t raw0 = smem_addr(smem + C::w), raw_bar = bar(RAW), empty = bar(EMPTY), full = bar(FULL);
        const uint32_t sl0 = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)C::SLOTS;
        const int blocks = p.K / QK - kt0 * 4;             // scale bytes of this CTA's columns
        int filled = 0;
        for (int i = cluster; i < tiles && !failed; i += clusters) {
            for (int k = 0; k < nk; k++) {
                uint32_t sfb[WB];
                there_now = there;
#pragma unroll
                for (int j = 0; j < WB; j++) sfb[j] = j < C::NR ? next[j < C::NR ? j : 0] : 0u;
                if (k + 1 < nk) {
                    load();
                } else if (i + clusters < tiles) {
                    rows_of(i + clusters);
                    load();
                }
                if (!mbar_wait(raw_bar + ring.st * 8, ring.turn, p.status)) failed = true;
                const uint32_t raw = raw0 + (uint32_t)(ring.st * C::NA * MX_TILE_BYTES);
                uint4 v[C::NA][4], sfa[C::NA];
#pragma unroll
                for (int a = 0; a < C::NA; a++) {
#pragma unroll
                    for (int j = 0; j < 4; j++) v[a][j] = lds128(raw + a * MX_TILE_BYTES + j * 2048 + (q * 32 + lane) * 16);
                    sfa[a] = lds128(raw + a * MX_TILE_BYTES + MX_TILE_CODES + lane * 16);
                }
                if (filled == C::NS) {
                    if (!failed && !mbar_wait(empty + freed.st * 8, freed.turn, p.status)) failed = true;
                    freed.next();
                } else {
                    filled++;
                }
                failed = __any_sync(0xffffffffu, failed);
                if (failed) break;
                fence_after();
                // bytes past the row's end belong to columns of zeros, but must not be NaN
                const int left = blocks - k * 4;
                const uint32_t mask = left >= 4 ? 0xffffffffu : (1u << (8 * left)) - 1u;
#pragma unroll
                for (int j = 0; j < C::NR; j++) sfb[j] &= there_now >> j & 1u ? mask : 0u;
                const uint32_t sl = sl0 + (uint32_t)(slot.st * C::SLOT);
#pragma unroll
                for (int a = 0; a < C::NA; a++) {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        uint32_t c[8];
                        spread8(v[a][j].x, c[0], c[1]);
                        spread8(v[a][j].y, c[2], c[3]);
                        spread8(v[a][j].z, c[4], c[5]);
                        spread8(v[a][j].w, c[6], c[7]);
                        write_tmem<8>(sl + (uint32_t)(a * 32 + j * 8), c);
                    }
                    const uint32_t s4[4] = {sfa[a].x, sfa[a].y, sfa[a].z, sfa[a].w};
                    write_tmem<4>(sl + (uint32_t)(C::NA * 32 + a * 4), s4);
                }
                write_tmem<WB>(sl + (uint32_t)(C::NA * 36), sfb);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + slot.st * 8);
                ring.next();
                slot.next();
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------------ sums, output
        set_registers<C::BIG, true>();
        const int q = warp & 3, half = (warp - 4) >> 2;    // tensor-memory lanes 32 q .., column chunks half, half + 2, ..
        int turn = 0;
        Ring<C::SETS> set;
        for (int i = cluster; i < tiles && !failed; i += clusters, turn++) {
            const Tile t = tile_at<BN>(p, where, i);
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
                    // two reads of tensor memory under way at a time
#pragma unroll
                    for (int j = 0; j < C::MINE; j += 2) {
                        uint32_t v[2][C::CW];
#pragma unroll
                        for (int x = 0; x < 2; x++)
                            if (j + x < C::MINE && 2 * (j + x) + half < cols) read_acc<C::CW>(at + (uint32_t)(2 * (j + x) * C::CW), v[x]);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                        for (int x = 0; x < 2; x++)
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
            if constexpr (!GATED) {
                if (n < p.N)
#pragma unroll
                    for (int j = 0; j < C::MINE; j++)
#pragma unroll
                        for (int c = 0; c < C::CW; c++) {
                            const int col = (2 * j + half) * C::CW + c;
                            if (col < t.n) {
                                const int64_t at = (int64_t)(t.r0 + col) * p.ldd + n;
                                if (p.bf16)
                                    static_cast<__nv_bfloat16 *>(p.dst)[at] = __float2bfloat16_rn(acc[0][j][c]);
                                else
                                    static_cast<float *>(p.dst)[at] = acc[0][j][c];
                            }
                        }
            } else {
                // a warp's 32 lanes are one block of 32 output values of each column's row; N is a
                // multiple of 32, so the block is there as a whole or not at all
                if (t.g * MX_TILE + 32 * q < p.N) {
                    uint8_t *const codes = p.codes + (int64_t)t.r0 * p.N + t.g * MX_TILE + 32 * q + (lane & ~3);
                    uint8_t *const scales = p.scales + (int64_t)t.r0 * p.So + t.g * 4 + q;
#pragma unroll
                    for (int j = 0; j < C::MINE; j++)
#pragma unroll
                        for (int c = 0; c < C::CW; c += 4) {
                            const int col = (2 * j + half) * C::CW + c;
                            if (col >= t.n) continue;
                            uint32_t word = 0;             // this lane's code in each of four columns
                            uint32_t bytes = 0;            // their scales
#pragma unroll
                            for (int x = 0; x < 4; x++) {
                                const float v = swish(acc[0][j][c + x]) * acc[1][j][c + x];
                                const int b = mx_scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu), false);
                                const float inv = mx_inverse(b);
                                word |= (inv == 0.0f ? 0u : e4m3x2(v * inv, 0.0f)) << (8 * x);
                                bytes |= (uint32_t)b << (8 * x);
                            }
                            // four lanes turn their 4 x 4 codes: lane l & 3 then has column l & 3's four
                            uint32_t other = __shfl_xor_sync(0xffffffffu, word, 1);
                            word = lane & 1 ? __byte_perm(other, word, 0x7351) : __byte_perm(word, other, 0x6240);
                            other = __shfl_xor_sync(0xffffffffu, word, 2);
                            word = lane & 2 ? __byte_perm(other, word, 0x7632) : __byte_perm(word, other, 0x5410);
                            const int mine = col + (lane & 3);
                            if (mine < t.n) {
                                *reinterpret_cast<uint32_t *>(codes + (int64_t)mine * p.N) = word;
                                if (lane < 4) scales[(int64_t)mine * p.So] = (uint8_t)(bytes >> (8 * lane));
                            }
                        }
                }
                // the scales' padding, by the warp of the row's last block
                const int last = p.N / QK - 1;
                if (t.g * 4 + q == last)
#pragma unroll
                    for (int j = 0; j < C::MINE; j++)
#pragma unroll
                        for (int c = 0; c < C::CW; c++) {
                            const int col = (2 * j + half) * C::CW + c;
                            if (col < t.n && last + 1 + lane < p.So) p.scales[(int64_t)(t.r0 + col) * p.So + last + 1 + lane] = 0;
                        }
            }
        }
    } else {
        set_registers<C::BIG, false>();
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

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
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
    st = encode(&mx, x.codes, x.rows, p.K, C::BOX);
    if (st != GQ_OK) return st;

    // K shared out where the tiles leave SMs idle, two stages a CTA at least
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

}  // namespace

gq_status launch_mx_product(const void *rep, const gq_mx_rows &x, const gq_expert_rows *plan, void *dst, int64_t ldd,
                            bool bf16, void *codes, uint8_t *scales, int64_t N, int64_t K, cudaStream_t s) {
    MxParams p{};
    p.status = device_status_word();
    if (!p.status) return fail(GQ_ERR_CUDA, "device status word unavailable");
    const bool gated = codes != nullptr;
    p.E = plan ? (int)plan->E : 1;
    p.R = plan ? (int)plan->R : (int)x.rows;
    p.offsets = plan ? plan->offsets : nullptr;
    p.rows = plan ? plan->rows : nullptr;
    p.N = (int)N, p.K = (int)K, p.bf16 = bf16, p.ldd = ldd, p.x_rows = x.rows;
    p.G = (int)((N + MX_TILE - 1) / MX_TILE), p.KT = (int)((K + MX_TILE - 1) / MX_TILE);
    p.S = (int)gq_mx_scale_cols(K), p.So = gated ? (int)gq_mx_scale_cols(N) : 0;
    p.dst = dst, p.codes = static_cast<uint8_t *>(codes), p.scales = scales, p.x_scales = x.scales;
    p.w = static_cast<const uint8_t *>(rep);
    p.x_codes = static_cast<const uint8_t *>(x.codes);

    // Rows per tile by the rows that an expert has on average (of the experts that can have any).
    const int64_t some = std::min<int64_t>(p.E, p.R), mean = (p.R + some - 1) / some;
    auto most = [&](int bn) { return ((plan ? some : 0) + (p.R + bn - 1) / bn) * p.G; };
    if (most(16) >= (1LL << 31)) return fail(GQ_ERR_INVALID_ARG, "R=%lld rows of N=%lld are too many", (long long)p.R, (long long)N);
    if (gated) {
        if (mean <= 16) return launch<16, true>(p, x, most(16), s);
        if (mean <= 64) return launch<64, true>(p, x, most(64), s);
        return launch<128, true>(p, x, most(128), s);
    }
    if (mean <= 16) return launch<16, false>(p, x, most(16), s);
    if (mean <= 64) return launch<64, false>(p, x, most(64), s);
    return launch<176, false>(p, x, most(176), s);
}

}  // namespace gq

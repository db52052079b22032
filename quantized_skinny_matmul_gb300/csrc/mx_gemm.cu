// mx_gemm.cu -- products of e4m3 blocks with 4-bit (e2m1) block weights on tcgen05, for one matrix
// or for the matrices of many experts, and the gated unit silu(gate) * up with its output in blocks.
//
// dst^T = W . X^T: a tile is 128 weight rows (the MMA's M, tensor-memory lanes) by up to BN rows of
// activations (its N, tensor-memory columns; an MMA is as wide as its tile's rows need, in steps of
// 16).  kind::mxf8f6f4 multiplies the codes as they are and each block of 32 by its two powers of
// two, so nothing is converted on the way:
//   warp 0     copies: the weights' tile by a tensor copy that spreads 16 packed 4-bit codes over 16
//              bytes (the form in which this kind reads them), its scales by a bulk copy, the
//              activations' codes by tensor copies of whole rows (gathered four rows at a time where a
//              plan names them);
//   warp 1     issues: per stage of 128 columns, copies of the scales into tensor memory and 4 MMAs
//              (8 for the gated unit, whose gate and up tiles share the activations);
//   warps 2, 3 bring the activations' scale bytes into the order that tensor memory wants;
//   warps 4 .. 11  take the sums over: the tensor cores' accumulators cut off what does not fit 24 bits, so
//              every 4 stages (512 columns) they are added, rounded, to f32 registers, while the
//              next stages go to the other half of the accumulators; then they store the tile.
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

constexpr int THREADS = 384;
constexpr int EPI_WARPS = 8;
constexpr int FLUSH = 4;                     // stages per take-over of the accumulators
constexpr int A_BYTES = MX_TILE * MX_TILE;   // a weight tile in shared memory: one byte's room per code
constexpr int MAX_E = 1024;
constexpr int MAX_STAGES = 8;

// BN: rows of activations per tile.  GATED: two weight tiles (gate, up) per stage.
template <int BN, bool GATED>
struct Cfg {
    static constexpr int NA = GATED ? 2 : 1;
    static constexpr int NB = (BN + 127) / 128;             // 512-byte pieces of activation scales
    static constexpr int ST = GATED ? 4 : BN <= 16 ? 6 : BN <= 64 ? 8 : 5;
    static constexpr int BOX = BN <= 16 ? 16 : 32;          // activation rows per tensor copy
    static constexpr int CW = BN <= 16 ? 8 : 16;            // columns per read of tensor memory
    static constexpr int CHUNKS = BN / CW;
    static constexpr int MINE = (CHUNKS + 1) / 2;           // chunks of a warpgroup
    static constexpr int MAX_SPLIT = BN <= 16 ? 4 : 1;
    // tensor memory: two sets of accumulators, then the scales of every stage
    static constexpr int ACC = NA * BN;
    static constexpr int SF = 2 * ACC;
    static constexpr int SF_STAGE = 4 * (NA + NB);
    static constexpr int COLS_USED = SF + ST * SF_STAGE;
    static constexpr int COLS = COLS_USED <= 128 ? 128 : COLS_USED <= 256 ? 256 : 512;
    static_assert(COLS_USED <= 512, "tensor memory");
    // shared memory from a 1024-aligned base
    static constexpr int B_STAGE = (BN + BOX - 1) / BOX * BOX * 128;
    static constexpr int a = 0;
    static constexpr int b = a + ST * NA * A_BYTES;
    static constexpr int sfa = b + ST * B_STAGE;
    static constexpr int sfb = sfa + ST * NA * MX_TILE_SCALES;
    static constexpr int part = sfb + ST * NB * 512;
    static constexpr int PART_BYTES = NA * BN * MX_TILE * 4;
    static constexpr int starts = part + (MAX_SPLIT - 1) * PART_BYTES;
    static constexpr int bars = starts + (MAX_E + 4) * 4;
    static constexpr int total = bars + 256;
    static_assert(total + 1024 <= 227 * 1024, "shared memory");
    static_assert(ST <= MAX_STAGES, "barriers");
};

enum : int {
    FULL = 0,
    EMPTY = FULL + MAX_STAGES,
    ACC_FULL = EMPTY + MAX_STAGES,
    ACC_EMPTY = ACC_FULL + 2,
    PART_FULL = ACC_EMPTY + 2,
    PART_EMPTY,
    NUM_BARS
};
static_assert(NUM_BARS * 8 + 8 <= 256, "barrier area");

struct MxParams {
    const uint8_t *w_scales;       // of all tiles
    const uint8_t *x_scales;
    const int32_t *offsets, *rows;
    void *dst;
    uint8_t *codes, *scales;       // gated: the output's
    unsigned int *status;
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
// 32 rows of 16 bytes, 8-row groups 128 bytes apart, no swizzle
__device__ __forceinline__ uint64_t scales_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}
// kind::mxf8f6f4: A e2m1 (5), B e4m3 (0), both K-major, scales ue8m0, f32 sums; scale byte `sf` of both
__device__ __forceinline__ uint32_t mx_idesc(int n, int sf) {
    return (uint32_t)sf << 4 | 5u << 7 | (uint32_t)(n >> 3) << 17 | 1u << 23 | (uint32_t)(MX_TILE >> 4) << 24 | (uint32_t)sf << 29;
}
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
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
template <int W>
__device__ __forceinline__ void read_acc(uint32_t taddr, float (&v)[W]) {
    uint32_t r[W];
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
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < W; i++) v[i] = __uint_as_float(r[i]);
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

// Tile `i` of the launch: expert e, weight rows 128 g .., activation rows r0 .. r0 + n - 1.
struct Tile {
    int e, g, r0, n;
};
template <int BN>
__device__ __forceinline__ Tile tile_at(const MxParams &p, const int32_t *starts, int i) {
    int lo = 0, hi = p.E;                                  // starts[e] * G <= i < starts[e + 1] * G
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] * p.G <= i)
            lo = mid;
        else
            hi = mid;
    }
    const int nt = starts[lo + 1] - starts[lo], local = i - starts[lo] * p.G;
    Tile t;
    t.e = lo;
    t.g = local / nt;
    const int k = local - t.g * nt, r0 = p.offsets ? p.offsets[lo] : 0, r1 = p.offsets ? p.offsets[lo + 1] : p.R;
    t.r0 = r0 + k * BN;
    t.n = min(BN, r1 - t.r0);
    return t;
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int BN, bool GATED>
__global__ void __launch_bounds__(THREADS, 1)
    mx_product_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const MxParams p) {
    using C = Cfg<BN, GATED>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::bars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + NUM_BARS);
    int32_t *starts = reinterpret_cast<int32_t *>(smem + C::starts);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = p.split, rank = (int)blockIdx.x % split, cluster = (int)blockIdx.x / split, clusters = (int)gridDim.x / split;
    auto bar = [&](int i) { return smem_addr(bars + i); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::ST; i++) {
            mbar_init(bar(FULL + i), 1 + (C::NB > 1 ? 2 : 1));
            mbar_init(bar(EMPTY + i), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(bar(ACC_FULL + i), 1);
            mbar_init(bar(ACC_EMPTY + i), EPI_WARPS);
        }
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
            if (e < p.E) starts[e] = before + s - tiles;
            before += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) starts[p.E] = before;
    }
    fence_before();
    __syncthreads();
    if (split > 1) cluster_sync();            // every CTA's barriers are there before others arrive on them
    fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tiles = starts[p.E] * p.G;
    const int kt0 = (int)((int64_t)p.KT * rank / split), nk = (int)((int64_t)p.KT * (rank + 1) / split) - kt0;
    bool failed = false;

    if (warp == 0) {
        // ------------------------------------------------------------------ copies
        int step = 0;
        for (int i = cluster; i < tiles && !failed; i += clusters) {
            const Tile t = tile_at<BN>(p, starts, i);
            const int boxes = (t.n + C::BOX - 1) / C::BOX, quads = (t.n + 3) / 4;
            int4 idx[C::NB];
            if (p.rows) {
#pragma unroll
                for (int u = 0; u < C::NB; u++) {
                    int r[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int c = (u * 32 + lane) * 4 + j;
                        r[j] = c < t.n ? p.rows[t.r0 + c] : (int)p.x_rows;
                        if (r[j] < 0 || r[j] > p.x_rows || (r[j] == p.x_rows && c < t.n)) {
                            atomicOr(p.status, STATUS_RANGE);
                            r[j] = (int)p.x_rows;                 // past the end: zeros
                        }
                    }
                    idx[u] = make_int4(r[0], r[1], r[2], r[3]);
                }
            }
            // (the weights' copy counts the bytes that it reads, not the room that it fills)
            const uint32_t bytes = (uint32_t)(C::NA * (MX_TILE_CODES + MX_TILE_SCALES) + (p.rows ? quads * 512 : boxes * C::BOX * 128));
            for (int k = 0; k < nk; k++, step++) {
                const int st = step % C::ST, kt = kt0 + k;
                if (step >= C::ST && !mbar_wait(bar(EMPTY + st), (uint32_t)((step / C::ST - 1) & 1), p.status)) failed = true;
                if (__any_sync(0xffffffffu, failed)) {
                    failed = true;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(FULL + st), bytes);
#pragma unroll
                    for (int a = 0; a < C::NA; a++) {
                        const int64_t tile = ((int64_t)(t.e * C::NA + a) * p.G + t.g) * p.KT + kt;
                        copy_2d(smem_addr(smem + C::a + (st * C::NA + a) * A_BYTES), &map_w, 0, (int)(tile * MX_TILE), bar(FULL + st));
                        bulk_g2s(smem_addr(smem + C::sfa + (st * C::NA + a) * MX_TILE_SCALES), p.w_scales + tile * MX_TILE_SCALES,
                                 MX_TILE_SCALES, bar(FULL + st));
                    }
                    if (!p.rows)
                        for (int u = 0; u < boxes; u++)
                            copy_2d(smem_addr(smem + C::b + st * C::B_STAGE + u * C::BOX * 128), &map_x, kt * MX_TILE, t.r0 + u * C::BOX,
                                    bar(FULL + st));
                }
                __syncwarp();
                if (p.rows) {
#pragma unroll
                    for (int u = 0; u < C::NB; u++)
                        if (u * 32 + lane < quads)
                            copy_rows4(smem_addr(smem + C::b + st * C::B_STAGE + (u * 32 + lane) * 512), &map_x, kt * MX_TILE, idx[u],
                                       bar(FULL + st));
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMAs
        int step = 0, chunk = 0;
        for (int i = cluster; i < tiles && !failed; i += clusters) {
            const Tile t = tile_at<BN>(p, starts, i);
            const int n = (t.n + 15) & ~15;
            for (int k = 0; k < nk; k++, step++) {
                const int st = step % C::ST, set = chunk & 1;
                if (k % FLUSH == 0 && chunk >= 2 && !mbar_wait(bar(ACC_EMPTY + set), (uint32_t)((chunk / 2 - 1) & 1), p.status))
                    failed = true;
                if (!failed && !mbar_wait(bar(FULL + st), (uint32_t)((step / C::ST) & 1), p.status)) failed = true;
                if (__any_sync(0xffffffffu, failed)) {
                    failed = true;
                    break;
                }
                fence_after();
                if (lane == 0) {
                    const uint32_t acc = tmem + (uint32_t)(set * C::ACC), sf = tmem + (uint32_t)(C::SF + st * C::SF_STAGE);
#pragma unroll
                    for (int a = 0; a < C::NA; a++)
                        copy_scales(sf + 4 * a, scales_desc(smem_addr(smem + C::sfa + (st * C::NA + a) * MX_TILE_SCALES)));
#pragma unroll
                    for (int u = 0; u < C::NB; u++)
                        if (u * 128 < n)
                            copy_scales(sf + 4 * (C::NA + u), scales_desc(smem_addr(smem + C::sfb + (st * C::NB + u) * 512)));
                    const uint64_t bd = operand_desc(smem_addr(smem + C::b + st * C::B_STAGE));
#pragma unroll
                    for (int a = 0; a < C::NA; a++) {
                        const uint64_t ad = operand_desc(smem_addr(smem + C::a + (st * C::NA + a) * A_BYTES));
#pragma unroll
                        for (int kk = 0; kk < 4; kk++)     // 32 columns: 32 bytes further in both operands
                            mma_mx(acc + a * BN, ad + (uint64_t)(kk * 2), bd + (uint64_t)(kk * 2), mx_idesc(n, kk), sf + 4 * a,
                                   sf + 4 * C::NA, k % FLUSH != 0 || kk > 0);
                    }
                    commit(bar(EMPTY + st));
                    if (k % FLUSH == FLUSH - 1 || k == nk - 1) commit(bar(ACC_FULL + set));
                }
                __syncwarp();
                if (k % FLUSH == FLUSH - 1 || k == nk - 1) chunk++;
            }
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------------ the activations' scales
        const int u = warp - 2;                            // rows 128 u .. of the tile
        if (u < C::NB) {
            int step = 0;
            for (int i = cluster; i < tiles && !failed; i += clusters) {
                const Tile t = tile_at<BN>(p, starts, i);
                const uint8_t *row[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int c = u * 128 + j * 32 + lane;
                    int64_t r = -1;
                    if (c < t.n) r = p.rows ? p.rows[t.r0 + c] : t.r0 + c;
                    row[j] = r >= 0 && r < p.x_rows ? p.x_scales + r * p.S : nullptr;
                }
                for (int k = 0; k < nk; k++, step++) {
                    const int st = step % C::ST, kt = kt0 + k;
                    uint32_t w[4];
                    // scale bytes past the row's end belong to columns of zeros, but must not be NaN
                    const int left = p.K / QK - kt * 4;
                    const uint32_t mask = left >= 4 ? 0xffffffffu : (1u << (8 * left)) - 1u;
#pragma unroll
                    for (int j = 0; j < 4; j++) w[j] = row[j] ? *reinterpret_cast<const uint32_t *>(row[j] + kt * 4) & mask : 0u;
                    if (step >= C::ST && !mbar_wait(bar(EMPTY + st), (uint32_t)((step / C::ST - 1) & 1), p.status)) failed = true;
                    if (__any_sync(0xffffffffu, failed)) {
                        failed = true;
                        break;
                    }
                    *reinterpret_cast<uint4 *>(smem + C::sfb + (st * C::NB + u) * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(FULL + st));
                }
            }
        }
    } else {
        // ------------------------------------------------------------------ sums, output
        const int q = warp & 3, half = (warp - 4) >> 2;    // tensor-memory lanes 32 q .., column chunks half, half + 2, ..
        int chunk = 0, turn = 0;
        for (int i = cluster; i < tiles && !failed; i += clusters, turn++) {
            const Tile t = tile_at<BN>(p, starts, i);
            const int cols = (t.n + C::CW - 1) / C::CW;    // chunks in use
            float acc[C::NA][C::MINE][C::CW];
#pragma unroll
            for (int a = 0; a < C::NA; a++)
#pragma unroll
                for (int j = 0; j < C::MINE; j++)
#pragma unroll
                    for (int c = 0; c < C::CW; c++) acc[a][j][c] = 0.0f;
            for (int k = 0; k < nk; k += FLUSH, chunk++) {
                const int set = chunk & 1;
                if (!failed && !mbar_wait(bar(ACC_FULL + set), (uint32_t)((chunk / 2) & 1), p.status)) failed = true;
                failed = __any_sync(0xffffffffu, failed);
                if (failed) break;
                fence_after();
#pragma unroll
                for (int a = 0; a < C::NA; a++)
#pragma unroll
                    for (int j = 0; j < C::MINE; j++)
                        if (2 * j + half < cols) {
                            float v[C::CW];
                            read_acc<C::CW>(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(set * C::ACC + a * BN + (2 * j + half) * C::CW), v);
#pragma unroll
                            for (int c = 0; c < C::CW; c++) acc[a][j][c] += v[c];
                        }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ACC_EMPTY + set));
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
                if (t.g * MX_TILE + 32 * q < p.N)
#pragma unroll
                    for (int j = 0; j < C::MINE; j++)
#pragma unroll
                        for (int c = 0; c < C::CW; c++) {
                            const int col = (2 * j + half) * C::CW + c;
                            if (col < t.n) {
                                const float gate = acc[0][j][c], v = gate / (1.0f + expf(-gate)) * acc[1][j][c];
                                const int b = mx_scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu), false);
                                const float inv = mx_inverse(b);
                                const int64_t r = t.r0 + col;
                                p.codes[r * p.N + n] = (uint8_t)(inv == 0.0f ? 0u : e4m3x2(v * inv, 0.0f));
                                if (lane == 0) p.scales[r * p.So + t.g * 4 + q] = (uint8_t)b;
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

gq_status encode(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t inner, int64_t outer, int64_t stride,
                 int box_rows) {
    std::call_once(g_encode_once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    if (!g_encode) return fail(GQ_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
    const cuuint64_t strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1u, 1u};
    const CUresult r = g_encode(map, type, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(GQ_ERR_CUDA, "cuTensorMapEncodeTiled (mx) failed (%d)", (int)r);
    return GQ_OK;
}

constexpr int MAX_DEV = 64;

template <int BN, bool GATED>
gq_status launch(MxParams p, const void *rep, const gq_mx_rows &x, int64_t tiles128, int64_t most_tiles, cudaStream_t s) {
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
    CUtensorMap mw, mx;
    st = encode(&mw, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, rep, MX_TILE, tiles128 * MX_TILE, MX_TILE / 2, MX_TILE);
    if (st != GQ_OK) return st;
    st = encode(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, x.codes, p.K, x.rows, p.K, p.rows ? 1 : C::BOX);
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
    return check_cuda(cudaLaunchKernelEx(&cfg, kernel, mw, mx, p), "mx product launch");
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
    const int64_t count = (int64_t)p.E * (gated ? 2 : 1), tiles128 = count * p.G * p.KT;
    p.w_scales = static_cast<const uint8_t *>(rep) + tiles128 * MX_TILE_CODES;

    // Rows per tile by the rows that an expert has on average (of the experts that can have any).
    const int64_t some = std::min<int64_t>(p.E, p.R), mean = (p.R + some - 1) / some;
    auto most = [&](int bn) { return ((plan ? some : 0) + (p.R + bn - 1) / bn) * p.G; };
    if (most(16) >= (1LL << 31)) return fail(GQ_ERR_INVALID_ARG, "R=%lld rows of N=%lld are too many", (long long)p.R, (long long)N);
    if (gated) {
        if (mean <= 16) return launch<16, true>(p, rep, x, tiles128, most(16), s);
        if (mean <= 64) return launch<64, true>(p, rep, x, tiles128, most(64), s);
        return launch<112, true>(p, rep, x, tiles128, most(112), s);
    }
    if (mean <= 16) return launch<16, false>(p, rep, x, tiles128, most(16), s);
    if (mean <= 64) return launch<64, false>(p, rep, x, tiles128, most(64), s);
    return launch<192, false>(p, rep, x, tiles128, most(192), s);
}

}  // namespace gq

// route.cu -- routing to experts: scores, the choice of top_k, and the rows sorted by expert.
//
// One warp per token; lane l holds the values of experts l, l + 32, .. as ordered 32-bit keys, whose lowest bits say which of
// the lane's experts it is, and sorts them; a choice then costs a warp-wide maximum of the lanes' first keys, and the lane that
// had it moves up.  Without a bias the order of the scores is the order of the logits.  Keys lack some bits, and with a bias
// (and for the groups' sums) f32 values carry a rounding error: where two values that decide something are closer
// than its bound (about one token in a hundred with a bias), the warp takes the 32 best candidates, one per lane, and
// ranks them by their values in 64 bits; where that does not settle it (the groups' sums are close, or more than
// 32 candidates are), it does the whole token in 64 bits.
//
// The plan is a counting sort, stable in the tokens.  Up to 32 tokens: one CTA does all of it.  More:
// each CTA counts the choices of its chunk of tokens per expert into the workspace (about one chunk
// per SM, so that the counts of all chunks, which every CTA of the second kernel reads, stay small), and the
// second kernel places each chunk's choices behind those of the chunks before it.  No atomics on
// memory, so nothing depends on timing.  Both are bound by instructions, not by memory: 8192 tokens, 8 of 256
// experts by sigmoid scores with a bias in 4 of 8 groups, take 27 us and 12 us (their bytes 1.4).
#include <algorithm>
#include <cfloat>

#include "mx.cuh"

namespace gq {
namespace {

constexpr int SOLO_TOKENS = 32;    // tokens that one CTA routes and sorts by itself

struct RouteParams {
    const void *logits;
    const float *bias;
    const int32_t *used;
    int32_t *ids;
    float *weights;
    int32_t *offsets, *rows, *pos;   // solo CTA only
    int32_t *counts;                 // [chunks][E], or nullptr
    unsigned int *status;
    int64_t ldl;
    int E, k, T, chunk, sigmoid, groups, top_groups, group_best, renormalize, bf16;
    int lanes, log_lanes;            // that look through a group
    int per_group;                   // E / groups
    float factor;
};

// Keys that order as their floats do; 0 is below all of them.
__device__ __forceinline__ uint32_t order32(float x) {
    const uint32_t b = __float_as_uint(x);
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unorder32(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k); }
__device__ __forceinline__ uint64_t order64(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ uint64_t warp_max64(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// The two largest of two pairs.
template <typename F>
__device__ __forceinline__ void best_two(F &a, F &b, F c, F d) {
    const F lo = a < c ? a : c;
    a = a < c ? c : a;
    b = b < d ? d : b;
    b = lo < b ? b : lo;
}

// Which groups take part, as a bit each, from the choice values in shared memory.  32 / P lanes look through a group, P the
// power of two from `groups` on; expert e's value is at e + (e / n) * (32 / P), so that lanes of different groups use
// different banks.  `gap` receives the distance between the worst group that takes part and the best that does not.
template <typename F>
__device__ __forceinline__ uint32_t best_groups(const F *c, int n, int groups, int log_lanes, int top, int best, int lane, F &gap) {
    const F none = -(F)INFINITY;
    const int g = lane >> log_lanes, lanes = 1 << log_lanes;
    F a = none, b = none;
    if (g < groups)
        for (int j = lane & (lanes - 1); j < n; j += lanes) best_two<F>(a, b, c[g * (n + lanes) + j], none);
    for (int d = 1; d < lanes; d <<= 1) {
        const F oa = __shfl_xor_sync(0xffffffffu, a, d), ob = __shfl_xor_sync(0xffffffffu, b, d);
        best_two<F>(a, b, oa, ob);
    }
    const F value = best == 2 && n > 1 ? a + b : a;
    int rank = 0;
    for (int h = 0; h < groups; h++) {
        const F v = __shfl_sync(0xffffffffu, value, h * lanes);
        rank += v > value || (v == value && h < g);
    }
    const bool in = g < groups && rank < top;
    // ranks are all different: the worst that takes part has rank top - 1, the best other rank top
    const uint32_t w = __ballot_sync(0xffffffffu, g < groups && rank == top - 1), o = __ballot_sync(0xffffffffu, g < groups && rank == top);
    gap = __shfl_sync(0xffffffffu, value, __ffs((int)w) - 1) - __shfl_sync(0xffffffffu, value, __ffs((int)o) - 1);
    // one bit per group
    uint32_t bits = __ballot_sync(0xffffffffu, in), out = 0;
    if (lanes == 1) return bits;
    for (int h = 0; h < groups; h++) out |= (bits >> (h * lanes) & 1u) << h;
    return out;
}

__device__ __forceinline__ double score64(const RouteParams &p, float z, float m, double sum) {
    if (p.sigmoid) return 1.0 / (1.0 + exp(-(double)z));
    return m == -INFINITY ? 0.0 : exp((double)z - (double)m) / sum;
}

// A logit or a bias as it counts: NaN as -infinity, +infinity as the largest finite number.  So no sum, difference or score of two
// such is NaN, but for the difference of two -infinities.
__device__ __forceinline__ float plain(float z) { return fminf(fmaxf(z, -INFINITY), FLT_MAX); }   // (fmaxf drops a NaN)
__device__ __forceinline__ float plain(__nv_bfloat16 z) { return plain(__bfloat162float(z)); }
__device__ __forceinline__ float logit(const RouteParams &p, int64_t t, int e) {
    return p.bf16 ? plain(static_cast<const __nv_bfloat16 *>(p.logits)[t * p.ldl + e]) : plain(static_cast<const float *>(p.logits)[t * p.ldl + e]);
}

// The sum of the exponentials of token t, in 64 bits.
__device__ __noinline__ double sum64(const RouteParams &p, int64_t t, float m, int lane) {
    double sum = 0.0;
    if (p.sigmoid || m == -INFINITY) return 1.0;
    for (int e = lane; e < p.E; e += 32) sum += exp((double)logit(p, t, e) - (double)m);
    return warp_sum(sum);
}

// Token t in 64 bits, from the start; lane j < k returns the j-th choice.  With groups the experts' values are formed once,
// in shared memory (a few microseconds: this GPU has few 64-bit units); without, again for each choice (for tokens with more
// than 32 values closer than f32 can tell).
__device__ __noinline__ int choose64(const RouteParams &p, int64_t t, float m, double sum, double *shared, int lane) {
    uint32_t allowed = 0xffffffffu;
    const int n = p.per_group;
    const bool grouped = p.top_groups < p.groups, sums = !p.bias && p.group_best == 2;
    // without a bias, and where no sums are compared, the logits decide
    auto value = [&](int e) {
        const float z = logit(p, t, e);
        return p.bias ? score64(p, z, m, sum) + (double)plain(p.bias[e]) : (double)z;
    };
    if (grouped) {
        for (int e = lane; e < p.E; e += 32) shared[e + e / n * p.lanes] = sums ? score64(p, logit(p, t, e), m, sum) : value(e);
        __syncwarp();
        double gap;
        allowed = best_groups<double>(shared, n, p.groups, p.log_lanes, p.top_groups, p.group_best, lane, gap);
        __syncwarp();
    }
    uint64_t last_key = ~0ull;
    int last = -1, id = -1;
    for (int j = 0; j < p.k; j++) {
        uint64_t key = 0;
        int at = 0x7fffffff;
        for (int e = lane; e < p.E; e += 32) {
            if (!(allowed >> (e / n) & 1u)) continue;
            const uint64_t c = order64((grouped && !sums ? shared[e + e / n * p.lanes] : value(e)) + 0.0);
            // behind the last choice in the order of values, then indices
            if ((c < last_key || (c == last_key && e > last)) && c > key) key = c, at = e;
        }
        const uint64_t top = warp_max64(key);
        if (top == 0) break;
        const int e = (int)__reduce_min_sync(0xffffffffu, key == top ? (uint32_t)at : 0x7fffffffu);
        if (lane == j) id = e;
        last_key = top;
        last = e;
    }
    return id;
}

// Sorts N keys of a lane, the largest first: a bitonic network.
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[N]) {
#pragma unroll
    for (int size = 2; size <= N; size *= 2)
#pragma unroll
        for (int step = size / 2; step > 0; step /= 2)
#pragma unroll
            for (int i = 0; i < N; i++) {
                const int j = i ^ step;
                if (j > i) {
                    const uint32_t hi = max(key[i], key[j]), lo = min(key[i], key[j]);
                    key[i] = (i & size) == 0 || size == N ? hi : lo;
                    key[j] = (i & size) == 0 || size == N ? lo : hi;
                }
            }
}

// One token.  Lane j < k returns the j-th choice.  z: the lane's logits; m and sum: their maximum and the sum of the
// exponentials (softmax); bias, group: of the lane's experts.
template <int V, typename T>
__device__ __forceinline__ int choose(const RouteParams &p, int64_t t, const float (&z)[V], const float (&bias)[V], const int (&group)[V], float m,
                                      float sum, double *shared, int lane) {
    // the lowest bits of a key: the lane's experts counted from the last, so that of equal values the lowest index is first
    constexpr uint32_t SLOT = V - 1;
    const bool grouped = p.top_groups < p.groups, sums = !p.bias && p.group_best == 2;
    const float inverse = p.sigmoid ? 1.0f : m == -INFINITY ? 0.0f : 1.0f / sum;
    // The fast exponential and reciprocal: a sigmoid is off by 2e-7 at most; a softmax score by its rounded argument and
    // sum, 2^-18 of the largest score at most.  Two values that differ by more than `tol` (and the rounding of the sums
    // with a bias) are in order.
    const float tol = p.sigmoid ? 0x1p-20f : inverse * 0x1p-17f;
    auto score = [&](float x) {
        float e, r;
        if (p.sigmoid) {
            asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
            asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
            return r;
        }
        if (m == -INFINITY) return 0.0f;
        asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"((x - m) * 1.4426950408889634f));
        return e * inverse;
    };
    float c[V];
#pragma unroll
    for (int i = 0; i < V; i++) c[i] = p.bias ? score(z[i]) + bias[i] : z[i];
    uint32_t allowed = 0xffffffffu;
    if (grouped) {
        float *values = reinterpret_cast<float *>(shared);
#pragma unroll
        for (int i = 0; i < V; i++)
            if (i * 32 + lane < p.E) values[i * 32 + lane + group[i] * p.lanes] = sums ? score(z[i]) : c[i];
        __syncwarp();
        float gap;
        allowed = best_groups<float>(values, p.per_group, p.groups, p.log_lanes, p.top_groups, p.group_best, lane, gap);
        __syncwarp();
        if (p.bias || sums) {
            float size = 0.0f;
            if (p.bias)
#pragma unroll
                for (int i = 0; i < V; i++) size = fmaxf(size, fabsf(c[i]));
            size = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(size)));
            // (two of the largest values would overflow in a sum of f32)
            if (!(gap > 2.0f * tol + 0x1p-20f * size) || size > 0x1p126f) return choose64(p, t, m, sum64(p, t, m, lane), shared, lane);
        }
    }
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; i++)
        key[i] = i * 32 + lane < p.E && (allowed >> group[i] & 1u) ? (order32(c[i] + 0.0f) & ~SLOT) | (SLOT - i) : 0u;
    sort_keys<V>(key);
    int id = -1;
    uint32_t mine = 0;                        // the lane's candidate
    int found = 0;
    auto next = [&] {                         // the best that is left goes to lane `found`; false if there is none
        const uint32_t top = __reduce_max_sync(0xffffffffu, key[0]);
        if (top <= SLOT) return false;
        // equal keys are of the same place in different lanes: the lowest lane has the lowest index
        const int from = __ffs((int)__ballot_sync(0xffffffffu, key[0] == top)) - 1;
        if (lane == found) id = (int)(SLOT - (top & SLOT)) * 32 + from, mine = top;
        if (lane == from) {
#pragma unroll
            for (int i = 0; i + 1 < V; i++) key[i] = key[i + 1];
            key[V - 1] = 0;
        }
        found++;
        return true;
    };
    while (found < p.k && next()) {
    }
    // bf16 logits without a bias: keys lack nothing
    if (!p.bias && sizeof(T) == 2) return id;
    // the choice after the last says how far it is from it
    const int chosen = found;
    const bool one_more = found < 32 && next();
    uint32_t after = __shfl_down_sync(0xffffffffu, mine, 1);
    if (chosen == 32) {                       // (all lanes are taken: the best that is left)
        const uint32_t top = __reduce_max_sync(0xffffffffu, key[0]);
        if (lane == 31) after = top;
    } else if (!one_more && lane == chosen - 1) {
        after = 0;
    }
    // a key's value is up to 32 units of the last place below its expert's
    auto apart = [&](uint32_t hi, uint32_t lo) {
        if (lo <= SLOT) return true;
        const float a = unorder32(hi & ~SLOT), b = unorder32(lo & ~SLOT);
        if (!p.bias) return (hi & ~SLOT) != (lo & ~SLOT);
        return a - b > tol + (0x1p-21f + V * 0x1p-23f) * (fabsf(a) + fabsf(b));
    };
    if (!__any_sync(0xffffffffu, lane < chosen && !apart(mine, after))) return id;
    // 32 candidates, ranked by their values in 64 bits
    while (found < 32 && next()) {
    }
    const double s = sum64(p, t, m, lane);
    double exact = -INFINITY;
    if (lane < found) {
        const float x = logit(p, t, id);
        exact = p.bias ? score64(p, x, m, s) + (double)plain(p.bias[id]) : (double)x;
    }
    int rank = 0;
    for (int j = 0; j < found; j++) {
        const double v = __shfl_sync(0xffffffffu, exact, j);
        const int e = __shfl_sync(0xffffffffu, id, j);
        rank += v > exact || (v == exact && e < id);
    }
    // what was not taken must be below the last choice
    const uint32_t left = __reduce_max_sync(0xffffffffu, key[0]);
    const uint32_t w = __ballot_sync(0xffffffffu, lane < found && rank == p.k - 1);
    if (!apart(__shfl_sync(0xffffffffu, mine, __ffs((int)w) - 1), left)) return choose64(p, t, m, s, shared, lane);
    // to the lanes of their ranks
    int out = -1;
    for (int j = 0; j < found; j++) {
        const int r = __shfl_sync(0xffffffffu, rank, j), e = __shfl_sync(0xffffffffu, id, j);
        if (r == lane && lane < p.k) out = e;
    }
    return out;
}

// Stable places for n choices in order, by all warps of the CTA; base[e] is where expert e's next row goes, and per_warp has room for
// a byte per expert and warp.  Each warp ranks 32 choices among themselves and counts them per expert; a prefix over
// the warps' counts gives each its base.
__device__ __forceinline__ void place(const int32_t *ids, int n, int64_t first, int k, int E, int32_t *base, uint8_t *per_warp, int32_t *rows,
                                      int32_t *pos) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    for (int i0 = 0; i0 < n; i0 += blockDim.x) {
        for (int j = threadIdx.x; j < (warps * E + 3) / 4; j += blockDim.x) reinterpret_cast<uint32_t *>(per_warp)[j] = 0;
        __syncthreads();
        const int i = i0 + threadIdx.x, e = i < n ? ids[i] : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        if (e >= 0 && rank == 0) per_warp[warp * E + e] = (uint8_t)__popc(same);
        __syncthreads();
        int at = 0;
        if (e >= 0) {
            at = base[e];
            for (int w = 0; w < warp; w++) at += per_warp[w * E + e];
        }
        if (i < n) {
            pos[first + i] = e < 0 ? -1 : at + rank;
            if (e >= 0) rows[at + rank] = (int32_t)((uint32_t)(first + i) / (uint32_t)k);
        }
        if (i0 + (int)blockDim.x < n) {
            __syncthreads();
            // the last warp of each expert moves its base
            for (int x = threadIdx.x; x < E; x += blockDim.x) {
                int all = 0;
                for (int w = 0; w < warps; w++) all += per_warp[w * E + x];
                base[x] += all;
            }
            __syncthreads();
        }
    }
}

// Exclusive sums of n counts in shared memory, in place, by one warp; returns the total.
__device__ __forceinline__ int scan(int32_t *counts, int n, int lane) {
    int total = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int v = i0 + lane < n ? counts[i0 + lane] : 0;
        int s = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += u;
        }
        if (i0 + lane < n) counts[i0 + lane] = total + s - v;
        total += __shfl_sync(0xffffffffu, s, 31);
    }
    __syncwarp();
    return total;
}

__device__ __forceinline__ int tokens_used(const int32_t *used, int T, unsigned int *status) {
    if (!used) return T;
    const int u = *used;
    if (u < 0 || u > T) atomicOr(status, STATUS_RANGE);
    return min(max(u, 0), T);
}

constexpr int route_threads(int V) { return V <= 8 ? 1024 : 512; }

// Dynamic shared memory: E counts, SOLO_TOKENS * k ids (solo), then, with groups, E doubles per warp.
template <int V, typename T>
__global__ void __launch_bounds__(route_threads(V)) route_kernel(const RouteParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    int32_t *counts = reinterpret_cast<int32_t *>(smem);
    const int words = (p.E + 3) / 4 * 4;
    int32_t *list = counts + words;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    // choice values by group, for warps that need them: E and a few more per group
    double *shared = reinterpret_cast<double *>(list + (p.pos ? (SOLO_TOKENS * p.k + 3) / 4 * 4 : 0)) + (size_t)warp * (p.E + p.groups * p.lanes);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) counts[e] = 0;
    int group[V];
#pragma unroll
    for (int i = 0; i < V; i++) group[i] = (i * 32 + lane) / (p.E / p.groups) & 31;
    pdl_wait();
    pdl_launch_dependents();
    float bias[V];
#pragma unroll
    for (int i = 0; i < V; i++) bias[i] = p.bias && i * 32 + lane < p.E ? plain(p.bias[i * 32 + lane]) : 0.0f;
    __syncthreads();
    const int used = tokens_used(p.used, p.T, p.status);
    const int t0 = blockIdx.x * p.chunk, t1 = min(t0 + p.chunk, p.T);
    const bool counted = p.counts || p.pos;
    for (int t = t0 + warp; t < t1; t += warps) {
        int id = -1;
        float w = 0.0f;
        if (t < used) {
            const T *row = static_cast<const T *>(p.logits) + t * p.ldl;
            float z[V], m = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; i++) {
                z[i] = i * 32 + lane < p.E ? plain(row[i * 32 + lane]) : -INFINITY;
                m = fmaxf(m, z[i]);
            }
            float sum = 1.0f;
            if (!p.sigmoid) {
                m = unorder32(__reduce_max_sync(0xffffffffu, order32(m)));
                sum = 0.0f;
                if (m > -INFINITY) {
#pragma unroll
                    for (int i = 0; i < V; i++) sum += expf(z[i] - m);
                    sum = warp_sum(sum);
                }
            }
            id = choose<V, T>(p, t, z, bias, group, m, sum, shared, lane);
            if (lane < p.k) {
                // (no value is NaN, so every place is filled; a mistake in that would not read out of bounds)
                GQ_DCHECK((uint32_t)id < (uint32_t)p.E, p.status);
                id = (uint32_t)id < (uint32_t)p.E ? id : -1;
                const float chosen = id < 0 ? -INFINITY : plain(row[id]);
                w = p.sigmoid ? 1.0f / (1.0f + expf(-chosen)) : m > -INFINITY ? expf(chosen - m) / sum : 0.0f;
            }
            if (p.renormalize) {
                const float all = warp_sum(w);
                if (all > 0.0f) w /= all;
            }
            w *= p.factor;
        }
        if (lane < p.k) {
            p.ids[(int64_t)t * p.k + lane] = id;
            p.weights[(int64_t)t * p.k + lane] = w;
            if (p.pos) list[(t - t0) * p.k + lane] = id;
            if (counted && id >= 0) atomicAdd(&counts[id], 1);
        }
    }
    if (!counted) return;
    __syncthreads();
    if (p.pos) {
        if (warp == 0) {
            const int total = scan(counts, p.E, lane);
            for (int e = lane; e < p.E; e += 32) p.offsets[e] = counts[e];
            if (lane == 0) p.offsets[p.E] = total;
        }
        __syncthreads();
        // (the choices are made: the groups' room serves the warps' counts)
        place(list, (t1 - t0) * p.k, 0, p.k, p.E, counts, reinterpret_cast<uint8_t *>(list + (SOLO_TOKENS * p.k + 3) / 4 * 4), p.rows, p.pos);
    } else {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.counts[(int64_t)blockIdx.x * p.E + e] = counts[e];
    }
}

// CTA c places the choices of chunk c.  Four threads sum an expert's counts over the chunks.
constexpr int PLAN_THREADS = 1024;
__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const int32_t *__restrict__ ids, const int32_t *__restrict__ counts,
                                                            int32_t *__restrict__ offsets, int32_t *__restrict__ rows,
                                                            int32_t *__restrict__ pos, int E, int k, int T, int chunk, int chunks) {
    extern __shared__ __align__(16) uint8_t smem[];
    int32_t *base = reinterpret_cast<int32_t *>(smem), *before = base + E;
    uint8_t *per_warp = reinterpret_cast<uint8_t *>(before + E);
    for (int e = threadIdx.x; e < 2 * E; e += PLAN_THREADS) base[e] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    const int parts = max(1, PLAN_THREADS / E);
    for (int x = threadIdx.x; x < E * parts; x += PLAN_THREADS) {
        const int e = x % E, part = x / E;
        int all = 0, mine = 0;
#pragma unroll 16
        for (int c = part; c < chunks; c += parts) {
            const int v = counts[(int64_t)c * E + e];
            all += v;
            mine += c < (int)blockIdx.x ? v : 0;
        }
        atomicAdd(&base[e], all);
        atomicAdd(&before[e], mine);
    }
    __syncthreads();
    {
        // exclusive sums over the experts: E <= PLAN_THREADS, one each
        __shared__ int32_t sums[32];
        const int e = threadIdx.x, lane = e & 31, warp = e >> 5, v = e < E ? base[e] : 0;
        int s = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += u;
        }
        if (lane == 31) sums[warp] = s;
        __syncthreads();
        if (warp == 0) {
            int t = sums[lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, t, d);
                if (lane >= d) t += u;
            }
            sums[lane] = t;
        }
        __syncthreads();
        if (warp > 0) s += sums[warp - 1];
        if (e < E) {
            if (blockIdx.x == 0) {
                offsets[e] = s - v;
                if (e == E - 1) offsets[E] = s;
            }
            base[e] = s - v + before[e];
        }
    }
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * chunk * k;
    const int n = (min((int)(blockIdx.x + 1) * chunk, T) - (int)blockIdx.x * chunk) * k;
    place(ids + first, n, first, k, E, base, per_warp, rows, pos);
}

template <int V>
gq_status route_launch(RouteParams p, int chunks, size_t fixed, cudaStream_t s) {
    // values by group in 64 bits; the solo CTA's counts of each warp (a byte per expert) lie over them
    const size_t per_warp = p.top_groups < p.groups ? (size_t)(p.E + p.groups * p.lanes) * 8 : p.pos ? (size_t)(p.E + 7) / 4 * 4 : 0;
    int warps = std::min(route_threads(V) / 32, p.chunk);
    if (per_warp) warps = std::max<int>(1, std::min<int64_t>(warps, (int64_t)((48 * 1024 - fixed) / per_warp)));
    warps = (p.chunk + (p.chunk + warps - 1) / warps - 1) / ((p.chunk + warps - 1) / warps);   // as many turns, no idle warps
    void *args[] = {&p};
    const void *fn = p.bf16 ? (const void *)route_kernel<V, __nv_bfloat16> : (const void *)route_kernel<V, float>;
    return launch_pdl(fn, dim3(chunks), dim3(32 * warps), fixed + warps * per_warp, s, args, "route launch");
}

}  // namespace

gq_status launch_route(const gq_router &r, const void *logits, int64_t ldl, bool bf16, const int32_t *used, int32_t *ids,
                       float *weights, int32_t *offsets, int32_t *rows, int32_t *pos, int64_t T, cudaStream_t s) {
    RouteParams p{};
    p.logits = logits, p.bias = r.bias, p.used = used, p.ids = ids, p.weights = weights, p.ldl = ldl;
    p.E = (int)r.E, p.k = (int)r.top_k, p.T = (int)T, p.sigmoid = r.score == GQ_SCORE_SIGMOID;
    p.groups = (int)r.groups, p.top_groups = (int)r.top_groups, p.group_best = (int)r.group_best;
    p.renormalize = r.renormalize != 0, p.bf16 = bf16, p.factor = r.factor;
    int P = 1;
    while (P < p.groups) P *= 2;
    p.lanes = 32 / P;
    while ((1 << p.log_lanes) < p.lanes) p.log_lanes++;
    p.per_group = p.E / p.groups;
    p.status = device_status_word();
    if (!p.status) return fail(GQ_ERR_CUDA, "device status word unavailable");
    const bool solo = pos && T <= SOLO_TOKENS;
    p.chunk = solo ? (int)T : (int)std::max<int64_t>(8, (T + sm_count() - 1) / sm_count());
    const int chunks = (int)((T + p.chunk - 1) / p.chunk);
    if (solo) {
        p.offsets = offsets, p.rows = rows, p.pos = pos;
    } else if (pos) {
        Workspace ws;
        gq_status st = get_workspace(s, 0, (size_t)chunks * p.E * 4, &ws);
        if (st != GQ_OK) return st;
        p.counts = reinterpret_cast<int32_t *>(ws.data);
    }
    const size_t fixed = (size_t)(p.E + 3) / 4 * 16 + (solo ? (size_t)(SOLO_TOKENS * p.k + 3) / 4 * 16 : 0);
    gq_status st;
    if (p.E <= 32) st = route_launch<1>(p, chunks, fixed, s);
    else if (p.E <= 64) st = route_launch<2>(p, chunks, fixed, s);
    else if (p.E <= 128) st = route_launch<4>(p, chunks, fixed, s);
    else if (p.E <= 256) st = route_launch<8>(p, chunks, fixed, s);
    else if (p.E <= 512) st = route_launch<16>(p, chunks, fixed, s);
    else st = route_launch<32>(p, chunks, fixed, s);
    if (st != GQ_OK || solo || !pos) return st;
    int E = p.E, k = p.k, TT = p.T, chunk = p.chunk, nch = chunks;
    const int32_t *cids = ids, *counts = p.counts;
    void *args[] = {&cids, &counts, &offsets, &rows, &pos, &E, &k, &TT, &chunk, &nch};
    return launch_pdl((const void *)plan_kernel, dim3(chunks), dim3(PLAN_THREADS), (size_t)E * 8 + (size_t)E * (PLAN_THREADS / 32) + 16, s, args, "plan launch");
}

}  // namespace gq

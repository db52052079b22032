// route.cu -- routing to experts: scores, the choice of top_k, and the rows sorted by expert.
//
// One warp per token; lane l holds the logits of experts l, l + 32, ..  A choice is made on ordered
// 32-bit keys, one warp-wide maximum and one minimum of indices per chosen expert.  Without a bias
// the order of the scores is the order of the logits, which are exact.  With one (and for the groups'
// sums) the f32 values carry a rounding error: where two values that decide something are closer than
// its bound, the warp does the token again in 64 bits (a few tokens in ten thousand).
//
// The plan is a counting sort, stable in the tokens.  Up to 32 tokens: one CTA does all of it.  More:
// each CTA counts the choices of its chunk of tokens per expert into the workspace (about one chunk
// per SM, so that the counts of all chunks, which every CTA of the second kernel reads, stay small), and the
// second kernel places each chunk's choices behind those of the chunks before it.  No atomics on
// memory, so nothing depends on timing.
#include <algorithm>

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

// Which groups take part, as a bit each, from the choice values c[e] in shared memory: lane g looks
// through group g.  `gap` receives the distance between the worst group that does and the best that
// does not.
template <typename F>
__device__ __forceinline__ uint32_t best_groups(const F *c, int E, int groups, int top, int best, int lane, F &gap) {
    const int n = E / groups;
    const F none = -(F)INFINITY;
    F a = none, b = none;
    if (lane < groups)
        for (int j = 0; j < n; j++) {
            int at = j + lane;                       // a start of its own: no two lanes in one bank
            if (at >= n) at %= n;
            const F v = c[lane * n + at];
            b = v > a ? a : v > b ? v : b;
            a = v > a ? v : a;
        }
    const F value = best == 2 && n > 1 ? a + b : a;
    int rank = 0;
    for (int g = 0; g < groups; g++) {
        const F v = __shfl_sync(0xffffffffu, value, g);
        rank += v > value || (v == value && g < lane);
    }
    const bool in = lane < groups && rank < top;
    F worst = in ? value : (F)INFINITY, other = !in && lane < groups ? value : none;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const F w = __shfl_xor_sync(0xffffffffu, worst, d), o = __shfl_xor_sync(0xffffffffu, other, d);
        worst = w < worst ? w : worst;
        other = o > other ? o : other;
    }
    gap = worst - other;
    return __ballot_sync(0xffffffffu, in);
}

// One token.  Lane j < k returns the j-th choice (its expert and logit); m and the sum of exponentials as
// the caller computed them.  F is float (with the checks of close values: `close` is set) or double.
template <int V, typename F>
__device__ __forceinline__ void choose(const RouteParams &p, const float (&z)[V], float m, F sum, F *shared, int lane, int &id,
                                       float &zid, bool &close) {
    constexpr bool FAST = sizeof(F) == 4;
    auto score = [&](float x) -> F {
        if (p.sigmoid) return (F)1 / ((F)1 + (FAST ? (F)expf(-x) : (F)exp(-(double)x)));
        return m == -INFINITY ? (F)0 : (FAST ? (F)expf(x - m) : (F)exp((double)x - (double)m)) / sum;
    };
    const bool grouped = p.top_groups < p.groups;
    // bounds of the f32 errors: a score's relative one, and a sum's
    const F rel = p.sigmoid ? (F)0x1p-21 : (F)0x1p-18;
    const F most = p.sigmoid ? (F)1 : m == -INFINITY ? (F)0 : (F)1 / sum;
    uint32_t allowed = 0xffffffffu;
    F c[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int e = i * 32 + lane;
        // without a bias, and where no sums are compared, the logits decide
        c[i] = p.bias ? (e < p.E ? score(z[i]) + (F)p.bias[e] : (F)0) : (F)z[i];
    }
    if (grouped) {
        const bool sums = !p.bias && p.group_best == 2;
#pragma unroll
        for (int i = 0; i < V; i++)
            if (i * 32 + lane < p.E) shared[i * 32 + lane] = sums ? score(z[i]) : c[i];
        __syncwarp();
        F gap;
        allowed = best_groups<F>(shared, p.E, p.groups, p.top_groups, p.group_best, lane, gap);
        __syncwarp();
        if (FAST && (p.bias || sums)) {
            float size = 0.0f;                       // the largest magnitude among the biases
            if (p.bias)
#pragma unroll
                for (int i = 0; i < V; i++)
                    if (i * 32 + lane < p.E) size = fmaxf(size, fabsf((float)c[i]));
            size = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(size)));
            close |= !((float)gap > 4.0f * (float)(rel * most) + 0x1p-20f * size);
        }
    }
    const int per_group = p.E / p.groups;
    using Key = typename std::conditional<FAST, uint32_t, uint64_t>::type;
    Key key[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int e = i * 32 + lane;
        const bool in = e < p.E && (!grouped || (allowed >> (e / per_group) & 1u));
        if constexpr (FAST)
            key[i] = in ? order32(c[i] + 0.0f) : 0u;
        else
            key[i] = in ? order64(c[i] + 0.0) : 0ull;
    }
    Key best = 0;
    int at = 0;
    auto local = [&] {
        best = 0;
#pragma unroll
        for (int i = 0; i < V; i++)
            if (key[i] > best) best = key[i], at = i;
    };
    local();
    float before = INFINITY;
    for (int j = 0; j <= p.k; j++) {
        // the choice after the last only says how far it is from it
        if (j == p.k && !(FAST && p.bias)) break;
        Key top;
        if constexpr (FAST)
            top = __reduce_max_sync(0xffffffffu, best);
        else
            top = warp_max64(best);
        if (top == 0) break;
        if constexpr (FAST) {
            if (p.bias) {
                const float v = unorder32(top);
                close |= !(before - v > 2.0f * (float)(rel * most) + 0x1p-21f * (fabsf(v) + (j ? fabsf(before) : 0.0f)));
                before = v;
            }
        }
        if (j == p.k) break;
        const int e = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)(at * 32 + lane) : 0xffffffffu);
        float mine = 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++)
            if (i == (e >> 5)) mine = z[i];
        const float chosen = __shfl_sync(0xffffffffu, mine, e & 31);
        if (lane == j) id = e, zid = chosen;
        if (lane == (e & 31)) {
#pragma unroll
            for (int i = 0; i < V; i++)
                if (i == (e >> 5)) key[i] = 0;
            local();
        }
        __syncwarp();
    }
}

// Stable places for n choices in order (32 at a time, by one warp): base[e] is where expert e's next row goes.
__device__ __forceinline__ void place(const int32_t *ids, int n, int64_t first, int k, int32_t *base, int32_t *rows,
                                      int32_t *pos, int lane) {
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const int e = i < n ? ids[i] : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const int r = e < 0 ? -1 : base[e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && (same >> lane) == 1u) base[e] = r + 1;      // the last lane of its expert
        __syncwarp();
        if (i < n) {
            pos[first + i] = r;
            if (r >= 0) rows[r] = (int32_t)((first + i) / k);
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
template <int V>
__global__ void __launch_bounds__(route_threads(V)) route_kernel(const RouteParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    int32_t *counts = reinterpret_cast<int32_t *>(smem);
    const int words = (p.E + 3) / 4 * 4;
    int32_t *list = counts + words;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    double *shared = reinterpret_cast<double *>(list + (p.pos ? (SOLO_TOKENS * p.k + 3) / 4 * 4 : 0)) + (size_t)warp * p.E;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) counts[e] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    const int used = tokens_used(p.used, p.T, p.status);
    const int t0 = blockIdx.x * p.chunk, t1 = min(t0 + p.chunk, p.T);
    const bool counted = p.counts || p.pos;
    for (int t = t0 + warp; t < t1; t += warps) {
        int id = -1;
        float w = 0.0f;
        if (t < used) {
            float z[V], m = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; i++) {
                const int e = i * 32 + lane;
                z[i] = -INFINITY;
                if (e < p.E)
                    z[i] = p.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[t * p.ldl + e])
                                  : static_cast<const float *>(p.logits)[t * p.ldl + e];
                if (isnan(z[i])) z[i] = -INFINITY;
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
            float zid = -INFINITY;
            bool close = false;
            choose<V, float>(p, z, m, sum, reinterpret_cast<float *>(shared), lane, id, zid, close);
            if (__any_sync(0xffffffffu, close)) {
                double sum64 = 1.0;
                if (!p.sigmoid && m > -INFINITY) {
                    sum64 = 0.0;
#pragma unroll 1
                    for (int i = 0; i < V; i++) {
                        float x = 0.0f;
#pragma unroll
                        for (int u = 0; u < V; u++)
                            if (u == i) x = z[u];
                        sum64 += exp((double)x - (double)m);
                    }
                    sum64 = warp_sum(sum64);
                }
                choose<V, double>(p, z, m, sum64, shared, lane, id, zid, close);
            }
            if (lane < p.k) w = p.sigmoid ? 1.0f / (1.0f + expf(-zid)) : m > -INFINITY ? expf(zid - m) / sum : 0.0f;
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
        if (warp != 0) return;
        const int total = scan(counts, p.E, lane);
        for (int e = lane; e < p.E; e += 32) p.offsets[e] = counts[e];
        if (lane == 0) p.offsets[p.E] = total;
        __syncwarp();
        place(list, (t1 - t0) * p.k, 0, p.k, counts, p.rows, p.pos, lane);
    } else {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.counts[(int64_t)blockIdx.x * p.E + e] = counts[e];
    }
}

// CTA c places the choices of chunk c.
__global__ void __launch_bounds__(256) plan_kernel(const int32_t *__restrict__ ids, const int32_t *__restrict__ counts,
                                                   int32_t *__restrict__ offsets, int32_t *__restrict__ rows,
                                                   int32_t *__restrict__ pos, int E, int k, int T, int chunk, int chunks) {
    extern __shared__ __align__(16) uint8_t smem[];
    int32_t *base = reinterpret_cast<int32_t *>(smem), *before = base + E;
    pdl_wait();
    pdl_launch_dependents();
    for (int e = threadIdx.x; e < E; e += 256) {
        int all = 0, mine = 0;
#pragma unroll 8
        for (int c = 0; c < chunks; c++) {
            const int v = counts[(int64_t)c * E + e];
            all += v;
            mine += c < (int)blockIdx.x ? v : 0;
        }
        base[e] = all;
        before[e] = mine;
    }
    __syncthreads();
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    const int total = scan(base, E, lane);
    for (int e = lane; e < E; e += 32) {
        if (blockIdx.x == 0) offsets[e] = base[e];
        base[e] += before[e];
    }
    if (blockIdx.x == 0 && lane == 0) offsets[E] = total;
    __syncwarp();
    const int64_t first = (int64_t)blockIdx.x * chunk * k;
    const int n = (min((int)(blockIdx.x + 1) * chunk, T) - (int)blockIdx.x * chunk) * k;
    place(ids + first, n, first, k, base, rows, pos, lane);
}

template <int V>
gq_status route_launch(RouteParams p, int chunks, size_t fixed, cudaStream_t s) {
    const size_t per_warp = p.top_groups < p.groups ? (size_t)p.E * 8 : 0;
    int warps = std::min(route_threads(V) / 32, p.chunk);
    if (per_warp) warps = std::max<int>(1, std::min<int64_t>(warps, (int64_t)((48 * 1024 - fixed) / per_warp)));
    warps = (p.chunk + (p.chunk + warps - 1) / warps - 1) / ((p.chunk + warps - 1) / warps);   // as many turns, no idle warps
    void *args[] = {&p};
    return launch_pdl((const void *)route_kernel<V>, dim3(chunks), dim3(32 * warps), fixed + warps * per_warp, s, args, "route launch");
}

}  // namespace

gq_status launch_route(const gq_router &r, const void *logits, int64_t ldl, bool bf16, const int32_t *used, int32_t *ids,
                       float *weights, int32_t *offsets, int32_t *rows, int32_t *pos, int64_t T, cudaStream_t s) {
    RouteParams p{};
    p.logits = logits, p.bias = r.bias, p.used = used, p.ids = ids, p.weights = weights, p.ldl = ldl;
    p.E = (int)r.E, p.k = (int)r.top_k, p.T = (int)T, p.sigmoid = r.score == GQ_SCORE_SIGMOID;
    p.groups = (int)r.groups, p.top_groups = (int)r.top_groups, p.group_best = (int)r.group_best;
    p.renormalize = r.renormalize != 0, p.bf16 = bf16, p.factor = r.factor;
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
    return launch_pdl((const void *)plan_kernel, dim3(chunks), dim3(256), (size_t)E * 8, s, args, "plan launch");
}

}  // namespace gq

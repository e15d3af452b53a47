// rowgroup.hip -- which rows go with which matrix: rows sorted by a group
// number (expert, adapter), and the top-k router that gives the numbers.
//
// Grouping is a stable counting sort of ids[rows] by id (ids outside
// [0, groups) are dropped), in chunks of consecutive rows:
//   count: per chunk, how many ids of each group (LDS, integer);
//   place: per chunk, base[g] = rows of smaller groups + rows of group g in
//          earlier chunks (every workgroup adds up all chunks' counts); then
//          blocks of ids in order.  Eight waves take consecutive ids each, 64
//          at a time: ids that are equal within the 64 find each other by
//          ballots over the id's bits, so a row's place is its wave's base +
//          earlier equal ids of the wave + equal lanes below.
// Sums of integers only: nothing depends on the order of the atomics.  Up to
// kGSingle rows are one chunk, counted inside the place kernel: one launch.
// The router counts its own choices (one launch less), and a decode step's
// few tokens are routed and placed by one workgroup, in one launch.
//
// Latency bounds all of this.  Measured (MI355X, kernel times): 16 tokens of
// 64 experts, top 8: 5.3 us in one launch (3.0 + 3.7 us as route and
// place); 8192 tokens of 128 experts, top 8: 8.3 + 5.0 us (6.2 + 3.2 + 14.0 us with a
// count kernel of its own and the counts added up one chunk after another).
#include "qg_launch.h"
#include "qg_rows.h"

namespace qg {

constexpr int kGThreads = 512;
constexpr int kGWaves = kGThreads / kWave;
constexpr int kGSingle = 2048;  // rows that one workgroup counts and places by itself

struct GroupParams {
    const int32_t* ids;
    int32_t rows, groups, chunk, chunks, bits;
    int32_t* offsets;
    int32_t* order;
    int32_t* pos;
    int32_t* counts;  // [chunks][groups], chunks > 1 only
};

__global__ __launch_bounds__(kGThreads) void group_count_kernel(GroupParams p) {
    __shared__ int hist[kMaxRowGroups];
    for (int g = threadIdx.x; g < p.groups; g += kGThreads) hist[g] = 0;
    lds_barrier();
    const int lo = blockIdx.x * p.chunk, hi = min(lo + p.chunk, p.rows);
    for (int i = lo + (int)threadIdx.x; i < hi; i += kGThreads) {
        const uint32_t id = (uint32_t)p.ids[i];
        if (id < (uint32_t)p.groups) atomicAdd(&hist[id], 1);
    }
    lds_barrier();
    for (int g = threadIdx.x; g < p.groups; g += kGThreads) p.counts[(int64_t)blockIdx.x * p.groups + g] = hist[g];
}

// Exclusive prefix of total[0..groups) into base (block-wide, 512 threads,
// two groups each); returns the sum.
__device__ __forceinline__ int scan_groups(const int* total, int* base, int groups, int* scratch) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = tid / kWave;
    const int g0 = 2 * tid;
    const int a = g0 < groups ? total[g0] : 0, b = g0 + 1 < groups ? total[g0 + 1] : 0;
    const int incl = wave_scan_incl(a + b);
    if (lane == kWave - 1) scratch[w] = incl;
    lds_barrier();
    int before = 0, all = 0;
    for (int q = 0; q < kGWaves; ++q) {
        if (q < w) before += scratch[q];
        all += scratch[q];
    }
    const int e = before + incl - (a + b);
    if (g0 < groups) base[g0] = e;
    if (g0 + 1 < groups) base[g0 + 1] = e + a;
    lds_barrier();
    return all;
}
static_assert(kMaxRowGroups == 2 * kGThreads, "two groups per thread");

// Places the ids [lo, hi): base[g] (LDS) is the next place of group g and is
// advanced; whist is [kGWaves][groups] of LDS.  S: steps of 64 ids per wave
// between two barriers.
template <int S, typename Ids>
__device__ __forceinline__ void place_ids(const GroupParams& p, const Ids& id_at, int lo, int hi, int* base, int* whist) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = tid / kWave;
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    for (int b0 = lo; b0 < hi; b0 += S * kGThreads) {
        int id[S], rank[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int i = b0 + (w * S + s) * kWave + lane;
            const int v = i < hi ? id_at(i) : -1;
            id[s] = (uint32_t)v < (uint32_t)p.groups ? v : -1;
        }
        for (int q = tid; q < kGWaves * p.groups; q += kGThreads) whist[q] = 0;
        lds_barrier();
        volatile int* mine = whist + w * p.groups;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const bool live = id[s] >= 0;
            uint64_t same = __ballot(live);
            for (int q = 0; q < p.bits; ++q) {
                const uint64_t one = __ballot((id[s] >> q) & 1);
                same &= ((id[s] >> q) & 1) ? one : ~one;
            }
            rank[s] = 0;
            if (live) {
                const int had = mine[id[s]];
                rank[s] = had + __popcll(same & below);
                // the last of the equal lanes writes the new count; every lane has read
                // the old one in the instruction before (one wave, in-order LDS)
                if ((same >> lane) == 1) mine[id[s]] = had + __popcll(same);
            }
        }
        lds_barrier();
        for (int g = tid; g < p.groups; g += kGThreads) {
            int run = base[g], c[kGWaves];
#pragma unroll
            for (int q = 0; q < kGWaves; ++q) c[q] = whist[q * p.groups + g];
#pragma unroll
            for (int q = 0; q < kGWaves; ++q) {
                whist[q * p.groups + g] = run;
                run += c[q];
            }
            base[g] = run;
        }
        lds_barrier();
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int i = b0 + (w * S + s) * kWave + lane;
            if (i < hi) {
                int at = -1;
                if (id[s] >= 0) {
                    at = whist[w * p.groups + id[s]] + rank[s];
                    p.order[at] = i;
                }
                p.pos[i] = at;
            }
        }
        lds_barrier();
    }
}

// All rows by one workgroup; total, base: [groups] of LDS.
template <typename Ids>
__device__ __forceinline__ void place_all(const GroupParams& p, const Ids& id_at, int* whist, int* base, int* total,
                                          int* scratch) {
    const int tid = threadIdx.x;
    for (int g = tid; g < p.groups; g += kGThreads) total[g] = 0;
    lds_barrier();
    for (int i = tid; i < p.rows; i += kGThreads) {
        const uint32_t id = (uint32_t)id_at(i);
        if (id < (uint32_t)p.groups) atomicAdd(&total[id], 1);
    }
    lds_barrier();
    const int all = scan_groups(total, base, p.groups, scratch);
    for (int g = tid; g < p.groups; g += kGThreads) p.offsets[g] = base[g];
    if (tid == 0) p.offsets[p.groups] = all;
    for (int i = all + tid; i < p.rows; i += kGThreads) p.order[i] = -1;
    lds_barrier();
    if (p.rows <= kGThreads) place_ids<1>(p, id_at, 0, p.rows, base, whist);
    else place_ids<4>(p, id_at, 0, p.rows, base, whist);
}

// total[g] and before[g] += the counts of all chunks and of those before this
// workgroup's: a thread adds W consecutive groups of every cs-th chunk.
template <int W>
__device__ __forceinline__ void sum_counts(const GroupParams& p, int* total, int* before) {
    typedef int vec __attribute__((ext_vector_type(W)));
    constexpr int U = 8;  // loads in flight
    const int units = p.groups / W, across = min(units, kGThreads), cs = kGThreads / across;
    const int c0 = (int)threadIdx.x / across;
    if (c0 >= cs) return;
    for (int u = (int)threadIdx.x % across; u < units; u += across) {
        const int32_t* at = p.counts + u * W;
        vec all = 0, mine = 0;
        for (int c = c0; c < p.chunks; c += U * cs) {
            vec v[U];
#pragma unroll
            for (int q = 0; q < U; ++q) v[q] = *reinterpret_cast<const vec*>(at + (int64_t)min(c + q * cs, p.chunks - 1) * p.groups);
#pragma unroll
            for (int q = 0; q < U; ++q) {
                if (c + q * cs < p.chunks) all += v[q];
                if (c + q * cs < (int)blockIdx.x) mine += v[q];
            }
        }
#pragma unroll
        for (int e = 0; e < W; ++e) {
            atomicAdd(&total[u * W + e], all[e]);
            atomicAdd(&before[u * W + e], mine[e]);
        }
    }
}

inline size_t group_lds(int groups) { return (size_t)(kGWaves + 2) * groups * sizeof(int); }

__global__ __launch_bounds__(kGThreads) void group_place_kernel(GroupParams p) {
    extern __shared__ int lds[];  // whist [kGWaves][groups] | base [groups] | total [groups]
    __shared__ int scratch[kGWaves];
    int* whist = lds;
    int* base = lds + kGWaves * p.groups;
    int* total = base + p.groups;
    const int tid = threadIdx.x;
    auto id_at = [&](int i) { return p.ids[i]; };
    if (p.chunks == 1) {
        place_all(p, id_at, whist, base, total, scratch);
        return;
    }
    // counts of all chunks, and of the chunks before this one (in whist, which
    // place_ids clears again)
    int* before = whist;
    for (int g = tid; g < p.groups; g += kGThreads) total[g] = before[g] = 0;
    lds_barrier();
    if (p.groups % 4 == 0) sum_counts<4>(p, total, before);
    else sum_counts<1>(p, total, before);
    lds_barrier();
    const int all = scan_groups(total, base, p.groups, scratch);
    if (blockIdx.x == 0) {
        for (int g = tid; g < p.groups; g += kGThreads) p.offsets[g] = base[g];
        if (tid == 0) p.offsets[p.groups] = all;
    }
    lds_barrier();
    for (int g = tid; g < p.groups; g += kGThreads) base[g] += before[g];
    const int lo = min((int)blockIdx.x * p.chunk, p.rows), hi = min(lo + p.chunk, p.rows);
    for (int i = max(all, lo) + tid; i < hi; i += kGThreads) p.order[i] = -1;
    lds_barrier();
    if (p.chunk <= kGThreads) place_ids<1>(p, id_at, lo, hi, base, whist);
    else place_ids<4>(p, id_at, lo, hi, base, whist);
}

// Chunks at most: every workgroup of the place kernel reads all their counts.
static int64_t max_chunks(int64_t groups) {
    const int64_t c = 32768 / groups;
    return c < 16 ? 16 : c > 256 ? 256 : c;
}
// Rows per chunk, a multiple of `unit`, at least `least`.
static void group_chunks(int64_t rows, int64_t groups, int64_t unit, int64_t least, int32_t* chunk, int32_t* chunks) {
    if (rows <= kGSingle) least = rows;
    int64_t per = (rows + max_chunks(groups) - 1) / max_chunks(groups);
    if (per < least) per = least;
    per = (per + unit - 1) / unit * unit;
    *chunk = (int32_t)per;
    *chunks = (int32_t)((rows + per - 1) / per);
}

size_t group_workspace(int64_t rows, int64_t groups) {
    return rows > kGSingle ? (size_t)max_chunks(groups) * (size_t)groups * sizeof(int32_t) : 0;
}

static GroupParams group_params(const GroupArgs& a) {
    GroupParams p;
    p.ids = a.ids;
    p.rows = (int32_t)a.rows;
    p.groups = a.groups;
    p.bits = 0;
    while ((1 << p.bits) < a.groups) ++p.bits;
    p.offsets = a.offsets;
    p.order = a.order;
    p.pos = a.pos;
    p.counts = static_cast<int32_t*>(a.ws);
    return p;
}

hipError_t launch_group_rows(const GroupArgs& a, hipStream_t st) {
    GroupParams p = group_params(a);
    group_chunks(a.rows, a.groups, 1, kGThreads, &p.chunk, &p.chunks);
    if (p.chunks > 1) group_count_kernel<<<p.chunks, kGThreads, 0, st>>>(p);
    group_place_kernel<<<p.chunks, kGThreads, group_lds(a.groups), st>>>(p);
    return hipGetLastError();
}

// ------------------------------------------------------------------ router
// One wave per token; lane l holds logits l, l + 64, ...  Each of the top_k
// rounds takes the largest key (an order-preserving integer of the fp32
// logit; 0: masked or already taken) over the wave and the lowest expert
// that holds it.  Softmax weights in fp32 around the largest logit.
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
    auto step = [&](int o) { v = max(v, (uint32_t)o); };
    step(dpp_mov<0xB1>((int)v));
    step(dpp_mov<0x4E>((int)v));
    step(dpp_mov<0x141>((int)v));
    step(dpp_mov<0x140>((int)v));
    step(dpp_mov<0x142, 0xA>((int)v));
    step(dpp_mov<0x143, 0xC>((int)v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum_all(float v) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wave_sum_to_lane63(v)), 63));
}
// ascending keys of fp32 values (equal values have equal keys: -0.0 as 0.0),
// 0 for -inf and NaN; +inf as the largest finite
__device__ __forceinline__ uint32_t logit_key(float f) {
    if (!(f > -__builtin_inff())) return 0u;
    if (f == 0.0f) return 0x80000000u;
    const uint32_t u = __float_as_uint(__builtin_fminf(f, 3.40282347e38f));
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

template <int XT, int NJ>
__device__ __forceinline__ void load_keys(const void* logits, int64_t t, int experts, uint32_t (&key)[NJ]) {
    const int lane = threadIdx.x & (kWave - 1);
    float l[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int64_t at = t * experts + min(lane + kWave * j, experts - 1);
        l[j] = XT == 0 ? static_cast<const float*>(logits)[at] : bf16_to_f32(static_cast<const uint16_t*>(logits)[at]);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) key[j] = lane + kWave * j < experts ? logit_key(l[j]) : 0u;
}

template <int NJ>
__device__ __forceinline__ void route_token(uint32_t (&key)[NJ], int top_k, bool renorm, int& my_id, float& my_w) {
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t best = key[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) best = max(best, key[j]);
    const uint32_t top = wave_umax(best);
    const float lmax = top ? key_logit(top) : 0.0f;
    float all = 0.0f;
    if (!renorm) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) all += key[j] ? expf(key_logit(key[j]) - lmax) : 0.0f;
        all = wave_sum_all(all);
    }
    my_id = -1;
    uint32_t my_key = 0, m = top;
    for (int r = 0; r < top_k; ++r) {
        if (r) {
            best = key[0];
#pragma unroll
            for (int j = 1; j < NJ; ++j) best = max(best, key[j]);
            m = wave_umax(best);
        }
        if (m == 0) break;
        bool found = false;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint64_t hit = __ballot(key[j] == m);
            if (!found && hit) {
                found = true;
                const int l = __builtin_ctzll(hit);
                if (lane == l) key[j] = 0;
                if (lane == r) {
                    my_id = l + kWave * j;
                    my_key = m;
                }
            }
        }
    }
    my_w = my_id >= 0 ? expf(key_logit(my_key) - lmax) : 0.0f;
    if (renorm) all = wave_sum_all(my_w);
    if (my_id >= 0) my_w = my_w / all;
}

constexpr int kRouteSmall = 64;  // tokens that one workgroup routes and places

struct RouteParams {
    const void* logits;
    int32_t tokens, top_k, renorm, per;  // per: tokens of a workgroup
    int32_t* ids;
    float* weights;
    GroupParams g;
};

// Tokens lo + w, lo + w + waves, ... below hi by wave w, the next one's logits
// requested before the choice; keep(pair, id) takes the choices.
template <int XT, int NJ, typename Keep>
__device__ __forceinline__ void route_tokens(const RouteParams& p, int lo, int hi, int waves, const Keep& keep) {
    const int lane = threadIdx.x & (kWave - 1);
    int t = lo + (int)threadIdx.x / kWave;
    if (t >= hi) return;
    uint32_t key[NJ];
    load_keys<XT, NJ>(p.logits, t, p.g.groups, key);
    for (;;) {
        const int next = t + waves;
        uint32_t ahead[NJ];
        load_keys<XT, NJ>(p.logits, min(next, hi - 1), p.g.groups, ahead);
        int id;
        float w;
        route_token<NJ>(key, p.top_k, p.renorm != 0, id, w);
        if (lane < p.top_k) {
            const int64_t at = (int64_t)t * p.top_k + lane;
            p.ids[at] = id;
            p.weights[at] = w;
            keep((int)at, id);
        }
        if (next >= hi) break;
        t = next;
#pragma unroll
        for (int j = 0; j < NJ; ++j) key[j] = ahead[j];
    }
}

// A chunk of tokens per workgroup, the choices counted (unless the place
// kernel's only workgroup counts them).
constexpr int kRWaves = 16, kRThreads = kRWaves * kWave;

template <int XT, int NJ>
__global__ __launch_bounds__(kRThreads) void route_kernel(RouteParams p) {
    __shared__ int hist[kMaxRowGroups];
    for (int g = threadIdx.x; g < p.g.groups; g += kRThreads) hist[g] = 0;
    lds_barrier();
    const int lo = (int)blockIdx.x * p.per, hi = min(lo + p.per, p.tokens);
    route_tokens<XT, NJ>(p, lo, hi, kRWaves, [&](int, int id) {
        if (id >= 0) atomicAdd(&hist[id], 1);
    });
    if (p.g.chunks == 1) return;
    lds_barrier();
    for (int g = threadIdx.x; g < p.g.groups; g += kRThreads)
        p.g.counts[(int64_t)blockIdx.x * p.g.groups + g] = hist[g];
}

// Few tokens: routed and placed by one workgroup.
template <int XT, int NJ>
__global__ __launch_bounds__(kGThreads) void route_small_kernel(RouteParams p) {
    extern __shared__ int lds[];
    __shared__ int scratch[kGWaves];
    __shared__ int ids[kGSingle];
    route_tokens<XT, NJ>(p, 0, p.tokens, kGWaves, [&](int at, int id) { ids[at] = id; });
    lds_barrier();
    int* base = lds + kGWaves * p.g.groups;
    place_all(p.g, [&](int i) { return ids[i]; }, lds, base, base + p.g.groups, scratch);
}

template <int XT, int NJ>
static void run_route(const RouteParams& p, hipStream_t st) {
    const size_t lds = group_lds(p.g.groups);
    if (p.per == 0) {
        route_small_kernel<XT, NJ><<<1, kGThreads, lds, st>>>(p);
    } else {
        route_kernel<XT, NJ><<<(p.tokens + p.per - 1) / p.per, kRThreads, 0, st>>>(p);
        group_place_kernel<<<p.g.chunks, kGThreads, lds, st>>>(p.g);
    }
}
template <int XT>
static void run_route(const RouteParams& p, hipStream_t st) {
    if (p.g.groups <= 64) run_route<XT, 1>(p, st);
    else if (p.g.groups <= 128) run_route<XT, 2>(p, st);
    else if (p.g.groups <= 256) run_route<XT, 4>(p, st);
    else run_route<XT, 16>(p, st);
}

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t st) {
    RouteParams p;
    p.logits = a.logits;
    p.tokens = (int32_t)a.tokens;
    p.top_k = a.top_k;
    p.renorm = a.renorm;
    p.ids = a.ids;
    p.weights = a.weights;
    p.g = group_params(a.group);
    // whole tokens per chunk, at least one per wave
    group_chunks(a.group.rows, a.group.groups, a.top_k, (int64_t)kRWaves * a.top_k, &p.g.chunk, &p.g.chunks);
    p.per = p.g.chunks > 1 ? p.g.chunk / a.top_k : a.tokens > kRouteSmall ? kRWaves : 0;
    if (a.xt == 0) run_route<0>(p, st);
    else run_route<1>(p, st);
    return hipGetLastError();
}

}  // namespace qg

// rowgroup.hip -- which rows go with which matrix: rows sorted by a group
// number (expert, adapter), and the top-k router that gives the numbers.
//
// Grouping is a stable counting sort of ids[rows] by id (ids outside
// [0, groups) are dropped), in chunks of up to 64 workgroups:
//   count: per chunk, how many ids of each group (LDS, integer);
//   place: per chunk, base[g] = rows of smaller groups + rows of group g in
//          earlier chunks; then blocks of 2048 ids in order.  Eight waves take
//          256 consecutive ids each, 64 at a time: ids that are equal within
//          the 64 find each other by ballots over the id's bits, so a row's
//          place is its wave's base + earlier equal ids of the wave + equal
//          lanes below.  Nothing depends on the order of atomics.
// A single chunk counts inside the place kernel: one launch.
#include "qg_launch.h"
#include "qg_rows.h"

namespace qg {

constexpr int kGThreads = 512;
constexpr int kGWaves = kGThreads / kWave;
constexpr int kGSteps = 4;                             // 64 ids per wave and step
constexpr int kGBlock = kGThreads * kGSteps;           // ids placed between two barriers
constexpr int kGMaxChunks = 64;

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
// advanced; whist is [kGWaves][groups] of LDS.
template <typename Ids>
__device__ __forceinline__ void place_ids(const GroupParams& p, const Ids& id_at, int lo, int hi, int* base, int* whist) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = tid / kWave;
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    for (int b0 = lo; b0 < hi; b0 += kGBlock) {
        for (int q = tid; q < kGWaves * p.groups; q += kGThreads) whist[q] = 0;
        lds_barrier();
        int id[kGSteps], rank[kGSteps];
        volatile int* mine = whist + w * p.groups;
#pragma unroll
        for (int s = 0; s < kGSteps; ++s) {
            const int i = b0 + (w * kGSteps + s) * kWave + lane;
            const int v = i < hi ? id_at(i) : -1;
            const bool live = (uint32_t)v < (uint32_t)p.groups;
            id[s] = live ? v : -1;
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
            int run = base[g];
            for (int q = 0; q < kGWaves; ++q) {
                const int c = whist[q * p.groups + g];
                whist[q * p.groups + g] = run;
                run += c;
            }
            base[g] = run;
        }
        lds_barrier();
#pragma unroll
        for (int s = 0; s < kGSteps; ++s) {
            const int i = b0 + (w * kGSteps + s) * kWave + lane;
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

__global__ __launch_bounds__(kGThreads) void group_place_kernel(GroupParams p) {
    extern __shared__ int lds[];  // whist [kGWaves][groups] | base [groups] | total [groups]
    __shared__ int scratch[kGWaves];
    int* whist = lds;
    int* base = lds + kGWaves * p.groups;
    int* total = base + p.groups;
    const int tid = threadIdx.x;
    const int lo = blockIdx.x * p.chunk, hi = min(lo + p.chunk, p.rows);
    if (p.chunks == 1) {
        for (int g = tid; g < p.groups; g += kGThreads) total[g] = 0;
        lds_barrier();
        for (int i = tid; i < p.rows; i += kGThreads) {
            const uint32_t id = (uint32_t)p.ids[i];
            if (id < (uint32_t)p.groups) atomicAdd(&total[id], 1);
        }
        lds_barrier();
        const int all = scan_groups(total, base, p.groups, scratch);
        for (int g = tid; g < p.groups; g += kGThreads) p.offsets[g] = base[g];
        if (tid == 0) p.offsets[p.groups] = all;
        for (int i = all + tid; i < p.rows; i += kGThreads) p.order[i] = -1;
    } else {
        for (int g = tid; g < p.groups; g += kGThreads) {
            int t = 0;
            for (int c = 0; c < p.chunks; ++c) t += p.counts[(int64_t)c * p.groups + g];
            total[g] = t;
        }
        lds_barrier();
        const int all = scan_groups(total, base, p.groups, scratch);
        if (blockIdx.x == 0) {
            for (int g = tid; g < p.groups; g += kGThreads) p.offsets[g] = base[g];
            if (tid == 0) p.offsets[p.groups] = all;
        }
        lds_barrier();
        for (int g = tid; g < p.groups; g += kGThreads) {
            int t = base[g];
            for (int c = 0; c < (int)blockIdx.x; ++c) t += p.counts[(int64_t)c * p.groups + g];
            base[g] = t;
        }
        for (int i = max(all, lo) + tid; i < hi; i += kGThreads) p.order[i] = -1;
        lds_barrier();
    }
    place_ids(p, [&](int i) { return p.ids[i]; }, lo, hi, base, whist);
}

static void group_chunks(int64_t rows, int32_t* chunk, int32_t* chunks) {
    const int64_t blocks = (rows + kGBlock - 1) / kGBlock;
    const int64_t per = (blocks + kGMaxChunks - 1) / kGMaxChunks;
    *chunk = (int32_t)(per * kGBlock);
    *chunks = (int32_t)((blocks + per - 1) / per);
}

size_t group_workspace(int64_t rows, int64_t groups) {
    int32_t chunk, chunks;
    group_chunks(rows, &chunk, &chunks);
    return chunks > 1 ? (size_t)chunks * (size_t)groups * sizeof(int32_t) : 0;
}

hipError_t launch_group_rows(const GroupArgs& a, hipStream_t st) {
    GroupParams p;
    p.ids = a.ids;
    p.rows = (int32_t)a.rows;
    p.groups = a.groups;
    group_chunks(a.rows, &p.chunk, &p.chunks);
    p.bits = 0;
    while ((1 << p.bits) < a.groups) ++p.bits;
    p.offsets = a.offsets;
    p.order = a.order;
    p.pos = a.pos;
    p.counts = static_cast<int32_t*>(a.ws);
    if (p.chunks > 1) group_count_kernel<<<p.chunks, kGThreads, 0, st>>>(p);
    const size_t lds = (size_t)(kGWaves + 2) * a.groups * sizeof(int);
    group_place_kernel<<<p.chunks, kGThreads, lds, st>>>(p);
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
__device__ __forceinline__ void route_token(const void* logits, int64_t t, int experts, int top_k, bool renorm,
                                            int& my_id, float& my_w) {
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t key[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = lane + kWave * j;
        key[j] = 0;
        if (e < experts) {
            const int64_t at = t * experts + e;
            key[j] = logit_key(XT == 0 ? static_cast<const float*>(logits)[at]
                                       : bf16_to_f32(static_cast<const uint16_t*>(logits)[at]));
        }
    }
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

struct RouteParams {
    const void* logits;
    int32_t tokens, experts, top_k, renorm;
    int32_t* ids;
    float* weights;
};

template <int XT, int NJ>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteParams p) {
    const int lane = threadIdx.x & (kWave - 1);
    const int t = blockIdx.x * kWaves + (int)threadIdx.x / kWave;
    if (t >= p.tokens) return;
    int id;
    float w;
    route_token<XT, NJ>(p.logits, t, p.experts, p.top_k, p.renorm != 0, id, w);
    if (lane < p.top_k) {
        p.ids[(int64_t)t * p.top_k + lane] = id;
        p.weights[(int64_t)t * p.top_k + lane] = w;
    }
}

template <int XT>
static void run_route(const RouteParams& p, hipStream_t st) {
    const int grid = (p.tokens + kWaves - 1) / kWaves;
    if (p.experts <= 64) route_kernel<XT, 1><<<grid, kThreads, 0, st>>>(p);
    else if (p.experts <= 128) route_kernel<XT, 2><<<grid, kThreads, 0, st>>>(p);
    else if (p.experts <= 256) route_kernel<XT, 4><<<grid, kThreads, 0, st>>>(p);
    else route_kernel<XT, 16><<<grid, kThreads, 0, st>>>(p);
}

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t st) {
    RouteParams p;
    p.logits = a.logits;
    p.tokens = (int32_t)a.tokens;
    p.experts = a.group.groups;
    p.top_k = a.top_k;
    p.renorm = a.renorm;
    p.ids = a.ids;
    p.weights = a.weights;
    if (a.xt == 0) run_route<0>(p, st);
    else run_route<1>(p, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_group_rows(a.group, st);
}

}  // namespace qg

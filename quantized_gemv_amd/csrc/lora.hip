// lora.hip -- low-rank adapters of many requests beside a shared projection:
//   y[t] += scale[g] B[g] (A[g] x[t]),  g the adapter of row t,
// for up to 8 matrices that read the same x (q, k, v; gate, up).
//
// Two launches.  shrink: v = A x; a workgroup takes 16 sorted rows (32 where the
// groups have that many: A is read half as often; two of 2048 x 2048, rank 128,
// 2048 rows: 57 -> 54 us) of one adapter, one part of k and one matrix, on
// v_mfma_f32_16x16x32_bf16 (exact products, fp32 sums), and stores its fp32
// partial sums [part][row][rank]; few rows would leave most CUs idle without
// the parts.  expand: the parts
// are added in order, scaled and split into three bf16 terms (hi + mid + lo,
// 24 bits: nothing of the fp32 value is lost), so that the product with B
// runs on the same matrix instructions; y is read, added to and written once.
//
// Few rows: the latency of two dependent launches (16 rows, rank 16, 4096 x
// 4096: 4.2 + 4.4 us).  Many: reading and writing y (4129 rows of 11008 fp32, a
// tenth of them without an adapter, rank 64: 72 us for 327 MB, 4.5 TB/s, after
// 17 us of shrink).
#include "qg_launch.h"
#include "qg_rows.h"

namespace qg {

typedef __bf16 lbf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kLMaxParts = 8;

struct LoraMatP {
    const uint16_t* a;
    const uint16_t* b;
    const float* scale;
    void* y;
    int32_t n, r;
    int64_t ws_at;  // floats: this matrix's partial sums [parts][rows][rpad]
};
struct LoraParams {
    LoraMatP m[kMaxGroupLaunch];
    const uint16_t* x;
    const int32_t* offsets;
    const int32_t* order;
    float* ws;
    int32_t count, groups, rows, x_rows, k, parts;
    int32_t rgroups;               // shrink: rank groups (the largest rank's)
    int32_t strips, strip_blocks;  // expand: strips of columns (the widest matrix's), blocks per strip
    int64_t block0;
};

// ------------------------------------------------------------------ shrink
// Eight waves share the part's k of up to four 16-row tiles of A (ranks 64 rg
// .. + 63, RT tiles); their sums meet in LDS.
constexpr int kSWaves = 8;
constexpr int kSThreads = kSWaves * kWave;
constexpr int kSRanks = 64;  // ranks of a workgroup

template <int RM, int RT>
__device__ __forceinline__ void shrink_tile(const LoraParams& p, const LoraMatP& m, const RowTile& t, int kpart, int rg,
                                            f32x4 (&red)[kSWaves][RM * 4][kWave]) {
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int share = kpart * kSWaves + wave, shares = p.parts * kSWaves;
    const int units = p.k / 32;
    const int c0 = (int)((int64_t)units * share / shares), c1 = (int)((int64_t)units * (share + 1) / shares);
    const uint16_t* x[RM];
    const uint16_t* a[RT];
    f32x4 acc[RM][RT];
#pragma unroll
    for (int s = 0; s < RM; ++s) {
        const int src = min(max(p.order[t.row0 + min(16 * s + i, t.rows - 1)], 0), p.x_rows - 1);
        x[s] = p.x + (int64_t)src * p.k + 8 * g;
#pragma unroll
        for (int q = 0; q < RT; ++q) acc[s][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int q = 0; q < RT; ++q)
        a[q] = m.a + ((int64_t)t.group * m.r + min(kSRanks * rg + 16 * q + i, m.r - 1)) * p.k + 8 * g;
    // the loads of several steps are requested together
    auto batch = [&](int c, auto steps) {
        constexpr int U = decltype(steps)::value;
        u32x4 xf[U][RM], af[U][RT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int s = 0; s < RM; ++s) xf[u][s] = *reinterpret_cast<const u32x4*>(x[s] + (c + u) * 32);
#pragma unroll
            for (int q = 0; q < RT; ++q) af[u][q] = *reinterpret_cast<const u32x4*>(a[q] + (c + u) * 32);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < RM; ++s)
#pragma unroll
                for (int q = 0; q < RT; ++q)
                    acc[s][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(lbf16x8, af[u][q]),
                                                                        __builtin_bit_cast(lbf16x8, xf[u][s]), acc[s][q], 0, 0, 0);
    };
    constexpr int U = RT == 4 ? 4 : 8;
    int c = c0;
    for (; c + U <= c1; c += U) batch(c, std::integral_constant<int, U>());
    for (; c + 2 <= c1; c += 2) batch(c, std::integral_constant<int, 2>());
    if (c < c1) batch(c, std::integral_constant<int, 1>());
#pragma unroll
    for (int s = 0; s < RM; ++s)
#pragma unroll
        for (int q = 0; q < RT; ++q) red[wave][s * RT + q][lane] = acc[s][q];
    lds_barrier();
    // wave w finishes row tile w / RT, rank tile w % RT
    const int rpad = (m.r + 15) / 16 * 16;
    const int row = 16 * (wave / RT) + i, rank = kSRanks * rg + 16 * (wave % RT);
    if (wave < RM * RT && rank < rpad) {
        f32x4 s = red[0][wave][lane];
#pragma unroll
        for (int w = 1; w < kSWaves; ++w) s += red[w][wave][lane];
        // lane l: sorted row l % 16 of the tile, ranks 4 (l / 16) + r of the tile
        if (row < t.rows)
            *reinterpret_cast<f32x4*>(p.ws + m.ws_at + ((int64_t)kpart * p.rows + t.row0 + row) * rpad + rank + 4 * g) = s;
    }
}

template <int RM>
__global__ __launch_bounds__(kSThreads) void lora_shrink_kernel(LoraParams p) {
    static_assert(RM * 4 <= kSWaves, "a wave per tile at the end");
    __shared__ f32x4 red[kSWaves][RM * 4][kWave];
    const GroupOffsets groups = request_groups(p.offsets, p.groups, 0);
    int64_t block = p.block0 + blockIdx.x;
    const int mi = (int)(block % p.count);
    block /= p.count;
    const int rg = (int)(block % p.rgroups);
    block /= p.rgroups;
    const LoraMatP& m = p.m[mi];
    const int ranks = m.r - kSRanks * rg;
    const int kpart = (int)(block % p.parts);
    const RowTile t = find_row_tile<16 * RM>(p.offsets, p.groups, p.rows, (int)(block / p.parts), group_tiles<16 * RM>(groups, p.rows, 0));
    if (t.rows <= 0 || ranks <= 0) return;
    if (ranks <= 16) shrink_tile<RM, 1>(p, m, t, kpart, rg, red);
    else if (ranks <= 32) shrink_tile<RM, 2>(p, m, t, kpart, rg, red);
    else shrink_tile<RM, 4>(p, m, t, kpart, rg, red);
}

// ------------------------------------------------------------------ expand
// A workgroup takes 16 MT sorted rows of one adapter and a strip of blocks of
// 64 CT columns of one matrix, each of its four waves all the rows and 16 CT
// columns of a block.  v is summed, scaled and split once per strip; the old y
// and B of a block are requested one block ahead; the products go through
// LDS so that y is read and written in whole rows of 64 CT columns.
constexpr int kXThreads = 256;

// y of many rows is read and written once: non-temporal (5% at 4129 x 11008).
// The few rows of a decode step stay in the caches for the next kernel.
template <bool NT, typename T>
__device__ __forceinline__ T load_y(const T* p) {
    return NT ? __builtin_nontemporal_load(p) : *p;
}
template <bool NT, typename T>
__device__ __forceinline__ void write_y(T v, T* p) {
    if constexpr (NT) __builtin_nontemporal_store(v, p);
    else *p = v;
}
// Four columns of y, aligned to their elements only (rows of any length start
// anywhere): one load or store all the same, the memory system takes them.
typedef float y4f __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t y4h __attribute__((ext_vector_type(2), aligned(2)));

template <int YT, int MT, int KC, int CT>
__global__ __launch_bounds__(kXThreads, MT == 1 ? 4 : 3) void lora_expand_kernel(LoraParams p) {
    constexpr int R = 16 * MT;                  // rows
    constexpr int KG = 4 * KC;                  // k groups of 8
    constexpr int kXCols = 64 * CT, kXLine = kXCols + 4;  // 4 floats longer: no bank conflicts
    constexpr int TPR = kXCols / 4;             // threads per row of y, 4 columns each
    constexpr int RPP = kXThreads / TPR;        // rows per pass of the workgroup
    constexpr int YR = R / RPP;                 // passes
    __shared__ u32x4 vsh[3 * KG * R];           // v: [term][k group of 8][row]
    __shared__ __attribute__((aligned(16))) float dsh[R * kXLine];
    const GroupOffsets groups = request_groups(p.offsets, p.groups, 0);
    const int64_t block = p.block0 + blockIdx.x;
    const int strip = (int)(block % p.strips), mi = (int)(block / p.strips % p.count);
    const LoraMatP& m = p.m[mi];
    const int n = m.n, r = m.r;
    const int nb1 = min((strip + 1) * p.strip_blocks, (n + kXCols - 1) / kXCols);
    int nb = strip * p.strip_blocks;
    const RowTile t = find_row_tile<R>(p.offsets, p.groups, p.rows, (int)(block / p.strips / p.count), group_tiles<R>(groups, p.rows, 0));
    if (t.rows <= 0 || nb >= nb1) return;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;

    typedef typename std::conditional<YT == 0, y4f, y4h>::type y_t;
    struct Block {
        u32x4 b[CT][KC];
        y_t y[YR];
    };
    // y: thread (row tid / TPR + RPP s, four columns from 4 (tid % TPR), at the
    // row's end its last four).  Every load is made, rows and columns past the
    // ends repeat others and are not stored: loads under branches would be
    // waited for one by one.
    const int ycol = 4 * (tid % TPR);
    int64_t yat[YR];
    int src[YR];
    uint32_t live = 0;
#pragma unroll
    for (int s = 0; s < YR; ++s) src[s] = p.order[t.row0 + min(tid / TPR + RPP * s, t.rows - 1)];
    __builtin_amdgcn_sched_barrier(0);  // all requested before one is used
#pragma unroll
    for (int s = 0; s < YR; ++s) {
        const bool in = src[s] >= 0 && src[s] < p.x_rows;
        live |= in && tid / TPR + RPP * s < t.rows ? 1u << s : 0u;
        yat[s] = in ? (int64_t)src[s] * n : 0;
    }
    auto load = [&](int block_n, Block& k) {
        const int n0 = block_n * kXCols;
        // B: lane (i, g) holds column i of a 16-column tile, ranks 8 (4 c + g) ..
        // + 7; past the rank the first ones again, against zeros of v
#pragma unroll
        for (int q = 0; q < CT; ++q) {
            const uint16_t* b = m.b + ((int64_t)t.group * n + min(n0 + 16 * (wave * CT + q) + i, n - 1)) * r;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const int at = (4 * c + g) * 8;
                k.b[q][c] = *reinterpret_cast<const u32x4*>(b + (at < r ? at : 0));
            }
        }
        const int at = min(n0 + ycol, n - 4);
#pragma unroll
        for (int s = 0; s < YR; ++s) {
            if constexpr (YT == 0) k.y[s] = load_y<MT != 1>(reinterpret_cast<const y_t*>(static_cast<const float*>(m.y) + yat[s] + at));
            else k.y[s] = load_y<MT != 1>(reinterpret_cast<const y_t*>(static_cast<const uint16_t*>(m.y) + yat[s] + at));
        }
    };
    auto finish = [&](int block_n, const Block& k) {
        const int n0 = block_n * kXCols;
        f32x4 acc[MT][CT];
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int q = 0; q < CT; ++q) acc[a][q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int w = 0; w < 3; ++w)
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    const lbf16x8 v = __builtin_bit_cast(lbf16x8, vsh[(w * KG + 4 * c + g) * R + 16 * a + i]);
#pragma unroll
                    for (int q = 0; q < CT; ++q)
                        acc[a][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(lbf16x8, k.b[q][c]), v, acc[a][q], 0, 0, 0);
                }
        // lane l holds row 16 a + l % 16, columns 16 (CT wave + q) + 4 (l / 16) + r
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int q = 0; q < CT; ++q)
                *reinterpret_cast<f32x4*>(dsh + (16 * a + i) * kXLine + 16 * (wave * CT + q) + 4 * g) = acc[a][q];
        lds_barrier();
        const int at = min(n0 + ycol, n - 4), skip = n0 + ycol - at;  // 4 and more: a piece past the end
#pragma unroll
        for (int s = 0; s < YR; ++s) {
            // the columns' products (those of a shifted piece start earlier, or in
            // the block before: not stored)
            const float* line = dsh + (tid / TPR + RPP * s) * kXLine;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float d = skip == 0 ? line[ycol + e] : line[max(at - n0 + e, 0)];
                if constexpr (YT == 0) v[e] = k.y[s][e] + d;
                else v[e] = ((e & 1) ? __uint_as_float(k.y[s][e >> 1] & 0xFFFF0000u) : bf16_to_f32(k.y[s][e >> 1] & 0xFFFFu)) + d;
            }
            if (!((live >> s) & 1)) continue;
            if (skip == 0) {
                if constexpr (YT == 0) {
                    const y_t o = {v[0], v[1], v[2], v[3]};
                    write_y<MT != 1>(o, reinterpret_cast<y_t*>(static_cast<float*>(m.y) + yat[s] + at));
                } else {
                    const y_t o = {any_f32_to_bf16(v[0]) | (any_f32_to_bf16(v[1]) << 16), any_f32_to_bf16(v[2]) | (any_f32_to_bf16(v[3]) << 16)};
                    write_y<MT != 1>(o, reinterpret_cast<y_t*>(static_cast<uint16_t*>(m.y) + yat[s] + at));
                }
            } else {
#pragma unroll
                for (int e = 1; e < 4; ++e) {
                    if (e >= skip) {
                        if constexpr (YT == 0) static_cast<float*>(m.y)[yat[s] + at + e] = v[e];
                        else static_cast<uint16_t*>(m.y)[yat[s] + at + e] = (uint16_t)any_f32_to_bf16(v[e]);
                    }
                }
            }
        }
        lds_barrier();  // dsh is written again by the next block
    };

    Block ka, kb;
    load(nb, ka);
    __builtin_amdgcn_sched_barrier(0);
    // v: the parts in order, scaled, as hi + mid + lo bf16 (24 bits), rows and
    // ranks past the ends zero
    const int rpad = (r + 15) / 16 * 16;
    const float scale = m.scale ? m.scale[t.group] : 1.0f;
    uint2* vh = reinterpret_cast<uint2*>(vsh);
#pragma unroll
    for (int q0 = 0; q0 < R * KC * 8; q0 += kXThreads) {
        const int q = q0 + tid;
        if (R * KC * 8 % kXThreads != 0 && q >= R * KC * 8) break;
        const int j4 = q % (KC * 8), row = q / (KC * 8);
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (4 * j4 < r && row < t.rows) {
            const float* at = p.ws + m.ws_at + (int64_t)(t.row0 + row) * rpad + 4 * j4;
            const int64_t step = (int64_t)p.rows * rpad;
            auto add = [&](auto most) {  // up to that many parts, requested together
                f32x4 part[decltype(most)::value];
#pragma unroll
                for (int s = 0; s < most; ++s) part[s] = *reinterpret_cast<const f32x4*>(at + min(s, p.parts - 1) * step);
                v = part[0];
#pragma unroll
                for (int s = 1; s < most; ++s) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] += s < p.parts ? part[s][e] : 0.0f;  // under a branch the loads would follow
                }
            };
            if (p.parts <= 2) add(std::integral_constant<int, 2>());
            else add(std::integral_constant<int, kLMaxParts>());
        }
        uint32_t term[3][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float f = v[e] * scale;
            term[0][e] = any_f32_to_bf16(f);  // NaN here is enough for the sum
            const float f1 = f - bf16_to_f32(term[0][e]);
            term[1][e] = f32_to_bf16(f1);
            term[2][e] = f32_to_bf16(f1 - bf16_to_f32(term[1][e]));
        }
#pragma unroll
        for (int w = 0; w < 3; ++w)
            vh[((w * KG + (j4 >> 1)) * R + row) * 2 + (j4 & 1)] =
                make_uint2(term[w][0] | (term[w][1] << 16), term[w][2] | (term[w][3] << 16));
    }
    lds_barrier();
    for (;;) {
        if (nb + 1 < nb1) load(nb + 1, kb);
        __builtin_amdgcn_sched_barrier(0);
        finish(nb, ka);
        if (++nb >= nb1) break;
        if (nb + 1 < nb1) load(nb + 1, ka);
        __builtin_amdgcn_sched_barrier(0);
        finish(nb, kb);
        if (++nb >= nb1) break;
    }
}

// 32 rows per workgroup where the groups have that many.  The host knows the
// groups there are, not those in use: 4096 rows of 12 adapters, rank 64, 4096 x
// 11008, take 147 us with 256 loaded (119 with 32 rows) and 105 with those 12; of
// rank 16, 4096 x 4096, with 1024 loaded 66 (32 rows: 82) and 43.
static bool tall_groups(int64_t rows, int64_t groups) { return rows >= 32 * groups; }
static int shrink_rows(int64_t rows, int64_t groups) { return tall_groups(rows, groups) ? 32 : 16; }

// Parts of k of the shrink: enough workgroups to fill the CUs, and a
// workgroup's own time kept short: 2048 of k at most (us with the expand, one
// part for all of k and this: 4129 rows, 8192 x 4096, rank 64: 81, 75; 700 rows
// of 100 adapters, two of 8192 x 1024: 24, 17; at 1024 of k 84 and 21).
static int lora_parts(int64_t rows, int64_t groups, int64_t k, int count, int rmax) {
    const int64_t blocks = max_row_tiles(rows, groups, shrink_rows(rows, groups)) * count * ((rmax + kSRanks - 1) / kSRanks);
    int64_t parts = (256 + blocks - 1) / blocks;
    if (parts < (k + 2047) / 2048) parts = (k + 2047) / 2048;
    const int64_t most = k / 32 / kSWaves;  // a matrix instruction per wave at least
    if (parts > most) parts = most;
    if (parts > kLMaxParts) parts = kLMaxParts;
    return (int)(parts < 1 ? 1 : parts);
}

size_t lora_workspace(int64_t rows, int64_t groups, int64_t k, int count, int rmax, int64_t padded_rank) {
    return (size_t)lora_parts(rows, groups, k, count, rmax) * (size_t)rows * (size_t)padded_rank * sizeof(float);
}

template <int YT, int MT, int KC, int CT>
static hipError_t run_expand(LoraParams& p, int64_t widest, hipStream_t st) {
    const int64_t blocks = (widest + 64 * CT - 1) / (64 * CT), tiles = max_row_tiles(p.rows, p.groups, 16 * MT) * p.count;
    // Strips as long as they can be with enough workgroups left (us with the
    // shrink, at 512, 1024, 2048, 4096, 8192 workgroups.  16 rows: 48 rows of 11008,
    // rank 16, 11.5 9.9 10.7 10.1 10.5; three of 500 x 4096, rank 32, 29 26 24 25 25;
    // 32 rows: three of 4096 x 4096, rank 16, 132 112 110 101 101; 1500 x 14336, rank
    // 32, 51 49 43 46 46; two of 2048 x 2048, rank 128, 50 51 53 53 53).
    int64_t per = blocks * tiles / (MT == 1 ? 1024 : 4096);
    per = per < 1 ? 1 : per > blocks ? blocks : per;
    p.strip_blocks = (int32_t)per;
    p.strips = (int32_t)((blocks + per - 1) / per);
    return launch_blocks(tiles * p.strips, kXThreads, [&](uint32_t grid, int64_t block0) {
        p.block0 = block0;
        lora_expand_kernel<YT, MT, KC, CT><<<grid, kXThreads, 0, st>>>(p);
    });
}
template <int YT>
static hipError_t launch_expand(LoraParams& p, int rmax, int64_t widest, hipStream_t st) {
    const bool tall = tall_groups(p.rows, p.groups);
    if (rmax <= 32) return tall ? run_expand<YT, 2, 1, 2>(p, widest, st) : run_expand<YT, 1, 1, 4>(p, widest, st);
    if (rmax <= 64) return tall ? run_expand<YT, 2, 2, 2>(p, widest, st) : run_expand<YT, 1, 2, 2>(p, widest, st);
    if (rmax <= 128) return tall ? run_expand<YT, 2, 4, 2>(p, widest, st) : run_expand<YT, 1, 4, 2>(p, widest, st);
    return tall ? run_expand<YT, 2, 8, 1>(p, widest, st) : run_expand<YT, 1, 8, 1>(p, widest, st);
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t st) {
    LoraParams p;
    p.x = a.x;
    p.offsets = a.offsets;
    p.order = a.order;
    p.ws = static_cast<float*>(a.ws);
    p.count = a.count;
    p.groups = a.groups;
    p.rows = (int32_t)a.rows;
    p.x_rows = (int32_t)a.x_rows;
    p.k = (int32_t)a.k;
    int64_t at = 0, widest = 0;
    int rmax = 0;
    for (int j = 0; j < a.count; ++j)
        if (a.m[j].r > rmax) rmax = a.m[j].r;
    p.parts = lora_parts(a.rows, a.groups, a.k, a.count, rmax);
    p.rgroups = (rmax + kSRanks - 1) / kSRanks;
    for (int j = 0; j < a.count; ++j) {
        const LoraMat& m = a.m[j];
        p.m[j] = {m.a, m.b, m.scale, m.y, (int32_t)m.n, m.r, at};
        at += (int64_t)p.parts * a.rows * ((m.r + 15) / 16 * 16);
        if (m.n > widest) widest = m.n;
    }
    const int tile = shrink_rows(a.rows, a.groups);
    const hipError_t e = launch_blocks(max_row_tiles(a.rows, a.groups, tile) * p.parts * p.rgroups * p.count, kSThreads,
                                       [&](uint32_t grid, int64_t block0) {
                                           p.block0 = block0;
                                           if (tile == 32) lora_shrink_kernel<2><<<grid, kSThreads, 0, st>>>(p);
                                           else lora_shrink_kernel<1><<<grid, kSThreads, 0, st>>>(p);
                                       });
    if (e != hipSuccess) return e;
    return a.yt == 0 ? launch_expand<0>(p, rmax, widest, st) : launch_expand<1>(p, rmax, widest, st);
}

}  // namespace qg

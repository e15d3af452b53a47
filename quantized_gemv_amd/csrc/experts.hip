// experts.hip -- int8 products grouped by expert, with ragged row counts.
//
// Rows i of the plan are sorted by expert; expert e holds rows offsets[e] ..
// offsets[e + 1] - 1, and
//   y[i][n] = (sum_k codes[e][n][k] x[src(i)][k]) / s_w[e][n]             (W8A16)
//   y[i][n] = (sum_k codes[e][n][k] xq[src(i)][k]) / (s_w[e][n] s_x[src]) (W8A8)
// with src(i) = order[i] / per_row.  SwiGLU launches compute a gate and an up
// product per output and store gate / (1 + exp(-gate)) * up.
#include "qg_gemm.h"
#include "qg_rows.h"

namespace qg {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kEUnit = 64;  // k per unit: 4 lane groups x 16 codes
constexpr int kEThreads = 256;
constexpr int kEWaves = kEThreads / kWave;

struct ExpertParams {
    const int8_t* codes[2];   // gate, up (or one matrix)
    const float* scale[2];
    const void* x;
    const float* s_x;
    const int32_t* offsets;
    const int32_t* order;
    void* y;
    int64_t expert_bytes;     // one expert's codes
    int32_t e, n, k, rows, x_rows;
    RowDiv per_row;
    int32_t tiled;            // 16-row tiled codes (else row-major); a 16-row tile is 16 k bytes in both
    int64_t block0;           // workgroups of earlier launches of the same product
    int32_t ntiles;           // workgroup tiles along n
};

// 16 int8 codes -> two bf16x8 (codes 0-7, 8-15), exact: fp32 by integer
// conversion, the upper halves of two fp32 values form a bf16 pair
__device__ __forceinline__ void codes_to_bf16(const u32x4& w, bf16x8& a0, bf16x8& a1) {
    uint32_t h[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t v = w[d];
        const float f0 = (float)(int)(int8_t)(v & 0xFFu);
        const float f1 = (float)(int)(int8_t)((v >> 8) & 0xFFu);
        const float f2 = (float)(int)(int8_t)((v >> 16) & 0xFFu);
        const float f3 = (float)(int)(int8_t)(v >> 24);
        h[2 * d] = __builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u);
        h[2 * d + 1] = __builtin_amdgcn_perm(__float_as_uint(f3), __float_as_uint(f2), 0x07060302u);
    }
    a0 = __builtin_bit_cast(bf16x8, u32x4{h[0], h[1], h[2], h[3]});
    a1 = __builtin_bit_cast(bf16x8, u32x4{h[4], h[5], h[6], h[7]});
}

__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + expf(-g)) * u; }

template <int YT>
__device__ __forceinline__ void store_y(void* y, int64_t at, float v) {
    if constexpr (YT == 0) static_cast<float*>(y)[at] = v;
    else static_cast<uint16_t*>(y)[at] = (uint16_t)any_f32_to_bf16(v);
}

// ------------------------------------------------------------------ streams
// Few rows per expert: the time goes into reading the chosen experts' codes.
// A workgroup multiplies sixteen sorted rows of one expert with 32 matrix
// rows (GLU: 16 of the gate and the same 16 of the up matrix); each of its
// four waves takes a quarter of k, two 16 x 16 tiles of
// v_mfma_f32_16x16x32_bf16 (or v_mfma_i32_16x16x64_i8) that share the x
// fragments, and their sums meet in LDS in order.  Tiled codes: two units of
// 64 k are on their way while one is multiplied, and the first codes are
// requested before the rows of x are known.  Codes are read in whole 128-byte lines
// (row-major: a pair of units at a time; tiled: blocks of 1 KB), once each:
// non-temporal.
//
// HBM bounds it.  Small workgroups with little in registers keep the most of
// them on a CU, so that one's start (tile search, row numbers) and end hide
// behind the others' loads.  Waves per workgroup x tiles per wave x units per
// step, us of four calls with few rows (180, 199, 100 and 88 MB of codes of the
// chosen experts):
// 4 x 2 x 1: 32.5, 32.8, 24.6, 25.0; 4 x 4 x 2: 34.1, 36.3, 26.1, 25.0;
// 8 x 4 x 2: 35.7, 45.0, 30.9, 29.2; 2 x 2 x 1: 33.9, 33.0, 25.0, 26.1.
// Row-major codes, two loads of 16 bytes per lane that read whole 128-byte
// lines: r1 holds row l % 8, r2 row 8 + l % 8, both chunk l / 8 of the line's
// eight.  The matrix instructions want row l % 16 and one chunk for all rows:
// lanes 8 apart exchange halves, after which r1 holds chunk 2 (l / 16) of row
// l % 16 and r2 the chunk after it.
__device__ __forceinline__ void line_halves(u32x4& r1, u32x4& r2) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int a = (int)r1[d], b = (int)r2[d];
        r1[d] = (uint32_t)__builtin_amdgcn_update_dpp(a, b, 0x128, 0xF, 0xC, false);  // row_ror:8 into lanes 8-15
        r2[d] = (uint32_t)__builtin_amdgcn_update_dpp(b, a, 0x128, 0xF, 0x3, false);  // and into lanes 0-7
    }
}

template <int ACT, int YT, bool GLU, bool TILED>
__global__ __launch_bounds__(kEThreads, 5) void experts_stream_kernel(ExpertParams p) {
    constexpr int NT = 2;
    constexpr int OT = GLU ? 1 : NT;      // 16-row output tiles
    constexpr int U = TILED ? 1 : 2;      // units loaded together: row-major lines hold two
    // sets of registers, D - 1 of them on their way while one is multiplied
    // (row-major: one set, loaded and multiplied, and more waves instead)
    constexpr int D = TILED ? 3 : 1;
    constexpr int XF = ACT == 0 ? 2 : 1;  // x loads per unit and 16 rows
    typedef typename std::conditional<ACT == 0, f32x4, i32x4>::type acc_t;
    __shared__ acc_t part[kEWaves][NT][kWave];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;  // weight row / x row, k group
    const GroupOffsets groups = request_groups(p.offsets, p.e, 0);
    const int64_t block = p.block0 + blockIdx.x;
    const int ot0 = (int)(block % p.ntiles) * OT;  // first 16-row output tile
    const RowTile t = find_row_tile<16>(p.offsets, p.e, p.rows, (int)(block / p.ntiles), group_tiles<16>(groups, p.rows, 0));
    if (t.rows <= 0) return;  // uniform over the workgroup

    const int pairs = p.k / (2 * kEUnit);
    const int c0 = 2 * (pairs * wave / kEWaves), c1 = 2 * (pairs * (wave + 1) / kEWaves);
    __amdgpu_buffer_rsrc_t rw[NT];
    uint32_t woff[NT][U];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        // rows past n: row-major codes repeat the last row; tiled codes are
        // padded to whole tiles; tiles past the last repeat it
        const int ot = min(ot0 + q % OT, (p.n - 1) / 16);
        rw[q] = make_rsrc(p.codes[GLU ? q : 0] + (int64_t)t.group * p.expert_bytes + (int64_t)ot * 16 * p.k,
                          (uint32_t)(16 * p.k));
#pragma unroll
        for (int u = 0; u < U; ++u)
            woff[q][u] = TILED ? (uint32_t)(lane * 16)
                               : (uint32_t)(min((lane & 7) + 8 * u, p.n - 1 - 16 * ot) * p.k + (lane >> 3) * 16);
    }
    struct Units {
        u32x4 w[NT][U], x[U][XF];
    };
    auto load_w = [&](int c, Units& s) {
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int u = 0; u < U; ++u)
                s.w[q][u] = __builtin_amdgcn_raw_buffer_load_b128(rw[q], woff[q][u], c * (TILED ? 1024 : 64), kCachePolicyNT);
    };
    Units s[D];
    if (D > 1 && c0 < c1) load_w(c0, s[0]);
    __builtin_amdgcn_sched_barrier(0);
    // this lane's x row (rows past the tile repeat its last)
    constexpr int kX = ACT == 0 ? 2 : 1;  // bytes of an x value
    const int at = t.row0 + min(i, t.rows - 1);
    const int src = min(p.order ? divide(max(p.order[at], 0), p.per_row) : at, p.x_rows - 1);
    const uint8_t* xrow = static_cast<const uint8_t*>(p.x) + (int64_t)src * p.k * kX + 16 * U * kX * g;
    auto load_x = [&](int c, Units& s) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int f = 0; f < XF; ++f)
                s.x[u][f] = *reinterpret_cast<const u32x4*>(xrow + (int64_t)c * (64 * kX) + 16 * (u * kX + f));
    };
    acc_t acc[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) acc[q] = acc_t{0, 0, 0, 0};
    auto multiply = [&](Units& s) {
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            if constexpr (!TILED) line_halves(s.w[q][0], s.w[q][1]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if constexpr (ACT == 0) {
                    bf16x8 w0, w1;
                    codes_to_bf16(s.w[q][u], w0, w1);
                    acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, __builtin_bit_cast(bf16x8, s.x[u][0]), acc[q], 0, 0, 0);
                    acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, __builtin_bit_cast(bf16x8, s.x[u][XF - 1]), acc[q], 0, 0, 0);
                } else {
                    acc[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, s.w[q][u]),
                                                                   __builtin_bit_cast(i32x4, s.x[u][0]), acc[q], 0, 0, 0);
                }
            }
        }
    };
    if (D > 1 && c0 < c1) {
        load_x(c0, s[0]);
#pragma unroll
        for (int d = 1; d < D - 1; ++d) {
            if (c0 + d * U < c1) {
                load_w(c0 + d * U, s[d]);
                load_x(c0 + d * U, s[d]);
            }
        }
    }
    // at the end wave w < OT finishes output tile w: its row scales are
    // requested now
    float sw[GLU ? 2 : 1][4];
    if (wave < OT) {
#pragma unroll
        for (int q = 0; q < (GLU ? 2 : 1); ++q)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                sw[q][r] = p.scale[q][(int64_t)t.group * p.n + min(16 * (ot0 + wave) + 4 * g + r, p.n - 1)];
    }
    auto step = [&](int c, int d, bool load) {  // d: c's set
        if (load) {
            load_w(c + (D - 1) * U, s[(d + D - 1) % D]);
            load_x(c + (D - 1) * U, s[(d + D - 1) % D]);
        }
        __builtin_amdgcn_sched_barrier(0);
        multiply(s[d]);
        __builtin_amdgcn_sched_barrier(0);
    };
    // no branch between the loads and their products: a load that may or may
    // not have been made is waited for as if it were the last one
    int c = c0;
    for (; c + (2 * D - 2) * U < c1; c += D * U)
#pragma unroll
        for (int d = 0; d < D; ++d) step(c + d * U, d, true);
#pragma unroll
    for (int d = 0; d < 2 * D - 2; ++d)
        if (c + d * U < c1) step(c + d * U, d % D, c + (d + D - 1) * U < c1);
#pragma unroll
    for (int q = 0; q < NT; ++q) part[wave][q][lane] = acc[q];
    lds_barrier();
    // lane l holds x row l % 16, matrix rows 4 (l / 16) + r
    if (wave >= OT || i >= t.rows) return;
    acc_t sum[GLU ? 2 : 1];
#pragma unroll
    for (int q = 0; q < (GLU ? 2 : 1); ++q) {
        sum[q] = part[0][GLU ? q : wave][lane];
#pragma unroll
        for (int w = 1; w < kEWaves; ++w) sum[q] += part[w][GLU ? q : wave][lane];
    }
    const float sx = ACT == 0 ? 1.0f : p.s_x[src];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int n = 16 * (ot0 + wave) + 4 * g + r;
        if (n < p.n) {
            float o[GLU ? 2 : 1];
#pragma unroll
            for (int q = 0; q < (GLU ? 2 : 1); ++q) {
                o[q] = (float)sum[q][r] / sw[q][r];
                if constexpr (ACT == 1) o[q] /= sx;  // one after the other: the scales' product may overflow
            }
            if constexpr (GLU) o[0] = swiglu(o[0], o[1]);
            store_y<YT>(p.y, (int64_t)(t.row0 + i) * p.n + n, o[0]);
        }
    }
}

template <int ACT, int YT, bool GLU, bool TILED>
static hipError_t run_stream(ExpertParams p, hipStream_t st) {
    const int out_tiles = (p.n + 15) / 16;
    p.ntiles = GLU ? out_tiles : (out_tiles + 1) / 2;
    return launch_blocks(max_row_tiles(p.rows, p.e, 16) * p.ntiles, kEThreads, [&](uint32_t grid, int64_t block0) {
        p.block0 = block0;
        experts_stream_kernel<ACT, YT, GLU, TILED><<<grid, kEThreads, 0, st>>>(p);
    });
}

// ------------------------------------------------------------------ tiles
// Many rows per expert: a 256-thread workgroup computes BM = 128 (or 32)
// sorted rows of one expert times 256 matrix rows (GLU: 128 of the gate and
// the same 128 of the up matrix); each of its four waves all BM rows times 64
// matrix rows, BM / 32 x 2 tiles of v_mfma_f32_32x32x16_bf16 (or
// v_mfma_i32_32x32x32_i8).  Two workgroups run on a CU (four of 32 rows).
//   x: gathered by direct global->LDS loads (per-lane row addresses) into a
//      ring of 4 stages of 128 bytes per row, shared by the four waves;
//      16-byte chunks permuted by the row (swz), free of bank conflicts.
//   codes: no two waves of a workgroup share any, so they go straight to
//      registers, 16 bytes per lane, one stage ahead, and are widened to bf16
//      there (exact).
// Waves multiply only the 32-row blocks that hold rows: a group's last tile
// costs what its rows need, to 32.  Tiles go expert by expert, kTall row tiles
// by all column tiles at a time, and each XCD takes one contiguous run of
// that order, so the tiles that run together share codes and rows in its L2.
//
// 2048 tokens, 8 experts of 2 x 11008 x 4096, bf16 x: 676 us, 1.09 PFLOP/s.
// What holds it, from runs with parts taken out (at 704 us): the matrix instructions alone
// take 453 us (the clock falls to 1.8 GHz under them), without the LDS reads
// 597, without the widening 651, with neither x nor codes loaded 466: the loads
// cost most.  They are not late (codes two stages ahead: no change) and not
// from far (the L2s miss 1 GB of 6.5 GB asked), so it is the L1s' and L2s' rate.
// Tried and slower: 256 rows by eight waves, one workgroup per CU (796: fewer
// bytes, but no second workgroup to cover the barrier), one, two, four row
// tiles at a time (808, 750, 726 against 715 with eight).  Loads between the
// products instead of before them and a raised wave priority: 3.5%.  y is
// stored as the products leave it, 128 bytes of two rows at a time: four columns
// of 32 rows at a time (operands swapped) was 3-10% slower, whole rows by way of
// LDS 2-4%.
constexpr int kTN = 256, kTThreads = 256, kTStages = 4;
constexpr int kTall = 8;  // row tiles that go through the column tiles together
constexpr size_t tile_lds(int bm) { return (size_t)kTStages * bm * 128 + bm * sizeof(float); }

template <int ACT>
struct TileAcc {
    typedef f32x16 type;
};
template <>
struct TileAcc<1> {
    typedef i32x16 type;
};

template <int ACT, int YT, bool GLU, bool TILED, int BM, int MA>
__device__ __forceinline__ void experts_tile(const ExpertParams& p, const RowTile& t, int n0, uint8_t* smem,
                                             const uint32_t (&xoff)[BM / 32], float sx_tid) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5;
    const int c0 = n0 + wave * (GLU ? 32 : 64);  // this wave's first output
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x, (uint32_t)((int64_t)p.x_rows * p.k * (ACT == 0 ? 2 : 1)));
    // this lane's matrix row of each 32-row block, as an offset from the
    // wave's first 16-row tile: rows past n repeat the last one (tiled codes:
    // the last 16-row tile)
    __amdgpu_buffer_rsrc_t rw[2];
    uint32_t woff[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int first = min(c0 + (GLU ? 0 : 32 * b), (p.n - 1) & ~15), row = c0 + (GLU ? 0 : 32 * b) + (lane & 31);
        rw[b] = make_rsrc(p.codes[GLU ? b : 0] + (int64_t)t.group * p.expert_bytes + (int64_t)first * p.k,
                          (uint32_t)(32 * p.k));
        if constexpr (TILED) woff[b] = (uint32_t)(min(row >> 4, (p.n - 1) >> 4) - (first >> 4)) * 16 * p.k + (lane & 15) * 16 + h * 256;
        else woff[b] = (uint32_t)(min(row, p.n - 1) - first) * p.k + h * 16;
    }
    // 16-code pieces of a stage: piece q of lane half h is k group 2 q + h
    constexpr int kPieces = ACT == 0 ? 2 : 4;
    constexpr int kUnit = TILED ? 1024 : 64, kPair = TILED ? 512 : 32;
    constexpr int kLoads = 2 * kPieces;
    struct Codes {
        u32x4 v[2][kPieces];
    };
    auto load_codes = [&](int c, int b, Codes& w) {
        const int at = c * (kPieces / 2 * kUnit);
#pragma unroll
        for (int q = 0; q < kPieces; ++q)
            w.v[b][q] = __builtin_amdgcn_raw_buffer_load_b128(rw[b], woff[b] + (q >> 1) * kUnit + (q & 1) * kPair, at, 0);
    };
    const int nk = p.k / (ACT == 0 ? 64 : 128);
    auto load_x = [&](int c, int first, int step) {
        const int at = min(c, nk - 1) * 128;
        uint8_t* dst = smem + (c % kTStages) * (BM * 128);
#pragma unroll
        for (int l = first; l < MA; l += step) dma16_buffer(rx, dst + (wave + 4 * l) * 1024, xoff[l], at);
    };
    typename TileAcc<ACT>::type acc[MA][2];
#pragma unroll
    for (int a = 0; a < MA; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0;

    const int xrow = (lane & 31) * 128, xswz = (lane >> 1) & 7;  // swz of a row: its chunk ^ xswz
    auto multiply = [&](int c, const Codes& w, const auto& between) {
        const uint8_t* xs = smem + (c % kTStages) * (BM * 128) + xrow;
        bf16x8 wb[2][2];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            between(q);
            const int chunk = ACT == 0 ? 4 * (q >> 1) + 2 * h + (q & 1) : 2 * q + h;
            u32x4 xf[MA];
#pragma unroll
            for (int a = 0; a < MA; ++a)
                xf[a] = *reinterpret_cast<const u32x4*>(xs + a * 32 * 128 + 16 * (chunk ^ xswz));
            if constexpr (ACT == 0) {
                if ((q & 1) == 0) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) codes_to_bf16(w.v[b][q >> 1], wb[b][0], wb[b][1]);
                }
#pragma unroll
                for (int a = 0; a < MA; ++a)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, xf[a]),
                                                                            wb[b][q & 1], acc[a][b], 0, 0, 0);
            } else {
#pragma unroll
                for (int a = 0; a < MA; ++a)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
                            __builtin_bit_cast(i32x4, xf[a]), __builtin_bit_cast(i32x4, w.v[b][q]), acc[a][b], 0, 0, 0);
            }
        }
    };

    // Step c issues the codes of stage c + 1, then the x of stage c + 3 (past
    // the end the last stage again, into a slot that is not read), always in
    // this order: at its start at most x of c + 1, codes of c and x of c + 2
    // may be outstanding, which leaves x of c landed.
    // the outputs' scales are requested here, before anything that is counted
    float sw[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
        sw[b] = p.scale[GLU ? b : 0][(int64_t)t.group * p.n + min(c0 + (GLU ? 0 : 32 * b) + (lane & 31), p.n - 1)];
    __builtin_amdgcn_sched_barrier(0);
    Codes wa, wb;
    load_x(0, 0, 1);
    load_x(1, 0, 1);
    __builtin_amdgcn_sched_barrier(0);
    load_codes(0, 0, wa);
    load_codes(0, 1, wa);
    __builtin_amdgcn_sched_barrier(0);
    load_x(2, 0, 1);
    __builtin_amdgcn_sched_barrier(0);
    // read after the barriers of the k loop
    if (ACT == 1 && tid < BM) reinterpret_cast<float*>(smem + kTStages * (BM * 128))[tid] = 1.0f / sx_tid;
    auto step = [&](int c, const Codes& now, Codes& next) {
        wait_vmcnt<kLoads + 2 * MA>();
        lds_barrier();  // every wave's share of x stage c is there, and no one reads stage c - 1 any more
        // the loads go between the products, so that no run of them holds the
        // matrix unit up: codes in front of quarters 0 and 1, x of 2 and 3
        const int wat = min(c + 1, nk - 1), xat = c + 3;
        __builtin_amdgcn_s_setprio(1);
        multiply(c, now, [&](int q) {
            __builtin_amdgcn_sched_barrier(0);
            if (q < 2) {
                load_codes(wat, q, next);
            } else {
                load_x(xat, q & 1, 2);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int c = 0; c + 1 < nk; c += 2) {
        step(c, wa, wb);
        step(c + 1, wb, wa);
    }
    if (ACT == 1 && (nk & 1)) step(nk - 1, wa, wb);  // k is a multiple of 128: bf16 stages come in pairs
    wait_vmcnt<0>();  // no load may land in LDS after the workgroup has ended

    // lane l holds output column l % 32 of each block, rows 8 (r / 4) + 4 (l / 32) + r % 4;
    // stores past the tile's rows fall outside the buffer's range and are dropped
    constexpr int kY = YT == 0 ? 4 : 2;
    const float* rsx = reinterpret_cast<const float*>(smem + kTStages * (BM * 128));
    const __amdgpu_buffer_rsrc_t ry =
        make_rsrc(static_cast<uint8_t*>(p.y) + (int64_t)t.row0 * p.n * kY, (uint32_t)(t.rows * p.n * kY));
    const uint32_t line = (uint32_t)(p.n * kY);
    uint32_t yoff[2];
    float rsw[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int col = c0 + (GLU ? 0 : 32 * b) + (lane & 31);
        yoff[b] = col < p.n ? (uint32_t)(4 * h) * line + (uint32_t)(col * kY) : 0x80000000u;
        rsw[b] = 1.0f / sw[b];
    }
#pragma unroll
    for (int a = 0; a < MA; ++a) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = a * 32 + 8 * (r >> 2) + (r & 3);
            const float sx = ACT == 0 ? 1.0f : rsx[row + 4 * h];
            float o[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                o[b] = (float)acc[a][b][r] * rsw[b];
                if constexpr (ACT == 1) o[b] *= sx;
            }
            if constexpr (GLU) o[0] = swiglu(o[0], o[1]);
#pragma unroll
            for (int b = 0; b < (GLU ? 1 : 2); ++b) {
                if constexpr (YT == 0) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o[b]), ry, yoff[b] + row * line, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)any_f32_to_bf16(o[b]), ry, yoff[b] + row * line, 0, 0);
            }
        }
    }
}

template <int ACT, int YT, bool GLU, bool TILED, int BM>
__global__ __launch_bounds__(kTThreads, BM == 32 ? 4 : 2) void experts_tile_kernel(ExpertParams p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the tile: consecutive workgroups go to different XCDs, each XCD gets a
    // contiguous run of the tiles there are (the grid is sized for the most
    // there can be)
    const GroupTiles first = group_tiles<BM>(request_groups(p.offsets, p.e, 0), p.rows, 0);
    const int64_t total = (int64_t)count_row_tiles<BM>(p.offsets, p.e, p.rows, first) * p.ntiles;
    const int64_t block = p.block0 + blockIdx.x, per = (total + 7) >> 3;
    const int64_t at = (block & 7) * per + (block >> 3);
    if ((block >> 3) >= per || at >= total) return;
    RowTile t = find_row_tile<BM>(p.offsets, p.e, p.rows, (int)(at / p.ntiles), first);
    if (t.rows <= 0) return;
    const int64_t r = at - (int64_t)t.before * p.ntiles;
    const int mt = (t.count + BM - 1) / BM;
    const int st = (int)(r / (kTall * (int64_t)p.ntiles));
    const int u = (int)(r - (int64_t)st * kTall * p.ntiles), tall = min(kTall, mt - kTall * st);
    const int m = kTall * st + u % tall;
    const int n0 = u / tall * (GLU ? kTN / 2 : kTN);
    t.row0 = t.first + m * BM;
    t.rows = min(BM, t.count - m * BM);

    // rows of x of this lane's loads and (the last) of this thread's s_x; rows
    // past the tile repeat its last.  All are requested before one is used.
    constexpr int kL = BM / 32;
    auto row_of = [&](int l) { return l < kL ? (wave + 4 * l) * 8 + (lane >> 3) : min(tid, BM - 1); };
    int src[kL + ACT];
#pragma unroll
    for (int l = 0; l < kL + ACT; ++l) src[l] = t.row0 + min(row_of(l), t.rows - 1);
    if (p.order) {
#pragma unroll
        for (int l = 0; l < kL + ACT; ++l) src[l] = p.order[src[l]];
#pragma unroll
        for (int l = 0; l < kL + ACT; ++l) src[l] = divide(max(src[l], 0), p.per_row);
    }
    uint32_t xsrc[kL];
#pragma unroll
    for (int l = 0; l < kL; ++l)
        xsrc[l] = (uint32_t)min(src[l], p.x_rows - 1) * (uint32_t)(p.k * (ACT == 0 ? 2 : 1)) + 16 * swz<8>(row_of(l), lane & 7);
    const float sx_tid = ACT == 1 ? p.s_x[min(src[kL + ACT - 1], p.x_rows - 1)] : 1.0f;
    if constexpr (BM == 32) {
        experts_tile<ACT, YT, GLU, TILED, BM, 1>(p, t, n0, smem, xsrc, sx_tid);
    } else {
        if (t.rows > 96) experts_tile<ACT, YT, GLU, TILED, BM, 4>(p, t, n0, smem, xsrc, sx_tid);
        else if (t.rows > 64) experts_tile<ACT, YT, GLU, TILED, BM, 3>(p, t, n0, smem, xsrc, sx_tid);
        else if (t.rows > 32) experts_tile<ACT, YT, GLU, TILED, BM, 2>(p, t, n0, smem, xsrc, sx_tid);
        else experts_tile<ACT, YT, GLU, TILED, BM, 1>(p, t, n0, smem, xsrc, sx_tid);
    }
}

template <int ACT, int YT, bool GLU, bool TILED, int BM>
static hipError_t run_tile(ExpertParams p, hipStream_t st) {
    auto kern = experts_tile_kernel<ACT, YT, GLU, TILED, BM>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)tile_lds(BM));
    if (e != hipSuccess) return e;
    const int per = GLU ? kTN / 2 : kTN;
    p.ntiles = (p.n + per - 1) / per;
    const int64_t blocks = (max_row_tiles(p.rows, p.e, BM) * p.ntiles + 7) / 8 * 8;
    return launch_blocks(blocks, kTThreads, [&](uint32_t grid, int64_t block0) {
        p.block0 = block0;
        kern<<<grid, kTThreads, tile_lds(BM), st>>>(p);
    });
}

template <int ACT, int YT, bool GLU>
static hipError_t run_kind(const ExpertParams& p, hipStream_t st) {
    // Streams up to nine rows per expert, tiles above.  Measured, us, stream and
    // 128-row tiles of a swiglu at 8, 12, 24 rows per expert:
    //                          64 of 1024 x 2048        16 of 2304 x 4096
    //   bf16 x, tiled codes    47 50, 58 51, 95 57      56 60, 69 62, 109 69
    //   bf16 x, row-major      57 58, 72 59, 114 63     67 98, 83 100, 132 106
    //   int8 x, tiled codes    44 47, 53 48, 84 52      53 66, 63 67, 96 70
    //   int8 x, row-major      48 51, 58 53, 93 57      55 91, 66 91, 104 95
    // (row-major codes of few wide experts would stay streams up to 16 rows: 97
    // 102 and 77 93.)  Where 128-row tiles do not fill the CUs, a workgroup's own
    // time decides: 32-row tiles then, or streams while all of them together read
    // few matrix rows.  Stream, 32-row, 128-row tiles (products) of 5 experts of
    // 440 x 2176 at 64, 256, 1024 rows each, and of 16 of 1024 x 2048 at 32, 128:
    //   bf16 x, tiled codes    12 17 32, 21 17 32, 68 30 35    19 17 28, 52 24 32
    //   bf16 x, row-major      13 21 32, 26 21 32, 80 38 33    24 21 28, 69 36 31
    //   int8 x, tiled codes    11 10 18, 18 11 19, 54 17 19    16 11 16, 42 17 19
    //   int8 x, row-major      11 19 23, 20 20 24, 62 36 25    19 20 22, 54 36 24
    // (the codes' layout is not asked: row-major ones would take 128-row tiles from
    // about 100 rows per expert on, at 256 rows of the second 51 and 25 with int8
    // x).  At 256 tiles of 128 rows and above the two tiles are even with tiled
    // codes (32 of 704 x 1024, 256 rows: 25 22), and with more of them 128 rows win.
    constexpr int kPer = GLU ? kTN / 2 : kTN;
    const bool fills = max_row_tiles(p.rows, p.e, 128) * ((p.n + kPer - 1) / kPer) >= 256;
    const int64_t streamed = max_row_tiles(p.rows, p.e, 16) * p.n * (GLU ? 2 : 1);
    // The tile kernel keeps 32-bit offsets into x and a tile's y; past them many
    // rows cost several times as much (8 experts of 1024 x 8192, bf16 x: 262016
    // rows 3.6 ms in tiles, 262144 rows 23.2 ms in streams).
    const bool small = (int64_t)p.x_rows * p.k * (ACT == 0 ? 2 : 1) < ((int64_t)1 << 32) && p.n < (1 << 21);
    if (p.rows <= 9 * (int64_t)p.e || (!fills && streamed < 28000) || !small)
        return p.tiled ? run_stream<ACT, YT, GLU, true>(p, st) : run_stream<ACT, YT, GLU, false>(p, st);
    if (!fills) return p.tiled ? run_tile<ACT, YT, GLU, true, 32>(p, st) : run_tile<ACT, YT, GLU, false, 32>(p, st);
    return p.tiled ? run_tile<ACT, YT, GLU, true, 128>(p, st) : run_tile<ACT, YT, GLU, false, 128>(p, st);
}
template <int ACT, int YT>
static hipError_t run_glu(const ExpertParams& p, bool glu, hipStream_t st) {
    return glu ? run_kind<ACT, YT, true>(p, st) : run_kind<ACT, YT, false>(p, st);
}

hipError_t launch_experts(const ExpertArgs& a, hipStream_t st) {
    ExpertParams p;
    p.codes[0] = a.codes;
    p.codes[1] = a.codes2;
    p.scale[0] = a.scale;
    p.scale[1] = a.scale2;
    p.x = a.x;
    p.s_x = a.s_x;
    p.offsets = a.offsets;
    p.order = a.order;
    p.y = a.y;
    p.e = (int32_t)a.e;
    p.n = (int32_t)a.n;
    p.k = (int32_t)a.k;
    p.rows = (int32_t)a.rows;
    p.x_rows = (int32_t)a.x_rows;
    p.per_row = row_div(a.per_row);
    p.expert_bytes = a.t16 ? (a.n + 15) / 16 * 16 * a.k : a.n * a.k;
    p.tiled = a.t16;
    const bool glu = a.codes2 != nullptr;
    if (a.act_int8) return a.yt == 0 ? run_glu<1, 0>(p, glu, st) : run_glu<1, 1>(p, glu, st);
    return a.yt == 0 ? run_glu<0, 0>(p, glu, st) : run_glu<0, 1>(p, glu, st);
}

// ------------------------------------------------------------------ combine
// A thread adds four consecutive outputs of a token over its slots, in slot
// order (fp32), so the result does not depend on the plan's order; the rows of
// up to eight slots are requested together.
struct CombineParams {
    CombineArgs a;
    int64_t nblocks, block0;
    int32_t cols;  // columns of a workgroup
};
// four columns, aligned to their elements only (rows of any length)
typedef float c4f __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t c4h __attribute__((ext_vector_type(2), aligned(2)));

template <int YT>
__global__ __launch_bounds__(kThreads) void combine_kernel(CombineParams p) {
    constexpr int S = 8;
    const CombineArgs& a = p.a;
    const int64_t block = p.block0 + blockIdx.x;
    const int64_t t = block / p.nblocks;
    const int64_t n0 = (block % p.nblocks) * p.cols + 4 * (int)threadIdx.x;
    if (n0 >= a.n) return;
    // at the row's end its last four columns (a row of fewer: past it, into the
    // workspace's padding); every load is made, slots and rows that are not
    // there repeat others and count as zero
    const int64_t at = max((int64_t)0, min(n0, a.n - 4)), skip = n0 - at;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < a.top_k; j0 += S) {
        f32x4 h[S];
        float w[S];
        int64_t row[S];
#pragma unroll
        for (int j = 0; j < S; ++j) {
            const int64_t slot = t * a.top_k + min(j0 + j, a.top_k - 1);
            row[j] = a.pos[slot];
            w[j] = a.weights[slot];
            if (j0 + j >= a.top_k || row[j] >= a.rows) row[j] = -1;
        }
#pragma unroll
        for (int j = 0; j < S; ++j) h[j] = *reinterpret_cast<const c4f*>(a.h + max(row[j], (int64_t)0) * a.n + at);
#pragma unroll
        for (int j = 0; j < S; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = row[j] >= 0 ? __builtin_fmaf(w[j], h[j][e], s[e]) : s[e];
    }
    const int64_t out = t * a.n + at;
    if (skip == 0 && a.n >= 4) {
        if constexpr (YT == 0) {
            *reinterpret_cast<c4f*>(static_cast<float*>(a.y) + out) = s;
        } else {
            *reinterpret_cast<c4h*>(static_cast<uint16_t*>(a.y) + out) =
                c4h{any_f32_to_bf16(s[0]) | (any_f32_to_bf16(s[1]) << 16), any_f32_to_bf16(s[2]) | (any_f32_to_bf16(s[3]) << 16)};
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e >= skip && at + e < a.n) store_y<YT>(a.y, out + e, s[e]);
    }
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t st) {
    CombineParams p;
    p.a = a;
    // one wave per workgroup where that leaves CUs without work
    const int threads = a.tokens * ((a.n + 1023) / 1024) < 1024 ? kWave : kThreads;
    p.cols = 4 * threads;
    p.nblocks = (a.n + p.cols - 1) / p.cols;
    return launch_blocks(a.tokens * p.nblocks, threads, [&](uint32_t grid, int64_t block0) {
        p.block0 = block0;
        if (a.yt == 0) combine_kernel<0><<<grid, threads, 0, st>>>(p);
        else combine_kernel<1><<<grid, threads, 0, st>>>(p);
    });
}

}  // namespace qg

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
constexpr int kEThreads = 512;
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
    int32_t e, n, k, rows, x_rows, per_row;
    int32_t row_stride, unit_stride, group_stride;  // bytes from row to row of a tile, unit to unit, k group to k group
    int32_t tiled;            // 16-row tiled codes (else row-major); a 16-row tile is 16 k bytes in both
    int64_t block0;           // workgroups of earlier launches of the same product
    int32_t ntiles;           // workgroup tiles along n
    int32_t split;            // waves of a workgroup that share a tile, each with a part of k
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
    else static_cast<uint16_t*>(y)[at] = (uint16_t)f32_to_bf16(v);
}

// Sixteen sorted rows of one expert times NT 16-row tiles of its matrix (GLU:
// NT / 2 tiles of the gate and the same of the up matrix) per wave; the
// workgroup's 8 waves take 8 / split groups of tiles and split parts of k
// each, summed through LDS in order.
template <int ACT, int YT, bool GLU>
__global__ __launch_bounds__(kEThreads) void experts_stream_kernel(ExpertParams p) {
    constexpr int NT = 4;
    constexpr int OT = GLU ? NT / 2 : NT;  // 16-row output tiles
    typedef typename std::conditional<ACT == 0, f32x4, i32x4>::type acc_t;
    __shared__ acc_t part[kEWaves][NT][kWave];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;  // weight row / x row, k group
    const int64_t block = p.block0 + blockIdx.x;
    const int nt = (int)(block % p.ntiles);
    const RowTile t = find_row_tile<16>(p.offsets, p.e, p.rows, (int)(block / p.ntiles));
    if (t.rows <= 0) return;  // uniform over the workgroup

    // this lane's x row (rows past the tile repeat its last)
    auto source = [&](int r) {
        const int at = t.row0 + min(r, t.rows - 1);
        const int src = p.order ? p.order[at] / p.per_row : at;
        return min(max(src, 0), p.x_rows - 1);
    };
    const int src = source(i);
    const uint8_t* xrow = static_cast<const uint8_t*>(p.x) + (int64_t)src * p.k * (ACT == 0 ? 2 : 1) + (ACT == 0 ? 32 : 16) * g;

    const int part_k = wave % p.split, grp = wave / p.split;
    const int ot0 = (nt * (kEWaves / p.split) + grp) * OT;  // first 16-row output tile
    const int units = p.k / kEUnit;
    const int c0 = (int)((int64_t)units * part_k / p.split), c1 = (int)((int64_t)units * (part_k + 1) / p.split);

    const int8_t* wrow[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        // rows past n: row-major codes repeat the last row; tiled codes are
        // padded to whole tiles, tiles past the last repeat it
        const int ot = min(ot0 + q % OT, (p.n - 1) / 16);
        const int row = p.tiled ? i : min(i, p.n - 1 - 16 * ot);
        wrow[q] = p.codes[GLU ? q / OT : 0] + (int64_t)t.group * p.expert_bytes + (int64_t)ot * 16 * p.k +
                  (int64_t)row * p.row_stride + g * p.group_stride;
    }
    acc_t acc[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) acc[q] = acc_t{0, 0, 0, 0};
    for (int c = c0; c < c1; ++c) {
        u32x4 w[NT];
#pragma unroll
        for (int q = 0; q < NT; ++q) w[q] = *reinterpret_cast<const u32x4*>(wrow[q] + (int64_t)c * p.unit_stride);
        if constexpr (ACT == 0) {
            const u32x4 xa = *reinterpret_cast<const u32x4*>(xrow + (int64_t)c * 128);
            const u32x4 xb = *reinterpret_cast<const u32x4*>(xrow + (int64_t)c * 128 + 16);
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                bf16x8 a0, a1;
                codes_to_bf16(w[q], a0, a1);
                acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, __builtin_bit_cast(bf16x8, xa), acc[q], 0, 0, 0);
                acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, __builtin_bit_cast(bf16x8, xb), acc[q], 0, 0, 0);
            }
        } else {
            const i32x4 xa = *reinterpret_cast<const i32x4*>(xrow + (int64_t)c * 64);
#pragma unroll
            for (int q = 0; q < NT; ++q)
                acc[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w[q]), xa, acc[q], 0, 0, 0);
        }
    }
    if (p.split > 1) {
#pragma unroll
        for (int q = 0; q < NT; ++q) part[wave][q][lane] = acc[q];
        lds_barrier();
        if (part_k != 0) return;
        for (int w = 1; w < p.split; ++w)
#pragma unroll
            for (int q = 0; q < NT; ++q) acc[q] += part[wave + w][q][lane];
    }
    // lane l holds x row l % 16, matrix rows 4 (l / 16) + r
    if (i >= t.rows) return;
    const float sx = ACT == 0 ? 1.0f : p.s_x[src];
#pragma unroll
    for (int q = 0; q < OT; ++q) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int n = 16 * (ot0 + q) + 4 * g + r;
            if (n < p.n) {
                const int64_t sw = (int64_t)t.group * p.n + n;
                float o = (float)acc[q][r] / (ACT == 0 ? p.scale[0][sw] : p.scale[0][sw] * sx);
                if constexpr (GLU) {
                    const float u = (float)acc[OT + q][r] / (ACT == 0 ? p.scale[1][sw] : p.scale[1][sw] * sx);
                    o = swiglu(o, u);
                }
                store_y<YT>(p.y, (int64_t)(t.row0 + i) * p.n + n, o);
            }
        }
    }
}

template <int ACT, int YT, bool GLU>
static hipError_t run_stream(ExpertParams p, hipStream_t st) {
    const int out_tiles = (p.n + 15) / 16, per_wave = GLU ? 2 : 4;
    p.split = 8;
    const int per_wg = per_wave * (kEWaves / p.split);
    p.ntiles = (out_tiles + per_wg - 1) / per_wg;
    return launch_blocks(max_row_tiles(p.rows, p.e, 16) * p.ntiles, kEThreads, [&](uint32_t grid, int64_t block0) {
        p.block0 = block0;
        experts_stream_kernel<ACT, YT, GLU><<<grid, kEThreads, 0, st>>>(p);
    });
}

// ------------------------------------------------------------------ tiles
// Many rows per expert: a 256-thread workgroup computes 128 sorted rows of one
// expert times 256 matrix rows (GLU: 128 of the gate and the same 128 of the
// up matrix); each of its four waves all 128 rows times 64 matrix rows, 4 x 2
// tiles of v_mfma_f32_32x32x16_bf16 (or v_mfma_i32_32x32x32_i8).  Two
// workgroups run on a CU.
//   x: gathered by direct global->LDS loads (per-lane row addresses) into a
//      ring of 4 stages of 128 bytes per row, shared by the four waves;
//      16-byte chunks permuted by the row (swz), free of bank conflicts.
//   codes: no two waves of a workgroup share any, so they go straight to
//      registers, 16 bytes per lane, one stage ahead, and are widened to bf16
//      there (exact).
// Waves multiply only the 32-row blocks that hold rows: a group's last tile
// costs what its rows need, to 32.  Tiles go expert by expert, four row tiles
// by all column tiles at a time, and each XCD takes one contiguous run of
// that order, so the tiles that run together share codes and rows in its L2.
constexpr int kTM = 128, kTN = 256, kTThreads = 256, kTStages = 4;
constexpr int kTStageBytes = kTM * 128;
constexpr size_t kTLds = (size_t)kTStages * kTStageBytes + kTM * sizeof(float);

template <int ACT>
struct TileAcc {
    typedef f32x16 type;
};
template <>
struct TileAcc<1> {
    typedef i32x16 type;
};

template <int ACT, int YT, bool GLU, bool TILED, int MA>
__device__ __forceinline__ void experts_tile(const ExpertParams& p, const RowTile& t, int n0, uint8_t* smem,
                                             const uint32_t (&xoff)[4]) {
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
    auto load_codes = [&](int c, Codes& w) {
        const int at = c * (kPieces / 2 * kUnit);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int q = 0; q < kPieces; ++q)
                w.v[b][q] = __builtin_amdgcn_raw_buffer_load_b128(rw[b], woff[b] + (q >> 1) * kUnit + (q & 1) * kPair, at, 0);
    };
    const int nk = p.k / (ACT == 0 ? 64 : 128);
    auto load_x = [&](int c) {
        const int at = min(c, nk - 1) * 128;
        uint8_t* dst = smem + (c % kTStages) * kTStageBytes;
#pragma unroll
        for (int l = 0; l < 4; ++l) dma16_buffer(rx, dst + (wave + 4 * l) * 1024, xoff[l], at);
    };
    typename TileAcc<ACT>::type acc[MA][2];
#pragma unroll
    for (int a = 0; a < MA; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0;

    const int xrow = (lane & 31) * 128, xswz = (lane >> 1) & 7;  // swz of a row: its chunk ^ xswz
    auto multiply = [&](int c, const Codes& w) {
        const uint8_t* xs = smem + (c % kTStages) * kTStageBytes + xrow;
        bf16x8 wb[2][2];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
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
    Codes wa, wb;
    load_x(0);
    load_x(1);
    __builtin_amdgcn_sched_barrier(0);
    load_codes(0, wa);
    __builtin_amdgcn_sched_barrier(0);
    load_x(2);
    __builtin_amdgcn_sched_barrier(0);
    auto step = [&](int c, const Codes& now, Codes& next) {
        wait_vmcnt<kLoads + 8>();
        lds_barrier();  // every wave's share of x stage c is there, and no one reads stage c - 1 any more
        load_codes(min(c + 1, nk - 1), next);
        __builtin_amdgcn_sched_barrier(0);
        load_x(c + 3);
        __builtin_amdgcn_sched_barrier(0);
        multiply(c, now);
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
    const float* rsx = reinterpret_cast<const float*>(smem + kTStages * kTStageBytes);
    const __amdgpu_buffer_rsrc_t ry =
        make_rsrc(static_cast<uint8_t*>(p.y) + (int64_t)t.row0 * p.n * kY, (uint32_t)(t.rows * p.n * kY));
    const uint32_t line = (uint32_t)(p.n * kY);
    uint32_t yoff[2];
    float rsw[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int col = c0 + (GLU ? 0 : 32 * b) + (lane & 31);
        yoff[b] = col < p.n ? (uint32_t)(4 * h) * line + (uint32_t)(col * kY) : 0x80000000u;
        rsw[b] = 1.0f / p.scale[GLU ? b : 0][(int64_t)t.group * p.n + min(col, p.n - 1)];
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
                else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)f32_to_bf16(o[b]), ry, yoff[b] + row * line, 0, 0);
            }
        }
    }
}

template <int ACT, int YT, bool GLU, bool TILED>
__global__ __launch_bounds__(kTThreads, 2) void experts_tile_kernel(ExpertParams p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the tile: consecutive workgroups go to different XCDs, each XCD gets a
    // contiguous run of the tiles there are (the grid is sized for the most
    // there can be)
    const int64_t total = (int64_t)count_row_tiles<kTM>(p.offsets, p.e, p.rows) * p.ntiles;
    const int64_t block = p.block0 + blockIdx.x, per = (total + 7) >> 3;
    const int64_t at = (block & 7) * per + (block >> 3);
    if ((block >> 3) >= per || at >= total) return;
    RowTile t = find_row_tile<kTM>(p.offsets, p.e, p.rows, (int)(at / p.ntiles));
    if (t.rows <= 0) return;
    const int64_t r = at - (int64_t)t.before * p.ntiles;
    const int mt = (t.count + kTM - 1) / kTM;
    const int st = (int)(r / (4 * (int64_t)p.ntiles));
    const int u = (int)(r - (int64_t)st * 4 * p.ntiles), tall = min(4, mt - 4 * st);
    const int m = 4 * st + u % tall;
    const int n0 = u / tall * (GLU ? kTN / 2 : kTN);
    t.row0 = t.first + m * kTM;
    t.rows = min(kTM, t.count - m * kTM);

    // rows past the tile repeat its last row
    auto source = [&](int row) {
        const int i = t.row0 + min(row, t.rows - 1);
        const int src = p.order ? p.order[i] / p.per_row : i;
        return min(max(src, 0), p.x_rows - 1);
    };
    uint32_t xsrc[4];
#pragma unroll
    for (int l = 0; l < 4; ++l) {
        const int row = (wave + 4 * l) * 8 + (lane >> 3);
        xsrc[l] = (uint32_t)source(row) * (uint32_t)(p.k * (ACT == 0 ? 2 : 1)) + 16 * swz<8>(row, lane & 7);
    }
    if constexpr (ACT == 1) {
        // read after the barriers of the k loop
        if (tid < kTM) reinterpret_cast<float*>(smem + kTStages * kTStageBytes)[tid] = 1.0f / p.s_x[source(tid)];
    }
    if (t.rows > 96) experts_tile<ACT, YT, GLU, TILED, 4>(p, t, n0, smem, xsrc);
    else if (t.rows > 64) experts_tile<ACT, YT, GLU, TILED, 3>(p, t, n0, smem, xsrc);
    else if (t.rows > 32) experts_tile<ACT, YT, GLU, TILED, 2>(p, t, n0, smem, xsrc);
    else experts_tile<ACT, YT, GLU, TILED, 1>(p, t, n0, smem, xsrc);
}

template <int ACT, int YT, bool GLU, bool TILED>
static hipError_t run_tile(ExpertParams p, hipStream_t st) {
    auto kern = experts_tile_kernel<ACT, YT, GLU, TILED>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)kTLds);
    if (e != hipSuccess) return e;
    const int per = GLU ? kTN / 2 : kTN;
    p.ntiles = (p.n + per - 1) / per;
    const int64_t blocks = (max_row_tiles(p.rows, p.e, kTM) * p.ntiles + 7) / 8 * 8;
    return launch_blocks(blocks, kTThreads, [&](uint32_t grid, int64_t block0) {
        p.block0 = block0;
        kern<<<grid, kTThreads, kTLds, st>>>(p);
    });
}

template <int ACT, int YT, bool GLU>
static hipError_t run_kind(const ExpertParams& p, hipStream_t st) {
    // the tile kernel keeps 32-bit offsets into x and a tile's y
    const bool small = (int64_t)p.x_rows * p.k * (ACT == 0 ? 2 : 1) < ((int64_t)1 << 32) && p.n < (1 << 21);
    if (p.rows <= 16 * (int64_t)p.e || !small) return run_stream<ACT, YT, GLU>(p, st);
    return p.tiled ? run_tile<ACT, YT, GLU, true>(p, st) : run_tile<ACT, YT, GLU, false>(p, st);
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
    p.per_row = a.per_row;
    p.expert_bytes = a.t16 ? (a.n + 15) / 16 * 16 * a.k : a.n * a.k;
    p.tiled = a.t16;
    p.row_stride = a.t16 ? 16 : (int32_t)a.k;
    p.unit_stride = a.t16 ? 1024 : 64;
    p.group_stride = a.t16 ? 256 : 16;
    const bool glu = a.codes2 != nullptr;
    if (a.act_int8) return a.yt == 0 ? run_glu<1, 0>(p, glu, st) : run_glu<1, 1>(p, glu, st);
    return a.yt == 0 ? run_glu<0, 0>(p, glu, st) : run_glu<0, 1>(p, glu, st);
}

// ------------------------------------------------------------------ combine
// One workgroup per token and 1024 outputs; a thread adds its 4 outputs over
// the token's slots in slot order (fp32), so the result does not depend on
// the plan's order.
struct CombineParams {
    CombineArgs a;
    int64_t nblocks, block0;
};
template <int YT>
__global__ __launch_bounds__(kThreads) void combine_kernel(CombineParams p) {
    const CombineArgs& a = p.a;
    const int64_t block = p.block0 + blockIdx.x;
    const int64_t t = block / p.nblocks;
    const int64_t n0 = (block % p.nblocks) * (4 * kThreads) + threadIdx.x;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < a.top_k; ++j) {
        const int64_t at = a.pos[t * a.top_k + j];
        if (at < 0 || at >= a.rows) continue;
        const float w = a.weights[t * a.top_k + j];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t n = n0 + q * kThreads;
            if (n < a.n) s[q] = __builtin_fmaf(w, a.h[at * a.n + n], s[q]);
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int64_t n = n0 + q * kThreads;
        if (n < a.n) store_y<YT>(a.y, t * a.n + n, s[q]);
    }
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t st) {
    CombineParams p;
    p.a = a;
    p.nblocks = (a.n + 4 * kThreads - 1) / (4 * kThreads);
    return launch_blocks(a.tokens * p.nblocks, kThreads, [&](uint32_t grid, int64_t block0) {
        p.block0 = block0;
        if (a.yt == 0) combine_kernel<0><<<grid, kThreads, 0, st>>>(p);
        else combine_kernel<1><<<grid, kThreads, 0, st>>>(p);
    });
}

}  // namespace qg

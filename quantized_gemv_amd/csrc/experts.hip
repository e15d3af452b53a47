// experts.hip -- int8 products grouped by expert, with ragged row counts.
//
// Rows i of the plan are sorted by expert; expert e holds rows offsets[e] ..
// offsets[e + 1] - 1, and
//   y[i][n] = (sum_k codes[e][n][k] x[src(i)][k]) / s_w[e][n]             (W8A16)
//   y[i][n] = (sum_k codes[e][n][k] xq[src(i)][k]) / (s_w[e][n] s_x[src]) (W8A8)
// with src(i) = order[i] / per_row.  SwiGLU launches compute a gate and an up
// product per output and store gate / (1 + exp(-gate)) * up.
#include "qg_launch.h"
#include "qg_rows.h"

namespace qg {

typedef __bf16 ebf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

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
__device__ __forceinline__ void codes_to_bf16(const u32x4& w, ebf16x8& a0, ebf16x8& a1) {
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
    a0 = __builtin_bit_cast(ebf16x8, u32x4{h[0], h[1], h[2], h[3]});
    a1 = __builtin_bit_cast(ebf16x8, u32x4{h[4], h[5], h[6], h[7]});
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
                ebf16x8 a0, a1;
                codes_to_bf16(w[q], a0, a1);
                acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, __builtin_bit_cast(ebf16x8, xa), acc[q], 0, 0, 0);
                acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, __builtin_bit_cast(ebf16x8, xb), acc[q], 0, 0, 0);
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

template <int ACT, int YT>
static hipError_t run_glu(const ExpertParams& p, bool glu, hipStream_t st) {
    return glu ? run_stream<ACT, YT, true>(p, st) : run_stream<ACT, YT, false>(p, st);
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

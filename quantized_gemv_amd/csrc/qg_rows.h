// qg_rows.h -- device pieces of the products whose matrix depends on the row
// (expert products, low-rank adapters) and of the grouping that plans them.
//
// A plan is offsets[groups + 1] and order[rows] on the device: the rows
// (tokens, or token / slot pairs) sorted by group.  The kernels never trust
// its contents: offsets are clamped into [0, rows] and made ascending,
// source rows into the matrix, so a wrong plan gives wrong numbers, never an
// access out of bounds.
#pragma once

#include "qg_device.h"

namespace qg {

// Round-to-nearest-even narrowing of any fp32 to bf16 bits, by the hardware's
// conversion: the bits of f32_to_bf16 on every finite and infinite value (all
// compared), and NaN stays NaN.  (The rounding sum of f32_to_bf16 would carry
// payloads from 0x7FFF8000 on over into a zero, and scales and weights come from
// outside with any payload.)
__device__ __forceinline__ uint32_t any_f32_to_bf16(float f) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

// Inclusive prefix sum over the wave (all 64 lanes active): DPP row shifts
// within the rows of 16, then the row totals carried up.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ int dpp_add(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROW_MASK, 0xF, false);
}
__device__ __forceinline__ int wave_scan_incl(int v) {
    v = dpp_add<0x111, 0xF>(v);  // row_shr:1
    v = dpp_add<0x112, 0xF>(v);  // row_shr:2
    v = dpp_add<0x114, 0xF>(v);  // row_shr:4
    v = dpp_add<0x118, 0xF>(v);  // row_shr:8
    v = dpp_add<0x142, 0xA>(v);  // row_bcast:15 into rows 1, 3
    v = dpp_add<0x143, 0xC>(v);  // row_bcast:31 into rows 2, 3
    return v;
}

// One tile of up to MT sorted rows of one group (rows == 0: no such tile),
// and the group it belongs to: its first row, its rows, and the tiles of the
// groups before it.
struct RowTile {
    int group, row0, rows;
    int first, count, before;
};

// 64 groups from `base`, one per lane: their rows, tiles of MT rows, and the
// tiles up to and with them (`before`: of the groups before base).
struct GroupTiles {
    int lo, hi, tiles, incl;
};
// request_groups only asks for the offsets (groups past the last are empty): a
// kernel does it first and takes its block number apart while they come, with no
// exit in between (16 rows with adapters of rank 16: 8.4 -> 8.0 us).
struct GroupOffsets {
    int lo, hi;
};
__device__ __forceinline__ GroupOffsets request_groups(const int32_t* __restrict__ offsets, int groups, int base) {
    const int g = base + (threadIdx.x & (kWave - 1));
    return {offsets[min(g, groups)], offsets[min(g + 1, groups)]};
}
template <int MT>
__device__ __forceinline__ GroupTiles group_tiles(const GroupOffsets& o, int rows, int before) {
    GroupTiles t;
    t.lo = min(max(o.lo, 0), rows);
    t.hi = min(max(o.hi, t.lo), rows);
    t.tiles = (t.hi - t.lo + MT - 1) / MT;
    t.incl = before + wave_scan_incl(t.tiles);
    return t;
}

// The tile-th tile of MT rows over all groups in ascending order, found by
// one wave (all lanes active; the result is uniform): lane l takes group
// base + l, the wave's prefix sum of their tile counts places the tile.
// Groups without rows have no tiles.  g: group_tiles of base 0.
template <int MT>
__device__ __forceinline__ RowTile find_row_tile(const int32_t* __restrict__ offsets, int groups, int rows, int tile,
                                                 GroupTiles g) {
    RowTile t = {0, 0, 0, 0, 0, 0};
    for (int base = 0;;) {
        const uint64_t hit = __ballot(tile >= g.incl - g.tiles && tile < g.incl);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            t.group = base + l;
            const int first = __builtin_amdgcn_readlane(g.lo, l);
            const int last = __builtin_amdgcn_readlane(g.hi, l);
            t.before = __builtin_amdgcn_readlane(g.incl, l) - __builtin_amdgcn_readlane(g.tiles, l);
            const int at = tile - t.before;
            t.first = first;
            t.count = last - first;
            t.row0 = first + at * MT;
            t.rows = min(MT, last - t.row0);
            break;
        }
        base += kWave;
        if (base >= groups) break;
        g = group_tiles<MT>(request_groups(offsets, groups, base), rows, __builtin_amdgcn_readlane(g.incl, kWave - 1));
    }
    t.group = __builtin_amdgcn_readfirstlane(t.group);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    t.first = __builtin_amdgcn_readfirstlane(t.first);
    t.count = __builtin_amdgcn_readfirstlane(t.count);
    t.before = __builtin_amdgcn_readfirstlane(t.before);
    return t;
}

// Tiles of MT rows over all groups (uniform; all lanes active); g as above.
template <int MT>
__device__ __forceinline__ int count_row_tiles(const int32_t* __restrict__ offsets, int groups, int rows, GroupTiles g) {
    for (int base = kWave; base < groups; base += kWave)
        g = group_tiles<MT>(request_groups(offsets, groups, base), rows, __builtin_amdgcn_readlane(g.incl, kWave - 1));
    return __builtin_amdgcn_readlane(g.incl, kWave - 1);
}

// v / d for 0 <= v < 2^31 and d in [1, 16] by one product: mul = 2^shift / d
// rounded up, 2^(shift - 31) >= d, so v (mul d - 2^shift) < 2^shift.
struct RowDiv {
    uint32_t mul;
    int32_t shift;
};
inline RowDiv row_div(int d) {
    int s = 31;
    while ((1 << (s - 31)) < d) ++s;
    return {(uint32_t)((((uint64_t)1 << s) + d - 1) / d), s};
}
__device__ __forceinline__ int divide(int v, const RowDiv& d) { return (int)(((uint64_t)(uint32_t)v * d.mul) >> d.shift); }

// Most tiles of MT rows that `rows` rows in `groups` groups can make: every
// group that has rows may end in a part tile.
inline int64_t max_row_tiles(int64_t rows, int64_t groups, int mt) {
    return rows / mt + (groups < rows ? groups : rows);
}

// A launch of `blocks` workgroups in pieces that keep the grid's work-items
// below 2^32: launch(grid, workgroups of the earlier pieces).
template <typename F>
inline hipError_t launch_blocks(int64_t blocks, int threads, const F& launch) {
    const int64_t most = (((int64_t)1 << 32) - 1) / threads;
    for (int64_t b = 0; b < blocks; b += most) launch((uint32_t)(blocks - b < most ? blocks - b : most), b);
    return hipGetLastError();
}

}  // namespace qg

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

// The tile-th tile of MT rows over all groups in ascending order, found by
// one wave (all lanes active; the result is uniform): lane l takes group
// base + l, the wave's prefix sum of their tile counts places the tile.
// Groups without rows have no tiles.
template <int MT>
__device__ __forceinline__ RowTile find_row_tile(const int32_t* __restrict__ offsets, int groups, int rows, int tile) {
    const int lane = threadIdx.x & (kWave - 1);
    RowTile t = {0, 0, 0, 0, 0, 0};
    int before = 0;
    for (int base = 0; base < groups; base += kWave) {
        const int g = base + lane;
        int lo = 0, hi = 0;
        if (g < groups) {
            lo = min(max(offsets[g], 0), rows);
            hi = min(max(offsets[g + 1], lo), rows);
        }
        const int tiles = (hi - lo + MT - 1) / MT;
        const int incl = before + wave_scan_incl(tiles);
        const uint64_t hit = __ballot(tile >= incl - tiles && tile < incl);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            t.group = base + l;
            const int first = __builtin_amdgcn_readlane(lo, l);
            const int last = __builtin_amdgcn_readlane(hi, l);
            t.before = __builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(tiles, l);
            const int at = tile - t.before;
            t.first = first;
            t.count = last - first;
            t.row0 = first + at * MT;
            t.rows = min(MT, last - t.row0);
            break;
        }
        before = __builtin_amdgcn_readlane(incl, kWave - 1);
    }
    t.group = __builtin_amdgcn_readfirstlane(t.group);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    t.first = __builtin_amdgcn_readfirstlane(t.first);
    t.count = __builtin_amdgcn_readfirstlane(t.count);
    t.before = __builtin_amdgcn_readfirstlane(t.before);
    return t;
}

// Tiles of MT rows over all groups (uniform; all lanes active).
template <int MT>
__device__ __forceinline__ int count_row_tiles(const int32_t* __restrict__ offsets, int groups, int rows) {
    const int lane = threadIdx.x & (kWave - 1);
    int sum = 0;
    for (int base = 0; base < groups; base += kWave) {
        const int g = base + lane;
        if (g < groups) {
            const int lo = min(max(offsets[g], 0), rows);
            sum += (min(max(offsets[g + 1], lo), rows) - lo + MT - 1) / MT;
        }
    }
    return wave_sum(sum);
}

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

// qg_fp8_plan.h -- which kernel multiplies e4m3 operands, from the sizes alone.
// Plain host code: a CPU test asks it which kernels a list of sizes reaches.
#pragma once

#include <cmath>
#include <cstdint>

namespace qg {

constexpr int64_t kCUs = 256;  // MI355X
constexpr int kMaxParts = 8;  // of k
constexpr int64_t kPlanBlock = 128;  // values of k under one step
constexpr int64_t kStreamTokens = 1 << 20;  // a stream's grid stays below 2^16 along the tokens
constexpr int64_t kMaxGroups = 1 << 23;     // and any launch below 2^32 threads

// Which kernel runs goes by what each is expected to take, in us, from the
// sizes alone.  A tile costs `step` per block of k where its CU has one, `more`
// for each further one that shares the CU or comes after it (measured with all
// CUs at work: clocks are lower then), and `start` per launch.  Taken at
// 4096 x 4096 x 16384 (bf16 y: XL 203 us, L 244, H 293, M 262, S 420), 128 x 4096 x 4096
// (XL 43, L 28, M 21, S 15), 1100 x 4096 x 4096 (L 32, H 27, M 34, S 45) and the shapes
// named below.
enum TileKind { kS, kM, kH, kL, kXL };
struct TileCost {
    int bm, bn;
    double start, step, more;
};
constexpr TileCost kNarrow[] = {{64, 64, 4.5, 0.31, 0.20}, {128, 128, 5, 0.58, 0.54}, {192, 128, 6, 0.74, 0.80},
                                {256, 128, 6, 0.90, 0.95}, {256, 256, 8, 1.42, 1.60}};
constexpr TileCost kWide[] = {{64, 64, 4.5, 0.47, 0.33}, {128, 128, 5, 0.98, 1.08}, {192, 128, 6, 1.28, 1.50},
                              {256, 128, 6, 1.70, 1.85}};

struct Fp8Plan {
    bool stream;
    int kind, parts;  // of a stream, 16-row tiles per workgroup
    int64_t cols;  // kXL: columns of tiles before `rest` takes over
    int rest;
    double us;
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline double tiles_us(const TileCost& t, int64_t tiles, double blocks) {
    const int64_t c = ceil_div(tiles, kCUs);
    return blocks * (t.step + (double)(c - 1) * t.more);
}

// A stream's workgroups of 16 `tiles` matrix rows: `own` us per k where each CU
// has one, `more` + `more_k` k for each further round of them, besides the reading
// of the matrix (fitted to 1000 sizes of up to 300 tokens, of which the three m <= 16 and
// the two for more miss the time by 6 % and 8 % on average).
struct StreamCost {
    int tiles;
    double own, more, more_k;
};
constexpr StreamCost kFew[] = {{1, 4.2e-4, 0.46, 3.6e-4}, {2, 6.4e-4, 0.49, 5.5e-4}, {4, 12.4e-4, 0.61, 11e-4}};
constexpr StreamCost kMany[] = {{1, 6.6e-4, 1.2, 6.0e-4}, {2, 8.0e-4, 0.82, 8.3e-4}};

// Rows per workgroup by the expected time (in tiles, 16, 32 and 64 rows: 16 x 11008 x
// 4096 11.2, 11.5, 10.2 us; 16 x 22016 x 4096 19.6, 16.5, 19.4; 64 x 4096 x 4096 10.0,
// 6.5, -).
inline double stream_us(int64_t m, int64_t n, int64_t k, int* tiles) {
    const double read = (double)n * (double)k / (m <= 16 ? 14e6 : 10.4e6);
    double best = 0.0;
    *tiles = 0;
    for (int i = 0; i < (m <= 16 ? 3 : 2); ++i) {
        const StreamCost& c = m <= 16 ? kFew[i] : kMany[i];
        const int64_t rounds = ceil_div(ceil_div(n, 16 * c.tiles) * ceil_div(m, m <= 16 ? 16 : 32), kCUs);
        const double us = 3 + read + c.own * (double)k + (double)(rounds - 1) * (c.more + c.more_k * (double)k);
        if (*tiles == 0 || us < best) {
            best = us;
            *tiles = c.tiles;
        }
    }
    return best;
}

// Parts of k: their fp32 sums are written and read again, by a second launch
// (300 x 4096 x 11008: H whole 58.6 us, in 2 parts 39.1, in 4 31.5; L in 4 35.6).
inline double join_us(int64_t m, int64_t n, int parts) {
    return parts == 1 ? 0.0 : 3.5 + 4.0 * parts * (double)m * (double)n / 3.5e6;
}

inline Fp8Plan plan_fp8(int64_t m, int64_t n, int64_t k, int yt) {
    Fp8Plan best = {true, 0, 1, 0, kL, 0.0};
    best.us = stream_us(m, n, k, &best.kind);
    if (m <= 16) return best;
    if (m > kStreamTokens) best.us = 1e300;
    const int64_t kb = k / kPlanBlock;
    const double read = (double)n * (double)k / 5e6;  // the matrix from memory
    const TileCost* cost = yt == 0 ? kWide : kNarrow;
    for (int kind = kS; kind <= (yt == 0 ? kL : kXL); ++kind) {
        const TileCost& t = cost[kind];
        const int64_t tiles = ceil_div(m, t.bm) * ceil_div(n, t.bn);
        for (int parts = 1; parts <= kMaxParts && parts <= kb; ++parts) {
            if (parts > 1 && tiles * (parts - 1) >= 2 * kCUs) break;  // CUs enough without
            if (tiles * parts >= kMaxGroups) break;
            const double us = t.start + fmax(tiles_us(t, tiles * parts, (double)ceil_div(kb, parts)), read) + join_us(m, n, parts);
            if (us < best.us) best = {false, kind, parts, n, kL, us};
        }
    }
    // whole rounds of XL, the rest of the matrix in L or H (2048 x 11008 x 4096: XL
    // 111 us, L 109, 32 columns of XL and 22 of L 96, of H 92)
    if (yt != 0) {
        const int64_t tm = ceil_div(m, cost[kXL].bm), tn = ceil_div(n, cost[kXL].bn), rounds = tm * tn / kCUs;
        const int64_t cols = rounds * kCUs / tm;
        for (int kind = kH; kind <= kL && cols >= 1 && cols < tn; ++kind) {
            const int64_t rest = ceil_div(m, cost[kind].bm) * ceil_div(n - cols * cost[kXL].bn, cost[kind].bn);
            const double us = cost[kXL].start + tiles_us(cost[kXL], tm * cols, (double)kb) +
                              (double)kb * (double)ceil_div(rest, kCUs) * cost[kind].more;
            if (us < best.us) best = {false, kXL, 1, cols, kind, us};
        }
    }
    return best;
}

}  // namespace qg

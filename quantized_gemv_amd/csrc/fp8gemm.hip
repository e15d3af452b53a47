// fp8gemm.hip -- product of e4m3 operands with an fp32 step per block of 128
// (gfx950).
//
//   y[m][n] = sum over blocks b of s_x[b][m] s_w[n / 128][b] P_b,
//   P_b     = sum of x[m][k] w[n][k] over the 128 k of block b.
//
// P_b comes from the matrix cores, its accumulator starting at 0; the steps go
// on in the vector unit, one multiply-add per output and block into fp32.  The
// matrix rows are operand A and the tokens operand B: a lane then holds four
// outputs of one token (column l % 16, rows 4 (l / 16) ..), so the product of
// the two steps is one value per lane and tile.  Lane l supplies 32 codes of
// row l % 16: the 16 bytes at 16 (l / 16) and those 64 further, for both
// operands, so the instruction's own pairing of k is the dot product whatever
// it is.
//
// Two instructions give P_b.  v_mfma_f32_16x16x128_f8f6f4 takes the codes as
// they are, at twice the rate of bf16, but is not exact: measured on MI355X, of
// eight products (eight consecutive k) each is cut off, towards zero, below
// 2^-13 of the largest's binade before they are added; the sums of eight add
// in fp32.  On codes of Gaussian values the result is off by 1.6e-5 of its
// size, at worst by 7 2^-13 of each eight's largest product.  For bf16 outputs
// (half a step: 3.9e-3) it serves where the matrix cores bound the time.
// Elsewhere, and for every fp32 output, the codes are widened to bf16, which
// holds every e4m3 value, and four v_mfma_f32_16x16x32_bf16 add exact products
// in fp32 (1.2e-8 on the same values).
#include "qg_fp8.h"
#include "qg_fp8_plan.h"
#include "qg_gemm.h"
#include "qg_launch.h"

namespace qg {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct Fp8Params {
    const uint8_t* codes;
    const float* s_w;
    const uint8_t* x;
    const float* s_x;
    int64_t M, N;
    int K, KB;  // KB = K / 128
    void* y;
    int yt;
    // tile kernels: the matrix rows from n1 on go in the second kind of tile; parts
    // of k, their sums [parts][M][ld] in fp32 where there is more than one
    int64_t n1;
    int tiles_m, tiles_n, tiles_m2, tiles_n2, parts;
    float* sums;
};

// 32 codes of a row as the matrix instructions take them.
template <bool WIDE>
struct Operand {
    i32x8 q;
};
template <>
struct Operand<true> {
    bf16x8 h[4];
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <bool WIDE>
__device__ __forceinline__ Operand<WIDE> operand(u32x4 a, u32x4 b) {
    Operand<WIDE> o;
    const uint32_t w[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (WIDE) {
            const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, false);
            const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, true);
            o.h[i >> 1][4 * (i & 1) + 0] = lo[0];
            o.h[i >> 1][4 * (i & 1) + 1] = lo[1];
            o.h[i >> 1][4 * (i & 1) + 2] = hi[0];
            o.h[i >> 1][4 * (i & 1) + 3] = hi[1];
        } else {
            o.q[i] = (int)w[i];
        }
    }
    return o;
}

template <bool WIDE>
__device__ __forceinline__ f32x4 block_product(const Operand<WIDE>& a, const Operand<WIDE>& b) {
    f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.h[i], b.h[i], d, 0, 0, 0);
    } else {
        d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.q, b.q, d, 0, 0, 0, 0, 0, 0);
    }
    return d;
}

// Where outputs go: rows of ld values, of which the first n exist; whole: every
// four columns from a multiple of 4 can be stored at once.
struct Out {
    void* y;
    int yt;  // 0: fp32, 1: bf16
    int64_t ld, n;
    bool whole;
};

// Four outputs of one token, columns n .. n + 3 (n < o.n).
__device__ __forceinline__ void store4(const Out& o, int64_t m, int64_t n, f32x4 v) {
    const int64_t at = m * o.ld + n;
    if (o.yt == 0) {
        float* y = static_cast<float*>(o.y) + at;
        if (o.whole) {
            *reinterpret_cast<f32x4*>(y) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < o.n) y[i] = v[i];
        }
    } else {
        uint16_t* y = static_cast<uint16_t*>(o.y) + at;
        if (o.whole) {
            *reinterpret_cast<uint2*>(y) = make_uint2(any_f32_to_bf16(v[0]) | (any_f32_to_bf16(v[1]) << 16),
                                                      any_f32_to_bf16(v[2]) | (any_f32_to_bf16(v[3]) << 16));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < o.n) y[i] = (uint16_t)any_f32_to_bf16(v[i]);
        }
    }
}
__device__ __forceinline__ Out output_of(const Fp8Params& p) { return {p.y, p.yt, p.N, p.N, (p.N & 3) == 0}; }

// ------------------------------------------------------------------ few tokens
// The time goes into reading the matrix once.  A workgroup multiplies 16 RT
// matrix rows with 16 MT tokens; its NW waves take the blocks of k in turn, U
// of them requested ahead, and their sums meet in LDS in wave order.  Rows are
// requested in whole lines, eight lanes to the 128 bytes of each, and pass
// through the wave's own LDS into the order of the matrix instruction (requested
// in that order, 16 bytes here and there: 16 x 22016 x 4096 row-major 22.5 against
// 19.0 us, 64 x 11008 x 4096 in tiles, where bf16 outputs now come from 64 x 64 tiles,
// 21.5 against 17.4); the next block is
// requested as soon as they are there.  Blocks past the last are requested past
// the end of the buffer, which reads zeros and moves nothing; their step is 0, as
// the last block's, which is read again for them, may be infinite.  ONCE: the
// matrix is read by this one pass and goes past the caches.
// A wave's LDS accesses before this come before those after it.
__device__ __forceinline__ void lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int MT, int RT, bool TILED, bool WIDE, int NW, int U, bool ONCE>
__global__ __launch_bounds__(64 * NW) void fp8_stream_kernel(Fp8Params p) {
    constexpr int kTurn = 128 * ((TILED ? 0 : RT) + MT), kRed = 64 * MT * RT;
    __shared__ u32x4 lds[NW][kTurn > kRed ? kTurn : kRed];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    u32x4* turn = lds[wave];
    const int r = lane & 15, g = lane >> 4;
    const int64_t tile0 = (int64_t)blockIdx.x * RT;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
    const int64_t rows_w = TILED ? (p.N + 15) / 16 * 16 : p.N;
    const int rw = (int)min((int64_t)16 * RT, rows_w - 16 * tile0);
    const int rx = (int)min((int64_t)16 * MT, p.M - m0);
    const uint32_t w_bytes = (uint32_t)rw * (uint32_t)p.K, x_bytes = (uint32_t)rx * (uint32_t)p.K;
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(p.codes + 16 * tile0 * p.K, w_bytes);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x + m0 * p.K, x_bytes);
    const float* sw = p.s_w + 16 * tile0 / kFp8Block * p.KB;
    // Row-major: lanes 8 i .. 8 i + 7 read the 128 bytes of row i, then of row 8 + i.
    uint32_t wo[RT], wo8[RT], xo[MT], xo8[MT];
    const float* sx[MT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        wo[t] = TILED ? (uint32_t)min(t, rw / 16 - 1) * 16u * (uint32_t)p.K + 16u * lane
                      : (uint32_t)min(16 * t + (lane >> 3), rw - 1) * (uint32_t)p.K + 16u * (lane & 7);
        wo8[t] = (uint32_t)min(16 * t + 8 + (lane >> 3), rw - 1) * (uint32_t)p.K + 16u * (lane & 7);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        xo[t] = (uint32_t)min(16 * t + (lane >> 3), rx - 1) * (uint32_t)p.K + 16u * (lane & 7);
        xo8[t] = (uint32_t)min(16 * t + 8 + (lane >> 3), rx - 1) * (uint32_t)p.K + 16u * (lane & 7);
        sx[t] = p.s_x + m0 + min(16 * t + r, rx - 1);
    }

    u32x4 wb[U][RT][2], xb[U][MT][2];
    float sb[U][MT], swb[U];
    auto request = [&](int u, int kb) {
        const bool in = kb < p.KB;
        const int kc = min(kb, p.KB - 1);
        const uint32_t ws = (uint32_t)kc * (TILED ? 2048u : 128u), xs = (uint32_t)kc * 128u;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const uint32_t o = in ? wo[t] + ws : w_bytes;
            const uint32_t o2 = !in ? w_bytes : TILED ? o + 1024u : wo8[t] + ws;
            wb[u][t][0] = ONCE ? load16_nt(wr, o) : load16(wr, o);
            wb[u][t][1] = ONCE ? load16_nt(wr, o2) : load16(wr, o2);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            xb[u][t][0] = load16(xr, in ? xo[t] + xs : x_bytes);
            xb[u][t][1] = load16(xr, in ? xo8[t] + xs : x_bytes);
            sb[u][t] = sx[t][(int64_t)kc * p.M];
        }
        swb[u] = sw[kc];
    };
    f32x4 acc[MT][RT];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < RT; ++b) acc[a][b] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < U; ++u) request(u, wave + NW * u);
    for (int kb = wave; kb < p.KB; kb += NW * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // Through LDS into the order of the matrix instruction; a wave's own part, so that
            // it waits for no other.
            auto put = [&](int t, const u32x4* v) __attribute__((always_inline)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = 8 * h + (lane >> 3);
                    turn[128 * t + 8 * row + swz<8>(row, lane & 7)] = v[h];
                }
            };
            auto get = [&](int t, u32x4* v) __attribute__((always_inline)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) v[h] = turn[128 * t + 8 * r + swz<8>(r, g + 4 * h)];
            };
            u32x4 fw[RT][2], fx[MT][2];
            float c[MT];
#pragma unroll
            for (int b = 0; b < RT; ++b) {
                if constexpr (TILED) {
                    fw[b][0] = wb[u][b][0];
                    fw[b][1] = wb[u][b][1];
                } else {
                    put(MT + b, wb[u][b]);
                }
            }
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                put(a, xb[u][a]);
                const float step = sb[u][a] * swb[u];
                c[a] = u == 0 || kb + NW * u < p.KB ? step : 0.0f;
            }
            request(u, kb + NW * (U + u));
            lds_order();
            if constexpr (!TILED)
#pragma unroll
                for (int b = 0; b < RT; ++b) get(MT + b, fw[b]);
#pragma unroll
            for (int a = 0; a < MT; ++a) get(a, fx[a]);
            lds_order();
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                const Operand<WIDE> bx = operand<WIDE>(fx[a][0], fx[a][1]);
#pragma unroll
                for (int b = 0; b < RT; ++b) {
                    const f32x4 d = block_product<WIDE>(operand<WIDE>(fw[b][0], fw[b][1]), bx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[a][b][i] = __builtin_fmaf(d[i], c[a], acc[a][b][i]);
                }
            }
        }
    }
    f32x4* red = reinterpret_cast<f32x4*>(turn);
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < RT; ++b) red[64 * (a * RT + b) + lane] = acc[a][b];
    __syncthreads();
    const Out o = output_of(p);
    for (int q = threadIdx.x; q < MT * RT * 64; q += 64 * NW) {
        const int t = q >> 6, l = q & 63;
        f32x4 v = reinterpret_cast<const f32x4*>(lds[0])[64 * t + l];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += reinterpret_cast<const f32x4*>(lds[w])[64 * t + l];
        const int64_t m = m0 + 16 * (t / RT) + (l & 15);
        const int64_t n = 16 * (tile0 + t % RT) + 4 * (l >> 4);
        if (m < p.M && n < p.N) store4(o, m, n, v);
    }
}

// ------------------------------------------------------------------ many tokens
// A workgroup of WAVES_M x WAVES_N waves computes BM tokens x BN matrix rows
// over KB / parts blocks of k.  Both operands go through STAGES LDS buffers of
// a block each, filled by direct global -> LDS loads; rows of 128 bytes are
// stored with their 16-byte chunks permuted by the row (swz), 16-row tiles as
// they are: both are read without bank conflicts.
//
// What bounds it is the loads into LDS (from the L2s about 65 bytes per ns and
// CU with all of them at work), so they never stop: a buffer is refilled in two
// parts while its block is still multiplied.  The matrix rows' fragments and
// those of the first part of a wave's tokens (half or fewer) are in registers
// first (a group of 16 tokens is read LA groups ahead); once every wave has them,
// that part is requested again (S1), the second part when that is read (S2), each
// about 1.5 blocks before it is wanted.  The loads are spread between the matrix
// instructions (at once, a wave would stand still until the address unit has
// taken all of them: 2.45 -> 2.57 PFLOP/s at 4096 x 4096 x 16384), and the
// products of kLag instructions ago take their steps beside them.
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_>
struct Fp8Tile {
    static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, STAGES = STAGES_;
    static constexpr int kNW = WAVES_M * WAVES_N;
    static constexpr int MT = BM / WAVES_M / 16, NT = BN / WAVES_N / 16;
    static constexpr int kCodes = (BM + BN) * kFp8Block;
    // Tiles of 16 tokens of a wave in the first part: half of them, or fewer where
    // that gives every wave as many loads.
    static constexpr int head() {
        int h = MT / 2;
        while (h * 2 * WAVES_M % kNW != 0) --h;
        return h;
    }
    static constexpr int H = head();
    static constexpr int kX1 = 2 * H * WAVES_M / kNW;         // 1 KB loads per wave: the first part's rows of x,
    static constexpr int kX2 = 2 * (MT - H) * WAVES_M / kNW;  // the second's,
    static constexpr int kW = BN / 8 / kNW;                   // all of the matrix's,
    static constexpr int kScaleLoads = BM / 64 + 1;  // and of all waves 64 steps of x each, then those of w
    static constexpr int kSL = (kScaleLoads + kNW - 1) / kNW;
    static constexpr int kScales = 256 * kScaleLoads;
    static constexpr int kFirst = kW + kX1 + kSL, kSecond = kX2;  // loads of a block's two parts
    static_assert(H > 0 && 2 * (MT - H) * WAVES_M % kNW == 0 && BN % (8 * kNW) == 0 && BM % 64 == 0 && kFp8Block % (BN / WAVES_N) == 0,
                  "whole loads per wave, one step of w per wave");
    static constexpr int kLds = STAGES * kCodes + (STAGES + 1) * kScales;
    static constexpr int kPerSimd = 160 * 1024 / kLds * kNW / 4;  // waves that the LDS has room for
};

template <class C, bool TILED, bool WIDE>
__device__ __forceinline__ void fp8_tile(const Fp8Params& p, uint8_t* smem, int64_t m0, int64_t n0, int kb0, int kb1,
                                         const Out& out) {
    constexpr int BM = C::BM, BN = C::BN, WAVES_M = C::WAVES_M, WAVES_N = C::WAVES_N, STAGES = C::STAGES;
    constexpr int MT = C::MT, NT = C::NT, NW = C::kNW;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;
    const int r = lane & 15, g = lane >> 4;

    const int rx = (int)min((int64_t)BM, p.M - m0);
    const int64_t rows_w = TILED ? (p.N + 15) / 16 * 16 : p.N;
    const int rw = (int)min((int64_t)BN, rows_w - n0);
    // This lane's 16 bytes at block 0 of each load: x's rows in two parts (every
    // wave row's first tokens, then the rest), w's rows or tiles.
    constexpr int R = BM / WAVES_M, H = C::H;  // tokens of a wave
    auto x_row = [&](int part, int l) {
        const int j = wave + NW * l, per = 2 * (part == 0 ? H : MT - H);
        return j / per * R + (part == 0 ? 0 : 16 * H) + 8 * (j % per);
    };
    uint32_t xo[2][C::kX1 > C::kX2 ? C::kX1 : C::kX2], wo[C::kW];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int l = 0; l < (h == 0 ? C::kX1 : C::kX2); ++l) {
            const int row = x_row(h, l) + (lane >> 3);
            xo[h][l] = (uint32_t)min(row, rx - 1) * (uint32_t)p.K + 16u * swz<8>(row, lane & 7);
        }
#pragma unroll
    for (int l = 0; l < C::kW; ++l) {
        const int b = wave + NW * l, row = 8 * b + (lane >> 3);
        wo[l] = TILED ? (uint32_t)min(b >> 1, rw / 16 - 1) * 16u * (uint32_t)p.K + 1024u * (b & 1) + 16u * lane
                      : (uint32_t)min(row, rw - 1) * (uint32_t)p.K + 16u * swz<8>(row, lane & 7);
    }
    const float* ssrc[C::kSL];
    int64_t sstr[C::kSL];
    int sdst[C::kSL];
#pragma unroll
    for (int l = 0; l < C::kSL; ++l) {
        const int sj = min(wave + NW * l, C::kScaleLoads - 1);
        if (sj < BM / 64) {
            ssrc[l] = p.s_x + m0 + min(64 * sj + lane, rx - 1);
            sstr[l] = p.M;
        } else {  // lanes past BN / 128 repeat the last: all in one line
            const int64_t nb = min(n0 / kFp8Block + min(lane, (BN - 1) / kFp8Block), (p.N - 1) / kFp8Block);
            ssrc[l] = p.s_w + nb * p.KB;
            sstr[l] = 1;
        }
        sdst[l] = STAGES * C::kCodes + 256 * sj;
    }
    // Blocks past the last are requested outside of empty buffers: nothing is
    // read, the loop has no branch, and every wait is for the same number of loads.
    const uint32_t x_bytes = (uint32_t)rx * (uint32_t)p.K, w_bytes = (uint32_t)rw * (uint32_t)p.K;
    auto issue_x = [&](int h, int l, int kb, int to) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x + m0 * p.K, kb < kb1 ? x_bytes : 0u);
        dma16_buffer(xr, smem + to * C::kCodes + x_row(h, l) * kFp8Block, xo[h][l], (uint32_t)kb * 128u);
    };
    // load i of a block's first part: w, half of x, the steps
    auto issue_first = [&](int i, int kb, int to, int sto) __attribute__((always_inline)) {
        if (i < C::kW) {
            const __amdgpu_buffer_rsrc_t wr = make_rsrc(p.codes + n0 * p.K, kb < kb1 ? w_bytes : 0u);
            dma16_buffer(wr, smem + to * C::kCodes + (BM / 8 + wave + NW * i) * 1024, wo[i],
                         (uint32_t)kb * (TILED ? 2048u : 128u));
        } else if (i < C::kW + C::kX1) {
            issue_x(0, i - C::kW, kb, to);
        } else {
            const int l = i - C::kW - C::kX1;
            dma4(ssrc[l] + (int64_t)min(kb, kb1 - 1) * sstr[l], smem + sdst[l] + sto * C::kScales);
        }
    };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int b = 0; b < MT; ++b) acc[a][b] = {0.0f, 0.0f, 0.0f, 0.0f};

    // Fragments and steps of a block, read from its LDS buffer.
    constexpr int LA = MT > 2 ? 2 : 1;
    constexpr int XR = MT % 4 == 0 ? 4 : MT % 3 == 0 ? 3 : 2;
    static_assert(MT % XR == 0 && XR > LA && H >= LA, "a whole turn of the ring per block");
    u32x4 fw[NT][2], fx[XR][2];
    float sx[XR], sw = 0.0f;
    // Rows 16 further have the same permutation, so a tile's address is one lane's
    // offset and a constant in the instruction (an offset per tile: 28 more additions
    // beside 32 matrix instructions, 4096 x 4096 x 16384 203 -> 212 us).
    const int xrow = wm * R + r, wrow = wn * (16 * NT) + r;
    const int xl = xrow * kFp8Block + 16 * swz<8>(xrow, g), xh = xrow * kFp8Block + 16 * swz<8>(xrow, g + 4);
    const int wl = BM * kFp8Block + (TILED ? wn * NT * 2048 + 16 * lane : wrow * kFp8Block + 16 * swz<8>(wrow, g));
    const int wh = TILED ? wl + 1024 : BM * kFp8Block + wrow * kFp8Block + 16 * swz<8>(wrow, g + 4);
    auto read_x = [&](const uint8_t* base, const uint8_t* sc, int b) __attribute__((always_inline)) {
        fx[b % XR][0] = *reinterpret_cast<const u32x4*>(base + xl + 2048 * b);
        fx[b % XR][1] = *reinterpret_cast<const u32x4*>(base + xh + 2048 * b);
        sx[b % XR] = *reinterpret_cast<const float*>(sc + 4 * xrow + 64 * b);
    };
    auto read_w = [&](const uint8_t* base, int a) __attribute__((always_inline)) {
        fw[a][0] = *reinterpret_cast<const u32x4*>(base + wl + 2048 * a);
        fw[a][1] = *reinterpret_cast<const u32x4*>(base + wh + 2048 * a);
    };
    auto read_sw = [&](const uint8_t* sc) {
        return reinterpret_cast<const float*>(sc)[BM + wn * (BN / WAVES_N) / kFp8Block];
    };

    // Block products wait in a ring for kLag steps before the vector unit
    // takes them up, so that neither waits for the other.
    constexpr int kLag = NT < 3 ? NT : 3, T = NT * MT;
    static_assert(T % 4 == 0, "ring of four");
    f32x4 d[4];
    float c_last = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = {0.0f, 0.0f, 0.0f, 0.0f};

    const uint8_t* scales = smem + STAGES * C::kCodes;
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
#pragma unroll
        for (int i = 0; i < C::kFirst; ++i) issue_first(i, kb0 + s, s, s);
#pragma unroll
        for (int i = 0; i < C::kSecond; ++i) issue_x(1, i, kb0 + s, s);
    }
    // The loads younger than the part that a wait is for: the first part of block
    // kb + 1 at S2 (after it the second of kb + 1, then pairs up to the first of
    // kb + STAGES), the second part of block kb at S1 likewise.
    constexpr int kAhead = (STAGES - 1) * (C::kFirst + C::kSecond);
    wait_vmcnt<kAhead + C::kSecond>();
    lds_barrier();
#pragma unroll
    for (int b = 0; b < LA; ++b) read_x(smem, scales, b);
#pragma unroll
    for (int a = 0; a < NT; ++a) read_w(smem, a);
    sw = read_sw(scales);

    constexpr int S1 = H - LA, S2 = MT - LA;
    int slot = 0, sslot = 0;  // of block kb; the steps have one buffer more, as they are read to the block's end
    for (int kb = kb0; kb < kb1; ++kb) {
        const uint8_t* here = smem + slot * C::kCodes;
        const uint8_t* shere = scales + sslot * C::kScales;
        const int freed = slot, sfree = sslot == 0 ? STAGES : sslot - 1;
        slot = slot + 1 == STAGES ? 0 : slot + 1;
        sslot = sslot == STAGES ? 0 : sslot + 1;
        const uint8_t* next = smem + slot * C::kCodes;
        const uint8_t* snext = scales + sslot * C::kScales;
        float sw_next = 0.0f;
        Operand<WIDE> w[NT];
#pragma unroll
        for (int b = 0; b < MT; ++b) {
            if (b == S1) {  // the second half of block kb has landed; its matrix rows and first half are read
                wait_vmcnt<kAhead>();
                lds_barrier();
            }
            if (b == S2) {  // the first part of block kb + 1 has landed; all of block kb is read
                wait_vmcnt<kAhead>();
                lds_barrier();
                sw_next = read_sw(snext);
            }
            const Operand<WIDE> x = operand<WIDE>(fx[b % XR][0], fx[b % XR][1]);
            const float c = sx[b % XR] * sw;
            if (b < MT - LA) read_x(here, shere, b + LA);
            else read_x(next, snext, b + LA - MT);
#pragma unroll
            for (int a = 0; a < NT; ++a) {
                if (b == 0) w[a] = operand<WIDE>(fw[a][0], fw[a][1]);
                const int t = b * NT + a, u = (t + T - kLag) % T;
                d[t & 3] = block_product<WIDE>(w[a], x);
                constexpr int n1 = (S2 - S1) * NT, n2 = (MT - S2) * NT;
                if (b >= S1 && b < S2) {
                    const int q = t - S1 * NT;
#pragma unroll
                    for (int i = q * C::kFirst / n1; i < (q + 1) * C::kFirst / n1; ++i)
                        issue_first(i, kb + STAGES, freed, sfree);
                } else if (b >= S2) {
                    const int q = t - S2 * NT;
#pragma unroll
                    for (int i = q * C::kSecond / n2; i < (q + 1) * C::kSecond / n2; ++i)
                        issue_x(1, i, kb + STAGES, freed);
                }
                if (b == MT - 1) read_w(next, a);
                const float cu = a < kLag ? c_last : c;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4& v = acc[u % NT][u / NT];
                    v[i] = __builtin_fmaf(d[u & 3][i], cu, v[i]);
                }
            }
            c_last = c;
            if constexpr (!WIDE) {
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a matrix instruction,
                    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // LDS reads,
                    __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);  // vector instructions
                }
            } else if (b == 0) {  // the matrix rows' conversions among the instructions (128x128, 64x64: 3-4% of the time)
                __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
#pragma unroll
                for (int i = 0; i < 4 * NT; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
                    if (i % 4 == 3) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                }
            } else {
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
#pragma unroll
                for (int i = 0; i < 4 * NT; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
                    if (i % 4 == 3) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        sw = sw_next;
    }
    wait_vmcnt<0>();  // no load into LDS outlives the workgroup
#pragma unroll
    for (int u = T - kLag; u < T; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4& v = acc[u % NT][u / NT];
            v[i] = __builtin_fmaf(d[u & 3][i], c_last, v[i]);
        }
#pragma unroll
    for (int b = 0; b < MT; ++b) {
        const int64_t m = m0 + wm * R + 16 * b + r;
#pragma unroll
        for (int a = 0; a < NT; ++a) {
            const int64_t n = n0 + wn * (16 * NT) + 16 * a + 4 * g;
            if (m < p.M && n < p.N) store4(out, m, n, acc[a][b]);
        }
    }
}

// Tile t of tiles_m x tiles_n, in supertiles of 4 token tiles: workgroups that
// follow one another, and so the XCD's that share an L2, read the same rows.
__device__ __forceinline__ void tile_at(int64_t t, int tiles_m, int tiles_n, int64_t& tm, int64_t& tn) {
    const int64_t per = 4 * (int64_t)tiles_n;
    const int64_t st = t / per, u = t - st * per;
    const int64_t h = min((int64_t)4, tiles_m - 4 * st);
    tm = 4 * st + u % h;
    tn = u / h;
}

// Tiles of kind A, then those of kind B for the matrix rows from n1 on.  Registers for
// as many waves as the LDS has room for: for more, 64 x 64 with widened codes moves sums
// to and from the accumulation registers (4096 x 4096 x 4096 190 -> 178 us).
template <class A, class B, bool TILED, bool WIDE>
__global__ __launch_bounds__(64 * A::kNW) __attribute__((amdgpu_waves_per_eu(2, A::kPerSimd))) void fp8_tile_kernel(Fp8Params p) {
    static_assert(A::kNW == B::kNW, "one size of workgroup");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[A::kLds > B::kLds ? A::kLds : B::kLds];
    const int64_t first = (int64_t)p.tiles_m * p.tiles_n * p.parts;
    int64_t tm, tn;
    if (blockIdx.x < first) {
        const int64_t w = xcd_run(blockIdx.x, first), tiles = (int64_t)p.tiles_m * p.tiles_n;
        const int part = (int)(w / tiles);
        tile_at(w - part * tiles, p.tiles_m, p.tiles_n, tm, tn);
        const int64_t ld = (p.N + 3) / 4 * 4;
        const Out o = p.parts == 1 ? output_of(p) : Out{p.sums + part * p.M * ld, 0, ld, ld, true};
        fp8_tile<A, TILED, WIDE>(p, smem, tm * A::BM, tn * A::BN, (int)((int64_t)p.KB * part / p.parts),
                                 (int)((int64_t)p.KB * (part + 1) / p.parts), o);
    } else if constexpr (!std::is_same<A, B>::value) {
        tile_at(xcd_run(blockIdx.x - first, gridDim.x - first), p.tiles_m2, p.tiles_n2, tm, tn);
        fp8_tile<B, TILED, WIDE>(p, smem, tm * B::BM, p.n1 + tn * B::BN, 0, p.KB, output_of(p));
    }
}

// The sums of the parts of k, added in their order.
__global__ __launch_bounds__(kThreads) void fp8_join_kernel(Fp8Params p) {
    const int64_t ld4 = (p.N + 3) / 4, chunks = p.M * ld4;
    const Out o = output_of(p);
    const f32x4* s = reinterpret_cast<const f32x4*>(p.sums);
    for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < chunks; c += (int64_t)gridDim.x * kThreads) {
        f32x4 v = s[c];
        for (int q = 1; q < p.parts; ++q) v += s[q * chunks + c];
        const int64_t m = c / ld4;
        store4(o, m, 4 * (c - m * ld4), v);
    }
}

template <int MT, int RT, bool WIDE, int NW, int U, bool ONCE>
hipError_t run_stream(const Fp8Params& p, bool t16, hipStream_t st) {
    const dim3 grid((uint32_t)((p.N + 16 * RT - 1) / (16 * RT)), (uint32_t)((p.M + 16 * MT - 1) / (16 * MT)));
    if (t16) fp8_stream_kernel<MT, RT, true, WIDE, NW, U, ONCE><<<grid, 64 * NW, 0, st>>>(p);
    else fp8_stream_kernel<MT, RT, false, WIDE, NW, U, ONCE><<<grid, 64 * NW, 0, st>>>(p);
    return hipGetLastError();
}

// cols: columns of tiles of kind A (all of them where that is enough).
template <class A, class B, bool WIDE>
hipError_t run_tiles(Fp8Params p, bool t16, hipStream_t st, int64_t cols, int parts) {
    if (parts > p.KB) return hipErrorInvalidValue;  // a part without a block has no steps to read
    p.tiles_m = (int)((p.M + A::BM - 1) / A::BM);
    p.tiles_n = (int)((p.N + A::BN - 1) / A::BN);
    p.tiles_m2 = p.tiles_n2 = 0;
    if (cols < p.tiles_n) {
        p.tiles_n = (int)cols;
        p.n1 = cols * A::BN;
        p.tiles_m2 = (int)((p.M + B::BM - 1) / B::BM);
        p.tiles_n2 = (int)((p.N - p.n1 + B::BN - 1) / B::BN);
    }
    p.parts = parts;
    const int64_t grid = (int64_t)p.tiles_m * p.tiles_n * parts + (int64_t)p.tiles_m2 * p.tiles_n2;
    if (t16) fp8_tile_kernel<A, B, true, WIDE><<<(uint32_t)grid, 64 * A::kNW, 0, st>>>(p);
    else fp8_tile_kernel<A, B, false, WIDE><<<(uint32_t)grid, 64 * A::kNW, 0, st>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || parts == 1) return e;
    const int64_t chunks = p.M * ((p.N + 3) / 4), want = (chunks + kThreads - 1) / kThreads;
    fp8_join_kernel<<<(uint32_t)(want < 4096 ? want : 4096), kThreads, 0, st>>>(p);
    return hipGetLastError();
}

typedef Fp8Tile<256, 256, 2, 4, 2> TileXL;
typedef Fp8Tile<256, 128, 4, 2, 2> TileL;
typedef Fp8Tile<192, 128, 2, 4, 2> TileH;
typedef Fp8Tile<128, 128, 2, 4, 2> TileM;
typedef Fp8Tile<64, 64, 2, 2, 4> TileS;

template <bool WIDE>
hipError_t run_plan(const Fp8Params& p, bool t16, const Fp8Plan& plan, hipStream_t st) {
    switch (plan.kind) {
        case kS: return run_tiles<TileS, TileS, WIDE>(p, t16, st, p.N, plan.parts);
        case kM: return run_tiles<TileM, TileM, WIDE>(p, t16, st, p.N, plan.parts);
        case kH: return run_tiles<TileH, TileH, WIDE>(p, t16, st, p.N, plan.parts);
        case kL: return run_tiles<TileL, TileL, WIDE>(p, t16, st, p.N, plan.parts);
        default: break;
    }
    if constexpr (WIDE) return hipErrorInvalidValue;  // no plan of fp32 outputs has it
    else if (plan.rest == kH) return run_tiles<TileXL, TileH, false>(p, t16, st, plan.cols, plan.parts);
    else return run_tiles<TileXL, TileL, false>(p, t16, st, plan.cols, plan.parts);
}

}  // namespace

size_t fp8_workspace(int64_t m, int64_t n, int64_t k, int yt) {
    const Fp8Plan plan = plan_fp8(m, n, k, yt);
    return plan.parts == 1 ? 0 : (size_t)plan.parts * (size_t)m * (size_t)((n + 3) / 4 * 4) * sizeof(float);
}

hipError_t launch_qgemm_fp8(const Fp8GemmArgs& a, hipStream_t st) {
    Fp8Params p = {};
    p.codes = a.codes;
    p.s_w = a.s_w;
    p.x = a.x;
    p.s_x = a.s_x;
    p.M = a.m;
    p.N = a.n;
    p.K = (int)a.k;
    p.KB = (int)(a.k / kFp8Block);
    p.y = a.y;
    p.yt = a.yt;
    p.sums = static_cast<float*>(a.ws);
    const Fp8Plan plan = plan_fp8(a.m, a.n, a.k, a.yt);
    if (!plan.stream) return a.yt == 0 ? run_plan<true>(p, a.t16, plan, st) : run_plan<false>(p, a.t16, plan, st);
    // Up to 32 tokens are one pass over the matrix: past the caches, which do not hold
    // it then (1 x 4096 x 4096 5.7 -> 5.3 us, 16 x 22016 x 4096 19.0 -> 17.2).
    if (a.m <= 16) {
        if (plan.kind == 4) return run_stream<1, 4, true, 8, 1, true>(p, a.t16, st);
        if (plan.kind == 2) return run_stream<1, 2, true, 8, 1, true>(p, a.t16, st);
        if (a.k > 4096) return run_stream<1, 1, true, 16, 1, true>(p, a.t16, st);  // 1 x 4096 x 11008 11.8 -> 11.2 us
        return run_stream<1, 1, true, 8, 2, true>(p, a.t16, st);
    }
    if (a.m <= 32) {
        if (plan.kind == 2) return run_stream<2, 2, true, 8, 1, true>(p, a.t16, st);
        return run_stream<2, 1, true, 8, 2, true>(p, a.t16, st);
    }
    if (plan.kind == 2) return run_stream<2, 2, true, 8, 1, false>(p, a.t16, st);
    return run_stream<2, 1, true, 8, 2, false>(p, a.t16, st);
}

}  // namespace qg

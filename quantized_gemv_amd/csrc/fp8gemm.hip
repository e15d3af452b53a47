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
    int tiles_m, tiles_n;
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

// Four outputs of one token, columns n .. n + 3 (those below N).
__device__ __forceinline__ void store4(const Fp8Params& p, int64_t m, int64_t n, f32x4 v) {
    const int64_t at = m * p.N + n;
    const bool whole = (p.N & 3) == 0;  // then n + 3 < N, and the address is a multiple of the store
    if (p.yt == 0) {
        float* y = static_cast<float*>(p.y) + at;
        if (whole) {
            *reinterpret_cast<f32x4*>(y) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < p.N) y[i] = v[i];
        }
    } else {
        uint16_t* y = static_cast<uint16_t*>(p.y) + at;
        if (whole) {
            *reinterpret_cast<uint2*>(y) = make_uint2(any_f32_to_bf16(v[0]) | (any_f32_to_bf16(v[1]) << 16),
                                                      any_f32_to_bf16(v[2]) | (any_f32_to_bf16(v[3]) << 16));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < p.N) y[i] = (uint16_t)any_f32_to_bf16(v[i]);
        }
    }
}

// ------------------------------------------------------------------ few tokens
// The time goes into reading the matrix once.  A workgroup multiplies 16 RT
// matrix rows with 16 MT tokens; its NW waves take the blocks of k in turn, U
// of them requested ahead, and their sums meet in LDS in wave order.  Blocks
// past the last are requested past the end of the buffer, which reads zeros
// and moves nothing.
template <int MT, int RT, bool TILED, bool WIDE, int NW, int U>
__global__ __launch_bounds__(64 * NW) void fp8_stream_kernel(Fp8Params p) {
    __shared__ f32x4 red[NW][MT * RT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    uint32_t wo[RT], xo[MT];
    const float* sx[MT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
        wo[t] = TILED ? (uint32_t)min(t, rw / 16 - 1) * 16u * (uint32_t)p.K + 16u * lane
                      : (uint32_t)min(16 * t + r, rw - 1) * (uint32_t)p.K + 16u * g;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int m = min(16 * t + r, rx - 1);
        xo[t] = (uint32_t)m * (uint32_t)p.K + 16u * g;
        sx[t] = p.s_x + m0 + m;
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
            wb[u][t][0] = load16(wr, o);
            wb[u][t][1] = load16(wr, in ? o + (TILED ? 1024u : 64u) : w_bytes);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const uint32_t o = in ? xo[t] + xs : x_bytes;
            xb[u][t][0] = load16(xr, o);
            xb[u][t][1] = load16(xr, in ? o + 64u : x_bytes);
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
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                const Operand<WIDE> bx = operand<WIDE>(xb[u][a][0], xb[u][a][1]);
                const float c = sb[u][a] * swb[u];
#pragma unroll
                for (int b = 0; b < RT; ++b) {
                    const f32x4 d = block_product<WIDE>(operand<WIDE>(wb[u][b][0], wb[u][b][1]), bx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[a][b][i] = __builtin_fmaf(d[i], c, acc[a][b][i]);
                }
            }
            request(u, kb + NW * (U + u));
        }
    }
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < RT; ++b) red[wave][a * RT + b][lane] = acc[a][b];
    __syncthreads();
    for (int q = threadIdx.x; q < MT * RT * 64; q += 64 * NW) {
        const int t = q >> 6, l = q & 63;
        f32x4 v = red[0][t][l];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += red[w][t][l];
        const int64_t m = m0 + 16 * (t / RT) + (l & 15);
        const int64_t n = 16 * (tile0 + t % RT) + 4 * (l >> 4);
        if (m < p.M && n < p.N) store4(p, m, n, v);
    }
}

// ------------------------------------------------------------------ many tokens
// A workgroup computes BM tokens x BN matrix rows; both operands go through a
// ring of STAGES LDS buffers of one block of k each, filled by direct
// global -> LDS loads.  Rows of 128 bytes are stored with their 16-byte chunks
// permuted by the row (swz), 16-row tiles as they are: both are read without
// bank conflicts.

template <int LPS, int MAXL>
__device__ __forceinline__ void wait_later(int later) {
    if constexpr (MAXL > 0) {
        if (later >= MAXL) wait_vmcnt<MAXL * LPS>();
        else wait_later<LPS, MAXL - 1>(later);
    } else {
        wait_vmcnt<0>();
    }
}

template <int BM_, int BN_, int WAVES_M, int WAVES_N, int STAGES>
struct Fp8Tile {
    static constexpr int BM = BM_, BN = BN_, kNW = WAVES_M * WAVES_N;
    static constexpr int MT = BM / WAVES_M / 16, NT = BN / WAVES_N / 16;
    static constexpr int kCodes = (BM + BN) * kFp8Block;
    static constexpr int kScaleLoads = BM / 64 + 1;  // 64 steps of x each, then those of w
    static constexpr int kStage = kCodes + 256 * kScaleLoads;
    static constexpr int kData = kCodes / 1024 / kNW;
    static constexpr int kLPS = kData + 1;
    static_assert(kCodes / 1024 % kNW == 0 && kScaleLoads <= kNW && BM % 64 == 0 && kFp8Block % (BN / WAVES_N) == 0,
                  "whole loads per wave, one step of w per wave");
    static constexpr int kLds = STAGES * kStage;
};

template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES, bool TILED, bool WIDE>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N) void fp8_tile_kernel(Fp8Params p) {
    typedef Fp8Tile<BM, BN, WAVES_M, WAVES_N, STAGES> C;
    constexpr int MT = C::MT, NT = C::NT, NW = C::kNW;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[C::kLds];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WAVES_N, wn = wave % WAVES_N;

    // tiles in supertiles of 4 token tiles, a contiguous run of them per XCD
    const int t = (int)xcd_run(blockIdx.x, gridDim.x);
    const int per = 4 * p.tiles_n;
    const int st = t / per, u = t - st * per;
    const int h = min(4, p.tiles_m - 4 * st);
    const int64_t m0 = (int64_t)(4 * st + u % h) * BM, n0 = (int64_t)(u / h) * BN;

    const int rx = (int)min((int64_t)BM, p.M - m0);
    const int64_t rows_w = TILED ? (p.N + 15) / 16 * 16 : p.N;
    const int rw = (int)min((int64_t)BN, rows_w - n0);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x + m0 * p.K, (uint32_t)rx * (uint32_t)p.K);
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(p.codes + n0 * p.K, (uint32_t)rw * (uint32_t)p.K);
    uint32_t off[C::kData];  // of this lane's 16 bytes at block 0; blocks of the stage: x's rows, then w's
#pragma unroll
    for (int l = 0; l < C::kData; ++l) {
        const int blk = wave + NW * l;
        const int row = 8 * blk + (lane >> 3);
        if (8 * blk < BM) {
            off[l] = (uint32_t)min(row, rx - 1) * (uint32_t)p.K + 16u * swz<8>(row, lane & 7);
        } else if (TILED) {
            const int b = blk - BM / 8;  // two 1 KB units per 16 rows
            off[l] = (uint32_t)min(b >> 1, rw / 16 - 1) * 16u * (uint32_t)p.K + 1024u * (b & 1) + 16u * lane;
        } else {
            off[l] = (uint32_t)min(row - BM, rw - 1) * (uint32_t)p.K + 16u * swz<8>(row - BM, lane & 7);
        }
    }
    // the steps: wave j < BM / 64 those of 64 tokens, the next one the matrix's
    const int sj = min(wave, C::kScaleLoads - 1);
    const float* ssrc;
    int64_t sstr;
    if (sj < BM / 64) {
        ssrc = p.s_x + m0 + min(64 * sj + lane, rx - 1);
        sstr = p.M;
    } else {
        const int64_t nb = min(n0 / kFp8Block + lane, (p.N - 1) / kFp8Block);
        ssrc = p.s_w + nb * p.KB;
        sstr = 1;
    }
    auto issue = [&](int kb) {
        uint8_t* base = smem + (kb % STAGES) * C::kStage;
#pragma unroll
        for (int l = 0; l < C::kData; ++l) {
            const int blk = wave + NW * l;
            const bool isx = 8 * blk < BM;
            dma16_buffer(isx ? xr : wr, base + blk * 1024, off[l], (uint32_t)kb * (!isx && TILED ? 2048u : 128u));
        }
        dma4(ssrc + kb * sstr, base + C::kCodes + 256 * sj);
    };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int b = 0; b < MT; ++b) acc[a][b] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (s < p.KB) issue(s);

    const int r = lane & 15, g = lane >> 4;
    for (int kb = 0; kb < p.KB; ++kb) {
        wait_later<C::kLPS, STAGES - 2>(min(STAGES - 2, p.KB - 1 - kb));
        lds_barrier();  // every wave's part of block kb is there, and block kb - 1 is read
        if (kb + STAGES - 1 < p.KB) issue(kb + STAGES - 1);
        const uint8_t* base = smem + (kb % STAGES) * C::kStage;
        const uint8_t* wbase = base + BM * kFp8Block;
        const float* sbase = reinterpret_cast<const float*>(base + C::kCodes);
        const float sw = sbase[BM + wn * (BN / WAVES_N) / kFp8Block];
        auto frag_x = [&](int b) {
            const int row = wm * (16 * MT) + 16 * b + r;
            return operand<WIDE>(*reinterpret_cast<const u32x4*>(base + row * kFp8Block + 16 * swz<8>(row, g)),
                           *reinterpret_cast<const u32x4*>(base + row * kFp8Block + 16 * swz<8>(row, g + 4)));
        };
        auto frag_w = [&](int a) {
            if constexpr (TILED) {
                const uint8_t* q = wbase + (wn * NT + a) * 2048 + 16 * lane;
                return operand<WIDE>(*reinterpret_cast<const u32x4*>(q), *reinterpret_cast<const u32x4*>(q + 1024));
            } else {
                const int row = wn * (16 * NT) + 16 * a + r;
                return operand<WIDE>(*reinterpret_cast<const u32x4*>(wbase + row * kFp8Block + 16 * swz<8>(row, g)),
                               *reinterpret_cast<const u32x4*>(wbase + row * kFp8Block + 16 * swz<8>(row, g + 4)));
            }
        };
        Operand<WIDE> fw[NT];
#pragma unroll
        for (int a = 0; a < NT; ++a) fw[a] = frag_w(a);
#pragma unroll
        for (int b = 0; b < MT; ++b) {
            const Operand<WIDE> fx = frag_x(b);
            const float c = sbase[wm * (16 * MT) + 16 * b + r] * sw;
#pragma unroll
            for (int a = 0; a < NT; ++a) {
                const f32x4 d = block_product<WIDE>(fw[a], fx);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[a][b][i] = __builtin_fmaf(d[i], c, acc[a][b][i]);
            }
        }
    }
#pragma unroll
    for (int b = 0; b < MT; ++b) {
        const int64_t m = m0 + wm * (16 * MT) + 16 * b + r;
#pragma unroll
        for (int a = 0; a < NT; ++a) {
            const int64_t n = n0 + wn * (16 * NT) + 16 * a + 4 * g;
            if (m < p.M && n < p.N) store4(p, m, n, acc[a][b]);
        }
    }
}

template <int MT, int RT, bool WIDE, int NW, int U>
hipError_t run_stream(const Fp8Params& p, bool t16, hipStream_t st) {
    const dim3 grid((uint32_t)((p.N + 16 * RT - 1) / (16 * RT)), (uint32_t)((p.M + 16 * MT - 1) / (16 * MT)));
    if (t16) fp8_stream_kernel<MT, RT, true, WIDE, NW, U><<<grid, 64 * NW, 0, st>>>(p);
    else fp8_stream_kernel<MT, RT, false, WIDE, NW, U><<<grid, 64 * NW, 0, st>>>(p);
    return hipGetLastError();
}

template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES, bool WIDE>
hipError_t run_tile(Fp8Params p, bool t16, hipStream_t st) {
    p.tiles_m = (int)((p.M + BM - 1) / BM);
    p.tiles_n = (int)((p.N + BN - 1) / BN);
    const uint32_t grid = (uint32_t)((int64_t)p.tiles_m * p.tiles_n);
    constexpr int T = 64 * WAVES_M * WAVES_N;
    if (t16) fp8_tile_kernel<BM, BN, WAVES_M, WAVES_N, STAGES, true, WIDE><<<grid, T, 0, st>>>(p);
    else fp8_tile_kernel<BM, BN, WAVES_M, WAVES_N, STAGES, false, WIDE><<<grid, T, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qgemm_fp8(const Fp8GemmArgs& a, hipStream_t st) {
    Fp8Params p;
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
    p.tiles_m = p.tiles_n = 0;
    if (a.m <= 16) return run_stream<1, 1, true, 8, 4>(p, a.t16, st);
    if (a.m <= 64) return run_stream<4, 1, true, 8, 2>(p, a.t16, st);
    if (a.yt == 0) return run_tile<256, 256, 2, 4, 2, true>(p, a.t16, st);
    return run_tile<256, 256, 2, 4, 2, false>(p, a.t16, st);
}

}  // namespace qg

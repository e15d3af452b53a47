// fp8rows.hip -- what stands between two products: the root-mean-square norm
// with the residual's addition, SwiGLU, and quantization to e4m3 in blocks of
// 128 (gfx950).
//
//   norm    h = x + r;  v = h / sqrt(sum h^2 / k + eps) * w
//   SwiGLU  v = g / (1 + exp(-g)) * u
//   as is   v = x
// and v goes out rounded (fp32, bf16), as int8 with 127 / max|v| of the row, or
// as e4m3 with the step of every 128 values.  All arithmetic is fp32; h is
// rounded for residual_out only, the norm goes on with the sum itself.
//
// HBM-bound for many rows, latency of one launch for few: every input is read
// once and kept in registers (8 consecutive values per lane and chunk, 16
// lanes to a block of 128), all loads are requested before the first is used.
#include "qg_fp8.h"
#include "qg_launch.h"

namespace qg {

namespace {

enum { kOpNone = 0, kOpNorm = 1, kOpSwiglu = 2 };
// The residual: none; its sum over an input; its sum in memory of its own, past
// the caches, as the products before its next use read more than they hold (4129 x
// 4096 bf16 26.4 -> 20.3 us, 8192 x 2048 26.2 -> 18.4; three sets of buffers in turn. With all
// of it in the caches, 2048 x 4096, 11.9 -> 13.3; in a layer with its products no difference.
// Over an input, whose lines are there already, 10.8 -> 11.4).
enum { kNone = 0, kInPlace = 1, kPast = 2 };

// g / (1 + exp(-g)) * u.  With t = -g log2(e) / 2 rounded, exp(-g) is 4^t (1 + d), where d =
// -g - 2 t ln 2 is what the rounding lost, and 2^t stays within fp32 for every gate that
// matters; 1 + exp(-g), scaled by 2^-32, has its reciprocal (0 from exp(-g) = 2^158 on).  With
// the hardware's 2^t and reciprocal (1 ulp each) the result is off by at most 10 half steps
// and, from ln 2, |g| / 21 more, besides the 2^-149 steps of 1 / (1 + exp(-g)).  d, the scale and
// the clamp (for infinite gates: -inf times 0 is NaN, as the quotient is) are 5 of 17 issue
// slots: 2048 x 11008 bf16 to e4m3 22.1 -> 24.1 us back to back, a feed-forward with its
// products the same within 1%.  Without them the error is 1.2 |g| half steps and gates
// below -87.3 give 0; 2^n and 2^rest apart, for 8.4 half steps in 23 slots, took 26.4 us.
__device__ __forceinline__ float swiglu_of(float g, float u) {
    constexpr float kScale = 2.32830644e-10f;  // 2^-32
    const float c = __builtin_amdgcn_fmed3f(g, -170.0f, 170.0f);
    const float t = c * -0.721347511f;
    const float d = __builtin_fmaf(t, -1.38629436f, -c);
    const float p = __builtin_amdgcn_exp2f(t);
    const float ps = p * kScale;
    const float den = __builtin_fmaf(__builtin_fmaf(ps, d, ps), p, kScale);
    return g * (__builtin_amdgcn_rcpf(den) * kScale) * u;
}

struct RowParams {
    const void* x;         // [rows][k], SwiGLU: [rows][2 k]
    const void* residual;  // [rows][k] or null
    void* residual_out;
    const void* weight;
    int wt, out;           // 0: fp32, 1: bf16 (weight, out); 2: int8, 3: e4m3 (out)
    float eps, inv_k;
    int64_t rows, k;
    void* y;
    float* s;
};

// Sum and maximum over the L lanes of a row, in every one of them.
template <int L>
__device__ __forceinline__ float lanes_sum(float v, float* scratch) {
    if constexpr (L == 16) {
        v += __int_as_float(dpp_mov<0xB1>(__float_as_int(v)));
        v += __int_as_float(dpp_mov<0x4E>(__float_as_int(v)));
        v += __int_as_float(dpp_mov<0x141>(__float_as_int(v)));
        v += __int_as_float(dpp_mov<0x140>(__float_as_int(v)));
        return v;
    } else {
        v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wave_sum_to_lane63(v)), 63));
        if constexpr (L > 64) {
            if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
            lds_barrier();
            v = scratch[0];
#pragma unroll
            for (int i = 1; i < L / 64; ++i) v += scratch[i];
            lds_barrier();
        }
        return v;
    }
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, uint32_t* scratch) {
    v = row16_max(v);
    if constexpr (L > 16) {
        v = max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
                max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
        if constexpr (L > 64) {
            if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
            lds_barrier();
            v = scratch[0];
#pragma unroll
            for (int i = 1; i < L / 64; ++i) v = max(v, scratch[i]);
            lds_barrier();
        }
    }
    return v;
}

// Operators that need the whole row (the norm; int8 outputs): L lanes hold a
// row of up to 8 L NP values.  L 16 and 64 put several rows into a workgroup.
template <int OP, int XT, int RES, int L, int NP>
__global__ __launch_bounds__(L < 256 ? 256 : L) void fp8_row_kernel(RowParams p) {
    constexpr int T = L < 256 ? 256 : L;
    constexpr int R = T / L;
    __shared__ float red[T / 64];
    const int lane = threadIdx.x % L;
    const int k8 = (int)(p.k / 8);
    int at[NP];  // first value of a chunk; lanes past the row read its last chunk and take zeros
    bool in[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const int c = lane + L * j;
        in[j] = c < k8;
        at[j] = 8 * (in[j] ? c : k8 - 1);
    }
    const int64_t groups = (p.rows + R - 1) / R;
    for (int64_t wg = xcd_run(blockIdx.x, gridDim.x); wg < groups; wg += gridDim.x) {
        const int64_t row0 = wg * R + threadIdx.x / L;
        const bool live = row0 < p.rows;
        const int64_t row = live ? row0 : p.rows - 1;
        float v[NP][8];
        // The weights as they stand, of either type: two loads, for bf16 the same
        // one; with the rest where there are registers for them (1 x 4096 3.1 -> 3.0
        // us, 4129 x 4096 5% less), else after the sum.
        constexpr bool kLate = L * NP > 2048;
        u32x4 rw[OP == kOpNorm ? NP : 1][2];
        auto weights = [&](int j) __attribute__((always_inline)) {
            const uint8_t* w = static_cast<const uint8_t*>(p.weight) + at[j] * (p.wt == 0 ? 4 : 2);
            rw[j][0] = *reinterpret_cast<const u32x4*>(w);
            rw[j][1] = *reinterpret_cast<const u32x4*>(w + (p.wt == 0 ? 16 : 0));
        };
        {
            Raw8<XT> rx[NP], rr[NP];
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                rx[j] = raw8<XT, OP == kOpSwiglu>(p.x, (OP == kOpSwiglu ? 2 : 1) * row * p.k + at[j]);
                if constexpr (OP == kOpSwiglu) rr[j] = raw8<XT, true>(p.x, (2 * row + 1) * p.k + at[j]);
                else if constexpr (RES != kNone) rr[j] = raw8<XT>(p.residual, row * p.k + at[j]);
            }
            if constexpr (OP == kOpNorm && !kLate) {
#pragma unroll
                for (int j = 0; j < NP; ++j) weights(j);
            }
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                values8<XT>(rx[j], v[j]);
                if constexpr (OP == kOpSwiglu || RES != kNone) {
                    float b[8];
                    values8<XT>(rr[j], b);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] = OP == kOpSwiglu ? swiglu_of(v[j][i], b[i]) : v[j][i] + b[i];
                    if constexpr (RES != kNone) {
                        if (live && in[j]) store8<RES == kPast>(p.residual_out, XT, row * p.k + at[j], v[j]);
                    }
                }
                // what a lane past the row has read may be residual_out already
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = in[j] ? v[j][i] : 0.0f;
            }
        }
        if constexpr (OP == kOpNorm) {
            auto sum_sq = [&](float by) {
                float t = 0.0f;
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    float a = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float h = v[j][i] * by;
                        a = __builtin_fmaf(h, h, a);
                    }
                    t += a;
                }
                return lanes_sum<L>(t, red);
            };
            const float mean = sum_sq(1.0f) * p.inv_k + p.eps;
            float f = 1.0f / __builtin_sqrtf(mean);
            // Squares above fp32's range (|h| from 1.8e19 on), or their mean with eps: again
            // with h 2^-80 and eps 2^-160.  Rows of 16 lanes share the branch.
            if (__any(!(mean <= 3.40282347e38f))) {
                constexpr float kSmall = 8.27180613e-25f;  // 2^-80
                const float small = sum_sq(kSmall) * p.inv_k + p.eps * kSmall * kSmall;
                if (!(mean <= 3.40282347e38f)) f = kSmall / __builtin_sqrtf(small);
            }
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                if constexpr (kLate) weights(j);
                float w32[8], w16[8];
                values8<0>(Raw8<0>{{rw[j][0], rw[j][1]}}, w32);
                values8<1>(Raw8<1>{{rw[j][0]}}, w16);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * f * (p.wt == 0 ? w32[i] : w16[i]);
            }
        }
        if (p.out <= 1) {
#pragma unroll
            for (int j = 0; j < NP; ++j)
                if (live && in[j]) store8(p.y, p.out, row * p.k + at[j], v[j]);
            continue;
        }
        uint32_t top[NP];
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            top[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top[j] = max(top[j], abs_bits(v[j][i]));
        }
        uint8_t* q = static_cast<uint8_t*>(p.y);
        if (p.out == 2) {
            uint32_t all = 0;
#pragma unroll
            for (int j = 0; j < NP; ++j) all = max(all, top[j]);
            all = lanes_max<L>(all, reinterpret_cast<uint32_t*>(red));
            const float s = all >= kInfBits ? __uint_as_float(kNanBits) : absmax_scale(__uint_as_float(all));
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                uint32_t o[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    o[h] = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[h] |= (uint32_t)(qcode(v[j][4 * h + i], s) & 0xFF) << (8 * i);
                }
                if (live && in[j]) *reinterpret_cast<uint2*>(q + row * p.k + at[j]) = make_uint2(o[0], o[1]);
            }
            if (live && lane == 0) p.s[row] = s;
        } else {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                float s, i;
                fp8_step(row16_max(top[j]), s, i);
                const uint2 o = fp8_codes8(v[j], i);
                if (live && in[j]) {
                    *reinterpret_cast<uint2*>(q + row * p.k + at[j]) = o;
                    if ((lane & 15) == 0) p.s[(int64_t)(at[j] / kFp8Block) * p.rows + row] = s;
                }
            }
        }
    }
}

// Operators whose blocks need nothing of the rest of their row: the rows as
// one run of chunks of 8, U of them per lane, 16 lanes to a block of 128.
template <int OP, int XT>
__global__ __launch_bounds__(kThreads) void fp8_flat_kernel(RowParams p, int64_t chunks) {
    constexpr int U = 2;
    const int64_t k8 = p.k / 8;
    const bool small = chunks <= 0xFFFFFFFFll;  // the quotient in 32 bits
    for (int64_t c0 = xcd_run(blockIdx.x, gridDim.x) * (kThreads * U) + threadIdx.x; c0 - threadIdx.x < chunks;
         c0 += (int64_t)gridDim.x * (kThreads * U)) {
        int64_t c[U], row[U], col[U];
        Raw8<XT> ra[U], rb[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            c[j] = min(c0 + j * kThreads, chunks - 1);
            row[j] = small ? (int64_t)((uint32_t)c[j] / (uint32_t)k8) : c[j] / k8;
            col[j] = c[j] - row[j] * k8;
            const int64_t e = 8 * (OP == kOpSwiglu ? 2 * row[j] * k8 + col[j] : c[j]);
            // SwiGLU's x, a product's output, is wanted no more: past the caches (4129 x 11008
            // bf16 to e4m3 45.7 -> 43.5 us, 2048 x 11008 to bf16 27.5 -> 23.7, to e4m3 24.0 either
            // way; 1000 x 11008, which fits in them, 12.2 -> 13.4; a feed-forward with its
            // products up to 1% less).
            ra[j] = raw8<XT, OP == kOpSwiglu>(p.x, e);
            if constexpr (OP == kOpSwiglu) rb[j] = raw8<XT, true>(p.x, e + p.k);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            float v[8];
            values8<XT>(ra[j], v);
            if constexpr (OP == kOpSwiglu) {
                float b[8];
                values8<XT>(rb[j], b);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = swiglu_of(v[i], b[i]);
            }
            const bool live = c0 + j * kThreads < chunks;
            if (p.out <= 1) {
                if (live) store8(p.y, p.out, 8 * c[j], v);
                continue;
            }
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[i]));
            float s, i;
            fp8_step(row16_max(top), s, i);
            const uint2 o = fp8_codes8(v, i);
            if (live) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + 8 * c[j]) = o;
                if ((threadIdx.x & 15) == 0) p.s[(col[j] >> 4) * p.rows + row[j]] = s;
            }
        }
    }
}

// Weights: a workgroup per block of 128 x 128, which stays in registers
// between its maximum and its codes.
template <int XT>
__global__ __launch_bounds__(kThreads) void fp8_weight_kernel(const void* w, int64_t n, int64_t k, uint8_t* codes,
                                                              float* scale) {
    __shared__ uint32_t red[kWaves];
    const int64_t kb = k / kFp8Block;
    const int64_t blocks = (n + kFp8Block - 1) / kFp8Block * kb;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int64_t ib = b / kb, jb = b - ib * kb;
        const int64_t col = jb * kFp8Block + 8 * (threadIdx.x & 15);
        Raw8<XT> r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // rows past the last repeat it
            const int64_t row = min(ib * kFp8Block + 16 * j + (threadIdx.x >> 4), n - 1);
            r[j] = raw8<XT>(w, row * k + col);
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v[8];
            values8<XT>(r[j], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[i]));
        }
        top = lanes_max<256>(top, red);
        float s, inv;
        fp8_step(top, s, inv);
        if (threadIdx.x == 0) scale[b] = s;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t row = ib * kFp8Block + 16 * j + (threadIdx.x >> 4);
            float v[8];
            values8<XT>(r[j], v);
            const uint2 o = fp8_codes8(v, inv);
            if (row < n) *reinterpret_cast<uint2*>(codes + row * k + col) = o;
        }
    }
}

// Workgroups of a launch: more than these are walked in turn (a launch's threads
// have to stay below 2^32).
constexpr int64_t kFewRows = 256;

uint32_t grid_of(int64_t want) { return (uint32_t)(want < (1 << 20) ? want : (1 << 20)); }

template <int OP, int XT, int RES, int L, int NP>
hipError_t run_rows(const RowParams& p, hipStream_t st) {
    constexpr int T = L < 256 ? 256 : L;
    const int64_t grid = (p.rows + T / L - 1) / (T / L);
    fp8_row_kernel<OP, XT, RES, L, NP><<<grid_of(grid), T, 0, st>>>(p);
    return hipGetLastError();
}

template <int OP, int XT, int RES>
hipError_t pick_rows(const RowParams& p, hipStream_t st) {
    const int64_t k8 = p.k / 8;
    if (k8 <= 16) return run_rows<OP, XT, RES, 16, 1>(p, st);
    if (k8 <= 64) return run_rows<OP, XT, RES, 64, 1>(p, st);
    if (k8 <= 256) return run_rows<OP, XT, RES, 256, 1>(p, st);
    // Few rows: a row's latency, so more lanes with fewer values in each (1 x 4096
    // 3.0 -> 2.6 us); many: lanes that all have work (2085 x 11008 in 512 lanes 20% less
    // than in 1024: 34.8 us).
    if (k8 <= 512) return p.rows <= kFewRows ? run_rows<OP, XT, RES, 512, 1>(p, st) : run_rows<OP, XT, RES, 256, 2>(p, st);
    if (k8 <= 768 && p.rows > kFewRows) return run_rows<OP, XT, RES, 256, 3>(p, st);
    if (k8 <= 1024) return run_rows<OP, XT, RES, 512, 2>(p, st);
    if (k8 <= 1536 && p.rows > kFewRows) return run_rows<OP, XT, RES, 512, 3>(p, st);
    if (k8 <= 2048) return run_rows<OP, XT, RES, 1024, 2>(p, st);
    if (k8 <= 3 * 1024) return run_rows<OP, XT, RES, 1024, 3>(p, st);
    return run_rows<OP, XT, RES, 1024, 4>(p, st);  // up to 32768 values
}

template <int OP>
hipError_t run_flat(const RowParams& p, int xt, hipStream_t st) {
    const int64_t chunks = p.rows * (p.k / 8);
    const int64_t grid = (chunks + 2 * kThreads - 1) / (2 * kThreads);
    if (xt == 0) fp8_flat_kernel<OP, 0><<<grid_of(grid), kThreads, 0, st>>>(p, chunks);
    else fp8_flat_kernel<OP, 1><<<grid_of(grid), kThreads, 0, st>>>(p, chunks);
    return hipGetLastError();
}

RowParams row_params(const RowArgs& a) {
    RowParams p;
    p.x = a.x;
    p.residual = a.residual;
    p.residual_out = a.residual_out;
    p.weight = a.weight;
    p.wt = a.wt;
    p.out = a.out;
    p.eps = a.eps;
    p.inv_k = 1.0f / (float)a.k;
    p.rows = a.rows;
    p.k = a.k;
    p.y = a.y;
    p.s = a.s;
    return p;
}

}  // namespace

hipError_t launch_rms_norm(const RowArgs& a, hipStream_t st) {
    const RowParams p = row_params(a);
    const int res = !a.residual ? kNone : a.residual_out == a.residual || a.residual_out == a.x ? kInPlace : kPast;
    if (res == kNone) return a.xt == 0 ? pick_rows<kOpNorm, 0, kNone>(p, st) : pick_rows<kOpNorm, 1, kNone>(p, st);
    if (res == kInPlace) return a.xt == 0 ? pick_rows<kOpNorm, 0, kInPlace>(p, st) : pick_rows<kOpNorm, 1, kInPlace>(p, st);
    return a.xt == 0 ? pick_rows<kOpNorm, 0, kPast>(p, st) : pick_rows<kOpNorm, 1, kPast>(p, st);
}

hipError_t launch_swiglu(const RowArgs& a, hipStream_t st) {
    const RowParams p = row_params(a);
    if (a.out != 2) return run_flat<kOpSwiglu>(p, a.xt, st);
    return a.xt == 0 ? pick_rows<kOpSwiglu, 0, kNone>(p, st) : pick_rows<kOpSwiglu, 1, kNone>(p, st);
}

hipError_t launch_quantize_fp8(const RowArgs& a, hipStream_t st) { return run_flat<kOpNone>(row_params(a), a.xt, st); }

hipError_t launch_quantize_fp8_weight(const void* w, int wt, int64_t n, int64_t k, uint8_t* codes, float* scale,
                                      hipStream_t st) {
    const int64_t grid = (n + kFp8Block - 1) / kFp8Block * (k / kFp8Block);
    if (wt == 0) fp8_weight_kernel<0><<<grid_of(grid), kThreads, 0, st>>>(w, n, k, codes, scale);
    else fp8_weight_kernel<1><<<grid_of(grid), kThreads, 0, st>>>(w, n, k, codes, scale);
    return hipGetLastError();
}

}  // namespace qg

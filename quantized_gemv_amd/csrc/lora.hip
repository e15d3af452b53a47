// lora.hip -- low-rank adapters of many requests beside a shared projection:
//   y[t] += scale[g] B[g] (A[g] x[t]),  g the adapter of row t,
// for up to 8 matrices that read the same x (q, k, v; gate, up).
//
// Two launches.  shrink: v = A x; a workgroup takes 16 sorted rows of one
// adapter, one part of k and one matrix, on v_mfma_f32_16x16x32_bf16 (exact
// products, fp32 sums), and stores its fp32 partial sums [part][row][rank];
// few rows would leave most CUs idle without the parts.  expand: the parts
// are added in order, scaled and split into three bf16 terms (hi + mid + lo,
// 24 bits: nothing of the fp32 value is lost), so that the product with B
// runs on the same matrix instructions; y is read, added to and written once.
#include "qg_launch.h"
#include "qg_rows.h"

namespace qg {

typedef __bf16 lbf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kLWaves = 4;
constexpr int kLThreads = kLWaves * kWave;

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
    int32_t nblocks;  // expand: blocks of columns, the same for every matrix (the widest one's)
    int64_t block0;
};

__device__ __forceinline__ int lora_source(const LoraParams& p, int at) { return p.order[at]; }

// RT: 16-row tiles of A (rank <= 16 RT)
template <int RT>
__device__ __forceinline__ void shrink_tile(const LoraParams& p, const LoraMatP& m, const RowTile& t, int kpart,
                                            f32x4 (&red)[kLWaves][16][kWave]) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
    const int i = lane & 15, g = lane >> 4;
    const int units = p.k / 32, shares = p.parts * kLWaves, share = kpart * kLWaves + wave;
    const int c0 = (int)((int64_t)units * share / shares), c1 = (int)((int64_t)units * (share + 1) / shares);
    const int src = min(max(lora_source(p, t.row0 + min(i, t.rows - 1)), 0), p.x_rows - 1);
    const uint16_t* x = p.x + (int64_t)src * p.k + 8 * g;
    const uint16_t* a[RT];
    f32x4 acc[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
        a[q] = m.a + ((int64_t)t.group * m.r + min(16 * q + i, m.r - 1)) * p.k + 8 * g;
        acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    for (int c = c0; c < c1; ++c) {
        const u32x4 xf = *reinterpret_cast<const u32x4*>(x + c * 32);
#pragma unroll
        for (int q = 0; q < RT; ++q) {
            const u32x4 af = *reinterpret_cast<const u32x4*>(a[q] + c * 32);
            acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(lbf16x8, af),
                                                             __builtin_bit_cast(lbf16x8, xf), acc[q], 0, 0, 0);
        }
    }
#pragma unroll
    for (int q = 0; q < RT; ++q) red[wave][q][lane] = acc[q];
    lds_barrier();
    const int rpad = (m.r + 15) / 16 * 16;
    for (int q = wave; q < rpad / 16; q += kLWaves) {
        f32x4 s = red[0][q][lane];
#pragma unroll
        for (int w = 1; w < kLWaves; ++w) s += red[w][q][lane];
        // lane l: sorted row l % 16, ranks 16 q + 4 (l / 16) + r
        if (i < t.rows)
            *reinterpret_cast<f32x4*>(p.ws + m.ws_at + ((int64_t)kpart * p.rows + t.row0 + i) * rpad + 16 * q + 4 * g) = s;
    }
}

__global__ __launch_bounds__(kLThreads) void lora_shrink_kernel(LoraParams p) {
    __shared__ f32x4 red[kLWaves][16][kWave];
    const int64_t block = p.block0 + blockIdx.x;
    const int mi = (int)(block % p.count), kpart = (int)(block / p.count % p.parts);
    const RowTile t = find_row_tile<16>(p.offsets, p.groups, p.rows, (int)(block / p.count / p.parts));
    if (t.rows <= 0) return;
    const LoraMatP& m = p.m[mi];
    if (m.r <= 16) shrink_tile<1>(p, m, t, kpart, red);
    else if (m.r <= 32) shrink_tile<2>(p, m, t, kpart, red);
    else if (m.r <= 64) shrink_tile<4>(p, m, t, kpart, red);
    else if (m.r <= 128) shrink_tile<8>(p, m, t, kpart, red);
    else shrink_tile<16>(p, m, t, kpart, red);
}

constexpr int kLCols = 256;  // columns per expand workgroup: 4 waves x 4 tiles of 16

template <int YT>
__global__ __launch_bounds__(kLThreads) void lora_expand_kernel(LoraParams p) {
    extern __shared__ u32x4 vsh[];  // [term][k group of 8][16 rows] bf16 x 8
    const int64_t block = p.block0 + blockIdx.x;
    const int nb = (int)(block % p.nblocks), mi = (int)(block / p.nblocks % p.count);
    const LoraMatP& m = p.m[mi];
    if (nb * kLCols >= m.n) return;
    const RowTile t = find_row_tile<16>(p.offsets, p.groups, p.rows, (int)(block / p.nblocks / p.count));
    if (t.rows <= 0) return;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
    const int i = lane & 15, g = lane >> 4;
    const int rpad = (m.r + 15) / 16 * 16, kg = (m.r + 31) / 32 * 4;  // k groups of 8, whole matrix instructions
    const float scale = m.scale ? m.scale[t.group] : 1.0f;
    uint16_t* vh = reinterpret_cast<uint16_t*>(vsh);
    for (int q = tid; q < kg * 8 * 16; q += kLThreads) {
        const int row = q & 15, j = q >> 4;
        float v = 0.0f;
        if (j < m.r && row < t.rows) {
            const float* at = p.ws + m.ws_at + (int64_t)(t.row0 + row) * rpad + j;
            for (int s = 0; s < p.parts; ++s) v += at[(int64_t)s * p.rows * rpad];
            v *= scale;
        }
        const uint32_t hi = f32_to_bf16(v);
        const float v1 = v - bf16_to_f32(hi);
        const uint32_t mid = f32_to_bf16(v1);
        const uint32_t lo = f32_to_bf16(v1 - bf16_to_f32(mid));
        const int slot = ((j >> 3) * 16 + row) * 8 + (j & 7);
        vh[slot] = (uint16_t)hi;
        vh[kg * 128 + slot] = (uint16_t)mid;
        vh[2 * kg * 128 + slot] = (uint16_t)lo;
    }
    lds_barrier();
    const int trow = i < t.rows ? lora_source(p, t.row0 + i) : -1;
    const bool live = trow >= 0 && trow < p.x_rows;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int n0 = nb * kLCols + (wave * 4 + q) * 16;
        if (n0 >= m.n) break;
        const uint16_t* b = m.b + ((int64_t)t.group * m.n + min(n0 + i, m.n - 1)) * m.r;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < kg; c += 4) {
            u32x4 bf = {0u, 0u, 0u, 0u};
            if ((c + g) * 8 < m.r) bf = *reinterpret_cast<const u32x4*>(b + (c + g) * 8);
#pragma unroll
            for (int term = 0; term < 3; ++term)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(lbf16x8, bf),
                    __builtin_bit_cast(lbf16x8, vsh[(term * kg + c + g) * 16 + i]), acc, 0, 0, 0);
        }
        if (live) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int n = n0 + 4 * g + r;
                if (n < m.n) {
                    const int64_t at = (int64_t)trow * m.n + n;
                    if constexpr (YT == 0) {
                        float* y = static_cast<float*>(m.y);
                        y[at] = y[at] + acc[r];
                    } else {
                        uint16_t* y = static_cast<uint16_t*>(m.y);
                        y[at] = (uint16_t)f32_to_bf16(bf16_to_f32(y[at]) + acc[r]);
                    }
                }
            }
        }
    }
}

static int lora_parts(int64_t rows, int64_t groups, int64_t k) {
    const int64_t tiles = max_row_tiles(rows, groups, 16);
    int64_t parts = (512 + tiles - 1) / tiles;
    const int64_t most = k / 32 / (2 * kLWaves);  // at least two matrix instructions deep per wave
    if (parts > most) parts = most;
    if (parts > 16) parts = 16;
    return (int)(parts < 1 ? 1 : parts);
}

size_t lora_workspace(int64_t rows, int64_t groups, int64_t k, int64_t padded_rank) {
    return (size_t)lora_parts(rows, groups, k) * (size_t)rows * (size_t)padded_rank * sizeof(float);
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
    p.parts = lora_parts(a.rows, a.groups, a.k);
    int64_t at = 0, widest = 0;
    int rmax = 0;
    for (int j = 0; j < a.count; ++j) {
        const LoraMat& m = a.m[j];
        p.m[j] = {m.a, m.b, m.scale, m.y, (int32_t)m.n, m.r, at};
        at += (int64_t)p.parts * a.rows * ((m.r + 15) / 16 * 16);
        if (m.n > widest) widest = m.n;
        if (m.r > rmax) rmax = m.r;
    }
    const int64_t tiles = max_row_tiles(a.rows, a.groups, 16);
    hipError_t e = launch_blocks(tiles * p.parts * p.count, kLThreads, [&](uint32_t grid, int64_t block0) {
        p.block0 = block0;
        lora_shrink_kernel<<<grid, kLThreads, 0, st>>>(p);
    });
    if (e != hipSuccess) return e;
    p.nblocks = (int32_t)((widest + kLCols - 1) / kLCols);
    const size_t lds = (size_t)3 * ((rmax + 31) / 32 * 4) * 16 * sizeof(u32x4);
    return launch_blocks(tiles * p.nblocks * p.count, kLThreads, [&](uint32_t grid, int64_t block0) {
        p.block0 = block0;
        if (a.yt == 0) lora_expand_kernel<0><<<grid, kLThreads, lds, st>>>(p);
        else lora_expand_kernel<1><<<grid, kLThreads, lds, st>>>(p);
    });
}

}  // namespace qg

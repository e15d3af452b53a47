// qg_fp8.h -- what the kernels of the 8-bit path between layers share: e4m3
// codes (OCP: 4 exponent bits, 3 mantissa bits, largest value 448, no
// infinities) in blocks of 128 with an fp32 step, and 8 values per lane.
#pragma once

#include "qg_device.h"
#include "qg_rows.h"

namespace qg {

constexpr int kFp8Block = 128;

// Absolute values are compared as the integers of their bits: the order is
// the same for numbers, infinities come above them and NaN above those, so one
// maximum finds the largest value and whether everything is finite.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kNanBits = 0x7FC00000u;

// The step of a block whose largest absolute value has the bits `top`, and
// its reciprocal: s = max(a / 448, 2^-126), i = 1 / s, both IEEE divisions.
// The bound keeps s normal and i finite; it acts on blocks below 5.3e-36 and on
// blocks of zeros.  A block that holds an infinity or NaN gets a NaN step (and
// so NaN codes): it reaches a product's sums as NaN.
__device__ __forceinline__ void fp8_step(uint32_t top, float& s, float& i) {
    s = __builtin_fmaxf(__uint_as_float(top) / 448.0f, 1.17549435e-38f);
    if (top >= kInfBits) s = __uint_as_float(kNanBits);
    i = 1.0f / s;
}

// Maximum over the 16 lanes of a DPP row, in all of them: quad swaps, then
// half-row and row mirrors.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = max(v, (uint32_t)dpp_mov<0xB1>((int)v));
    v = max(v, (uint32_t)dpp_mov<0x4E>((int)v));
    v = max(v, (uint32_t)dpp_mov<0x141>((int)v));
    v = max(v, (uint32_t)dpp_mov<0x140>((int)v));
    return v;
}

// Eight values times i as e4m3 codes, to nearest even (the hardware's
// conversion; |v i| <= 448 up to rounding, which the conversion takes to 448).
__device__ __forceinline__ uint2 fp8_codes8(const float v[8], float i) {
    uint2 o;
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * i, v[1] * i, 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * i, v[3] * i, a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * i, v[5] * i, 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * i, v[7] * i, b, true);
    o.x = (uint32_t)a;
    o.y = (uint32_t)b;
    return o;
}

// Eight consecutive values as they stand in memory: one 16-byte load of bf16,
// two of fp32.  PAST: past the caches.
template <int XT>
struct Raw8 {
    u32x4 w[XT == 0 ? 2 : 1];
};
template <int XT, bool PAST = false>
__device__ __forceinline__ Raw8<XT> raw8(const void* base, int64_t e) {
    Raw8<XT> r;
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(base) + e * (XT == 0 ? 4 : 2));
    r.w[0] = PAST ? __builtin_nontemporal_load(p) : p[0];
    if constexpr (XT == 0) r.w[1] = PAST ? __builtin_nontemporal_load(p + 1) : p[1];
    return r;
}
template <int XT>
__device__ __forceinline__ void values8(const Raw8<XT>& r, float v[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (XT == 0) {
            v[j] = __uint_as_float(r.w[0][j]);
            v[4 + j] = __uint_as_float(r.w[1][j]);
        } else {
            v[2 * j] = __uint_as_float(r.w[0][j] << 16);
            v[2 * j + 1] = __uint_as_float(r.w[0][j] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ u32x4 bf16_pack8(const float v[8]) {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = any_f32_to_bf16(v[2 * j]) | (any_f32_to_bf16(v[2 * j + 1]) << 16);
    return o;
}
// Eight values at element e of a float output (0: fp32, 1: bf16).  PAST: past
// the caches.
template <bool PAST = false>
__device__ __forceinline__ void store8(void* y, int yt, int64_t e, const float v[8]) {
    if (yt == 0) {
        u32x4* p = reinterpret_cast<u32x4*>(static_cast<float*>(y) + e);
        u32x4 a, b;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = __float_as_uint(v[j]);
            b[j] = __float_as_uint(v[4 + j]);
        }
        if constexpr (PAST) {
            __builtin_nontemporal_store(a, p);
            __builtin_nontemporal_store(b, p + 1);
        } else {
            p[0] = a;
            p[1] = b;
        }
    } else {
        u32x4* p = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(y) + e);
        if constexpr (PAST) __builtin_nontemporal_store(bf16_pack8(v), p);
        else *p = bf16_pack8(v);
    }
}

// Workgroup number -> position in the work, so that each of the 8 XCDs (to
// which consecutive workgroups go in turn) gets a contiguous run: neighbours
// then share an L2.
__device__ __forceinline__ int64_t xcd_run(int64_t b, int64_t g) {
    const int64_t per = g >> 3;
    return b < (per << 3) ? (b & 7) * per + (b >> 3) : b;
}

}  // namespace qg

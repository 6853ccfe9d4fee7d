// Device-side helpers of the layer operators: unaligned vector access, bf16 packing, and the MXFP8 form that
// activations are kept in.
//
// MXFP8: the values of a row in blocks of 32 consecutive columns (the last block may be shorter), each an
// E4M3 code (sign | 4 exponent bits, bias 7 | 3 mantissa bits, 0x7F and 0xFF NaN) times the block's E8M0
// scale, a byte b that stands for 2^(b - 127) (255: NaN). The scale written is the smallest power of two,
// at least 2^-127, with max|v| <= 448 * scale: nothing saturates, so every value is within half an E4M3 step
// (a relative 2^-4, or 2^-10 scales for the values below 2^-6 scales). A block of zeros gets b = 0. A block
// that holds a NaN or an infinity gets b = 255 and codes 0x7F: all its values read as NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "codec.hpp"

namespace nvfp4 {

constexpr int kMxBlock = 32;

// Global memory is read and written at any byte alignment (the target's unaligned access mode), so a row
// of odd length costs masks at its end only.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_any __attribute__((aligned(1), may_alias));
typedef u32x2 u32x2_any __attribute__((aligned(1), may_alias));
typedef uint16_t u16_any __attribute__((aligned(1), may_alias));
typedef uint32_t u32_any __attribute__((aligned(1), may_alias));
typedef uint16_t u16_lds __attribute__((may_alias));  // two scale bytes of those that a wave has stored in LDS as dwords

__device__ __forceinline__ uint4 load16(const void *p) {
    const u32x4 v = *static_cast<const u32x4_any *>(p);
    return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ uint2 load8b(const void *p) {
    const u32x2 v = *static_cast<const u32x2_any *>(p);
    return make_uint2(v.x, v.y);
}
__device__ __forceinline__ uint32_t load4(const void *p) { return *static_cast<const u32_any *>(p); }
__device__ __forceinline__ uint32_t load2b(const void *p) { return *static_cast<const u16_any *>(p); }
__device__ __forceinline__ void store16(void *p, uint4 v) {
    *static_cast<u32x4_any *>(p) = u32x4{v.x, v.y, v.z, v.w};
}
__device__ __forceinline__ void store8b(void *p, uint2 v) { *static_cast<u32x2_any *>(p) = u32x2{v.x, v.y}; }

// Two binary32 values rounded to bf16 (nearest, ties to even) in one dword.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}

// ------------------------------------------------------------------------- eight values of a row

// A value the compiler has to take as new: what was computed from it before is computed again from it after, and
// not kept in registers meanwhile.
__device__ __forceinline__ void renew(uint32_t &v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void renew(uint4 &v) { renew(v.x), renew(v.y), renew(v.z), renew(v.w); }

// Eight consecutive values as they lie in memory: bf16 (one 16-byte load) or fp32 (two).
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    uint4 a;
    // the first n (0..8) of the eight; the rest read as zeros
    __device__ __forceinline__ void load(const uint16_t *p, int n) {
        if (n >= 8) {
            a = load16(p);
        } else {
            uint32_t d[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) d[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
            a = make_uint4(d[0], d[1], d[2], d[3]);
        }
    }
    __device__ __forceinline__ void get(float v[8]) const {
        const uint32_t d[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(d[i]), v[2 * i + 1] = bf16_hi(d[i]);
    }
    __device__ __forceinline__ void again() { renew(a); }
};
template <>
struct Raw8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p, int n) {
        if (n >= 8) {
            a = load16(p);
            b = load16(p + 4);
        } else {
            uint32_t d[8] = {};
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) d[i] = __float_as_uint(p[i]);
            a = make_uint4(d[0], d[1], d[2], d[3]);
            b = make_uint4(d[4], d[5], d[6], d[7]);
        }
    }
    __device__ __forceinline__ void get(float v[8]) const {
        const uint32_t d[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(d[i]);
    }
    __device__ __forceinline__ void again() {}  // the values are what lies in memory
};

// The first n (0..8) of eight values, rounded once to the memory's type.
__device__ __forceinline__ void put8(uint16_t *p, const float v[8], int n) {
    const uint32_t d[4] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    if (n >= 8) {
        store16(p, make_uint4(d[0], d[1], d[2], d[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) p[i] = (uint16_t)(d[i >> 1] >> (16 * (i & 1)));
    }
}
__device__ __forceinline__ void put8(float *p, const float v[8], int n) {
    if (n >= 8) {
        store16(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
        store16(p + 4,
                make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) p[i] = v[i];
    }
}

// --------------------------------------------------------------------------------------- MXFP8

// Scale byte of a block whose largest magnitude has the binary32 pattern `amax` (sign clear). 448 is
// 1.75 * 2^8: a significand above 1.75 moves to the next power of two, which the addition's carry does.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
    if (amax >= 0x7F800000u) return 255u;
    const uint32_t b = (amax + 0x1FFFFFu) >> 23;
    return b < 8u ? 0u : b - 8u;
}

// 2^(b - 127); NaN for 255.
__device__ __forceinline__ float mx_scale_value(uint32_t b) {
    return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7FC00000u : b << 23);
}

// Eight values to E4M3 codes under scale byte `sb`. Multiplying by the inverse power of two (2^127 down to
// 2^-120 for the bytes that mx_scale_byte gives) is exact or far below the smallest code.
__device__ __forceinline__ uint2 mx_encode8(const float v[8], uint32_t sb) {
    if (sb == 255u) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    const float r = __uint_as_float((254u - sb) << 23);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * r, v[1] * r, lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * r, v[3] * r, lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * r, v[5] * r, hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * r, v[7] * r, hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// Four codes of a dword times a scale value.
__device__ __forceinline__ void mx_decode4(uint32_t c, float s, float v[4]) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    v[0] = a.x * s, v[1] = a.y * s, v[2] = b.x * s, v[3] = b.y * s;
}

// Largest magnitude (binary32 pattern, sign clear; NaN patterns order above infinity) of eight values.
__device__ __forceinline__ uint32_t amax8(const float v[8]) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
}

// Maximum over the four lanes of a quad (all four must be active).
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
}

// The lane's eight values (n of them in the row, 0..8) of a 32-value block held by a quad, to memory: codes
// at `codes`, the block's scale byte by the quad's first lane at `scale`.
// WHOLE: n is 0 or 8.
template <bool WHOLE = false>
__device__ __forceinline__ void mx_put8(uint8_t *codes, uint8_t *scale, const float v[8], int n, int lane) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (WHOLE ? n > 0 : i < n) ? v[i] : 0.0f;  // past the row: no part in the maximum
    const uint32_t sb = mx_scale_byte(quad_max(amax8(w)));
    const uint2 c = mx_encode8(w, sb);
    if (n >= 8) {
        store8b(codes, c);
    } else if (!WHOLE) {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) codes[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
    if ((lane & 3) == 0 && n > 0) *scale = (uint8_t)sb;
}

// Eight values of an MXFP8 row (they lie in one block): the raw bytes, then the values.
struct RawMx8 {
    uint2 c;
    uint32_t sb;
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scale, int n) {
        c = make_uint2(0u, 0u);
        sb = 0u;
        if (n >= 8) {
            c = load8b(codes);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) (i < 4 ? c.x : c.y) |= (uint32_t)codes[i] << (8 * (i & 3));
        }
        if (n > 0) sb = *scale;
    }
    __device__ __forceinline__ void get(float v[8]) const {
        const float s = mx_scale_value(sb);
        mx_decode4(c.x, s, v);
        mx_decode4(c.y, s, v + 4);
    }
    __device__ __forceinline__ void again() { renew(c.x), renew(c.y), renew(sb); }
};

}  // namespace nvfp4

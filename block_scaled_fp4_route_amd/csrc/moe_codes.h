// Block-scaled e2m1 codes in registers: from values (exact rounding) and to the
// 16-bit operands of the matrix instructions (exact decoding).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_rows.h"

namespace moe {

constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ u4w ld_b128(rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u4w, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// The E4M3 byte nearest to a / 6 (ties to even, at most 448), a >= 0 finite.
__device__ __forceinline__ uint32_t e4m3_sixth(float a) {
    // near the result: a * fp32(1/6) is off by 2^-23 of a at most, so the byte
    // it rounds to is the nearest one or its neighbour; which one is decided
    // by comparing a with 6 times the borders, exactly
    const float q = fminf(a * 0.16666667f, 448.0f);
    uint32_t b = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false) & 0x7Fu;
    const float v = e4m3_to_f32(b);
    const float up = e4m3_to_f32(min(b + 1u, 0x7Eu)), down = e4m3_to_f32(b ? b - 1u : 0u);
    const float hi = 3.0f * (v + up), lo = 3.0f * (v + down);  // 6 times the middle: exact
    const bool odd = b & 1u;
    if (b < 0x7Eu && (a > hi || (a == hi && odd))) b++;
    else if (b > 0u && (a < lo || (a == lo && odd))) b--;
    return b;
}

// Codes of eight values (times the exact power of two p) under the scale s,
// as one word, and the values they stand for (without p).
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float p, float s, float (&q)[8]) {
    const float b0 = 0.25f * s, b1 = 0.75f * s, b2 = 1.25f * s, b3 = 1.75f * s, b4 = 2.5f * s, b5 = 3.5f * s, b6 = 5.0f * s;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float m = fabsf(v[i]) * p;
        const uint32_t c = (uint32_t)(m > b0) + (m >= b1) + (m > b2) + (m >= b3) + (m > b4) + (m >= b5) + (m > b6);
        w |= (c | (__float_as_uint(v[i]) >> 31 << 3)) << (4 * i);
    }
    const f2v d0 = fp4x2<0>(w), d1 = fp4x2<1>(w), d2 = fp4x2<2>(w), d3 = fp4x2<3>(w);
    q[0] = d0.x; q[1] = d0.y; q[2] = d1.x; q[3] = d1.y;
    q[4] = d2.x; q[5] = d2.y; q[6] = d3.x; q[7] = d3.y;
    return w;
}

// The same for s = 1: times p, which is exact, the conversion instruction rounds
// as the definition does (nearest, ties to the even code, above 6 to 6, the sign
// kept), at a third of the comparisons' instructions.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float p, float (&q)[8]) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * p, v[1] * p, 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * p, v[3] * p, 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * p, v[5] * p, 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * p, v[7] * p, 1.0f, 3);
    const f2v d0 = fp4x2<0>(w), d1 = fp4x2<1>(w), d2 = fp4x2<2>(w), d3 = fp4x2<3>(w);
    q[0] = d0.x; q[1] = d0.y; q[2] = d1.x; q[3] = d1.y;
    q[4] = d2.x; q[5] = d2.y; q[6] = d3.x; q[7] = d3.y;
    return w;
}

__device__ __forceinline__ uint32_t max_mag(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
}

// The shared exponent X of an MXFP4 block whose largest magnitude has the bits
// `top` (finite): floor(log2) - 2, with ceil one more where the largest is above
// 1.5 times its power of two (6 = 1.5 2^2).
__device__ __forceinline__ int mx_exponent(uint32_t top, bool ceil) {
    const int X = (int)(top >> 23) - 129 + (ceil && (top & 0x7FFFFFu) > 0x400000u ? 1 : 0);
    return max(-127, min(125, X));
}

// ---------------------------------------------------------------------------
// Operands of the matrix instructions. Every e2m1 code times its scale has at
// most 6 significant bits: exact in bf16 (UE8M0 scales down to 2^-127: the
// values are subnormal bf16), and with an E4M3 scale, 2^-10 to 2688, in fp16.
constexpr int kNvBf16 = 0, kMxBf16 = 1, kNvF16 = 2, kCodes = 3;

// What a scale byte is to decode_op.
template <int MODE>
__device__ __forceinline__ float scale_op(uint32_t b) {
    if constexpr (MODE == kMxBf16) return __uint_as_float((b & 0xFFu) << 23);  // its exponent goes to the conversion
    else return e4m3_to_f32(b & 0xFFu);
}
// Eight codes -> eight 16-bit values.
template <int MODE>
__device__ __forceinline__ u4w decode_op(uint32_t w, float s) {
    u4w o;
    if constexpr (MODE == kMxBf16) {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    } else if constexpr (MODE == kNvBf16) {
        const f2v a = fp4x2<0>(w), b = fp4x2<1>(w), c = fp4x2<2>(w), d = fp4x2<3>(w);
        const f2v p[4] = {{a.x * s, a.y * s}, {b.x * s, b.y * s}, {c.x * s, c.y * s}, {d.x * s, d.y * s}};
#pragma unroll
        for (int i = 0; i < 4; i++) o[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p[i], bf2));
    } else {
        const hf2 ss = {(_Float16)s, (_Float16)s};
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * ss);
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * ss);
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * ss);
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * ss);
    }
    return o;
}

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 hf8 __attribute__((ext_vector_type(8)));
typedef int i8v __attribute__((ext_vector_type(8)));

// c + A B over 32 of the sum: A's row and B's column are lane % 16, a lane holds
// the eight of the sum at lane / 16; c: column lane % 16, rows 4 (lane / 16) + r.
template <bool F16>
__device__ __forceinline__ f4v mma16(u4w a, u4w b, f4v c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(hf8, a), __builtin_bit_cast(hf8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}
// The same over 128 codes, 32 a lane, each lane's under one UE8M0 byte.
__device__ __forceinline__ f4v mma16_codes(u4w a, u4w b, f4v c, uint32_t sa, uint32_t sb) {
    const i8v A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i8v B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

}  // namespace moe

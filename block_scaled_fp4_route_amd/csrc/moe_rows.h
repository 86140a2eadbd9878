// Eight consecutive elements of a row in any of the activation types (F32,
// BF16, F16), as fp32 in registers: one or two 16-byte accesses a lane. Stores
// round once, to nearest even; an fp32 value above the largest fp16 or bf16
// one becomes infinite, as the type has it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_learn.h"

namespace moe {

typedef uint32_t u2w __attribute__((ext_vector_type(2)));
typedef uint32_t u4w __attribute__((ext_vector_type(4)));
typedef _Float16 hf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

template <int DT>
struct Act;
template <>
struct Act<kActF32> {
    static constexpr int size = 4;
};
template <>
struct Act<kActBf16> {
    static constexpr int size = 2;
};
template <>
struct Act<kActF16> {
    static constexpr int size = 2;
};

// What a lane holds of eight elements as they lie in memory.
template <int DT>
struct Raw8 {
    u4w w[Act<DT>::size / 2];
};
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const void* row, size_t at) {
    Raw8<DT> r;
    const u4w* p = reinterpret_cast<const u4w*>(static_cast<const char*>(row) + at * Act<DT>::size);
#pragma unroll
    for (int i = 0; i < Act<DT>::size / 2; i++) r.w[i] = p[i];
    return r;
}
template <int DT>
__device__ __forceinline__ void unpack8(const Raw8<DT>& r, float (&v)[8]) {
    if constexpr (DT == kActF32) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = __uint_as_float(r.w[i / 4][i % 4]);
    } else if constexpr (DT == kActBf16) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = bf16_lo(r.w[0][i]);
            v[2 * i + 1] = bf16_hi(r.w[0][i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t w = r.w[0][i];  // a bit_cast of the vector's element itself reads element 0
            const hf2 h = __builtin_bit_cast(hf2, w);
            v[2 * i] = (float)h[0];
            v[2 * i + 1] = (float)h[1];
        }
    }
}
template <int DT>
__device__ __forceinline__ Raw8<DT> pack8(const float (&v)[8]) {
    Raw8<DT> r;
    if constexpr (DT == kActF32) {
#pragma unroll
        for (int i = 0; i < 8; i++) r.w[i / 4][i % 4] = __float_as_uint(v[i]);
    } else if constexpr (DT == kActBf16) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            r.w[0][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{v[2 * i], v[2 * i + 1]}), bf2));
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            r.w[0][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{v[2 * i], v[2 * i + 1]}), hf2));
    }
    return r;
}
template <int DT>
__device__ __forceinline__ void store8(void* row, size_t at, const Raw8<DT>& r) {
    u4w* p = reinterpret_cast<u4w*>(static_cast<char*>(row) + at * Act<DT>::size);
#pragma unroll
    for (int i = 0; i < Act<DT>::size / 2; i++) p[i] = r.w[i];
}

// 2^e as fp32, -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

}  // namespace moe

// Quantisation to block-scaled e2m1 codes (gfx950): a matrix of fp32, bf16 or
// fp16 values to NVFP4 (an E4M3 scale for 16 codes, and a power of two for
// each row if the caller wants one) or MXFP4 (a UE8M0 scale for 32 codes), and
// the values that the codes stand for.
//
// Nothing is divided. A block's exponent comes from the bits of its largest
// magnitude. A magnitude m goes to code c where the borders between codes
// (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5) times the scale s lie on the right
// sides of m: a border has at most 3 significant bits, an E4M3 scale 4, so
// the product is exact in fp32 and so is m times a power of two (MXFP4's scale
// is one: the conversion instruction does the rest). The E4M3
// scale nearest to amax / 6 is found the same way: 6 times the border between
// two E4M3 values has 7 bits. The result is therefore the definition's, bit
// for bit, with no case that a rounded quotient would decide.
//
// Memory bounds it: every value read once (a row with an exponent of its own
// stays in registers between its two uses), codes, scales and values written
// once: 8192 x 2560 fp32 to MXFP4 with its values 35 us, 5.1 TB/s, as fast as a
// copy. Small matrices are a launch: 640 x 2560 bf16 with row exponents 5.5 us.
// NVFP4 counts seven comparisons a value: 8192 x 2560 with row exponents and values
// takes 28.6 us in bf16 where MXFP4 takes 17.1, and 37.6 in fp32 against 35.1.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_codes.h"
#include "moe_rows.h"
#include "moe_serve.h"

namespace moe {
namespace {

constexpr int kRowExpMin = -100, kRowExpMax = 116;  // so that every decoded value is a normal bf16, and finite

struct QuantArgs {
    const char* x;
    size_t ldx;  // bytes
    uint32_t rows, c8;  // c8: pieces of 8 in a row
    int8_t* row_exp;
    uint8_t *codes, *scales;
    char* values;
    size_t ldv;  // bytes
    int rule;
};

// One piece of 8 values, its block's lanes beside it (2 of NVFP4, 4 of MXFP4;
// all of them active). re: the row's exponent.
template <int DT, int FMT>
__device__ __forceinline__ void quant_piece(const QuantArgs& a, uint32_t row, uint32_t c, const float (&v)[8], int re) {
    constexpr int L = Fmt<FMT>::G / 8;
    uint32_t top = max_mag(v);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
    const bool bad = top >= kInfBits;  // an infinity or a NaN: the whole block decodes to NaN
    uint32_t byte;
    float p, s, back;  // magnitudes times p against s; decoded times s times back
    if constexpr (FMT == kFmtNvfp4) {
        p = exp2i(-re);
        back = exp2i(re);
        byte = bad ? 0x7Fu : e4m3_sixth(__uint_as_float(top) * p);
        s = e4m3_to_f32(byte);
    } else {
        const int X = mx_exponent(top, a.rule == kScaleCeil);
        byte = bad ? 0xFFu : top == 0u ? 0u : (uint32_t)(X + 127);
        p = exp2i(-X);
        s = 1.0f;
        back = ue8m0_to_f32(byte);
    }
    float q[8];
    uint32_t w;
    if constexpr (FMT == kFmtNvfp4) w = codes8(v, p, s, q);
    else w = codes8(v, p, q);
    if (bad || (FMT == kFmtNvfp4 && byte == 0u)) {  // all codes zero (under a scale of 0, every border is 0)
        w = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            w |= bad ? 0u : __float_as_uint(v[i]) >> 31 << (4 * i + 3);
            q[i] = bad ? __uint_as_float(0x7FC00000u) : copysignf(0.0f, v[i]);
        }
    }
    const size_t at = (size_t)row * a.c8 + c;
    if (a.codes) reinterpret_cast<uint32_t*>(a.codes)[at] = w;
    if (a.scales && (c & (L - 1)) == 0) a.scales[at / L] = (uint8_t)byte;
    if (a.values) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            q[i] = q[i] * s * back;
            if (DT == kActF16) q[i] = q[i] > 65504.f ? 65504.f : q[i] < -65504.f ? -65504.f : q[i];
        }
        store8<DT>(a.values + (size_t)row * a.ldv, 8 * (size_t)c, pack8<DT>(q));
    }
}

// Blocks on their own: a lane a piece, whole blocks in or out of the matrix.
template <int DT, int FMT>
__global__ __launch_bounds__(256) void k_fp4_quant(QuantArgs a) {
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    const uint32_t row = i / a.c8, c = i - row * a.c8;
    if (row >= a.rows) return;
    float v[8];
    unpack8<DT>(load8<DT>(a.x + (size_t)row * a.ldx, 8 * (size_t)c), v);
    quant_piece<DT, FMT>(a, row, c, v, 0);
}

// NVFP4 with row exponents: NT threads take a row (64: four rows a workgroup,
// 256: one). The first kHeld pieces of a lane stay in registers, further ones
// are read again (longer rows: out of the cache).
constexpr int kHeld = 4;
constexpr uint32_t kRowsAtOnce = 1u << 25;
template <int DT, int NT>
__global__ __launch_bounds__(256) void k_fp4_quant_rows(QuantArgs a) {
    __shared__ uint32_t tops[4];
    const uint32_t t = threadIdx.x & (NT - 1), row = NT == 64 ? blockIdx.x * 4u + wave_id() : blockIdx.x;
    if (NT == 64 && row >= a.rows) return;
    const char* xr = a.x + (size_t)row * a.ldx;
    float v[kHeld][8];
    uint32_t top = 0;
    auto look = [&](const float (&u)[8]) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t m = __float_as_uint(u[i]) & 0x7FFFFFFFu;
            top = max(top, m < kInfBits ? m : 0u);
        }
    };
    Raw8<DT> raw[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; j++)
        if (t + NT * j < a.c8) raw[j] = load8<DT>(xr, 8 * (size_t)(t + NT * j));
#pragma unroll
    for (int j = 0; j < kHeld; j++)
        if (t + NT * j < a.c8) {
            unpack8<DT>(raw[j], v[j]);
            look(v[j]);
        }
    for (uint32_t c = t + NT * kHeld; c < a.c8; c += NT) {
        float u[8];
        unpack8<DT>(load8<DT>(xr, 8 * (size_t)c), u);
        look(u);
    }
    top = wave_max_u32(top);
    if (NT == 256) {
        if ((threadIdx.x & 63) == 0) tops[wave_id()] = top;
        __syncthreads();
        top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    }
    // the smallest e with top <= 2688 2^e = 1.3125 2^(11 + e)
    int e = (int)(top >> 23) - 138 + ((top & 0x7FFFFFu) > 0x280000u ? 1 : 0);
    e = top == 0u ? 0 : max(kRowExpMin, min(kRowExpMax, e));
    if (t == 0) a.row_exp[row] = (int8_t)e;
#pragma unroll
    for (int j = 0; j < kHeld; j++)
        if (t + NT * j < a.c8) quant_piece<DT, kFmtNvfp4>(a, row, t + NT * j, v[j], e);
    for (uint32_t c = t + NT * kHeld; c < a.c8; c += NT) {
        float u[8];
        unpack8<DT>(load8<DT>(xr, 8 * (size_t)c), u);
        quant_piece<DT, kFmtNvfp4>(a, row, c, u, e);
    }
}

template <int DT>
hipError_t quant(int fmt, const QuantArgs& a, hipStream_t s) {
    if (a.row_exp && a.c8 <= 64 * kHeld) {
        // a launch has less than 2^32 threads: 64 a row, so more rows than kRowsAtOnce go out in several
        for (uint32_t at = 0; at < a.rows; at += kRowsAtOnce) {
            QuantArgs b = a;
            const size_t pieces = (size_t)at * a.c8;
            b.rows = a.rows - at < kRowsAtOnce ? a.rows - at : kRowsAtOnce;
            b.x += at * a.ldx;
            b.row_exp += at;
            if (b.codes) b.codes += 4 * pieces;
            if (b.scales) b.scales += pieces / 2;  // two pieces a block
            if (b.values) b.values += at * a.ldv;
            hipLaunchKernelGGL((k_fp4_quant_rows<DT, 64>), dim3((b.rows + 3) / 4), dim3(256), 0, s, b);
            const hipError_t r = hipGetLastError();
            if (r != hipSuccess) return r;
        }
    } else if (a.row_exp) {
        hipLaunchKernelGGL((k_fp4_quant_rows<DT, 256>), dim3(a.rows), dim3(256), 0, s, a);
    } else {
        const dim3 grid((unsigned)(((size_t)a.rows * a.c8 + 255) / 256));
        if (fmt == kFmtNvfp4)
            hipLaunchKernelGGL((k_fp4_quant<DT, kFmtNvfp4>), grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_fp4_quant<DT, kFmtMxfp4>), grid, dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp4_quant(int dtype, int fmt, int rule, const void* x, size_t ldx, int rows, int cols,
                            int8_t* row_exp, uint8_t* codes, uint8_t* scales, void* values, size_t ldv, hipStream_t s) {
    const size_t es = dtype == kActF32 ? 4 : 2;
    const QuantArgs a = {static_cast<const char*>(x), ldx * es, (uint32_t)rows, (uint32_t)cols / 8, row_exp, codes, scales,
                         static_cast<char*>(values), ldv * es, rule};
    if (dtype == kActF32) return quant<kActF32>(fmt, a, s);
    return dtype == kActBf16 ? quant<kActBf16>(fmt, a, s) : quant<kActF16>(fmt, a, s);
}

}  // namespace moe

// Products of a few activation rows with a matrix stored in 4 bits (gfx950):
// y = base + x W^T for up to 64 tokens, W read once.
//
//  * up to 4 tokens (k_fp4_gemv): a wave has 4 rows of W, a lane 8 codes of each
//    per 512; x sits in LDS as fp32, products and sums on the vector units.
//  * up to 64 (k_fp4_few): a wave has one or two blocks of 16 rows, its share of
//    the sum, and all tokens, 16 at a time as columns of a matrix instruction:
//    the codes are decoded once in registers, where they are an operand already,
//    and the tokens' values come from L2. The waves' sums meet in LDS.
//
// 2560 x 8192 NVFP4 (11.8 MB): 1 token 6.5 us (launch, loads and sums over the
// lanes are one chain, 1.8 TB/s), 4 tokens 11.4 (four times the products). 16
// tokens of fp32 19 us, 64 35: each workgroup reads every token's parts, 250 MB
// from L2 at 64. 64 tokens rounded to MXFP4 9 us: an eleventh
// of those bytes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_codes.h"
#include "moe_device.h"
#include "moe_internal.h"
#include "moe_rows.h"
#include "moe_serve.h"

namespace moe {
namespace {

struct FewArgs {
    const char* x;           // activations, their parts (P K values a row), or codes
    size_t ldx;              // bytes
    const uint8_t* xs;       // kCodes: scale bytes [T][K / 32]
    int T, K, N;
    Fp4Matrix w;
    const char* base;
    char* y;
    size_t ldbase, ldy;      // bytes
    bool round_x;            // k_fp4_gemv: round x to MXFP4 first
};

__device__ __forceinline__ uint32_t ld_b16(rsrc_t r, uint32_t off) { return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0); }

template <int DT>
__device__ __forceinline__ float get1(const char* p, size_t i) {
    if constexpr (DT == kActF32) return reinterpret_cast<const float*>(p)[i];
    else if constexpr (DT == kActBf16) return (float)reinterpret_cast<const __bf16*>(p)[i];
    else return (float)reinterpret_cast<const _Float16*>(p)[i];
}
template <int DT>
__device__ __forceinline__ void put1(char* p, size_t i, float v) {
    if constexpr (DT == kActF32) reinterpret_cast<float*>(p)[i] = v;
    else if constexpr (DT == kActBf16) reinterpret_cast<__bf16*>(p)[i] = (__bf16)v;
    else reinterpret_cast<_Float16*>(p)[i] = (_Float16)v;
}

// ---------------------------------------------------------------------------
// Up to 4 tokens

constexpr int kGemvRows = 4;     // rows of a wave: 32 loads of codes and scales on their way
constexpr int kGemvChunk = 4096; // of the sum in LDS at a time

// x[chunk] of every token as fp32 in LDS: [token][half][piece of 8] quads, so
// that a wave reads 64 pieces' halves without bank conflicts.
template <int DT, int TT>
__device__ __forceinline__ void stage(const FewArgs& a, int k0, f4v (*lds)[2][kGemvChunk / 8]) {
    const int n8 = min(kGemvChunk, a.K - k0) / 8;
    for (int t = 0; t < TT; t++) {
        const char* row = a.x + (size_t)min(t, a.T - 1) * a.ldx;  // a token behind the last one loads and becomes zeros
        for (int p = threadIdx.x; p < kGemvChunk / 8; p += 256) {  // all lanes stay: a block's four share its maximum
            float v[8];
            const bool in = p < n8 && t < a.T;
            unpack8<DT>(load8<DT>(row, in ? (size_t)k0 + 8 * p : 0), v);
            if (a.round_x) {
                uint32_t top = max_mag(v);
                top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
                top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
                const int X = mx_exponent(top, false);
                float q[8];
                codes8(v, exp2i(-X), q);
                const float s = X == -127 ? __uint_as_float(0x00400000u) : exp2i(X);
#pragma unroll
                for (int j = 0; j < 8; j++) v[j] = top >= kInfBits ? __uint_as_float(0x7FC00000u) : q[j] * s;
            }
            lds[t][0][p] = in ? f4v{v[0], v[1], v[2], v[3]} : f4v{0.f, 0.f, 0.f, 0.f};
            lds[t][1][p] = in ? f4v{v[4], v[5], v[6], v[7]} : f4v{0.f, 0.f, 0.f, 0.f};
        }
    }
}

template <int FMT, int DT, int TT>
__global__ __launch_bounds__(256) void k_fp4_gemv(FewArgs a) {
    constexpr int R = kGemvRows, NI = kGemvChunk / 512, G8 = Fmt<FMT>::G / 8;
    __shared__ f4v xs[TT][2][kGemvChunk / 8];
    const int lane = threadIdx.x & 63, r0 = (blockIdx.x * 4 + wave_id()) * R, rows = min(R, a.N - r0);
    const uint32_t cb = (uint32_t)a.K / 2, sb = (uint32_t)a.K / Fmt<FMT>::G;
    const int rb = max(rows, 1), at = rows > 0 ? r0 : 0;  // a wave behind the last row loads from the first and stores nothing
    const rsrc_t rc = make_rsrc(a.w.codes + (size_t)at * cb, (uint32_t)rb * cb), rs = make_rsrc(a.w.scales + (size_t)at * sb, (uint32_t)rb * sb);
    float acc[R][TT];
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int t = 0; t < TT; t++) acc[r][t] = 0.0f;
    for (int k0 = 0; k0 < a.K; k0 += kGemvChunk) {
        const uint32_t p0 = k0 / 8, n8 = min(kGemvChunk, a.K - k0) / 8;
        uint32_t c[NI][R], s[NI][R];
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const uint32_t p = lane + 64 * i;
#pragma unroll
            for (int r = 0; r < R; r++) {
                const bool on = p < n8 && r < rows;
                c[i][r] = ld_b32(rc, on ? r * cb + 4 * (p0 + p) : kOOB);
                s[i][r] = ld_b8(rs, on ? r * sb + (p0 + p) / G8 : kOOB);
            }
        }
        if (k0) __syncthreads();
        stage<DT, TT>(a, k0, xs);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NI; i++) {
            if (64u * i < n8) {
                f4v x[TT][2];
#pragma unroll
                for (int t = 0; t < TT; t++) {
                    x[t][0] = xs[t][0][lane + 64 * i];
                    x[t][1] = xs[t][1][lane + 64 * i];
                }
#pragma unroll
                for (int r = 0; r < R; r++) {
                    float v[8];
                    if constexpr (FMT == kFmtMxfp4) {
                        const float e = __uint_as_float(s[i][r] << 23);
                        const f2v d0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i][r], e, 0), d1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i][r], e, 1);
                        const f2v d2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i][r], e, 2), d3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i][r], e, 3);
                        v[0] = d0.x; v[1] = d0.y; v[2] = d1.x; v[3] = d1.y;
                        v[4] = d2.x; v[5] = d2.y; v[6] = d3.x; v[7] = d3.y;
                    } else {
                        const float e = e4m3_to_f32(s[i][r]);
                        const f2v d0 = fp4x2<0>(c[i][r]), d1 = fp4x2<1>(c[i][r]), d2 = fp4x2<2>(c[i][r]), d3 = fp4x2<3>(c[i][r]);
                        v[0] = d0.x * e; v[1] = d0.y * e; v[2] = d1.x * e; v[3] = d1.y * e;
                        v[4] = d2.x * e; v[5] = d2.y * e; v[6] = d3.x * e; v[7] = d3.y * e;
                    }
#pragma unroll
                    for (int t = 0; t < TT; t++)
#pragma unroll
                        for (int j = 0; j < 8; j++) acc[r][t] = fmaf(v[j], x[t][j / 4][j % 4], acc[r][t]);
                }
            }
        }
    }
    float mine = 0.0f;  // lane 4 t + r keeps that sum
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int t = 0; t < TT; t++) {
            const float v = wave_sum(acc[r][t]);
            if (lane == R * t + r) mine = v;
        }
    const int t = lane / R, n = r0 + lane % R;
    if (t < TT && t < a.T && n < a.N) {
        if (a.w.row_exp) mine = ldexpf(mine, a.w.row_exp[n]);
        if (a.base) mine += get1<DT>(a.base + (size_t)t * a.ldbase, n);
        put1<DT>(a.y + (size_t)t * a.ldy, n, mine);
    }
}

// ---------------------------------------------------------------------------
// Up to 64 tokens

// MODE: how the codes become operands; P: parts of an activation; NG: groups of
// 16 tokens; RB: row blocks of a wave. A wave takes the blocks wave, wave + NW,
// ... of 128 of the sum; within one, lane l holds 32 codes of row l % 16 and the
// same 32 values of token l % 16 (those of sum index 32 (l / 16) .. + 31), which
// four matrix instructions use 8 at a time: the order of a sum's terms is free
// as long as both operands have the same.
template <int MODE, int P, int NG, int RB, int DT>
__global__ __launch_bounds__(512) void k_fp4_few(FewArgs a) {
    constexpr bool NV = MODE == kNvBf16 || MODE == kNvF16;
    constexpr int G = NV ? 16 : 32;
    __shared__ f4v part[8][RB][NG][64];
    const int lane = threadIdx.x & 63, wave = wave_id(), nw = blockDim.x >> 6;
    const int li = lane & 15, lg = lane >> 4, n0 = blockIdx.x * 16 * RB, rows = min(16 * RB, a.N - n0);
    const uint32_t cb = (uint32_t)a.K / 2, sb = (uint32_t)a.K / G, ldx = (uint32_t)a.ldx;
    const rsrc_t rc = make_rsrc(a.w.codes + (size_t)n0 * cb, rows * cb), rs = make_rsrc(a.w.scales + (size_t)n0 * sb, rows * sb);
    const rsrc_t rx = make_rsrc(a.x, (uint32_t)(a.T - 1) * ldx + (MODE == kCodes ? cb : (uint32_t)a.K * P * 2));
    const rsrc_t rxs = make_rsrc(MODE == kCodes ? a.xs : nullptr, MODE == kCodes ? (uint32_t)a.T * sb : 0u);
    f4v acc[RB][NG];
#pragma unroll
    for (int i = 0; i < RB; i++)
#pragma unroll
        for (int g = 0; g < NG; g++) acc[i][g] = f4v{0.f, 0.f, 0.f, 0.f};
    struct Wts {
        u4w c[RB];
        uint32_t s[RB];
    };
    auto fetch = [&](int b, Wts& q) {
        const uint32_t k = 128u * b + 32u * lg;
#pragma unroll
        for (int i = 0; i < RB; i++) {
            const uint32_t r = 16 * i + li;
            const bool on = (int)r < rows && k < (uint32_t)a.K;
            q.c[i] = ld_b128(rc, on ? r * cb + k / 2 : kOOB);
            q.s[i] = NV ? ld_b16(rs, on ? r * sb + k / 16 : kOOB) : ld_b8(rs, on ? r * sb + k / 32 : kOOB);
        }
    };
    auto work = [&](int b, const Wts& q) {
        const uint32_t k = 128u * b + 32u * lg;
        if constexpr (MODE == kCodes) {
#pragma unroll
            for (int g = 0; g < NG; g++) {
                const uint32_t t = 16 * g + li;
                const bool on = (int)t < a.T && k < (uint32_t)a.K;
                const u4w x = ld_b128(rx, on ? t * ldx + k / 2 : kOOB);
                const uint32_t s = ld_b8(rxs, on ? t * sb + k / 32 : kOOB);
#pragma unroll
                for (int i = 0; i < RB; i++) acc[i][g] = mma16_codes(q.c[i], x, acc[i][g], q.s[i], s);
            }
        } else {
            u4w w[RB][4];
#pragma unroll
            for (int i = 0; i < RB; i++)
#pragma unroll
                for (int s = 0; s < 4; s++) w[i][s] = decode_op<MODE>(q.c[i][s], scale_op<MODE>(NV && s >= 2 ? q.s[i] >> 8 : q.s[i]));
#pragma unroll
            for (int p = 0; p < P; p++)
#pragma unroll
                for (int g = 0; g < NG; g++) {
                    const uint32_t t = 16 * g + li;
                    const bool on = (int)t < a.T && k < (uint32_t)a.K;
                    const uint32_t o = on ? t * ldx + ((uint32_t)p * a.K + k) * 2 : kOOB;
                    u4w x[4];
#pragma unroll
                    for (int s = 0; s < 4; s++) x[s] = ld_b128(rx, on ? o + 16 * s : kOOB);
#pragma unroll
                    for (int s = 0; s < 4; s++)
#pragma unroll
                        for (int i = 0; i < RB; i++) acc[i][g] = mma16<MODE == kNvF16>(w[i][s], x[s], acc[i][g]);
                }
        }
    };
    const int nb = (a.K + 127) / 128;
    Wts q0, q1;
    fetch(wave, q0);  // blocks behind the last one: zeros
    for (int b = wave; b < nb; b += 2 * nw) {
        fetch(b + nw, q1);
        work(b, q0);
        fetch(b + 2 * nw, q0);
        if (b + nw < nb) work(b + nw, q1);
    }
#pragma unroll
    for (int i = 0; i < RB; i++)
#pragma unroll
        for (int g = 0; g < NG; g++) part[wave][i][g][lane] = acc[i][g];
    __syncthreads();
    for (int u = threadIdx.x; u < RB * NG * 64; u += blockDim.x) {
        const int l = u & 63, g = u / 64 % NG, i = u / (64 * NG);
        const int t = 16 * g + (l & 15), n = n0 + 16 * i + 4 * (l >> 4);
        if (t >= a.T || n >= a.N) continue;
        f4v v = part[0][i][g][l];
        for (int w = 1; w < nw; w++) v += part[w][i][g][l];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            float o = v[j];
            if (a.w.row_exp) o = ldexpf(o, a.w.row_exp[n + j]);
            if (a.base) o += get1<DT>(a.base + (size_t)t * a.ldbase, n + j);
            v[j] = o;
        }
        char* y = a.y + (size_t)t * a.ldy + (size_t)n * Act<DT>::size;
        if constexpr (DT == kActF32) {
            *reinterpret_cast<f4v*>(y) = v;
        } else {
            uint2 o;
            if constexpr (DT == kActBf16)
                o = make_uint2(__builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{v[0], v[1]}), bf2)),
                               __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{v[2], v[3]}), bf2)));
            else
                o = make_uint2(__builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{v[0], v[1]}), hf2)),
                               __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{v[2], v[3]}), hf2)));
            *reinterpret_cast<uint2*>(y) = o;
        }
    }
}

template <int MODE, int P, int DT>
hipError_t few(const FewArgs& a, hipStream_t s) {
    // enough waves that each has two or three blocks of the sum
    const int nb = (a.K + 127) / 128;
    const dim3 block(nb >= 16 ? 512 : nb >= 4 ? 256 : 128);
    if (a.T <= 16)
        hipLaunchKernelGGL((k_fp4_few<MODE, P, 1, 1, DT>), dim3((a.N + 15) / 16), block, 0, s, a);
    else if (a.T <= 32)
        hipLaunchKernelGGL((k_fp4_few<MODE, P, 2, 2, DT>), dim3((a.N + 31) / 32), block, 0, s, a);
    else
        hipLaunchKernelGGL((k_fp4_few<MODE, P, 4, 2, DT>), dim3((a.N + 31) / 32), block, 0, s, a);
    return hipGetLastError();
}

template <int FMT, int DT>
hipError_t gemv(const FewArgs& a, hipStream_t s) {
    const dim3 grid((a.N + 4 * kGemvRows - 1) / (4 * kGemvRows)), block(256);
    if (a.T == 1) hipLaunchKernelGGL((k_fp4_gemv<FMT, DT, 1>), grid, block, 0, s, a);
    else if (a.T == 2) hipLaunchKernelGGL((k_fp4_gemv<FMT, DT, 2>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_fp4_gemv<FMT, DT, 4>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp4_gemv(int K, int N, int fmt, int dtype, const void* x, size_t ldx, int T, const Fp4Matrix& w,
                           bool round_x, const void* base, size_t ldbase, void* y, size_t ldy, hipStream_t s) {
    const size_t es = dtype == kActF32 ? 4 : 2;
    const FewArgs a = {static_cast<const char*>(x), ldx * es, nullptr, T, K, N, w, static_cast<const char*>(base),
                       static_cast<char*>(y), ldbase * es, ldy * es, round_x};
    if (fmt == kFmtNvfp4) {
        if (dtype == kActF32) return gemv<kFmtNvfp4, kActF32>(a, s);
        return dtype == kActBf16 ? gemv<kFmtNvfp4, kActBf16>(a, s) : gemv<kFmtNvfp4, kActF16>(a, s);
    }
    if (dtype == kActF32) return gemv<kFmtMxfp4, kActF32>(a, s);
    return dtype == kActBf16 ? gemv<kFmtMxfp4, kActBf16>(a, s) : gemv<kFmtMxfp4, kActF16>(a, s);
}

hipError_t launch_fp4_few(int K, int N, int fmt, int dtype, const void* x, size_t ldx_bytes, const uint8_t* x_scales, int T,
                          const Fp4Matrix& w, const void* base, size_t ldbase, void* y, size_t ldy, hipStream_t s) {
    const size_t es = dtype == kActF32 ? 4 : 2;
    const FewArgs a = {static_cast<const char*>(x), ldx_bytes, x_scales, T, K, N, w, static_cast<const char*>(base),
                       static_cast<char*>(y), ldbase * es, ldy * es, false};
    if (x_scales) {
        if (dtype == kActF32) return few<kCodes, 1, kActF32>(a, s);
        return dtype == kActBf16 ? few<kCodes, 1, kActBf16>(a, s) : few<kCodes, 1, kActF16>(a, s);
    }
    if (fmt == kFmtNvfp4) {
        if (dtype == kActF32) return few<kNvBf16, 3, kActF32>(a, s);
        return dtype == kActBf16 ? few<kNvBf16, 1, kActBf16>(a, s) : few<kNvF16, 1, kActF16>(a, s);
    }
    if (dtype == kActF32) return few<kMxBf16, 3, kActF32>(a, s);
    return dtype == kActBf16 ? few<kMxBf16, 1, kActBf16>(a, s) : few<kMxBf16, 2, kActF16>(a, s);
}

}  // namespace moe

// Products with a matrix stored in block-scaled 4 bits (gfx950):
//   y = base + x W^T   and, for training what lies before a frozen W,
//   dx = dx_base + dy W.
//
// Activations kept: W becomes 16-bit values once (every e2m1 code times its
// scale has at most 6 significant bits: exact in bf16, and NVFP4's in fp16),
// the activations enter with all their bits as P bf16 parts laid side by side
// along the sum, x = p1 + p2 + p3 (bf16: itself; fp16: 2 parts, or itself
// where W is fp16; fp32: 3), and one 16-bit product over P K runs on the
// matrix units. Activations rounded to MXFP4 beside an MXFP4 matrix: both go
// to the scaled FP4 matrix instructions as codes, never widened.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_rows.h"
#include "moe_serve.h"

namespace moe {
namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 hf8 __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef int i8v __attribute__((ext_vector_type(8)));

constexpr int kBf16 = 0, kF16 = 1, kFp4 = 2;  // operands of the product
constexpr int kStepBytes = 128;               // of a row in one step of the sum

// Parts of an activation on the way of `dtype`, W as 16-bit `kind`.
int act_kind(int fmt, int dtype, bool backward) {
    // rows with exponents of their own keep them apart only where the sum does
    // not run over the rows
    return fmt == kFmtNvfp4 && dtype == kActF16 && !backward ? kF16 : kBf16;
}
int act_parts(int dtype, int kind) { return dtype == kActF32 ? 3 : dtype == kActF16 && kind == kBf16 ? 2 : 1; }

// ---------------------------------------------------------------------------
// Operands

// Eight codes times their scale, as fp32.
__device__ __forceinline__ void decode8(uint32_t w, float s, float (&v)[8]) {
    const f2v d0 = fp4x2<0>(w), d1 = fp4x2<1>(w), d2 = fp4x2<2>(w), d3 = fp4x2<3>(w);
    v[0] = d0.x * s; v[1] = d0.y * s; v[2] = d1.x * s; v[3] = d1.y * s;
    v[4] = d2.x * s; v[5] = d2.y * s; v[6] = d3.x * s; v[7] = d3.y * s;
}

// W as 16-bit values [N][K] (row exponents left out).
template <int FMT, int KIND>
__global__ __launch_bounds__(256) void k_fp4_widen(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                   size_t pieces, u4w* __restrict__ out) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= pieces) return;
    float v[8];
    decode8(codes[i], scale_to_f32<FMT>(scales[i / (Fmt<FMT>::G / 8)]), v);
    out[i] = KIND == kF16 ? pack8<kActF16>(v).w[0] : pack8<kActBf16>(v).w[0];
}

// W^T as bf16 [K][N], row exponents included. A workgroup turns 64 rows x 64
// columns in LDS.
template <int FMT>
__global__ __launch_bounds__(256) void k_fp4_widen_t(Fp4Matrix w, int K, int N, uint16_t* __restrict__ out) {
    __shared__ uint16_t t[64][72];  // [k][n]; 144-byte rows
    const int n0 = blockIdx.x * 64, k0 = blockIdx.y * 64, tid = threadIdx.x;
#pragma unroll
    for (int q = 0; q < 2; q++) {  // 64 rows of 8 pieces
        const int r = (tid >> 3) + 32 * q, c = tid & 7, n = n0 + r, k = k0 + 8 * c;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (n < N && k < K) {
            const size_t i = ((size_t)n * K + k) / 8;
            float s = scale_to_f32<FMT>(w.scales[i / (Fmt<FMT>::G / 8)]);
            decode8(reinterpret_cast<const uint32_t*>(w.codes)[i], s, v);
            if (w.row_exp) {
                const float e = exp2i(w.row_exp[n]);
#pragma unroll
                for (int j = 0; j < 8; j++) v[j] *= e;
            }
        }
        const u4w p = pack8<kActBf16>(v).w[0];
#pragma unroll
        for (int j = 0; j < 8; j++) t[8 * c + j][r] = (uint16_t)(p[j / 2] >> (16 * (j & 1)));
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; q++) {
        const int r = (tid >> 3) + 32 * q, c = tid & 7, k = k0 + r, n = n0 + 8 * c;
        if (k < K && n < N) *reinterpret_cast<u4w*>(out + (size_t)k * N + n) = *reinterpret_cast<const u4w*>(&t[r][8 * c]);
    }
}

// The high 16 bits of v as a bf16 value, NaN kept.
__device__ __forceinline__ uint32_t bf16_cut(float v) { return v != v ? 0x7FC0u : __float_as_uint(v) >> 16; }

// x [T][K] as P bf16 parts [T][P][K], cut, not rounded (no part overflows, and
// three hold 24 bits down to 2^-133). The parts behind an infinity or a NaN
// are 0.
template <int DT>
__global__ __launch_bounds__(256) void k_fp4_parts(const char* __restrict__ x, size_t ldx, size_t pieces, int k8,
                                                   u4w* __restrict__ out) {
    constexpr int P = DT == kActF32 ? 3 : 2;
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= pieces) return;
    const size_t t = i / (uint32_t)k8, c = i - t * k8;
    float v[8];
    unpack8<DT>(load8<DT>(x + t * ldx, 8 * c), v);
#pragma unroll
    for (int p = 0; p < P; p++) {
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            h[j] = bf16_cut(v[j]);
            v[j] = fabsf(v[j]) < INFINITY ? v[j] - __uint_as_float(h[j] << 16) : 0.0f;
        }
        out[(t * P + p) * k8 + c] = u4w{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
    }
}

// Scale bytes for the scaled product: [K / 256 steps][rows up to a whole tile][8], within a step's
// 8 blocks the even ones first (lanes 0-31 of a wave hold the even blocks of a
// step, lanes 32-63 the odd ones: a lane's four bytes are one word). Blocks
// behind the row's end are 0.
__device__ __forceinline__ int scale_place(int b) { return (b & 1) * 4 + (b >> 1 & 3); }
constexpr size_t tile_rows(size_t rows) { return (rows + 127) / 128 * 128; }
__global__ __launch_bounds__(256) void k_fp4_scale_panel(const uint8_t* __restrict__ scales, int rows, int nb,
                                                         uint8_t* __restrict__ out) {
    const int r = blockIdx.x * 256 + threadIdx.x, st = blockIdx.y;
    if (r >= rows) return;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const int b = 8 * st + j;
        if (b < nb) w[scale_place(j) / 4] |= (uint32_t)scales[(size_t)r * nb + b] << (8 * (scale_place(j) % 4));
    }
    *reinterpret_cast<uint2*>(out + ((size_t)st * tile_rows(rows) + r) * 8) = make_uint2(w[0], w[1]);
}

// ---------------------------------------------------------------------------
// C = A B^T, both row-major along the sum. A workgroup of 4 waves has a tile of
// 128 x 128; a step is 128 bytes of every row (64 16-bit values or 256 codes),
// loaded from memory straight into one of two LDS buffers while the other is
// multiplied. A row's eight 16-byte chunks sit in LDS at chunk ^ (row & 7), so
// that the reads of eight neighbouring rows' same chunk hit all banks once; the
// loads pick their chunk accordingly.
struct MmArgs {
    const char *a, *b;
    size_t lda, ldb;        // bytes between rows
    uint32_t wa, wb;        // bytes of a row (A's parts together; B starts again at its end)
    int M, N, steps;
    const uint8_t *sa, *sb; // kFp4: scale panels [steps][M or N][8]
    const int8_t* row_exp;  // of B's rows, or null
    const char* base;
    char* y;
    size_t ldbase, ldy;     // bytes
    int nt;                 // tiles along N
};

template <int N>
__device__ __forceinline__ void ring_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int KIND>
__device__ __forceinline__ f16v mma(u4w a, u4w b, f16v c) {
    if constexpr (KIND == kBf16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(hf8, a), __builtin_bit_cast(hf8, b), c, 0, 0, 0);
}
template <int KS>
__device__ __forceinline__ f16v mma4(u4w a, u4w b, f16v c, uint32_t sa, uint32_t sb) {
    const i8v A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i8v B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, KS, (int)sa, KS, (int)sb);
}

template <int KIND, int DT>
__global__ __launch_bounds__(256, 2) void k_fp4_mm(MmArgs g) {
    constexpr int BM = 128, BN = 128, MI = 2, NI = 2;
    constexpr int SC = KIND == kFp4 ? (BM + BN) * 8 : 0;       // scale bytes of a step
    constexpr int STEP = (BM + BN) * kStepBytes + SC;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STEP];
    const int lane = threadIdx.x & 63, wave = wave_id(), wm = wave >> 1, wn = wave & 1;
    const int m0 = blockIdx.x / g.nt * BM, n0 = blockIdx.x % g.nt * BN;
    const int am = min(BM, g.M - m0), bn = min(BN, g.N - n0);
    const rsrc_t rA = make_rsrc(g.a + (size_t)m0 * g.lda, (uint32_t)(am - 1) * (uint32_t)g.lda + g.wa);
    const rsrc_t rB = make_rsrc(g.b + (size_t)n0 * g.ldb, (uint32_t)(bn - 1) * (uint32_t)g.ldb + g.wb);
    // this lane's loads: 4 of each operand, row 8 (4 wave + i) + lane / 8
    const uint32_t ch = (uint32_t)((lane & 7) ^ (lane >> 3)) * 16u;
    uint32_t ka = ch, kb = ch;  // byte within the row
    while (kb >= g.wb) kb -= g.wb;
    uint32_t oa[4], ob[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int r = 8 * (4 * wave + i) + (lane >> 3);
        oa[i] = r < am ? (uint32_t)r * (uint32_t)g.lda : kOOB;
        ob[i] = r < bn ? (uint32_t)r * (uint32_t)g.ldb : kOOB;
    }
    auto to_lds = [](rsrc_t r, uint8_t* to, uint32_t off) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, off, 0, 0, 0);
    };
    auto issue = [&](int s, uint8_t* to) {
        const bool on = ka < g.wa;
#pragma unroll
        for (int i = 0; i < 4; i++) to_lds(rA, to + 1024 * (4 * wave + i), on && oa[i] != kOOB ? oa[i] + ka : kOOB);
#pragma unroll
        for (int i = 0; i < 4; i++)
            to_lds(rB, to + BM * kStepBytes + 1024 * (4 * wave + i), on && ob[i] != kOOB ? ob[i] + kb : kOOB);
        ka += kStepBytes;
        kb += kStepBytes;
        while (kb >= g.wb) kb -= g.wb;
        if constexpr (KIND == kFp4) {
            if (wave < 2) {  // 1 KB: 128 rows of 8 bytes
                const uint8_t* p = wave ? g.sb + ((size_t)s * tile_rows(g.N) + n0) * 8 : g.sa + ((size_t)s * tile_rows(g.M) + m0) * 8;
                to_lds(make_rsrc(p, 1024), to + (BM + BN) * kStepBytes + wave * BM * 8, 16u * lane);
            }
        }
    };
    f16v acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int j = 0; j < NI; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;
    const int lr = lane & 31, lh = lane >> 5;
    auto at = [&](int row, int c) { return (uint32_t)row * kStepBytes + (uint32_t)((c ^ (row & 7)) * 16); };
    auto multiply = [&](const uint8_t* from) {
        const uint8_t* fb = from + BM * kStepBytes;
        uint32_t sa[MI], sb[NI];
        if constexpr (KIND == kFp4) {
            const uint8_t* fs = from + (BM + BN) * kStepBytes;
#pragma unroll
            for (int i = 0; i < MI; i++) sa[i] = *reinterpret_cast<const uint32_t*>(fs + (64 * wm + 32 * i + lr) * 8 + 4 * lh);
#pragma unroll
            for (int j = 0; j < NI; j++)
                sb[j] = *reinterpret_cast<const uint32_t*>(fs + (BM + 64 * wn + 32 * j + lr) * 8 + 4 * lh);
        }
#pragma unroll
        for (int ks = 0; ks < 4; ks++) {
            u4w a[MI], b[NI];
#pragma unroll
            for (int i = 0; i < MI; i++) a[i] = *reinterpret_cast<const u4w*>(from + at(64 * wm + 32 * i + lr, 2 * ks + lh));
#pragma unroll
            for (int j = 0; j < NI; j++) b[j] = *reinterpret_cast<const u4w*>(fb + at(64 * wn + 32 * j + lr, 2 * ks + lh));
#pragma unroll
            for (int i = 0; i < MI; i++)
#pragma unroll
                for (int j = 0; j < NI; j++) {
                    if constexpr (KIND == kFp4) {
                        if (ks == 0) acc[i][j] = mma4<0>(a[i], b[j], acc[i][j], sa[i], sb[j]);
                        if (ks == 1) acc[i][j] = mma4<1>(a[i], b[j], acc[i][j], sa[i], sb[j]);
                        if (ks == 2) acc[i][j] = mma4<2>(a[i], b[j], acc[i][j], sa[i], sb[j]);
                        if (ks == 3) acc[i][j] = mma4<3>(a[i], b[j], acc[i][j], sa[i], sb[j]);
                    } else {
                        acc[i][j] = mma<KIND>(a[i], b[j], acc[i][j]);
                    }
                }
        }
    };
    issue(0, lds);
    for (int s = 0; s < g.steps; s++) {
        ring_barrier<0>();  // step s is there, and every wave is done with step s - 1
        if (s + 1 < g.steps) issue(s + 1, lds + ((s + 1) & 1) * STEP);
        multiply(lds + (s & 1) * STEP);
    }
    // acc[i][j][r]: row 8 (r / 4) + 4 lh + r % 4, column lr
#pragma unroll
    for (int j = 0; j < NI; j++) {
        const int n = n0 + 64 * wn + 32 * j + lr;
        if (n >= g.N) continue;
        const int e = g.row_exp ? g.row_exp[n] : 0;
#pragma unroll
        for (int i = 0; i < MI; i++)
#pragma unroll
            for (int r = 0; r < 16; r++) {
                const int m = m0 + 64 * wm + 32 * i + 8 * (r / 4) + 4 * lh + r % 4;
                if (m >= g.M) continue;
                float v = ldexpf(acc[i][j][r], e);
                const size_t es = Act<DT>::size;
                if constexpr (DT == kActF32) {
                    if (g.base) v += *reinterpret_cast<const float*>(g.base + (size_t)m * g.ldbase + n * es);
                    *reinterpret_cast<float*>(g.y + (size_t)m * g.ldy + n * es) = v;
                } else if constexpr (DT == kActBf16) {
                    if (g.base) v += (float)*reinterpret_cast<const __bf16*>(g.base + (size_t)m * g.ldbase + n * es);
                    *reinterpret_cast<__bf16*>(g.y + (size_t)m * g.ldy + n * es) = (__bf16)v;
                } else {
                    if (g.base) v += (float)*reinterpret_cast<const _Float16*>(g.base + (size_t)m * g.ldbase + n * es);
                    *reinterpret_cast<_Float16*>(g.y + (size_t)m * g.ldy + n * es) = (_Float16)v;
                }
            }
    }
}

template <int KIND>
hipError_t mm(int dtype, MmArgs& g, hipStream_t s) {
    g.nt = (g.N + 127) / 128;
    const dim3 grid((unsigned)((g.M + 127) / 128) * g.nt);
    if (dtype == kActF32) hipLaunchKernelGGL((k_fp4_mm<KIND, kActF32>), grid, dim3(256), 0, s, g);
    else if (dtype == kActBf16) hipLaunchKernelGGL((k_fp4_mm<KIND, kActBf16>), grid, dim3(256), 0, s, g);
    else hipLaunchKernelGGL((k_fp4_mm<KIND, kActF16>), grid, dim3(256), 0, s, g);
    return hipGetLastError();
}

// A's operand of a 16-bit product over K: the activations themselves, or their
// parts in the workspace.
hipError_t activations(int dtype, int P, const void* x, size_t ldx, int T, int K, char* parts, MmArgs& g, hipStream_t s) {
    const size_t es = dtype == kActF32 ? 4 : 2, pieces = (size_t)T * (K / 8);
    g.wa = (uint32_t)P * K * 2u;
    if (P == 1) {
        g.a = static_cast<const char*>(x);
        g.lda = ldx * es;
        return hipSuccess;
    }
    const dim3 grid((unsigned)((pieces + 255) / 256));
    if (dtype == kActF32)
        hipLaunchKernelGGL(k_fp4_parts<kActF32>, grid, dim3(256), 0, s, static_cast<const char*>(x), ldx * es, pieces, K / 8,
                           reinterpret_cast<u4w*>(parts));
    else
        hipLaunchKernelGGL(k_fp4_parts<kActF16>, grid, dim3(256), 0, s, static_cast<const char*>(x), ldx * es, pieces, K / 8,
                           reinterpret_cast<u4w*>(parts));
    g.a = parts;
    g.lda = g.wa;
    return hipGetLastError();
}

}  // namespace

size_t fp4_ws_bytes(int K, int N, int fmt, int dtype, int T, bool backward) {
    const int sum = backward ? N : K, P = act_parts(dtype, act_kind(fmt, dtype, backward));
    const size_t kept = align256((size_t)K * N * 2) + (P > 1 ? align256((size_t)T * P * sum * 2) : 0);
    if (backward || fmt != kFmtMxfp4) return kept;
    const size_t steps = (K + 255) / 256;
    const size_t rounded = align256((size_t)T * K / 2) + align256((size_t)T * K / 32) + steps * 8 * (tile_rows(T) + tile_rows(N));
    return kept > rounded ? kept : rounded;
}

hipError_t launch_fp4_apply(int K, int N, int fmt, int dtype, const void* x, size_t ldx, int T, const Fp4Matrix& w,
                            bool round_x, const void* base, size_t ldbase, void* y, size_t ldy, void* ws,
                            hipStream_t s) {
    const size_t es = dtype == kActF32 ? 4 : 2;
    if (T <= kGemvMaxT) return launch_fp4_gemv(K, N, fmt, dtype, x, ldx, T, w, round_x, base, ldbase, y, ldy, s);
    char* p = static_cast<char*>(ws);
    MmArgs g = {};
    g.M = T;
    g.N = N;
    g.row_exp = w.row_exp;
    g.base = static_cast<const char*>(base);
    g.y = static_cast<char*>(y);
    g.ldbase = ldbase * es;
    g.ldy = ldy * es;
    hipError_t r;
    if (round_x) {
        const int steps = (K + 255) / 256;
        uint8_t* codes = reinterpret_cast<uint8_t*>(p);
        uint8_t* scales = codes + align256((size_t)T * K / 2);
        uint8_t* sa = scales + align256((size_t)T * K / 32);
        uint8_t* sb = sa + steps * 8 * tile_rows(T);
        r = launch_fp4_quant(dtype, kFmtMxfp4, kScaleFloor, x, ldx, T, K, nullptr, codes, scales, nullptr, 0, s);
        if (r != hipSuccess) return r;
        if (T <= kFewMaxT) return launch_fp4_few(K, N, fmt, dtype, codes, K / 2, scales, T, w, base, ldbase, y, ldy, s);
        hipLaunchKernelGGL(k_fp4_scale_panel, dim3((T + 255) / 256, steps), dim3(256), 0, s, scales, T, K / 32, sa);
        if ((r = hipGetLastError()) != hipSuccess) return r;
        hipLaunchKernelGGL(k_fp4_scale_panel, dim3((N + 255) / 256, steps), dim3(256), 0, s, w.scales, N, K / 32, sb);
        if ((r = hipGetLastError()) != hipSuccess) return r;
        g.a = reinterpret_cast<const char*>(codes);
        g.b = reinterpret_cast<const char*>(w.codes);
        g.lda = g.ldb = g.wa = g.wb = (uint32_t)K / 2;
        g.sa = sa;
        g.sb = sb;
        g.steps = steps;
        return mm<kFp4>(dtype, g, s);
    }
    const int kind = act_kind(fmt, dtype, false), P = act_parts(dtype, kind);
    if ((r = activations(dtype, P, x, ldx, T, K, p + align256((size_t)K * N * 2), g, s)) != hipSuccess) return r;
    if (T <= kFewMaxT) return launch_fp4_few(K, N, fmt, dtype, g.a, g.lda, nullptr, T, w, base, ldbase, y, ldy, s);
    const size_t pieces = (size_t)N * (K / 8);
    const dim3 grid((unsigned)((pieces + 255) / 256));
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(w.codes);
    u4w* wide = reinterpret_cast<u4w*>(p);
    if (kind == kF16)
        hipLaunchKernelGGL((k_fp4_widen<kFmtNvfp4, kF16>), grid, dim3(256), 0, s, codes, w.scales, pieces, wide);
    else if (fmt == kFmtNvfp4)
        hipLaunchKernelGGL((k_fp4_widen<kFmtNvfp4, kBf16>), grid, dim3(256), 0, s, codes, w.scales, pieces, wide);
    else
        hipLaunchKernelGGL((k_fp4_widen<kFmtMxfp4, kBf16>), grid, dim3(256), 0, s, codes, w.scales, pieces, wide);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    g.b = p;
    g.ldb = g.wb = (uint32_t)K * 2;
    g.steps = (int)((g.wa + kStepBytes - 1) / kStepBytes);
    return kind == kF16 ? mm<kF16>(dtype, g, s) : mm<kBf16>(dtype, g, s);
}

hipError_t launch_fp4_backward(int K, int N, int fmt, int dtype, const void* dy, size_t lddy, int T,
                               const Fp4Matrix& w, const void* dx_base, size_t lddxb, void* dx, size_t lddx, void* ws,
                               hipStream_t s) {
    const size_t es = dtype == kActF32 ? 4 : 2;
    char* p = static_cast<char*>(ws);
    MmArgs g = {};
    g.M = T;
    g.N = K;
    g.base = static_cast<const char*>(dx_base);
    g.y = static_cast<char*>(dx);
    g.ldbase = lddxb * es;
    g.ldy = lddx * es;
    const dim3 grid((N + 63) / 64, (K + 63) / 64);
    if (fmt == kFmtNvfp4)
        hipLaunchKernelGGL(k_fp4_widen_t<kFmtNvfp4>, grid, dim3(256), 0, s, w, K, N, reinterpret_cast<uint16_t*>(p));
    else
        hipLaunchKernelGGL(k_fp4_widen_t<kFmtMxfp4>, grid, dim3(256), 0, s, w, K, N, reinterpret_cast<uint16_t*>(p));
    hipError_t r = hipGetLastError();
    if (r != hipSuccess) return r;
    const int P = act_parts(dtype, kBf16);
    if ((r = activations(dtype, P, dy, lddy, T, N, p + align256((size_t)K * N * 2), g, s)) != hipSuccess) return r;
    g.b = p;
    g.ldb = g.wb = (uint32_t)N * 2;
    g.steps = (int)((g.wa + kStepBytes - 1) / kStepBytes);
    return mm<kBf16>(dtype, g, s);
}

}  // namespace moe

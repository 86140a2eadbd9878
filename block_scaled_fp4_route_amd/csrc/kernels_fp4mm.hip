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
//
// Large products are bound by the matrix units: 8192 x 8192 x 2560 in bf16 takes
// 308-322 us, about 15 of them the join and 16 W (the product alone about 285, 1.2
// PFLOP/s; 344-349 under the profiler). As codes the product takes 116-121 us under
// the profiler (2.9 PFLOP/s), 29% of the matrix rate: steps of 256 codes take 2 us where the
// products alone would take 0.85, and a tile has ten of them between its ring's
// filling and its way out; neither bank conflicts (none) nor a longer ring
// changed it. Products of few tiles are bound by their steps' latency: 311 tokens of
// 640 x 2560 fp32 14 us for 30 steps.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_codes.h"
#include "moe_device.h"
#include "moe_internal.h"
#include "moe_rows.h"
#include "moe_serve.h"

namespace moe {
namespace {

typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int kBf16 = 0, kF16 = 1, kFp4 = 2;  // operands of the product

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

// W as 16-bit values [N][K] (row exponents left out), 256 pieces of 8 a workgroup.
template <int FMT, int KIND>
__device__ __forceinline__ void widen(const Fp4Matrix& w, int K, int N, uint32_t b, u4w* __restrict__ out) {
    const size_t i = (size_t)b * 256 + threadIdx.x;
    if (i >= (size_t)N * (K / 8)) return;
    float v[8];
    decode8(reinterpret_cast<const uint32_t*>(w.codes)[i], scale_to_f32<FMT>(w.scales[i / (Fmt<FMT>::G / 8)]), v);
    out[i] = KIND == kF16 ? pack8<kActF16>(v).w[0] : pack8<kActBf16>(v).w[0];
}

// W^T as bf16 [K][N], row exponents included. A workgroup turns 64 rows x 64
// columns in LDS.
template <int FMT>
__device__ __forceinline__ void widen_t(const Fp4Matrix& w, int K, int N, uint32_t b, uint16_t* __restrict__ out) {
    __shared__ uint16_t t[64][72];  // [k][n]; 144-byte rows
    const int nt = (N + 63) / 64, n0 = (int)(b % nt) * 64, k0 = (int)(b / nt) * 64, tid = threadIdx.x;
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
struct Acts {
    const char* x;
    size_t ldx;  // bytes
    int T, K;
    u4w* out;
};
template <int DT>
__device__ __forceinline__ void parts(const Acts& x, uint32_t b, uint32_t groups) {
    constexpr int P = DT == kActF32 ? 3 : 2;
    const uint32_t k8 = (uint32_t)x.K / 8;
    const size_t pieces = (size_t)x.T * k8;
    for (size_t i = (size_t)b * 256 + threadIdx.x; i < pieces; i += (size_t)groups * 256) {
        const size_t t = i / k8, c = i - t * k8;
        float v[8];
        unpack8<DT>(load8<DT>(x.x + t * x.ldx, 8 * c), v);
#pragma unroll
        for (int p = 0; p < P; p++) {
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                h[j] = bf16_cut(v[j]);
                v[j] = fabsf(v[j]) < INFINITY ? v[j] - __uint_as_float(h[j] << 16) : 0.0f;
            }
            x.out[(t * P + p) * k8 + c] = u4w{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
        }
    }
}

// Both operands in one launch (the second would cost 3 us): the first nw
// workgroups take W, the others the activations, where those need parts (DT; -1:
// not). TURN: W^T.
constexpr int kNoParts = -1;
template <int FMT, int KIND, bool TURN, int DT>
__global__ __launch_bounds__(256) void k_fp4_operands(Fp4Matrix w, int K, int N, uint32_t nw, char* out, Acts x) {
    if (blockIdx.x < nw) {
        if constexpr (TURN) widen_t<FMT>(w, K, N, blockIdx.x, reinterpret_cast<uint16_t*>(out));
        else widen<FMT, KIND>(w, K, N, blockIdx.x, reinterpret_cast<u4w*>(out));
    } else if constexpr (DT != kNoParts) {
        parts<DT>(x, blockIdx.x - nw, gridDim.x - nw);
    }
}
template <int DT>
__global__ __launch_bounds__(256) void k_fp4_parts(Acts x) {
    parts<DT>(x, blockIdx.x, gridDim.x);
}

// Scale bytes for the scaled product: [K / 256 steps][rows up to a whole
// tile][8], within a step's eight blocks the even ones first (lanes 0-31 of a
// wave hold the even blocks of a step, lanes 32-63 the odd ones: a lane's four
// bytes are one word). Blocks behind the row's end are 0.
__host__ __device__ constexpr size_t tile_rows(size_t rows) { return (rows + 255) / 256 * 256; }
__device__ __forceinline__ int scale_place(int b) { return (b & 1) * 4 + (b >> 1 & 3); }
struct Panel {
    const uint8_t* scales;
    int rows;
    uint8_t* out;
};
// The first `split` workgroups along x make a's panel, the others b's.
__global__ __launch_bounds__(256) void k_fp4_scale_panels(Panel a, Panel b, int split, int nb) {
    const bool first = (int)blockIdx.x < split;
    const uint8_t* __restrict__ scales = first ? a.scales : b.scales;
    uint8_t* __restrict__ out = first ? a.out : b.out;
    const int rows = first ? a.rows : b.rows;
    const int r = ((int)blockIdx.x - (first ? 0 : split)) * 256 + threadIdx.x, st = blockIdx.y;
    if (r >= rows) return;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const int k = 8 * st + j;
        if (k < nb) w[scale_place(j) / 4] |= (uint32_t)scales[(size_t)r * nb + k] << (8 * (scale_place(j) % 4));
    }
    *reinterpret_cast<uint2*>(out + (st * tile_rows(rows) + r) * 8) = make_uint2(w[0], w[1]);
}

// ---------------------------------------------------------------------------
// C = A B^T, both row-major along the sum. A step is 128 bytes of every row of
// the tile (64 16-bit values or 256 codes), loaded from memory straight into a
// ring of LDS buffers. A row's eight 16-byte chunks sit in LDS at chunk ^ (row /
// 2 & 7), so that the reads of 16 neighbouring rows' same chunk hit all banks
// once; the loads pick their chunk accordingly.
//
// Tiles: 256 x 256 by eight waves of 128 x 64 where they fill the chip. A
// compute unit takes 64 bytes a cycle from memory and 128 from LDS: a step's
// loads are half, its reads three quarters of its 2048 cycles of matrix
// instructions (256 x 128 by four waves, two workgroups a compute unit, steps of
// 64 bytes: loads three quarters; 415 us against 418 where the larger tiles
// leave a quarter of the chip idle in the last round, 127 against 112 where they
// do not). 128 x 128 and 64 x 64 where there are too few of those.
struct MmArgs {
    const char *a, *b;
    size_t lda, ldb;        // bytes between rows
    uint32_t wa, wb;        // bytes of a row (A's parts together; B starts again at its end)
    int M, N, wide;         // wide: a row's bytes in the sum, all parts
    const uint8_t *sa, *sb; // kFp4: scale panels [K / 256][rows up to a whole tile][8]
    const int8_t* row_exp;  // of B's rows, or null
    const char* base;
    char* y;
    size_t ldbase, ldy;     // bytes
    int mt, nt;             // tiles
    int full, split;        // the first `full` are whole; each other one has `split` workgroups, a part of the sum each
    float* part;            // their sums [tile - full][split][BM][BN]
};

template <int N>
__device__ __forceinline__ void ring_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16 or 4 bytes a lane from memory straight into LDS, the lanes' side by side.
__device__ __forceinline__ void to_lds16(rsrc_t r, uint8_t* to, uint32_t off, uint32_t step) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, off, step, 0, 0);
}
__device__ __forceinline__ void to_lds4(rsrc_t r, uint8_t* to, uint32_t off, uint32_t step) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 4, off, step, 0, 0);
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

// The place of tile number seq.
__device__ __forceinline__ void tile_at(int seq, int mt, int nt, int& m, int& n) {
    const int per = 4 * nt, grp = seq / per, gm = min(4, mt - 4 * grp), in = seq % per;
    m = 4 * grp + in % gm;
    n = in / gm;
}

// BM x BN by waves of 32 MI x 32 NI, a ring of R steps.
template <int KIND, int DT, int BM, int BN, int MI, int NI, int R>
__global__ __launch_bounds__(64 * (BM / (32 * MI)) * (BN / (32 * NI))) void k_fp4_mm(MmArgs g) {
    constexpr int WN = BN / (32 * NI), WAVES = BM / (32 * MI) * WN;
    constexpr int SB = 128, CH = SB / 16, RP = 64 / CH;                         // bytes and chunks of a row in a step; rows of a load
    constexpr int SC = KIND == kFp4 ? (BM + BN) * 8 : 0;                        // scale bytes of a step
    constexpr int LA = BM / RP / WAVES, LB = BN / RP / WAVES, LS = SC / 256 / WAVES, LOADS = LA + LB + LS;  // loads of a wave and step
    constexpr int STEP = (BM + BN) * SB + SC;
    constexpr int OUT = 32 * (32 * NI * 4 + 16);                                // a wave's 32 rows on their way out, fp32
    constexpr int LDS = R * STEP > WAVES * OUT ? R * STEP : WAVES * OUT;
    static_assert(LA * RP * WAVES == BM && LB * RP * WAVES == BN && LS * 256 * WAVES == SC && LOADS * (R - 1) < 64, "tile");
    __shared__ __attribute__((aligned(16))) uint8_t lds[LDS];
    const int steps = (g.wide + SB - 1) / SB;
    const int lane = threadIdx.x & 63, wave = wave_id(), wm = wave / WN, wn = wave % WN;
    // workgroups go to the eight XCDs in turn: each takes a run of the tiles, which
    // go down four tiles of M before the next of N, so that the workgroups of an
    // XCD share rows of both operands in its L2
    int m0, n0, s0 = 0, s1 = steps, piece = -1;
    {
        const int b = blockIdx.x, x = b % 8, q = g.full / 8, r = g.full % 8;
        int seq = x * q + min(x, r) + b / 8;
        if (b >= g.full) {
            piece = b - g.full;
            seq = g.full + piece / g.split;
            s0 = (int)((int64_t)(piece % g.split) * steps / g.split);
            s1 = (int)((int64_t)(piece % g.split + 1) * steps / g.split);
        }
        tile_at(seq, g.mt, g.nt, m0, n0);
        m0 *= BM;
        n0 *= BN;
    }
    const int am = min(BM, g.M - m0), bn = min(BN, g.N - n0);
    const rsrc_t rA = make_rsrc(g.a + (size_t)m0 * g.lda, (uint32_t)(am - 1) * (uint32_t)g.lda + g.wa);
    const rsrc_t rB = make_rsrc(g.b + (size_t)n0 * g.ldb, (uint32_t)(bn - 1) * (uint32_t)g.ldb + g.wb);
    // this lane's loads: row RP (L wave + i) + lane / CH, chunk lane % CH ^ swizzle;
    // with eight chunks, every second load's is another by 4
    const uint32_t ch = (uint32_t)((lane % CH) ^ (lane >> 4)) * 16u;
    uint32_t oa[LA], ob[LB];
#pragma unroll
    for (int i = 0; i < LA; i++) {
        const int r = RP * (LA * wave + i) + lane / CH;
        oa[i] = r < am ? (uint32_t)r * (uint32_t)g.lda + ((LA * wave + i) & 1 ? ch ^ 64u : ch) : kOOB;
    }
#pragma unroll
    for (int i = 0; i < LB; i++) {
        const int r = RP * (LB * wave + i) + lane / CH;
        ob[i] = r < bn ? (uint32_t)r * (uint32_t)g.ldb + ((LB * wave + i) & 1 ? ch ^ 64u : ch) : kOOB;
    }
    uint32_t kb = (uint32_t)s0 * SB % g.wb;  // B's byte of the next step to be loaded
    // Every step issues the same loads; those behind the last one read nothing.
    // The step goes into the scalar offset, so that a load costs no arithmetic,
    // unless a row of A ends within the step, or one of B.
    auto issue = [&](int s, uint8_t* to) {
        const uint32_t ka = (uint32_t)s * SB;
        if constexpr (KIND == kFp4) {  // both rows are as long (and with the second path its operands do not fit the registers)
#pragma unroll
            for (int i = 0; i < LA; i++) {
                const uint32_t c = (LA * wave + i) & 1 ? ch ^ 64u : ch;
                to_lds16(rA, to + 1024 * (LA * wave + i), ka + c < g.wa && oa[i] != kOOB ? oa[i] + ka : kOOB, 0);
            }
#pragma unroll
            for (int i = 0; i < LB; i++) {
                const uint32_t c = (LB * wave + i) & 1 ? ch ^ 64u : ch;
                to_lds16(rB, to + BM * SB + 1024 * (LB * wave + i), ka + c < g.wa && ob[i] != kOOB ? ob[i] + ka : kOOB, 0);
            }
        } else if (ka + SB <= g.wa && kb + SB <= g.wb) {
#pragma unroll
            for (int i = 0; i < LA; i++) to_lds16(rA, to + 1024 * (LA * wave + i), oa[i], ka);
#pragma unroll
            for (int i = 0; i < LB; i++) to_lds16(rB, to + BM * SB + 1024 * (LB * wave + i), ob[i], kb);
        } else {
            int l = lane;
            asm volatile("" : "+v"(l));  // nothing of this rare path is kept in registers over the loop
            auto off = [&](int q, int rows, uint32_t ld, uint32_t at, uint32_t end) {
                const int r = RP * q + l / CH;
                const uint32_t c = (uint32_t)((l % CH) ^ (l >> 4) ^ (q & 1 ? 4 : 0)) * 16u;
                return r < rows && ka + c < g.wa ? (uint32_t)r * ld + (at + c) % end : kOOB;
            };
#pragma unroll
            for (int i = 0; i < LA; i++) to_lds16(rA, to + 1024 * (LA * wave + i), off(LA * wave + i, am, (uint32_t)g.lda, ka, g.wa), 0);
#pragma unroll
            for (int i = 0; i < LB; i++) to_lds16(rB, to + BM * SB + 1024 * (LB * wave + i), off(LB * wave + i, bn, (uint32_t)g.ldb, kb, g.wb), 0);
        }
        kb += SB;
        while (kb >= g.wb) kb -= g.wb;
        if constexpr (KIND == kFp4) {  // rows of 8 bytes: A's, then B's
            const size_t ss = min(s, steps - 1);
#pragma unroll
            for (int i = 0; i < LS; i++) {
                const int q = LS * wave + i;  // 256 bytes, 32 rows, each
                const bool ofa = q < BM / 32;
                const uint8_t* p = ofa ? g.sa + (ss * tile_rows(g.M) + m0) * 8 : g.sb + (ss * tile_rows(g.N) + n0) * 8;
                to_lds4(make_rsrc(p, (ofa ? BM : BN) * 8), to + (BM + BN) * SB + 256 * q, 4u * lane, 256u * (ofa ? q : q - BM / 32));
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
    const int lr = lane & 31, lh = lane >> 5, am0 = 32 * MI * wm, bn0 = 32 * NI * wn;
    auto at = [&](int row, int c) { return (uint32_t)row * SB + (uint32_t)((c ^ (row >> 1 & 7)) * 16); };
    struct Frags {
        u4w a[MI], b[NI];
    };
    struct Scales {
        uint32_t a[MI], b[NI];
    };
    auto read = [&](const uint8_t* from, int ks, Frags& f) {
#pragma unroll
        for (int i = 0; i < MI; i++) f.a[i] = *reinterpret_cast<const u4w*>(from + at(am0 + 32 * i + lr, 2 * ks + lh));
#pragma unroll
        for (int j = 0; j < NI; j++) f.b[j] = *reinterpret_cast<const u4w*>(from + BM * SB + at(bn0 + 32 * j + lr, 2 * ks + lh));
    };
    auto read_scales = [&](const uint8_t* from, Scales& q) {
        const uint8_t* fs = from + (BM + BN) * SB + 4 * lh;
#pragma unroll
        for (int i = 0; i < MI; i++) q.a[i] = *reinterpret_cast<const uint32_t*>(fs + (am0 + 32 * i + lr) * 8);
#pragma unroll
        for (int j = 0; j < NI; j++) q.b[j] = *reinterpret_cast<const uint32_t*>(fs + (BM + bn0 + 32 * j + lr) * 8);
    };
    // B first: rows of the result are B's, a lane's column is a row of A
    auto rows = [&](auto KS, int i0, int i1, const Frags& f, const Scales& q) {
        constexpr int ks = decltype(KS)::value;
#pragma unroll
        for (int i = i0; i < i1; i++)
#pragma unroll
            for (int j = 0; j < NI; j++) {
                if constexpr (KIND == kFp4) acc[i][j] = mma4<ks>(f.b[j], f.a[i], acc[i][j], q.b[j], q.a[i]);
                else acc[i][j] = mma<KIND>(f.b[j], f.a[i], acc[i][j]);
            }
    };
    auto multiply = [&](auto KS, const Frags& f, const Scales& q) {
        __builtin_amdgcn_sched_barrier(0);  // the next reads go out before the products
        rows(KS, 0, MI, f, q);
        __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int s = 0; s < R; s++) issue(s0 + s, lds + s * STEP);
    ring_barrier<(R - 1) * LOADS>();  // step 0 is there
    Frags f0, f1;
    Scales q0, q1;
    read(lds, 0, f0);
    if constexpr (KIND == kFp4) read_scales(lds, q0);
    int cur = 0;  // s % R
    // a step's four products, each with the fragments of the next on their
    // way. Before the last, the next step is there, every wave has read all of
    // this one, and its buffer takes step s + R.
    auto step = [&](int s, const Scales& q, Scales& next) {
        uint8_t* buf = lds + cur * STEP;
        cur = cur + 1 == R ? 0 : cur + 1;
        read(buf, 1, f1);
        multiply(std::integral_constant<int, 0>{}, f0, q);
        read(buf, 2, f0);
        multiply(std::integral_constant<int, 1>{}, f1, q);
        read(buf, 3, f1);
        multiply(std::integral_constant<int, 2>{}, f0, q);
        ring_barrier<(R - 2) * LOADS>();
        if constexpr (KIND == kFp4) {  // (in two parts its operands do not fit the registers)
            issue(s + R, buf);
            read(lds + cur * STEP, 0, f0);
            read_scales(lds + cur * STEP, next);
            multiply(std::integral_constant<int, 3>{}, f1, q);
            return;
        }
        read(lds + cur * STEP, 0, f0);
        __builtin_amdgcn_sched_barrier(0);
        rows(std::integral_constant<int, 3>{}, 0, MI / 2, f1, q);
        __builtin_amdgcn_sched_barrier(0);
        issue(s + R, buf);  // between products, so that these do not wait for it
        __builtin_amdgcn_sched_barrier(0);
        rows(std::integral_constant<int, 3>{}, MI / 2, MI, f1, q);
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int s = s0; s < s1; s += 2) {
        step(s, q0, q1);
        if (s + 1 < s1) step(s + 1, q1, q0);
    }
    ring_barrier<0>();  // no load still writes LDS, and every wave has read its last step
    // acc[i][j][r]: row m = lr of A's 32, column n = 8 (r / 4) + 4 lh + r % 4 of
    // B's 32. Through LDS, so that a row's 32 NI columns leave side by side.
    float* out = reinterpret_cast<float*>(lds + wave * OUT);
    constexpr int ROW = 32 * NI + 4, PIECES = 4 * NI, PER = 64 / PIECES;  // floats of a row, its pieces of 8, rows at a time
    const int pc = lane % PIECES, n = n0 + bn0 + 8 * pc;
    float e[8];
#pragma unroll
    for (int q = 0; q < 8; q++) e[q] = g.row_exp && n < g.N ? exp2i(g.row_exp[n + q]) : 1.0f;
#pragma unroll
    for (int i = 0; i < MI; i++) {
#pragma unroll
        for (int j = 0; j < NI; j++)
#pragma unroll
            for (int q = 0; q < 4; q++)
                *reinterpret_cast<f4v*>(out + lr * ROW + 32 * j + 8 * q + 4 * lh) =
                    f4v{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // a wave's own region: its reads come behind its writes
#pragma unroll
        for (int u = 0; u < 32 / PER; u++) {
            const int row = u * PER + lane / PIECES, m = m0 + am0 + 32 * i + row;
            const f4v lo = *reinterpret_cast<const f4v*>(out + row * ROW + 8 * pc), hi = *reinterpret_cast<const f4v*>(out + row * ROW + 8 * pc + 4);
            if (piece >= 0) {
                float* to = g.part + ((size_t)piece * BM + am0 + 32 * i + row) * BN + bn0 + 8 * pc;
                *reinterpret_cast<f4v*>(to) = lo;
                *reinterpret_cast<f4v*>(to + 4) = hi;
            } else if (m < g.M && n < g.N) {
                float v[8];
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    v[q] = lo[q] * e[q];
                    v[4 + q] = hi[q] * e[4 + q];
                }
                if (g.base) {
                    float o[8];
                    unpack8<DT>(load8<DT>(g.base + (size_t)m * g.ldbase, n), o);
#pragma unroll
                    for (int q = 0; q < 8; q++) v[q] += o[q];
                }
                store8<DT>(g.y + (size_t)m * g.ldy, n, pack8<DT>(v));
            }
        }
        asm volatile("" ::: "memory");
    }
}

// The split tiles' parts, added in order: a thread 8 columns of a row.
template <int DT, int B>
__global__ __launch_bounds__(256) void k_fp4_join(MmArgs g) {
    const int tile = blockIdx.x / (B * B / 8 / 256), at = blockIdx.x % (B * B / 8 / 256) * 256 + threadIdx.x, row = at / (B / 8), c = at % (B / 8) * 8;
    int m, n;
    tile_at(g.full + tile, g.mt, g.nt, m, n);
    m = m * B + row;
    n = n * B + c;
    if (m >= g.M || n >= g.N) return;
    const float* p = g.part + ((size_t)tile * g.split * B + row) * B + c;
    f4v lo = *reinterpret_cast<const f4v*>(p), hi = *reinterpret_cast<const f4v*>(p + 4);
    for (int i = 1; i < g.split; i++) {
        lo += *reinterpret_cast<const f4v*>(p + (size_t)i * B * B);
        hi += *reinterpret_cast<const f4v*>(p + (size_t)i * B * B + 4);
    }
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; q++) v[q] = (q < 4 ? lo[q % 4] : hi[q % 4]) * (g.row_exp ? exp2i(g.row_exp[n + q]) : 1.0f);
    if (g.base) {
        float o[8];
        unpack8<DT>(load8<DT>(g.base + (size_t)m * g.ldbase, n), o);
#pragma unroll
        for (int q = 0; q < 8; q++) v[q] += o[q];
    }
    store8<DT>(g.y + (size_t)m * g.ldy, n, pack8<DT>(v));
}

constexpr int kCus = 256;                       // workgroups of a round of the large tiles
constexpr int kLargeFrom = 192;                 // tiles of a size that is worth it
constexpr int kMiddleFrom = 48, kMiddleSteps = 64;  // tiles and steps from which 128 x 128 tiles have their sums split
constexpr int kSmallGroups = 512;               // workgroups of the smaller tiles, where the sum is split
constexpr int kMaxSplit = 8, kMaxSmallSplit = 16;
// Bytes of parts that a product may leave: one round of large tiles, or all the
// smaller ones. None falls as M grows.
size_t part_bytes(int M, int N) {
    auto tiles = [&](size_t b) { return ((size_t)M + b - 1) / b * ((N + b - 1) / b); };
    if (tiles(256) >= kLargeFrom) return (size_t)kCus * 256 * 256 * 4;
    if (tiles(128) >= kMiddleFrom) return (size_t)kSmallGroups * 128 * 128 * 4;
    const size_t small = tiles(64) * kMaxSmallSplit;
    return (small < kSmallGroups ? small : kSmallGroups) * 64 * 64 * 4;
}

template <int KIND, int DT>
hipError_t mm_tiles(MmArgs& g, hipStream_t s) {
    auto tiles = [&](int bm, int bn) {
        g.mt = (g.M + bm - 1) / bm;
        g.nt = (g.N + bn - 1) / bn;
        return g.full = g.mt * g.nt;
    };
    // A last round of few tiles costs as much as a full one: each takes several
    // workgroups, and their sums are joined by a launch of their own (8192 x 2560
    // of 8192: 320 tiles on 256 compute units, 415 us whole, 305 split). Not where
    // few steps are saved: the parts are written and read, and the launch costs 4 us.
    auto cut = [&](int rest, int split, int least) {
        const int steps = g.wide / 128;
        while (split > 1 && steps / split < 4) split--;
        if (rest && split > 1 && steps - steps / split >= least) {
            g.split = split;
            g.full -= rest;
            return rest;
        }
        return 0;
    };
    g.split = 1;
    int parts = 0;
    hipError_t r;
    if (tiles(256, 256) >= kLargeFrom) {
        const int rest = g.full % kCus;
        parts = cut(rest, rest ? (kCus / rest < kMaxSplit ? kCus / rest : kMaxSplit) : 1, 24);
        hipLaunchKernelGGL((k_fp4_mm<KIND, DT, 256, 256, 4, 2, 2>), dim3(g.full + parts * g.split), dim3(512), 0, s, g);
        if ((r = hipGetLastError()) != hipSuccess || !parts) return r;
        hipLaunchKernelGGL((k_fp4_join<DT, 256>), dim3(parts * (256 * 256 / 8 / 256)), dim3(256), 0, s, g);
    } else if (tiles(128, 128) >= kLargeFrom) {
        // whole from 192 tiles on. For fp32 activations, three times the steps, that
        // is too early: 192 tiles of a sum of 8192 take 285 us whole and 211 in two
        // parts each, of 2560 98 and 77, 220 tiles 292 and 227; in bf16 192 take 87 and
        // 92, 220 101 and 95, 256 91 and 102
        hipLaunchKernelGGL((k_fp4_mm<KIND, DT, 128, 128, 2, 2, 2>), dim3(g.full), dim3(256), 0, s, g);
    } else if (const int big = tiles(128, 128); big >= kMiddleFrom && g.wide >= 128 * kMiddleSteps) {
        // long sums: the operands are read half as often as by 64 x 64 tiles, which
        // is worth the larger parts (300 tokens of 8192 x 2560 back to the input,
        // fp32: 122 us in 64 x 64 tiles, 75 so; 1000 of 2560 x 2048 bf16, 40
        // steps: 30 and 34)
        const int split = kSmallGroups / big;
        parts = cut(big, split, 20);
        hipLaunchKernelGGL((k_fp4_mm<KIND, DT, 128, 128, 2, 2, 2>), dim3(g.full + parts * g.split), dim3(256), 0, s, g);
        if ((r = hipGetLastError()) != hipSuccess || !parts) return r;
        hipLaunchKernelGGL((k_fp4_join<DT, 128>), dim3(parts * (128 * 128 / 8 / 256)), dim3(256), 0, s, g);
    } else {
        const int all = tiles(64, 64), split = kSmallGroups / all;
        parts = cut(all, split < kMaxSmallSplit ? split : kMaxSmallSplit, 20);
        hipLaunchKernelGGL((k_fp4_mm<KIND, DT, 64, 64, 1, 1, 4>), dim3(g.full + parts * g.split), dim3(256), 0, s, g);
        if ((r = hipGetLastError()) != hipSuccess || !parts) return r;
        hipLaunchKernelGGL((k_fp4_join<DT, 64>), dim3(parts * (64 * 64 / 8 / 256)), dim3(256), 0, s, g);
    }
    return hipGetLastError();
}
template <int KIND>
hipError_t mm(int dtype, MmArgs& g, hipStream_t s) {
    if (dtype == kActF32) return mm_tiles<KIND, kActF32>(g, s);
    return dtype == kActBf16 ? mm_tiles<KIND, kActBf16>(g, s) : mm_tiles<KIND, kActF16>(g, s);
}

// A's operand of a 16-bit product over K: the activations themselves, or their
// parts in the workspace, which are still to be made (workgroups for them; 0: none).
uint32_t activations(int dtype, int P, const void* x, size_t ldx, int T, int K, char* at, MmArgs& g, Acts& acts) {
    const size_t es = dtype == kActF32 ? 4 : 2, groups = ((size_t)T * (K / 8) + 255) / 256;
    acts = {static_cast<const char*>(x), ldx * es, T, K, reinterpret_cast<u4w*>(at)};
    g.wa = (uint32_t)P * K * 2u;
    g.a = P == 1 ? acts.x : at;
    g.lda = P == 1 ? acts.ldx : g.wa;
    return P == 1 ? 0 : (uint32_t)(groups < (1u << 22) ? groups : 1u << 22);
}

// W (TURN: W^T) widened to `out`, and the activations' parts.
template <int FMT, int KIND, bool TURN>
hipError_t operands(const Fp4Matrix& w, int K, int N, char* out, int dtype, uint32_t na, const Acts& acts, hipStream_t s) {
    const uint32_t nw = TURN ? (uint32_t)((N + 63) / 64) * ((K + 63) / 64) : (uint32_t)(((size_t)N * (K / 8) + 255) / 256);
    const dim3 grid(nw + na), block(256);
    if (!na) hipLaunchKernelGGL((k_fp4_operands<FMT, KIND, TURN, kNoParts>), grid, block, 0, s, w, K, N, nw, out, acts);
    else if (dtype == kActF32) hipLaunchKernelGGL((k_fp4_operands<FMT, KIND, TURN, kActF32>), grid, block, 0, s, w, K, N, nw, out, acts);
    else if constexpr (KIND == kBf16 && (TURN || FMT == kFmtMxfp4))
        hipLaunchKernelGGL((k_fp4_operands<FMT, KIND, TURN, kActF16>), grid, block, 0, s, w, K, N, nw, out, acts);
    return hipGetLastError();
}

}  // namespace

// Behind the reserved bytes: nothing more for the vector kernel; the activations'
// parts, or codes and scales, for up to kFewMaxT tokens; split sums, the widened W
// and the parts, or codes, scales and their panels, for more tokens and backward.
size_t fp4_ws_bytes(int K, int N, int fmt, int dtype, int T, bool backward) {
    if (T <= kGemvMaxT && !backward) return kCounterBytes;
    const bool few = T <= kFewMaxT && !backward;
    const int sum = backward ? N : K, P = act_parts(dtype, act_kind(fmt, dtype, backward));
    const size_t sums = kCounterBytes + (few ? 0 : part_bytes(T, backward ? K : N));
    const size_t kept = sums + (few ? 0 : align256((size_t)K * N * 2)) + (P > 1 ? align256((size_t)T * P * sum * 2) : 0);
    if (backward || fmt != kFmtMxfp4) return kept;
    const size_t steps = (K + 255) / 256;
    const size_t rounded = sums + align256((size_t)T * K / 2) + align256((size_t)T * K / 32) + (few ? 0 : steps * 8 * (tile_rows(T) + tile_rows(N)));
    return kept > rounded ? kept : rounded;
}

hipError_t launch_fp4_apply(int K, int N, int fmt, int dtype, const void* x, size_t ldx, int T, const Fp4Matrix& w,
                            bool round_x, const void* base, size_t ldbase, void* y, size_t ldy, void* ws,
                            hipStream_t s) {
    const size_t es = dtype == kActF32 ? 4 : 2;
    if (T <= kGemvMaxT) return launch_fp4_gemv(K, N, fmt, dtype, x, ldx, T, w, round_x, base, ldbase, y, ldy, s);
    char* p = static_cast<char*>(ws) + kCounterBytes;
    MmArgs g = {};
    g.M = T;
    g.N = N;
    g.part = reinterpret_cast<float*>(p);
    if (T > kFewMaxT) p += part_bytes(T, N);
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
        const int split = (T + 255) / 256;
        hipLaunchKernelGGL(k_fp4_scale_panels, dim3(split + (N + 255) / 256, steps), dim3(256), 0, s, Panel{scales, T, sa},
                           Panel{w.scales, N, sb}, split, K / 32);
        if ((r = hipGetLastError()) != hipSuccess) return r;
        g.a = reinterpret_cast<const char*>(codes);
        g.b = reinterpret_cast<const char*>(w.codes);
        g.lda = g.ldb = g.wa = g.wb = (uint32_t)K / 2;
        g.sa = sa;
        g.sb = sb;
        g.wide = K / 2;
        return mm<kFp4>(dtype, g, s);
    }
    const int kind = act_kind(fmt, dtype, false), P = act_parts(dtype, kind);
    Acts acts;
    const uint32_t na = activations(dtype, P, x, ldx, T, K, T <= kFewMaxT ? p : p + align256((size_t)K * N * 2), g, acts);
    if (T <= kFewMaxT) {
        if (na) {
            if (dtype == kActF32) hipLaunchKernelGGL(k_fp4_parts<kActF32>, dim3(na), dim3(256), 0, s, acts);
            else hipLaunchKernelGGL(k_fp4_parts<kActF16>, dim3(na), dim3(256), 0, s, acts);
            if ((r = hipGetLastError()) != hipSuccess) return r;
        }
        return launch_fp4_few(K, N, fmt, dtype, g.a, g.lda, nullptr, T, w, base, ldbase, y, ldy, s);
    }
    if (kind == kF16) r = operands<kFmtNvfp4, kF16, false>(w, K, N, p, dtype, na, acts, s);
    else if (fmt == kFmtNvfp4) r = operands<kFmtNvfp4, kBf16, false>(w, K, N, p, dtype, na, acts, s);
    else r = operands<kFmtMxfp4, kBf16, false>(w, K, N, p, dtype, na, acts, s);
    if (r != hipSuccess) return r;
    g.b = p;
    g.ldb = g.wb = (uint32_t)K * 2;
    g.wide = (int)g.wa;
    return kind == kF16 ? mm<kF16>(dtype, g, s) : mm<kBf16>(dtype, g, s);
}

hipError_t launch_fp4_backward(int K, int N, int fmt, int dtype, const void* dy, size_t lddy, int T,
                               const Fp4Matrix& w, const void* dx_base, size_t lddxb, void* dx, size_t lddx, void* ws,
                               hipStream_t s) {
    const size_t es = dtype == kActF32 ? 4 : 2;
    char* p = static_cast<char*>(ws) + kCounterBytes;
    MmArgs g = {};
    g.M = T;
    g.N = K;
    g.part = reinterpret_cast<float*>(p);
    p += part_bytes(T, K);
    g.base = static_cast<const char*>(dx_base);
    g.y = static_cast<char*>(dx);
    g.ldbase = lddxb * es;
    g.ldy = lddx * es;
    Acts acts;
    const uint32_t na = activations(dtype, act_parts(dtype, kBf16), dy, lddy, T, N, p + align256((size_t)K * N * 2), g, acts);
    const hipError_t r = fmt == kFmtNvfp4 ? operands<kFmtNvfp4, kBf16, true>(w, K, N, p, dtype, na, acts, s)
                                          : operands<kFmtMxfp4, kBf16, true>(w, K, N, p, dtype, na, acts, s);
    if (r != hipSuccess) return r;
    g.b = p;
    g.ldb = g.wb = (uint32_t)N * 2;
    g.wide = (int)g.wa;
    return mm<kBf16>(dtype, g, s);
}

}  // namespace moe

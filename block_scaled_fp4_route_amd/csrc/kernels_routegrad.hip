// The gradient of the routing, for gfx950. With w the softmax over the chosen
// k logits and dw the gradient of the loss at w:
//   ds[t][j] = w[t][j] (dw[t][j] - sum_i w[t][i] dw[t][i])
//   G        = dlogits_in + ds scattered to the chosen experts (masked tokens: 0)
//   dx       = G Wr        [T][H], over E
//   dWr      = G^T x       [E][H], over T
// Two forms of the two products, chosen by their size (pair_form), the first
// also by the caller (accumulate's bit 8, MOE_FP32_PRODUCTS):
//   fp32  k_rg_logits writes G, k_rg_gemm runs both products as one launch on
//         v_mfma_f32_16x16x4_f32.
//   pair  operands as pairs of fp16 parts (see pair_exp): k_rg_prep writes G
//         and the parts of G's rows, x and Wr in the order in which the
//         products load them, k_rg_gt those of G's columns, and k_rg_pair
//         runs both products as one launch on v_mfma_f32_32x32x16_f16.
// Where a product's long axis was split, k_rg_reduce adds its parts in order.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_learn.h"

namespace moe {

namespace {

constexpr int kTM = 64, kTN = 64, kTK = 32;  // tile of the products in fp32 form
constexpr int kPairCols = 128;                 // columns of a tile in pair form
constexpr int kMaxPart = 1024;                 // rows of a part of a product's long axis

// Multiplications (T E H) from which the products run by pairs of fp16 parts.
// The parts cost a fixed 15 us or so (their panels written and read, two more
// launches). Whole calls, fp32 against pairs, E = 512, H = 2560: T = 64 15
// against 29 us, 311 31 against 35, 409 (the limit) 35 against 37, 700 45
// against 42, 1200 74 against 63, 2451 124 against 82, 8191 376 against 201;
// E = 384, H = 4096: T = 311 27 against 42, 450 39 against 44.
// And only above 64 experts: up to there one fp32 tile holds all of them, so
// that x passes through the product once, and making its parts costs more than
// they save. T x E x H, fp32 against pairs: 8191 x 8 x 4096 112 against 157 us,
// x 32 113 against 158, x 64 132 against 164; 8191 x 64 x 1024 54 against 57;
// 2048 x 64 x 8192 92 against 94; 32768 x 8 x 4096 322 against 538; 2^20 x 64
// x 256 1222 against 2021. Above, pairs are from 17% slower to 1.9 times as
// fast: 8191 x 66 x 4096 150 against 170, 2^20 x 96 x 512 2779 against 3259,
// 8191 x 128 x 4096 167 against 178, x 2560 134 against 119, x 1024 87 against
// 60, 8191 x 256 x 4096 306 against 205.
constexpr int64_t kPairFrom = (int64_t)1 << 29;
bool pair_form(int H, int E, int T) { return E > kTM && (int64_t)T * E * H >= kPairFrom; }

typedef _Float16 h2v __attribute__((ext_vector_type(2)));
typedef _Float16 h8v __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));  // a chunk: 8 consecutive k of one row or column, one part

struct RgPlan {
    int BM;               // 0: fp32 form; else the pair form with tiles of BM rows
    int Ep;               // columns of G in the workspace (E rounded up to kTK, zero-padded)
    int mt, nt;           // dx: row tiles; both: column tiles
    int et;               // dWr: row tiles
    int sx, sw;           // parts of the long axis of dx (over E) and dWr (over T)
    int kx, kw;           // its length in a part (multiples of kTK; pair form: powers of 2)
    size_t g, egr, egc, ex, ew, ga, gt, xb, wb, px, pw, total;
};

// fp32: the fp32 form at every size (its regions are a part of the other one's).
RgPlan rg_plan(int H, int E, int T, bool fp32 = false) {
    RgPlan p = {};
    p.Ep = (E + kTK - 1) / kTK * kTK;
    if (!fp32 && pair_form(H, E, T)) {
        p.nt = H / kPairCols;
        // 256-row tiles read less per product; 128-row ones where the larger
        // would leave compute units idle (E = 512, H = 2560: 240 larger tiles
        // 62 us against 52 for T = 2451, 360 larger ones 71 against 78 for T = 4096)
        const int64_t large = ((int64_t)(T + 255) / 256 + (E + 255) / 256) * p.nt;
        p.BM = large >= 320 ? 256 : 128;
    } else {
        p.nt = H / kTN;
    }
    const int tm = p.BM ? p.BM : kTM;
    p.mt = (T + tm - 1) / tm;
    p.et = (E + tm - 1) / tm;
    if (p.BM) {
        auto split = [](int64_t tiles, int64_t len, int& parts, int& per) {
            per = kMaxPart;
            while (per > 64 && tiles * ((len + per - 1) / per) < 64) per /= 2;
            parts = (int)((len + per - 1) / per);
        };
        split((int64_t)p.mt * p.nt, E, p.sx, p.kx);
        split((int64_t)p.et * p.nt, T, p.sw, p.kw);
    } else {
        // parts until one workgroup per compute unit has work, of two steps
        // at least, and none above kMaxPart
        auto split = [](int64_t tiles, int64_t len, int& parts, int& per) {
            parts = 1;
            per = kTK;
            if (tiles < 1 || len < 1) return;  // no tokens
            int64_t n = (256 + tiles - 1) / tiles;
            if ((len + kMaxPart - 1) / kMaxPart > n) n = (len + kMaxPart - 1) / kMaxPart;
            const int64_t most = (len + 2 * kTK - 1) / (2 * kTK);
            if (n > most) n = most;
            if (n < 1) n = 1;
            int64_t l = (len + n - 1) / n;
            l = (l + kTK - 1) / kTK * kTK;
            per = (int)l;
            parts = (int)((len + l - 1) / l);
        };
        split((int64_t)p.mt * p.nt, E, p.sx, p.kx);
        split((int64_t)p.et * p.nt, T, p.sw, p.kw);
    }
    size_t o = kCounterBytes;
    auto take = [&o](size_t bytes) {
        const size_t at = o;
        o += align256(bytes);
        return at;
    };
    // The regions grow with T, so that fewer tokens never need more (parts and
    // tiles do not: a sum in fewer parts, a larger tile). Tokens x parts of dx:
    // a sum is split only below 512 tiles x parts of 64 x 64, or 128 of 128 x
    // 128, in parts of 64 at least; parts of dWr: likewise, or 1024 tokens each.
    auto up = [](size_t a, size_t b) { return (a + b - 1) / b; };
    const size_t tall = up(T, 1024) * 1024, ke = up(E, 64), most = ((size_t)1 << 21) / H;
    const size_t px = ke > 1 ? (ke * T < most ? ke * T : most) : 0;
    size_t pw = up(256, ke * (H / 64));
    if ((1 << 14) / (up(E, 256) * H) > pw) pw = (1 << 14) / (up(E, 256) * H);
    if (up(T, 1024) > pw) pw = up(T, 1024);
    if (up(T, 64) < pw) pw = up(T, 64);
    p.g = take((size_t)T * p.Ep * 4);
    if (p.BM) {
        p.egr = take((size_t)T * 4);
        p.egc = take(pw * p.Ep * 4);
        p.ex = take(pw * H * 4);
        p.ew = take(ke * H * 4);
        p.ga = take(up(T, 256) * 256 * p.Ep * 4);
        p.gt = take(tall * up(E, 256) * 256 * 4);
        p.xb = take(tall * H * 4);
        p.wb = take(up(E, 1024) * 1024 * H * 4);
    }
    p.px = take(px * H * 4);
    p.pw = take(pw > 1 ? pw * E * H * 4 : 0);
    p.total = o;
    return p;
}

// Adds the routing's part to one token's row of G, lane i of which holds the
// columns col(0), col(1), ... (one wave; lanes below k hold the token's
// routing). In increasing j, so an expert named twice adds in that order. An
// index outside [0, E) makes the row NaN.
template <int NV, class COL>
__device__ __forceinline__ void add_routing(float (&v)[NV], COL col, int E, int k, int me, float mw, float md) {
    const int lane = threadIdx.x & 63;
    const float dot = wave_sum(lane < k ? mw * md : 0.0f);
    const float ds = mw * (md - dot);
    for (int j = 0; j < k; j++) {
        const int e = __builtin_amdgcn_readlane(me, j);
        const float d = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ds), j));
#pragma unroll
        for (int i = 0; i < NV; i++) v[i] += col(i) == e ? d : 0.0f;
    }
    if (__ballot(lane < k && (unsigned)me >= (unsigned)E))
#pragma unroll
        for (int i = 0; i < NV; i++) v[i] = __builtin_nanf("");
}

// ---------------------------------------------------------------------------
// fp32 form

// grid ceil(T / 4), 256 threads: one wave per token; lane owns columns
// lane + 64 i (i < NV). dout may be din: a wave loads its row before it writes
// it, and no other wave touches it.
template <int NV>
__global__ __launch_bounds__(256) void k_rg_logits(const float* din, const int32_t* __restrict__ idx,
                                                   const float* __restrict__ w, const float* __restrict__ dw,
                                                   const uint8_t* __restrict__ mask, int T, int E, int Ep, int k,
                                                   float* __restrict__ G, float* dout) {
    const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + wave_id();
    if (t >= T) return;
    const bool on = !mask || mask[t], live = dw && lane < k;
    float v[NV];
    const int me = live ? idx[(size_t)t * k + lane] : 0;
    const float mw = live ? w[(size_t)t * k + lane] : 0.0f, md = live ? dw[(size_t)t * k + lane] : 0.0f;
    auto col = [lane](int i) { return lane + 64 * i; };
#pragma unroll
    for (int i = 0; i < NV; i++) v[i] = din && col(i) < E ? din[(size_t)t * E + col(i)] : 0.0f;
    if (dw) add_routing<NV>(v, col, E, k, me, mw, md);
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int e = col(i);
        if (e >= E || !on) v[i] = 0.0f;
        if (e < Ep) G[(size_t)t * Ep + e] = v[i];
        if (dout && e < E) dout[(size_t)t * E + e] = v[i];
    }
}

struct RgArgs {
    const float* G;
    int Ep;
    const float* Wr;
    const float* x;
    const uint8_t* mask;
    int T, E, H;
    float *dx, *dWr;  // outputs, or the parts [s][rows][H]
    int acc_x, acc_w;
    int sx, sw, kx, kw, mt, nt, et, nx;  // nx: workgroups of dx
};

// One 64 x 64 tile of C[M][H] = A B over [k0, k1). A(m, k) is G[m][k] (dx: KMAJ
// false) or G[k][m] (dWr: KMAJ true); B rows are rows of Wr (dx) or x (dWr).
// Both operands go through LDS as [k][m] and [k][n], two steps of 32 k in turn.
// In every wave lane (i = lane % 16, q = lane / 16) reads 2 consecutive m (n) of
// row k + q at once: MFMA (a, b) then covers the rows 2 i + a and columns 2 i +
// b of the wave's 32 x 32 square. Small tiles: what runs in this form has few
// of them, and splitting the sums instead costs their parts' traffic. Bound by
// latency at few tokens (8 us at T = 1). 311 x 384 x 4096 26 us, 75 TFLOP/s,
// half of the fp32 matrix rate: its 704 tiles all run at once, in 10 to 12 steps
// each, so that their starts and ends count. Then by that rate: 2451 x 512 x
// 2560 (on request) 124 us a call, 104 TFLOP/s.
constexpr int kLdsRow = kTM + 4;
constexpr int kLdsStep = 2 * kTK * kLdsRow;

template <bool KMAJ>
__device__ __forceinline__ void rg_tile(const RgArgs& a, int tile, int part, float* lds) {
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
    const int M = KMAJ ? a.E : a.T;                 // rows of C
    const int klen = KMAJ ? a.T : a.E;              // length of the sum
    const int m0 = tile / a.nt * kTM, n0 = tile % a.nt * kTN;
    const int per = KMAJ ? a.kw : a.kx;
    const int k0 = part * per, k1 = max(k0, min(klen, k0 + per)), len = k1 - k0;
    const float* B = KMAJ ? a.x : a.Wr;
    const bool masked = KMAJ && a.mask;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32, li = lane & 15, lq = lane >> 4;
    f4v acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) acc[i][j] = f4v{0.f, 0.f, 0.f, 0.f};
    // Loads through buffer resources over this part's rows: what lies behind
    // them reads 0 and no load waits for a branch. (H is a multiple of 64, G's
    // rows are padded to whole steps.)
    const rsrc_t rB = make_rsrc(B + (size_t)k0 * a.H, (uint32_t)len * (uint32_t)a.H * 4u);
    const rsrc_t rA = KMAJ ? make_rsrc(a.G + (size_t)k0 * a.Ep, (uint32_t)len * (uint32_t)a.Ep * 4u)
                           : make_rsrc(a.G + (size_t)m0 * a.Ep, (uint32_t)min(kTM, M - m0) * (uint32_t)a.Ep * 4u);
    const rsrc_t rm = make_rsrc(masked ? a.mask + k0 : nullptr, masked ? (uint32_t)len : 0u);
    const int br = tid / 16, bc = tid % 16 * 4;  // B (and A by rows of k): rows br + 16 i, columns bc
    const int ar = tid / 8, ac = tid % 8 * 4;    // A by rows of m: rows ar + 32 i, columns ac
    const uint32_t oa = KMAJ ? (m0 + bc < a.Ep ? (uint32_t)(m0 + bc) * 4u : kOOB) : (uint32_t)(ar * a.Ep + ac) * 4u;
    f4v ra[2], rb[2];
    uint32_t keep[2];
    auto fetch = [&](int k) {  // k from the part's start
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t row = (uint32_t)(k + br + 16 * i);
            rb[i] = __builtin_bit_cast(f4v, __builtin_amdgcn_raw_buffer_load_b128(
                                                rB, row * (uint32_t)a.H * 4u + (uint32_t)(n0 + bc) * 4u, 0, 0));
            keep[i] = masked ? ld_b8(rm, row) : 1u;
            const uint32_t q = KMAJ ? row * (uint32_t)a.Ep * 4u + oa
                                    : oa + (uint32_t)(32 * i * a.Ep + k0 + k) * 4u;
            ra[i] = __builtin_bit_cast(f4v, __builtin_amdgcn_raw_buffer_load_b128(rA, q, 0, 0));
        }
    };
    auto put = [&](float* As) {
        float* Bs = As + kTK * kLdsRow;
#pragma unroll
        for (int i = 0; i < 2; i++) {
#pragma unroll
            for (int j = 0; j < 4; j++) rb[i][j] = keep[i] ? rb[i][j] : 0.0f;
            *reinterpret_cast<f4v*>(Bs + (br + 16 * i) * kLdsRow + bc) = rb[i];
            if (KMAJ) {
                *reinterpret_cast<f4v*>(As + (br + 16 * i) * kLdsRow + bc) = ra[i];
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) As[(ac + j) * kLdsRow + ar + 32 * i] = ra[i][j];
            }
        }
    };
    if (len > 0) {
        fetch(0);
        put(lds);
        if (kTK < len) fetch(kTK);
        int cur = 0;
        for (int k = 0; k < len; k += kTK, cur ^= 1) {
            __syncthreads();  // step k is in LDS, and everybody is done with the step before
            const float *As = lds + cur * kLdsStep, *Bs = As + kTK * kLdsRow;
            if (k + kTK < len) put(lds + (cur ^ 1) * kLdsStep);
            if (k + 2 * kTK < len) fetch(k + 2 * kTK);
#pragma unroll
            for (int kk = 0; kk < kTK; kk += 4) {
                const f2v fa = *reinterpret_cast<const f2v*>(As + (kk + lq) * kLdsRow + wm + 2 * li);
                const f2v fb = *reinterpret_cast<const f2v*>(Bs + (kk + lq) * kLdsRow + wn + 2 * li);
#pragma unroll
                for (int i = 0; i < 2; i++)
#pragma unroll
                    for (int j = 0; j < 2; j++)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[i], fb[j], acc[i][j], 0, 0, 0);
            }
        }
    }
    const int parts = KMAJ ? a.sw : a.sx;
    float* C = (KMAJ ? a.dWr : a.dx) + (parts > 1 ? (size_t)part * M * a.H : 0);
    const bool add = parts == 1 && (KMAJ ? a.acc_w : a.acc_x);
    const int n = n0 + wn + 2 * li;
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int m = m0 + wm + 2 * (lq * 4 + q) + i;
            if (m < M) {
                f2v* c = reinterpret_cast<f2v*>(C + (size_t)m * a.H + n);
                f2v v = {acc[i][0][q], acc[i][1][q]};
                if (add) {
                    const f2v o = *c;
                    v.x += o.x;
                    v.y += o.y;
                }
                *c = v;
            }
        }
}

__global__ __launch_bounds__(256) void k_rg_gemm(RgArgs a) {
    __shared__ __align__(16) float lds[2 * kLdsStep];
    const int b = blockIdx.x;
    if (b < a.nx)
        rg_tile<false>(a, b % (a.mt * a.nt), b / (a.mt * a.nt), lds);
    else
        rg_tile<true>(a, (b - a.nx) % (a.et * a.nt), (b - a.nx) / (a.et * a.nt), lds);
}

// ---------------------------------------------------------------------------
// Pair form
//
// v_mfma_f32_32x32x16_f16 runs at 16 times the rate of the fp32 form, so an
// operand a is taken as 2^e (h + l): e brings the largest finite magnitude of
// its row (or column, whichever does not run along the sum; within a part of
// the sum) into [2^14, 2^15), h = fp16(a 2^-e), l = fp16(a 2^-e - h), both to
// nearest. h + l is a up to 2^-22 of it, except that values below 2^-17 of
// that largest one lose more (half the smallest step of l is 2^-25, 2^-39 of
// the largest). Each product is h h' + h l' + l h' (l l' is at most 2^-22 of
// it), summed in fp32: 3 2^-22 of every product at most, where the roundings
// of an fp32 sum of K products may take K 2^-24. A value that is infinite or
// NaN makes the outputs it reaches NaN.

__device__ __forceinline__ float finite_mag(float v) {
    const float a = fabsf(v);
    return a < INFINITY ? a : 0.0f;
}
// e for a largest finite magnitude m; 2^-e is a normal fp32 (rows below
// 2^-111 keep smaller parts).
__device__ __forceinline__ int pair_exp(float m) {
    const int e = (int)(__float_as_uint(m) >> 23) - 127 - 14;
    return m == 0.0f ? 0 : max(e, -125);
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Eight values -> the chunks of their parts.
__device__ __forceinline__ void pair8(const float (&v)[8], float scale, u4v& h, u4v& l) {
#pragma unroll
    for (int q = 0; q < 4; q++) {
        const float a = v[2 * q] * scale, b = v[2 * q + 1] * scale;
        const h2v hp = __builtin_convertvector((f2v{a, b}), h2v);
        const h2v lp = __builtin_convertvector((f2v{a - (float)hp[0], b - (float)hp[1]}), h2v);
        h[q] = __builtin_bit_cast(uint32_t, hp);
        l[q] = __builtin_bit_cast(uint32_t, lp);
    }
}

// Position of column n in its operand: within 64, even columns first, so that
// a lane of a product ends with two neighbouring columns; the pairs in an order
// in which the eight threads of make_panel that share a row of chunks write 128
// bytes in a row at once. Lane i of a product has pair pair_of(i).
__device__ __forceinline__ int place(int n) {
    const int p = n / 2 % 32;
    return n / 64 * 64 + n % 2 * 32 + p / 16 * 16 + p % 2 * 8 + p / 2 % 8;
}
__device__ __forceinline__ int pair_of(int i) { return i / 16 * 16 + i % 8 * 2 + i / 8 % 2; }

// The parts of a matrix whose rows run along the sum: out[part][2][kw / 8][W]
// chunks from p [rows][cols]. A workgroup of NT = 2^ntl threads (at least
// kw) takes the kw = 2^kwl rows of a part and 32 NT / kw columns, each thread
// 8 rows and 4 columns: it holds them in registers while the columns' maxima are found, so memory is
// read once and written once. Rows behind the end and masked ones are loaded
// (from the last row) and become zeros.
struct Panel {
    const float* p;
    const uint8_t* mask;  // rows that do not count, or null
    int rows, cols;       // cols a multiple of 32
    int kwl, ntl, W;
    u4v* out;
    int* e;               // exponents [part][cols]
    int cb, nb;           // workgroups per part, and all
};
__device__ __forceinline__ void make_panel(const Panel& j, int b, f4v (*red)[8]) {
    const int kw = 1 << j.kwl, part = b / j.cb, tid = threadIdx.x, wave = wave_id(), c4 = tid & 7;
    const int sub = tid >> j.kwl, r8 = (tid & (kw - 1)) >> 3;
    const int col = ((b % j.cb << (j.ntl - j.kwl)) + sub) * 32 + 4 * c4, r0 = part * kw + 8 * r8;
    const bool in = col < j.cols;
    f4v v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int r = min(r0 + i, j.rows - 1);
        v[i] = *reinterpret_cast<const f4v*>(j.p + (size_t)r * j.cols + (in ? col : 0));
    }
    // a wave has 64 rows: each lane looks at one of them
    const int mr = r0 - 8 * (tid / 8 % 8) + (tid & 63);
    const unsigned long long on = __ballot(mr < j.rows && (!j.mask || j.mask[min(mr, j.rows - 1)]));
    const uint32_t mine = (uint32_t)(on >> (tid / 8 % 8 * 8)) & 0xFFu;
    f4v m = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            if (!(mine >> i & 1)) v[i][q] = 0.0f;
            m[q] = fmaxf(m[q], finite_mag(v[i][q]));
        }
#pragma unroll
    for (int q = 0; q < 4; q++)
#pragma unroll
        for (int o = 8; o < 64; o <<= 1) m[q] = fmaxf(m[q], __shfl_xor(m[q], o, 64));
    if ((tid & 63) < 8) red[wave][c4] = m;
    __syncthreads();
    const int nw = kw / 64;
    for (int i = 0; i < nw; i++) {
        const f4v o = red[sub * nw + i][c4];
#pragma unroll
        for (int q = 0; q < 4; q++) m[q] = fmaxf(m[q], o[q]);
    }
    if (!in) return;
    u4v* out = j.out + (size_t)part * (kw / 4) * j.W;
#pragma unroll
    for (int q = 0; q < 4; q++) {
        const int e = pair_exp(m[q]);
        if (r8 == 0) j.e[(size_t)part * j.cols + col + q] = e;
        float c[8];
#pragma unroll
        for (int i = 0; i < 8; i++) c[i] = v[i][q];
        u4v h, l;
        pair8(c, pow2i(-e), h, l);
        out[(size_t)r8 * j.W + place(col + q)] = h;
        out[(size_t)(kw / 8 + r8) * j.W + place(col + q)] = l;
    }
}

// grid ng + panels of x + panels of Wr, 1024 threads or fewer. The first ng
// workgroups make G (a wave two tokens, a lane the columns 8 lane + 512 c + i):
// in fp32 for k_rg_gt (unless dout serves), and its rows' parts ga [tile][2][Ep / 8][BM].
// Everything a wave needs is loaded before its mask bytes are looked at, and
// before it writes (dout may be din; no other wave uses its two rows' values).
template <int NC>
__global__ __launch_bounds__(1024) void k_rg_prep(const float* din, const int32_t* __restrict__ idx,
                                                  const float* __restrict__ w, const float* __restrict__ dw,
                                                  const uint8_t* __restrict__ mask, int T, int E, int Ep, int k,
                                                  int vec, float* __restrict__ G, float* dout, u4v* __restrict__ ga,
                                                  int BM, int* __restrict__ egr, int ng, Panel px, Panel pw) {
    __shared__ f4v red[16][8];
    if ((int)blockIdx.x >= ng) {
        const int b = (int)blockIdx.x - ng;
        if (b < px.nb) make_panel(px, b, red); else make_panel(pw, b - px.nb, red);
        return;
    }
    constexpr int NV = 8 * NC;
    const int lane = threadIdx.x & 63, t0 = (int)(blockIdx.x * (blockDim.x >> 6) + wave_id()) * 2;
    auto col = [lane](int i) { return 8 * lane + i / 8 * 512 + i % 8; };
    float v[2][NV], mw[2], md[2];
    int me[2];
    bool on[2];
#pragma unroll
    for (int u = 0; u < 2; u++) {
        const size_t t = min(t0 + u, T - 1);
        on[u] = !mask || mask[t];
        me[u] = 0;
        mw[u] = md[u] = 0.0f;
        if (dw && lane < k) {
            me[u] = idx[t * k + lane];
            mw[u] = w[t * k + lane];
            md[u] = dw[t * k + lane];
        }
#pragma unroll
        for (int i = 0; i < NV; i++) v[u][i] = 0.0f;
        if (din) {
            if (vec) {  // E % 8 == 0: a lane's eight columns are all in or all out
#pragma unroll
                for (int c = 0; c < NC; c++)
                    if (col(8 * c) < E) {
                        const f4v* p = reinterpret_cast<const f4v*>(din + t * E + col(8 * c));
                        const f4v a = p[0], b = p[1];
#pragma unroll
                        for (int q = 0; q < 4; q++) {
                            v[u][8 * c + q] = a[q];
                            v[u][8 * c + 4 + q] = b[q];
                        }
                    }
            } else {
#pragma unroll
                for (int i = 0; i < NV; i++)
                    if (col(i) < E) v[u][i] = din[t * E + col(i)];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < 2; u++) {
        const int t = t0 + u;
        if (t >= T) break;
        if (dw) add_routing<NV>(v[u], col, E, k, me[u], mw[u], md[u]);
        float rm = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (!on[u] || col(i) >= E) v[u][i] = 0.0f;
            rm = fmaxf(rm, finite_mag(v[u][i]));
        }
        const int e = pair_exp(wave_max(rm));
        if (lane == 0) egr[t] = e;
        const float scale = pow2i(-e);
        u4v* tile = ga + (size_t)(t / BM) * (Ep / 4) * BM + t % BM;
#pragma unroll
        for (int c = 0; c < NC; c++) {
            const int c0 = col(8 * c);
            if (c0 >= Ep) continue;
            float o[8];
#pragma unroll
            for (int q = 0; q < 8; q++) o[q] = v[u][8 * c + q];
            if (G) {
                f4v* g = reinterpret_cast<f4v*>(G + (size_t)t * Ep + c0);
                g[0] = f4v{o[0], o[1], o[2], o[3]};
                g[1] = f4v{o[4], o[5], o[6], o[7]};
            }
            if (ga) {
                u4v h, l;
                pair8(o, scale, h, l);
                tile[(size_t)(c0 / 8) * BM] = h;
                tile[(size_t)(Ep / 8 + c0 / 8) * BM] = l;
            }
            if (dout) {
                if (vec) {
                    if (c0 < E) {
                        f4v* d = reinterpret_cast<f4v*>(dout + (size_t)t * E + c0);
                        d[0] = f4v{o[0], o[1], o[2], o[3]};
                        d[1] = f4v{o[4], o[5], o[6], o[7]};
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 8; q++)
                        if (c0 + q < E) dout[(size_t)t * E + c0 + q] = o[q];
                }
            }
        }
    }
}

// The parts of G's columns.
__global__ __launch_bounds__(1024) void k_rg_gt(Panel pg) {
    __shared__ f4v red[16][8];
    make_panel(pg, blockIdx.x, red);
}

// An operand of a product tile: chunks [2][KC][W], the tile's columns from
// `off`.
struct PairIn {
    const u4v* p;
    int KC, W, off;
};

// Wait until at most N vector memory operations of this wave are outstanding
// (they complete in issue order) and its LDS reads are done, then a workgroup
// barrier: the loads go from memory straight into LDS, so no register tells
// the compiler when they are there.
template <int N>
__device__ __forceinline__ void ring_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

struct PairArgs {
    const u4v *ga, *gt, *xb, *wb;
    const int *egr, *egc, *ex, *ew;
    int T, Tk, E, Ep, H;                 // Tk: T rounded up to kTK
    float *dx, *dWr;                     // outputs, or the parts [s][rows][H]
    int acc_x, acc_w;
    int sx, sw, kx, kw, mt, nt, et, nx;  // nx: workgroups of dx
};

// Steps of the ring of a tile, 24 KB (BM 256) or 16 KB (BM 128) each: two or
// three workgroups fit a compute unit, so that one multiplies while another
// starts or writes its tile (before the squares of 128 x 64, a ring of 6 with
// one workgroup: 175 us against 166 at 8191 x 512 x 2560; now 140 us, 129
// GFLOP of 16-bit products at 920 TFLOP/s, where a large library bf16 product
// reaches 1206).
constexpr int kRing = 3;

// One tile of BM x 128 of C, four waves of BM / 2 x 64, in steps of 16 k. LDS
// is a ring of steps, each as chunks [2][2][BM] of A and [2][2][128] of B.
// While the matrix instructions of step s run from one set of registers, the
// fragments of step s + 1 are read into the other, and the steps up to
// s + kRing are on their way from memory. The wave's square is as large as
// the registers allow: LDS feeds 128 bytes a cycle, and 128 x 64 needs 48 KB
// per workgroup and step where the matrix units take 768 cycles, 64 x 64
// 64 KB.
template <int BM>
__device__ __forceinline__ void pair_tile(const PairIn& A, const PairIn& B, int steps, const int* __restrict__ ea,
                                          const int* __restrict__ eb, bool permuted, int m0, int M, int n0, int H,
                                          float* C, bool add, u4v* lds) {
    constexpr int R = kRing, MI = BM / 64, NA = BM / 64, NB = 2, NI = NA + NB;  // NI: 1 KB loads of a wave and step
    constexpr int STEP = 4 * BM + 4 * 128;
    int* exps = reinterpret_cast<int*>(lds + R * STEP);  // of the tile's rows and columns
    const int lane = threadIdx.x & 63, wave = wave_id(), wm = wave >> 1, wn = wave & 1;
    const rsrc_t rA = make_rsrc(A.p, (uint32_t)A.KC * (uint32_t)A.W * 32u);
    const rsrc_t rB = make_rsrc(B.p, (uint32_t)B.KC * (uint32_t)B.W * 32u);
    uint32_t oa[NA], ob[NB];  // byte offsets of the wave's loads at step 0
#pragma unroll
    for (int i = 0; i < NA; i++) {
        const int q = wave + 4 * i, row = q / (BM / 64), seg = q % (BM / 64);  // row: part, chunk of the step
        oa[i] = ((uint32_t)((row >> 1) * A.KC + (row & 1)) * (uint32_t)A.W + (uint32_t)(A.off + 64 * seg + lane)) * 16u;
    }
#pragma unroll
    for (int i = 0; i < NB; i++) {
        const int q = wave + 4 * i, row = q / 2, seg = q % 2;
        ob[i] = ((uint32_t)((row >> 1) * B.KC + (row & 1)) * (uint32_t)B.W + (uint32_t)(B.off + 64 * seg + lane)) * 16u;
    }
    const uint32_t da = (uint32_t)A.W * 32u, db = (uint32_t)B.W * 32u;  // two chunk rows a step
    // every step issues the same loads; those behind the last one read nothing
    auto issue = [&](int s, u4v* to) {
        const bool on = s < steps;
#pragma unroll
        for (int i = 0; i < NA; i++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rA, (__attribute__((address_space(3))) void*)(to + 64 * (wave + 4 * i)), 16,
                on ? oa[i] + (uint32_t)s * da : kOOB, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < NB; i++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rB, (__attribute__((address_space(3))) void*)(to + 4 * BM + 64 * (wave + 4 * i)), 16,
                on ? ob[i] + (uint32_t)s * db : kOOB, 0, 0, 0);
    };
    struct Frags {
        h8v a[2][MI], b[2][2];
    };
    const int pa = (lane >> 5) * BM + 32 * MI * wm + (lane & 31), pb = 4 * BM + (lane >> 5) * 128 + 64 * wn + (lane & 31);
    auto read = [&](const u4v* from, Frags& f) {
#pragma unroll
        for (int t = 0; t < 2; t++) {
#pragma unroll
            for (int i = 0; i < MI; i++) f.a[t][i] = __builtin_bit_cast(h8v, from[pa + 2 * t * BM + 32 * i]);
#pragma unroll
            for (int j = 0; j < 2; j++) f.b[t][j] = __builtin_bit_cast(h8v, from[pb + 2 * t * 128 + 32 * j]);
        }
    };
    f16v acc[MI][2];
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;
    auto multiply = [&](const Frags& f) {
#pragma unroll
        for (int t = 0; t < 3; t++)  // l h', h l', h h'
#pragma unroll
            for (int i = 0; i < MI; i++)
#pragma unroll
                for (int j = 0; j < 2; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.a[t == 0][i], f.b[t == 1][j], acc[i][j], 0, 0, 0);
    };
    const int er = (int)threadIdx.x < BM ? ea[min(m0 + (int)threadIdx.x, M - 1)] : 0;
    const int ec = (int)threadIdx.x < 128 ? eb[n0 + threadIdx.x] : 0;
    if ((int)threadIdx.x < BM) exps[threadIdx.x] = er;
    if ((int)threadIdx.x < 128) exps[BM + threadIdx.x] = ec;
#pragma unroll
    for (int s = 0; s < R; s++) issue(s, lds + s * STEP);
    ring_barrier<(R - 1) * NI>();  // step 0 is there
    Frags f0, f1;
    read(lds, f0);
    int at = 0;  // s % R
    auto next = [](int q) { return q + 1 == R ? 0 : q + 1; };
    // step s from f, the fragments of step s + 1 into g: step s + 1 is there
    // and every wave has read step s, whose place the load of step s + R takes
    auto turn = [&](int s, const Frags& f, Frags& g) {
        ring_barrier<(R - 2) * NI>();
        issue(s + R, lds + at * STEP);
        at = next(at);
        read(lds + at * STEP, g);
        __builtin_amdgcn_sched_barrier(0);  // the reads go out before the products, not when g is needed
        multiply(f);
    };
    for (int s = 0; s < steps; s += 2) {  // steps are even
        turn(s, f0, f1);
        turn(s + 1, f1, f0);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const int nl = 64 * wn + 2 * pair_of(lane & 31), n = n0 + nl, e0 = exps[BM + nl], e1 = exps[BM + nl + 1];
    auto row = [&](int i, int r) {  // of the workgroup's tile
        const int q = 8 * (r / 4) + 4 * (lane >> 5) + r % 4;  // of the MFMA tile
        return 32 * MI * wm + (permuted ? i / 2 * 64 + 2 * pair_of(q) + i % 2 : 32 * i + q);
    };
    C += (size_t)m0 * H + n;
    const int rows = M - m0;
#pragma unroll
    for (int i = 0; i < MI; i++) {
        f2v old[16];
#pragma unroll
        for (int r = 0; r < 16; r++)
            old[r] = add ? *reinterpret_cast<const f2v*>(C + (size_t)min(row(i, r), rows - 1) * H) : f2v{0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 16; r++) {
            const int m = row(i, r), em = exps[m];
            f2v v = {ldexpf(acc[i][0][r], em + e0), ldexpf(acc[i][1][r], em + e1)};
            if (add) {
                v.x += old[r].x;
                v.y += old[r].y;
            }
            if (m < rows) *reinterpret_cast<f2v*>(C + (size_t)m * H) = v;
        }
    }
}

// The products' tiles: those of dWr first (their sums are the longer ones),
// then those of dx. Consecutive tiles share rows of A, so each XCD (workgroups
// go to the eight in turn) takes a run of each product's.
template <int BM>
__global__ __launch_bounds__(256, 2) void k_rg_pair(PairArgs a) {
    // One array: with a second one beside it the compiler waits for every load
    // in flight before each LDS read.
    __shared__ u4v lds[kRing * (4 * BM + 4 * 128) + (BM + 128) / 4];
    const int nw = (int)gridDim.x - a.nx;
    // tile number at place i of the launch among n, for the XCD of workgroup g
    auto turn = [](int n, int i, int g) {
        const int x0 = (g - i) % 8;  // XCD of place 0
        const int x = (i + x0) % 8, q = n / 8, r = n % 8, first = (x - x0 + 8) % 8;
        return first * q + min(first, r) + i / 8;
    };
    const bool w = (int)blockIdx.x < nw;
    const int b = w ? turn(nw, blockIdx.x, blockIdx.x) : turn(a.nx, (int)blockIdx.x - nw, blockIdx.x);
    if (w) {
        const int tile = b % (a.et * a.nt), part = b / (a.et * a.nt), m = tile / a.nt * BM, c = tile % a.nt * 128;
        const int KC = a.kw / 8, W = a.et * BM;
        const PairIn A = {a.gt + (size_t)part * 2 * KC * W, KC, W, m};
        const PairIn B = {a.xb + (size_t)part * 2 * KC * a.H, KC, a.H, c};
        pair_tile<BM>(A, B, min(a.kw, a.Tk - part * a.kw) / 16, a.egc + (size_t)part * a.Ep, a.ex + (size_t)part * a.H,
                      true, m, a.E, c, a.H, a.dWr + (a.sw > 1 ? (size_t)part * a.E * a.H : 0), a.sw == 1 && a.acc_w, lds);
    } else {
        const int tile = b % (a.mt * a.nt), part = b / (a.mt * a.nt), m = tile / a.nt * BM, c = tile % a.nt * 128;
        const PairIn A = {a.ga + (size_t)(tile / a.nt) * (a.Ep / 4) * BM + (size_t)part * (a.kx / 8) * BM, a.Ep / 8, BM, 0};
        const PairIn B = {a.wb + (size_t)part * (a.kx / 4) * a.H, a.kx / 8, a.H, c};
        pair_tile<BM>(A, B, min(a.kx, a.Ep - part * a.kx) / 16, a.egr, a.ew + (size_t)part * a.H, false, m, a.T, c, a.H,
                      a.dx + (a.sx > 1 ? (size_t)part * a.T * a.H : 0), a.sx == 1 && a.acc_x, lds);
    }
}

// out (+)= the parts, in increasing order. A thread adds all parts of its four
// outputs: 9 us at 512 x 2560 outputs of 8 parts; 117 us where 256 outputs have
// 1024 (2^20 tokens of one expert, 995 us in all).
__global__ __launch_bounds__(256) void k_rg_reduce(const f4v* __restrict__ px, int sx, size_t nx, f4v* dx, int acc_x,
                                                   const f4v* __restrict__ pw, int sw, size_t nw, f4v* dWr,
                                                   int acc_w) {
    size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    const f4v* p = px;
    f4v* out = dx;
    int parts = sx, add = acc_x;
    size_t n = nx;
    if (i >= nx) {
        i -= nx;
        p = pw;
        out = dWr;
        parts = sw;
        add = acc_w;
        n = nw;
        if (i >= nw) return;
    }
    f4v v = p[i];
#pragma unroll 4
    for (int s = 1; s < parts; s++) v += p[(size_t)s * n + i];
    if (add) v += out[i];
    out[i] = v;
}

}  // namespace

size_t route_backward_ws_bytes(int H, int E, int T) { return rg_plan(H, E, T).total; }

hipError_t launch_route_backward(int H, int E, int k, const float* x, int T, const float* Wr, const int32_t* idx,
                                 const float* w, const float* dw, const uint8_t* mask, const float* dlogits_in,
                                 float* dlogits_out, float* dx, float* dWr, int accumulate, void* ws, hipStream_t s) {
    if (T == 0 && (!dWr || accumulate & 2)) return hipSuccess;  // no tokens: zeros for dWr at most
    const RgPlan p = rg_plan(H, E, T, accumulate & 8);
    char* base = reinterpret_cast<char*>(ws);
    float* G = reinterpret_cast<float*>(base + p.g);
    const int nx = dx && T > 0 ? p.mt * p.nt * p.sx : 0, nw = dWr ? p.et * p.nt * p.sw : 0;
    const int acc_x = accumulate & 1, acc_w = (accumulate >> 1) & 1;
    float* ox = p.sx > 1 ? reinterpret_cast<float*>(base + p.px) : dx;
    float* ow = p.sw > 1 ? reinterpret_cast<float*>(base + p.pw) : dWr;
    hipError_t r = hipSuccess;
    if (p.BM && nx + nw) {
        int *egr = reinterpret_cast<int*>(base + p.egr), *egc = reinterpret_cast<int*>(base + p.egc);
        int *ex = reinterpret_cast<int*>(base + p.ex), *ew = reinterpret_cast<int*>(base + p.ew);
        u4v *ga = reinterpret_cast<u4v*>(base + p.ga), *gt = reinterpret_cast<u4v*>(base + p.gt);
        u4v *xb = reinterpret_cast<u4v*>(base + p.xb), *wb = reinterpret_cast<u4v*>(base + p.wb);
        // dlogits_out has G as the workspace would, where E needs no padding
        // (k_rg_gt reads it with 16-byte loads)
        const bool own_g = !dlogits_out || p.Ep != E || reinterpret_cast<uintptr_t>(dlogits_out) % 16;
        const float* Gp = own_g ? G : dlogits_out;
        float* Gw = own_g && nw ? G : nullptr;
        auto panel = [](const float* m, const uint8_t* mk, int rows, int cols, int kw, int nt, int parts, int W, u4v* out,
                        int* e, bool used) {
            Panel q = {m, mk, rows, cols, 0, 0, W, out, e, 0, 0};
            while ((1 << q.kwl) < kw) q.kwl++;
            while ((1 << q.ntl) < nt) q.ntl++;
            const int width = 32 * (nt / kw);
            q.cb = (cols + width - 1) / width;
            q.nb = used ? q.cb * parts : 0;
            return q;
        };
        const int nt = p.kw > p.kx ? p.kw : p.kx;  // threads: one panel's at least
        const Panel px = panel(x, mask, T, H, p.kw, nt, p.sw, H, xb, ex, nw > 0);
        const Panel pw = panel(Wr, nullptr, E, H, p.kx, nt, p.sx, H, wb, ew, nx > 0);
        const Panel pg = panel(Gp, nullptr, T, p.Ep, p.kw, p.kw, p.sw, p.et * p.BM, gt, egc, nw > 0);
        const int ng = (T + nt / 32 - 1) / (nt / 32);
        const int vec = E % 8 == 0 && (reinterpret_cast<uintptr_t>(dlogits_in) | reinterpret_cast<uintptr_t>(dlogits_out)) % 16 == 0;
#define RP(NC)                                                                                                       \
    hipLaunchKernelGGL((k_rg_prep<NC>), dim3(ng + px.nb + pw.nb), dim3(nt), 0, s, dlogits_in, idx, w, dw, mask, T, E, \
                       p.Ep, k, vec, Gw, dlogits_out, nx ? ga : nullptr, p.BM, egr, ng, px, pw)
        if (p.Ep <= 512) RP(1); else RP(2);
#undef RP
        if ((r = hipGetLastError()) != hipSuccess) return r;
        if (nw) {
            hipLaunchKernelGGL(k_rg_gt, dim3(pg.nb), dim3(p.kw), 0, s, pg);
            if ((r = hipGetLastError()) != hipSuccess) return r;
        }
        const PairArgs a = {ga, gt, xb, wb, egr, egc, ex, ew, T, (T + kTK - 1) / kTK * kTK, E, p.Ep, H, ox, ow,
                            acc_x, acc_w, p.sx, p.sw, p.kx, p.kw, p.mt, p.nt, p.et, nx};
        if (p.BM == 256)
            hipLaunchKernelGGL((k_rg_pair<256>), dim3(nx + nw), dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_rg_pair<128>), dim3(nx + nw), dim3(256), 0, s, a);
    } else {
        if (T > 0) {
            const dim3 grid((T + 3) / 4), block(256);
#define RL(NV)                                                                                                     \
    hipLaunchKernelGGL((k_rg_logits<NV>), grid, block, 0, s, dlogits_in, idx, w, dw, mask, T, E, p.Ep, k, G, dlogits_out)
            if (p.Ep <= 256) RL(4); else if (p.Ep <= 512) RL(8); else RL(16);
#undef RL
            if ((r = hipGetLastError()) != hipSuccess) return r;
        }
        if (nx + nw == 0) return hipSuccess;
        const RgArgs a = {G, p.Ep, Wr, x, mask, T, E, H, ox, ow, acc_x, acc_w,
                          p.sx, p.sw, p.kx, p.kw, p.mt, p.nt, p.et, nx};
        hipLaunchKernelGGL(k_rg_gemm, dim3(nx + nw), dim3(256), 0, s, a);
    }
    if ((r = hipGetLastError()) != hipSuccess) return r;
    const size_t qx = nx && p.sx > 1 ? (size_t)T * H / 4 : 0, qw = nw && p.sw > 1 ? (size_t)E * H / 4 : 0;
    if (qx + qw) {
        hipLaunchKernelGGL(k_rg_reduce, dim3((unsigned)((qx + qw + 255) / 256)), dim3(256), 0, s,
                           reinterpret_cast<const f4v*>(base + p.px), p.sx, qx, reinterpret_cast<f4v*>(dx), acc_x,
                           reinterpret_cast<const f4v*>(base + p.pw), p.sw, qw, reinterpret_cast<f4v*>(dWr), acc_w);
        r = hipGetLastError();
    }
    return r;
}

}  // namespace moe

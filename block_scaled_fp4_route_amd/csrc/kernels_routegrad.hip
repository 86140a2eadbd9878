// The gradient of the routing, for gfx950. With w the softmax over the chosen
// k logits and dw the gradient of the loss at w:
//   ds[t][j] = w[t][j] (dw[t][j] - sum_i w[t][i] dw[t][i])
//   G        = dlogits_in + ds scattered to the chosen experts (masked tokens: 0)
//   dx       = G Wr        [T][H], over E
//   dWr      = G^T x       [E][H], over T
// k_rg_logits writes G (one wave per token), k_rg_gemm runs both products as
// one launch, and k_rg_reduce adds the parts of products whose long axis was
// split. Everything in fp32: operands, v_mfma_f32_16x16x4_f32, sums.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_learn.h"

namespace moe {

namespace {

constexpr int kTM = 128, kTN = 128, kTK = 32;  // tile of the products
constexpr int kLogitRows = 32;                 // tokens of a workgroup of k_rg_logits (pair form): a word of bits
constexpr int kMaxRows = 128;                  // rows of a workgroup's column maxima

// Multiplications (T E H) from which the products run by pairs of fp16 parts.
constexpr int64_t kPairFrom = (int64_t)1 << 24;

struct RgPlan {
    int MW;               // 0: fp32 form; else the pair form with tiles of 128 MW rows
    int gb, xb, wb;       // parts of the column maxima of G, x and Wr
    int Ep;               // columns of G in the workspace (E rounded up to kTK, zero-padded)
    int mt, nt;           // dx: row tiles; both: column tiles
    int et;               // dWr: row tiles
    int sx, sw;           // parts of the long axis of dx (over E) and dWr (over T)
    int kx, kw;           // its length in a part (multiples of kTK)
    size_t g, exps, max, px, pw, total;
};

RgPlan rg_plan(int H, int E, int T) {
    RgPlan p;
    p.Ep = (E + kTK - 1) / kTK * kTK;
    p.nt = (H + kTN - 1) / kTN;
    p.MW = 0;
    if ((int64_t)T * E * H >= kPairFrom) {
        // 256-row tiles read less per product; 128-row ones where the larger
        // would leave compute units idle
        const int64_t large = ((int64_t)(T + 255) / 256 + (E + 255) / 256) * p.nt;
        p.MW = large >= 512 ? 2 : 1;
    }
    const int tm = p.MW ? 128 * p.MW : kTM;
    p.mt = (T + tm - 1) / tm;
    p.et = (E + tm - 1) / tm;
    // parts of the long axis until one workgroup per compute unit has work, of
    // two steps at least, and none above 1024
    auto split = [](int64_t tiles, int64_t len, int& parts, int& per) {
        parts = 1;
        per = kTK;
        if (tiles < 1 || len < 1) return;  // no tokens
        int64_t n = (256 + tiles - 1) / tiles;
        if (len / 1024 > n) n = len / 1024;
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
    size_t o = kCounterBytes;
    auto take = [&o](size_t bytes) {
        const size_t at = o;
        o += align256(bytes);
        return at;
    };
    p.g = take((size_t)T * p.Ep * 4);
    p.gb = (T + kLogitRows - 1) / kLogitRows;
    p.xb = (T + kMaxRows - 1) / kMaxRows;
    p.wb = (E + kMaxRows - 1) / kMaxRows;
    p.exps = take(p.MW ? ((size_t)T + p.gb + p.Ep + 2 * (size_t)H) * 4 : 0);
    p.max = take(p.MW ? ((size_t)p.gb * p.Ep + ((size_t)p.xb + p.wb) * H) * 4 : 0);
    p.px = take(p.sx > 1 ? (size_t)p.sx * T * H * 4 : 0);
    p.pw = take(p.sw > 1 ? (size_t)p.sw * E * H * 4 : 0);
    p.total = o;
    return p;
}

// One tile of C[M][H] = A B over [k0, k1). A(m, k) is G[m][k] (dx: KMAJ
// false) or G[k][m] (dWr: KMAJ true); B rows are rows of Wr (dx) or x (dWr).
// Both operands go through LDS as [k][m] and [k][n]. In every wave lane
// (i = lane % 16, q = lane / 16) reads 4 consecutive m (n) of row k + q in
// one 16-byte read: MFMA (a, b) then covers the rows 4 i + a and columns
// 4 i + b of the wave's 64 x 64 square, and a lane ends with 4 consecutive
// columns of each of its rows.
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
    // pair form: exponents of G's rows and columns, x's and Wr's columns; a bit per token that counts
    const int *egr, *egc, *ex, *ew;
    const uint32_t* keep;
};

constexpr int kLdsRow = kTM + 4;

template <bool KMAJ>
__device__ __forceinline__ void rg_tile(const RgArgs& a, int tile, int part, float* lds) {
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
    const int M = KMAJ ? a.E : a.T;                 // rows of C
    const int klen = KMAJ ? a.T : a.E;              // length of the sum
    const int m0 = tile / a.nt * kTM, n0 = tile % a.nt * kTN;
    const int per = KMAJ ? a.kw : a.kx;
    const int k0 = part * per, k1 = min(klen, k0 + per);
    const float* B = KMAJ ? a.x : a.Wr;
    const uint8_t* mask = KMAJ ? a.mask : nullptr;
    float* As = lds;
    float* Bs = lds + kTK * kLdsRow;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64, li = lane & 15, lq = lane >> 4;
    f4v acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = f4v{0.f, 0.f, 0.f, 0.f};
    const f4v zero = {0.f, 0.f, 0.f, 0.f};
    f4v ra[4], rb[4];
    auto fetch = [&](int k) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int p = tid + 256 * i;
            // B: 32 float4 per row of 128
            const int kr = k + p / 32, n = n0 + p % 32 * 4;
            rb[i] = kr < k1 && n < a.H && (!mask || mask[kr])
                        ? *reinterpret_cast<const f4v*>(B + (size_t)kr * a.H + n)
                        : zero;
            if (KMAJ) {  // G rows are tokens: 32 float4 per row of 128 experts
                const int m = m0 + p % 32 * 4;
                ra[i] = kr < k1 && m < a.Ep ? *reinterpret_cast<const f4v*>(a.G + (size_t)kr * a.Ep + m) : zero;
            } else {     // 8 float4 per row of 32 experts
                const int m = m0 + p / 8, kk = k + p % 8 * 4;
                ra[i] = m < M && kk < a.Ep ? *reinterpret_cast<const f4v*>(a.G + (size_t)m * a.Ep + kk) : zero;
            }
        }
    };
    fetch(k0);
    for (int k = k0; k < k1; k += kTK) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int p = tid + 256 * i;
            *reinterpret_cast<f4v*>(Bs + p / 32 * kLdsRow + p % 32 * 4) = rb[i];
            if (KMAJ) {
                *reinterpret_cast<f4v*>(As + p / 32 * kLdsRow + p % 32 * 4) = ra[i];
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) As[(p % 8 * 4 + j) * kLdsRow + p / 8] = ra[i][j];
            }
        }
        __syncthreads();
        if (k + kTK < k1) fetch(k + kTK);
#pragma unroll
        for (int kk = 0; kk < kTK; kk += 4) {
            const f4v fa = *reinterpret_cast<const f4v*>(As + (kk + lq) * kLdsRow + wm + 4 * li);
            const f4v fb = *reinterpret_cast<const f4v*>(Bs + (kk + lq) * kLdsRow + wn + 4 * li);
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[i], fb[j], acc[i][j], 0, 0, 0);
        }
    }
    const int parts = KMAJ ? a.sw : a.sx;
    float* C = (KMAJ ? a.dWr : a.dx) + (parts > 1 ? (size_t)part * M * a.H : 0);
    const bool add = parts == 1 && (KMAJ ? a.acc_w : a.acc_x);
    const int n = n0 + wn + 4 * li;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int m = m0 + wm + 4 * (lq * 4 + q) + i;
            if (m < M && n < a.H) {
                f4v* c = reinterpret_cast<f4v*>(C + (size_t)m * a.H + n);
                f4v v = {acc[i][0][q], acc[i][1][q], acc[i][2][q], acc[i][3][q]};
                if (add) v += *c;
                *c = v;
            }
        }
}

__global__ __launch_bounds__(256) void k_rg_gemm(RgArgs a) {
    __shared__ __align__(16) float lds[2 * kTK * kLdsRow];
    const int b = blockIdx.x;
    if (b < a.nx)
        rg_tile<false>(a, b % (a.mt * a.nt), b / (a.mt * a.nt), lds);
    else
        rg_tile<true>(a, (b - a.nx) % (a.et * a.nt), (b - a.nx) / (a.et * a.nt), lds);
}

// ---------------------------------------------------------------------------
// The products by pairs of fp16 parts.
//
// v_mfma_f32_32x32x16_f16 runs at 16 times the rate of the fp32 form, so an
// operand a is taken as 2^e (h + l): e brings the largest finite magnitude of
// its row (or column, whichever does not run along the sum) into [2^14, 2^15),
// h = fp16(a 2^-e), l = fp16(a 2^-e - h), both to nearest. h + l is a up to
// 2^-22 of it, except that values below 2^-17 of that largest one lose more
// (half the smallest step of l is 2^-25, 2^-39 of the largest). Each product
// is h h' + h l' + l h' (l l' is at most 2^-22 of it), summed in fp32: 3 2^-22
// of every product at most, where the roundings of an fp32 sum of K products
// may take K 2^-24.
// A value that is infinite or NaN makes the outputs it reaches NaN.

// Largest finite magnitude, as the bits of an fp32 (0 if there is none).
__device__ __forceinline__ float finite_mag(float v) {
    const float a = fabsf(v);
    return a < INFINITY ? a : 0.0f;
}
// e of the pair form for a row whose largest finite magnitude is m; 2^-e is a
// normal fp32 (a row below 2^-111 keeps smaller parts).
__device__ __forceinline__ int pair_exp(float m) {
    const int e = (int)(__float_as_uint(m) >> 23) - 127 - 14;
    return m == 0.0f ? 0 : max(e, -125);
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Each column's largest finite magnitude over kMaxRows rows: 256 columns and
// 16 x 8 rows a workgroup of 1024, every load of a lane in flight at once
// (rows behind the end and masked ones are loaded and left out).
struct MaxJob {
    const float* p;
    const uint8_t* mask;  // rows that do not count, or null
    int rows, cols;       // cols a multiple of 256
    float* part;          // [ceil(rows / kMaxRows)][cols]
    int nb;               // workgroups
};
__device__ __forceinline__ void col_max(const MaxJob& j, int b, float (*red)[256]) {
    const int cb = j.cols / 256, c = b % cb * 256, wave = wave_id(), lane = threadIdx.x & 63;
    const int r0 = b / cb * kMaxRows + wave * 8;
    f4v v[8];
    bool on[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int r = min(r0 + i, j.rows - 1);
        v[i] = *reinterpret_cast<const f4v*>(j.p + (size_t)r * j.cols + c + 4 * lane);
        on[i] = r0 + i < j.rows && (!j.mask || j.mask[r]);
    }
    f4v m = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
        for (int q = 0; q < 4; q++) m[q] = fmaxf(m[q], on[i] ? finite_mag(v[i][q]) : 0.0f);
    *reinterpret_cast<f4v*>(&red[wave][4 * lane]) = m;
    __syncthreads();
    if (threadIdx.x < 256) {
        float a = red[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < 16; i++) a = fmaxf(a, red[i][threadIdx.x]);
        j.part[(size_t)(b / cb) * j.cols + c + threadIdx.x] = a;
    }
}

// G: one wave per token, a lane the columns lane + 64 i (i < NV). Fp32 form:
// 4 tokens a workgroup of 256. Pair form (PAIR): 32 tokens a workgroup of
// 1024, which also writes the exponent of each row, its tokens' column maxima
// and a word that says which of them count; further workgroups make the
// column maxima of x and Wr. Rows that do not count are loaded and left out:
// a load that waits for its mask byte doubles the latency.
template <int NV, bool PAIR>
__global__ __launch_bounds__(PAIR ? 1024 : 256) void k_rg_logits(
    const float* __restrict__ din, const int32_t* __restrict__ idx, const float* __restrict__ w,
    const float* __restrict__ dw, const uint8_t* __restrict__ mask, int T, int E, int Ep, int k, float* __restrict__ G,
    float* dout, int* __restrict__ egr, uint32_t* __restrict__ keep, float* __restrict__ gpart, int ng, MaxJob jx,
    MaxJob jw) {
    __shared__ __align__(16) float red[PAIR ? 16 : 1][256];  // column maxima: of x and Wr, or as bits of G
    uint32_t* gm = reinterpret_cast<uint32_t*>(red);
    __shared__ uint32_t kept;
    if constexpr (PAIR) {
        if ((int)blockIdx.x >= ng) {
            const int b = (int)blockIdx.x - ng;
            if (b < jx.nb) col_max(jx, b, red); else col_max(jw, b - jx.nb, red);
            return;
        }
        for (int e = threadIdx.x; e < Ep; e += 1024) gm[e] = 0;
        if (threadIdx.x == 0) kept = 0;
        __syncthreads();
    }
    const int lane = threadIdx.x & 63, wave = wave_id();
    constexpr int PER = PAIR ? 2 : 1;  // tokens of a wave
    const int t0 = (int)blockIdx.x * (PAIR ? kLogitRows : 4) + wave * PER;
    float v[PER][NV], mw[PER], md[PER];
    int me[PER];
    bool on[PER];
#pragma unroll
    for (int u = 0; u < PER; u++) {
        const size_t t = min(t0 + u, T - 1);
        on[u] = t0 + u < T && (!mask || mask[t]);
        me[u] = 0;
        mw[u] = md[u] = 0.0f;
        if (dw && lane < k) {
            me[u] = idx[t * k + lane];
            mw[u] = w[t * k + lane];
            md[u] = dw[t * k + lane];
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int e = lane + 64 * i;
            v[u][i] = din && e < E ? din[t * E + e] : 0.0f;
        }
    }
#pragma unroll
    for (int u = 0; u < PER; u++) {
        const int t = t0 + u;
        if (t >= T) break;
        if (dw) {
            const float dot = wave_sum(lane < k ? mw[u] * md[u] : 0.0f);
            const float ds = mw[u] * (md[u] - dot);
            for (int j = 0; j < k; j++) {  // in increasing j, so an expert named twice adds in that order
                const int e = __builtin_amdgcn_readlane(me[u], j);
                const float d = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ds), j));
#pragma unroll
                for (int i = 0; i < NV; i++) v[u][i] += lane + 64 * i == e ? d : 0.0f;
            }
            if (__ballot(lane < k && (unsigned)me[u] >= (unsigned)E))
#pragma unroll
                for (int i = 0; i < NV; i++) v[u][i] = __builtin_nanf("");
        }
        float rm = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int e = lane + 64 * i;
            if (e >= E || !on[u]) v[u][i] = 0.0f;
            if (e < Ep) G[(size_t)t * Ep + e] = v[u][i];
            if (dout && e < E) dout[(size_t)t * E + e] = v[u][i];
            if constexpr (PAIR) {
                const float a = finite_mag(v[u][i]);
                rm = fmaxf(rm, a);
                if (e < Ep) atomicMax(&gm[e], __float_as_uint(a));
            }
        }
        if constexpr (PAIR) {
            rm = wave_max(rm);
            if (lane == 0) {
                egr[t] = pair_exp(rm);
                if (on[u]) atomicOr(&kept, 1u << (t & 31));
            }
        }
    }
    if constexpr (PAIR) {
        __syncthreads();
        for (int e = threadIdx.x; e < Ep; e += 1024) gpart[(size_t)blockIdx.x * Ep + e] = __uint_as_float(gm[e]);
        if (threadIdx.x == 0) keep[blockIdx.x] = kept;
    }
}

// grid ceil(columns / 16) of the jobs in turn, 1024 threads: exponents of the
// columns from the parts' maxima (cols are multiples of 16).
struct ExpJob {
    const float* part;
    int rows, cols;
    int* e;
    int nb;
};
__global__ __launch_bounds__(1024) void k_rg_exps(ExpJob a, ExpJob b, ExpJob c) {
    __shared__ float red[64][17];
    int blk = blockIdx.x;
    ExpJob j = a;
    if (blk >= a.nb) {
        blk -= a.nb;
        j = b;
        if (blk >= b.nb) {
            blk -= b.nb;
            j = c;
        }
    }
    const int col = threadIdx.x & 15, g = threadIdx.x >> 4, cc = blk * 16 + col;
    float m = 0.0f;
#pragma unroll 4
    for (int r = g; r < j.rows; r += 64) m = fmaxf(m, j.part[(size_t)r * j.cols + cc]);
    red[g][col] = m;
    __syncthreads();
#pragma unroll
    for (int h = 32; h >= 1; h >>= 1) {
        if (g < h) red[g][col] = fmaxf(red[g][col], red[g + h][col]);
        __syncthreads();
    }
    if (g == 0) j.e[cc] = pair_exp(red[0][col]);
}

typedef _Float16 h8v __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef uint32_t u2v __attribute__((ext_vector_type(2)));

// Two values (already scaled) -> their packed h and l parts.
typedef _Float16 h2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void pair2(float a, float b, uint32_t& h, uint32_t& l) {
    const h2v hp = __builtin_convertvector((f2v{a, b}), h2v);
    const h2v lp = __builtin_convertvector((f2v{a - (float)hp[0], b - (float)hp[1]}), h2v);
    h = __builtin_bit_cast(uint32_t, hp);
    l = __builtin_bit_cast(uint32_t, lp);
}

// One tile of 128 MW x 128 of C = A B over [k0, k1), as rg_tile. LDS holds
// chunks of 8 consecutive k of one row (column) of either part; a row m of A
// from G[k][m], and a column n of B, sits at position
// 128 (n / 128) + 32 (n % 4) + n / 4 % 32, so that threads with neighbouring
// float4 of a memory row write neighbouring chunks, MFMA j covers the columns
// 4 i + j, and a lane of C ends with 4 consecutive columns of each row. Wave w
// has the 32 MW positions of rows from 32 MW w and all 128 columns.
template <int MW, bool KMAJ>
__device__ __forceinline__ void rg_pair_tile(const RgArgs& a, int tile, int part, u4v* lds) {
    constexpr int MT = 128 * MW;
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
    const int M = KMAJ ? a.E : a.T, klen = KMAJ ? a.T : a.E;
    const int m0 = tile / a.nt * MT, n0 = tile % a.nt * kTN;
    const int per = KMAJ ? a.kw : a.kx;
    const int k0 = part * per, k1 = min(klen, k0 + per);
    const float* B = KMAJ ? a.x : a.Wr;
    const int* eb = KMAJ ? a.ex : a.ew;       // exponents of B's columns
    const int* ea = KMAJ ? a.egc : a.egr;     // exponents of A's rows
    u4v* As = lds;               // [2][4][MT]
    u4v* Bs = lds + 8 * MT;      // [2][4][128]
    f16v acc[MW][4];
#pragma unroll
    for (int i = 0; i < MW; i++)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;

    // B: thread (n2 = tid % 64, kc = tid / 64) has columns 2 n2, 2 n2 + 1 of
    // the 8 rows of chunk kc (H is a multiple of 256: columns are whole)
    const int bn = tid % 64 * 2, bk = wave * 8;
    const float sb0 = pow2i(-eb[n0 + bn]), sb1 = pow2i(-eb[n0 + bn + 1]);
    u2v rb[8];
    // A from G[k][m]: the same with MW times 2 columns; A from G[m][k]: rows
    // tid % 16 + 16 (tid / 64) + 64 i, chunk tid / 16 % 4
    const int an = tid % 64 * 2 * MW;
    const int am = tid % 16 + tid / 64 * 16, ac = tid / 16 % 4 * 8;
    float sa[2 * MW];
#pragma unroll
    for (int i = 0; i < 2 * MW; i++) {
        const int m = KMAJ ? m0 + an + i : m0 + am + 64 * i;
        sa[i] = pow2i(-ea[min(m, (KMAJ ? a.Ep : M) - 1)]);
    }
    // Loads go through buffer resources over the rows of this part: offsets
    // behind them (rows past k1 or M, rows that do not count, columns past
    // Ep) read 0, so no load waits for a branch.
    const rsrc_t rB = make_rsrc(B + (size_t)k0 * a.H, (uint32_t)(k1 - k0) * (uint32_t)a.H * 4u);
    const rsrc_t rA = KMAJ ? make_rsrc(a.G + (size_t)k0 * a.Ep, (uint32_t)(k1 - k0) * (uint32_t)a.Ep * 4u)
                           : make_rsrc(a.G + (size_t)m0 * a.Ep, (uint32_t)min(MT, M - m0) * (uint32_t)a.Ep * 4u);
    const uint32_t ob = (uint32_t)(n0 + bn) * 4u;
    const uint32_t oa = KMAJ ? (m0 + an < a.Ep ? (uint32_t)(m0 + an) * 4u : kOOB) : (uint32_t)(am * a.Ep + ac) * 4u;
    u4v ra4[KMAJ ? (MW == 2 ? 8 : 1) : 4 * MW];  // a row's columns, or the halves of a row's chunk
    u2v ra2[KMAJ && MW == 1 ? 8 : 1];
    auto fetch = [&](int k) {
        const uint32_t kp = KMAJ ? a.keep[k / 32] >> bk : 0xFFu;  // k0 is a multiple of 32
#pragma unroll
        for (int r = 0; r < 8; r++) {
            const uint32_t row = (uint32_t)(k - k0 + bk + r);
            const uint32_t o = kp >> r & 1u ? row * (uint32_t)a.H * 4u : kOOB;
            rb[r] = __builtin_bit_cast(u2v, __builtin_amdgcn_raw_buffer_load_b64(rB, o + ob, 0, 0));
            if constexpr (KMAJ) {
                const uint32_t q = row * (uint32_t)a.Ep * 4u + oa;
                if constexpr (MW == 2)
                    ra4[r] = __builtin_bit_cast(u4v, __builtin_amdgcn_raw_buffer_load_b128(rA, q, 0, 0));
                else
                    ra2[r] = __builtin_bit_cast(u2v, __builtin_amdgcn_raw_buffer_load_b64(rA, q, 0, 0));
            }
        }
        if constexpr (!KMAJ) {
#pragma unroll
            for (int i = 0; i < 2 * MW; i++) {
                const uint32_t q = oa + (uint32_t)(64 * i * a.Ep + k) * 4u;
                ra4[2 * i] = __builtin_bit_cast(u4v, __builtin_amdgcn_raw_buffer_load_b128(rA, q, 0, 0));
                ra4[2 * i + 1] = __builtin_bit_cast(u4v, __builtin_amdgcn_raw_buffer_load_b128(rA, q + 16u, 0, 0));
            }
        }
    };
    // element r of the chunk of A's i-th row or column
    auto elem = [&](int i, int r) -> float {
        uint32_t b;
        if constexpr (!KMAJ)
            b = ra4[2 * i + r / 4][r % 4];
        else if constexpr (MW == 2)
            b = ra4[r][i];
        else
            b = ra2[r][i];
        return __uint_as_float(b);
    };
    auto put = [&](u4v* to, int plane, int at, const float (&v)[8]) {  // a chunk of both parts
        u4v h, l;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            uint32_t hq, lq;
            pair2(v[2 * q], v[2 * q + 1], hq, lq);
            h[q] = hq;
            l[q] = lq;
        }
        to[at] = h;
        to[plane + at] = l;
    };
    auto place = [](int n) { return n / 128 * 128 + n % 4 * 32 + n / 4 % 32; };
    fetch(k0);
    for (int k = k0; k < k1; k += kTK) {
        __syncthreads();
        {
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; r++) v[r] = __uint_as_float(rb[r].x) * sb0;
            put(Bs, 4 * 128, bk / 8 * 128 + place(bn), v);
#pragma unroll
            for (int r = 0; r < 8; r++) v[r] = __uint_as_float(rb[r].y) * sb1;
            put(Bs, 4 * 128, bk / 8 * 128 + place(bn + 1), v);
#pragma unroll
            for (int i = 0; i < 2 * MW; i++) {
#pragma unroll
                for (int r = 0; r < 8; r++) v[r] = elem(i, r) * sa[i];
                put(As, 4 * MT, KMAJ ? bk / 8 * MT + place(an + i) : ac / 8 * MT + am + 64 * i, v);
            }
        }
        __syncthreads();
        if (k + kTK < k1) fetch(k + kTK);
#pragma unroll
        for (int ks = 0; ks < 2; ks++) {
            const int kc = 2 * ks + (lane >> 5), p = lane & 31;
            h8v fa[2][MW], fb[2][4];
#pragma unroll
            for (int t = 0; t < 2; t++) {
#pragma unroll
                for (int i = 0; i < MW; i++)
                    fa[t][i] = __builtin_bit_cast(h8v, As[(4 * t + kc) * MT + 32 * (MW * wave + i) + p]);
#pragma unroll
                for (int j = 0; j < 4; j++) fb[t][j] = __builtin_bit_cast(h8v, Bs[(4 * t + kc) * 128 + 32 * j + p]);
            }
#pragma unroll
            for (int i = 0; i < MW; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[1][i], fb[0][j], acc[i][j], 0, 0, 0);
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[0][i], fb[1][j], acc[i][j], 0, 0, 0);
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[0][i], fb[0][j], acc[i][j], 0, 0, 0);
                }
        }
    }
    const int parts = KMAJ ? a.sw : a.sx;
    float* C = (KMAJ ? a.dWr : a.dx) + (parts > 1 ? (size_t)part * M * a.H : 0);
    const bool add = parts == 1 && (KMAJ ? a.acc_w : a.acc_x);
    const int n = n0 + 4 * (lane & 31);
    int en[4];
#pragma unroll
    for (int j = 0; j < 4; j++) en[j] = eb[n + j];
#pragma unroll
    for (int i = 0; i < MW; i++)
#pragma unroll
        for (int r = 0; r < 16; r++) {
            // row of the MFMA tile, then of the workgroup's tile
            const int pr = 32 * (MW * wave + i) + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
            const int m = m0 + (KMAJ ? pr / 128 * 128 + pr % 32 * 4 + pr % 128 / 32 : pr);
            if (m >= M) continue;
            const int em = ea[m];
            f4v* c = reinterpret_cast<f4v*>(C + (size_t)m * a.H + n);
            f4v v;
#pragma unroll
            for (int j = 0; j < 4; j++) v[j] = ldexpf(acc[i][j][r], em + en[j]);
            if (add) v += *c;
            *c = v;
        }
}

// The products' tiles: those of dWr first (their sums are the longer ones),
// then those of dx. Consecutive tiles share rows of A, so each XCD (workgroups
// go to the eight in turn) takes a run of them.
template <int MW>
__global__ __launch_bounds__(256, 2) void k_rg_pair(RgArgs a) {
    __shared__ u4v lds[8 * 128 * MW + 8 * 128];
    const int n = gridDim.x, q = n / 8, r = n % 8, xcd = blockIdx.x % 8, i = blockIdx.x / 8;
    const int b = xcd * q + min(xcd, r) + i;
    const int nw = n - a.nx;
    if (b < nw)
        rg_pair_tile<MW, true>(a, b % (a.et * a.nt), b / (a.et * a.nt), lds);
    else
        rg_pair_tile<MW, false>(a, (b - nw) % (a.mt * a.nt), (b - nw) / (a.mt * a.nt), lds);
}

// out (+)= the parts, in increasing order.
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
    const RgPlan p = rg_plan(H, E, T);
    char* base = reinterpret_cast<char*>(ws);
    float* G = reinterpret_cast<float*>(base + p.g);
    hipError_t r = hipSuccess;
    RgArgs a = {};
    a.G = G;
    a.Ep = p.Ep;
    a.Wr = Wr;
    a.x = x;
    a.mask = mask;
    a.T = T;
    a.E = E;
    a.H = H;
    a.acc_x = accumulate & 1;
    a.acc_w = (accumulate >> 1) & 1;
    a.sx = p.sx;
    a.sw = p.sw;
    a.kx = p.kx;
    a.kw = p.kw;
    a.mt = p.mt;
    a.nt = p.nt;
    a.et = p.et;
    a.dx = p.sx > 1 ? reinterpret_cast<float*>(base + p.px) : dx;
    a.dWr = p.sw > 1 ? reinterpret_cast<float*>(base + p.pw) : dWr;
    a.nx = dx && T > 0 ? p.mt * p.nt * p.sx : 0;
    const int nw = dWr ? p.et * p.nt * p.sw : 0;
    int* egr = reinterpret_cast<int*>(base + p.exps);
    uint32_t* keep = reinterpret_cast<uint32_t*>(egr + T);
    int *egc = egr + T + p.gb, *ex = egc + p.Ep, *ew = ex + H;
    float* gpart = reinterpret_cast<float*>(base + p.max);
    float *xpart = gpart + (size_t)p.gb * p.Ep, *wpart = xpart + (size_t)p.xb * H;
    const bool products = a.nx + nw > 0;
    const bool pair = p.MW && products;
    if (T > 0) {
        const int cb = H / 256;
        const MaxJob jx = {x, mask, T, H, xpart, pair && dWr ? p.xb * cb : 0};
        const MaxJob jw = {Wr, nullptr, E, H, wpart, pair && dx ? p.wb * cb : 0};
        const int ng = pair ? p.gb : (T + 3) / 4;
#define RL(NV)                                                                                                     \
    if (pair)                                                                                                      \
        hipLaunchKernelGGL((k_rg_logits<NV, true>), dim3(ng + jx.nb + jw.nb), dim3(1024), 0, s, dlogits_in, idx, w, dw, \
                           mask, T, E, p.Ep, k, G, dlogits_out, egr, keep, gpart, ng, jx, jw);                             \
    else                                                                                                           \
        hipLaunchKernelGGL((k_rg_logits<NV, false>), dim3(ng), dim3(256), 0, s, dlogits_in, idx, w, dw, mask, T, E,  \
                           p.Ep, k, G, dlogits_out, egr, keep, gpart, ng, jx, jw)
        if (p.Ep <= 256) { RL(4); } else if (p.Ep <= 512) { RL(8); } else { RL(16); }
#undef RL
        if ((r = hipGetLastError()) != hipSuccess) return r;
    }
    if (!products) return hipSuccess;
    if (pair) {
        const ExpJob jg = {gpart, p.gb, p.Ep, egc, dWr ? p.Ep / 16 : 0};
        const ExpJob jx = {xpart, p.xb, H, ex, dWr ? H / 16 : 0}, jw = {wpart, p.wb, H, ew, dx ? H / 16 : 0};
        hipLaunchKernelGGL(k_rg_exps, dim3(jg.nb + jx.nb + jw.nb), dim3(1024), 0, s, jg, jx, jw);
        if ((r = hipGetLastError()) != hipSuccess) return r;
        a.egr = egr;
        a.keep = keep;
        a.egc = egc;
        a.ex = ex;
        a.ew = ew;
        if (p.MW == 2)
            hipLaunchKernelGGL((k_rg_pair<2>), dim3(a.nx + nw), dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_rg_pair<1>), dim3(a.nx + nw), dim3(256), 0, s, a);
    } else {
        hipLaunchKernelGGL(k_rg_gemm, dim3(a.nx + nw), dim3(256), 0, s, a);
    }
    if ((r = hipGetLastError()) != hipSuccess) return r;
    const size_t qx = a.nx && p.sx > 1 ? (size_t)T * H / 4 : 0, qw = dWr && p.sw > 1 ? (size_t)E * H / 4 : 0;
    if (qx + qw) {
        hipLaunchKernelGGL(k_rg_reduce, dim3((unsigned)((qx + qw + 255) / 256)), dim3(256), 0, s,
                           reinterpret_cast<const f4v*>(base + p.px), p.sx, qx, reinterpret_cast<f4v*>(dx), a.acc_x,
                           reinterpret_cast<const f4v*>(base + p.pw), p.sw, qw, reinterpret_cast<f4v*>(dWr), a.acc_w);
        r = hipGetLastError();
    }
    return r;
}

}  // namespace moe

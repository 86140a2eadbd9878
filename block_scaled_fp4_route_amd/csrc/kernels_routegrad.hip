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
#include <stdint.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_learn.h"

namespace moe {

namespace {

constexpr int kTM = 128, kTN = 128, kTK = 32;  // tile of the products

struct RgPlan {
    int Ep;               // columns of G in the workspace (E rounded up to kTK, zero-padded)
    int mt, nt;           // dx: row tiles; both: column tiles
    int et;               // dWr: row tiles
    int sx, sw;           // parts of the long axis of dx (over E) and dWr (over T)
    int kx, kw;           // its length in a part (multiples of kTK)
    size_t g, px, pw, total;
};

RgPlan rg_plan(int H, int E, int T) {
    RgPlan p;
    p.Ep = (E + kTK - 1) / kTK * kTK;
    p.mt = (T + kTM - 1) / kTM;
    p.nt = (H + kTN - 1) / kTN;
    p.et = (E + kTM - 1) / kTM;
    // parts until two workgroups per compute unit have work, at least two
    // steps each, and none much longer than the other product's
    auto split = [](int64_t tiles, int64_t len, int& parts, int& per) {
        parts = 1;
        per = kTK;
        if (tiles < 1 || len < 1) return;  // no tokens
        int64_t n = (512 + tiles - 1) / tiles;
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
    p.px = take(p.sx > 1 ? (size_t)p.sx * T * H * 4 : 0);
    p.pw = take(p.sw > 1 ? (size_t)p.sw * E * H * 4 : 0);
    p.total = o;
    return p;
}

// grid ceil(T / 4), 256 threads: one wave per token; lane owns columns
// lane + 64 i (i < NV).
template <int NV>
__global__ __launch_bounds__(256) void k_rg_logits(const float* __restrict__ din, const int32_t* __restrict__ idx,
                                                   const float* __restrict__ w, const float* __restrict__ dw,
                                                   const uint8_t* __restrict__ mask, int T, int E, int Ep, int k,
                                                   float* __restrict__ G, float* dout) {
    const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + wave_id();
    if (t >= T) return;
    float v[NV];
    const bool on = !mask || mask[t];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int e = lane + 64 * i;
        v[i] = on && din && e < E ? din[(size_t)t * E + e] : 0.0f;
    }
    if (on && dw) {
        const bool live = lane < k;
        const int me = live ? idx[(size_t)t * k + lane] : 0;
        const float mw = live ? w[(size_t)t * k + lane] : 0.0f;
        const float md = live ? dw[(size_t)t * k + lane] : 0.0f;
        const float dot = wave_sum(live ? mw * md : 0.0f);
        const float ds = live ? mw * (md - dot) : 0.0f;
        const bool bad = __ballot(live && (unsigned)me >= (unsigned)E) != 0;
        for (int j = 0; j < k; j++) {  // in increasing j, so an expert named twice adds in that order
            const int e = __builtin_amdgcn_readlane(me, j);
            const float d = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ds), j));
#pragma unroll
            for (int i = 0; i < NV; i++) v[i] += lane + 64 * i == e ? d : 0.0f;
        }
        if (bad)
#pragma unroll
            for (int i = 0; i < NV; i++) v[i] = __builtin_nanf("");
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int e = lane + 64 * i;
        if (e < Ep) G[(size_t)t * Ep + e] = e < E ? v[i] : 0.0f;
        if (dout && e < E) dout[(size_t)t * E + e] = v[i];
    }
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
    if (T > 0) {
        const dim3 grid((T + 3) / 4), block(256);
#define RL(NV)                                                                                                     \
    hipLaunchKernelGGL((k_rg_logits<NV>), grid, block, 0, s, dlogits_in, idx, w, dw, mask, T, E, p.Ep, k, G, dlogits_out)
        if (p.Ep <= 256) RL(4); else if (p.Ep <= 512) RL(8); else RL(16);
#undef RL
        if ((r = hipGetLastError()) != hipSuccess) return r;
    }
    RgArgs a = {G, p.Ep, Wr, x, mask, T, E, H, nullptr, nullptr, accumulate & 1, (accumulate >> 1) & 1,
                p.sx, p.sw, p.kx, p.kw, p.mt, p.nt, p.et, 0};
    a.dx = p.sx > 1 ? reinterpret_cast<float*>(base + p.px) : dx;
    a.dWr = p.sw > 1 ? reinterpret_cast<float*>(base + p.pw) : dWr;
    a.nx = dx && T > 0 ? p.mt * p.nt * p.sx : 0;
    const int nw = dWr ? p.et * p.nt * p.sw : 0;
    if (a.nx + nw == 0) return hipSuccess;
    hipLaunchKernelGGL(k_rg_gemm, dim3(a.nx + nw), dim3(256), 0, s, a);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    const size_t ex = dx && p.sx > 1 ? (size_t)T * H / 4 : 0, ew = dWr && p.sw > 1 ? (size_t)E * H / 4 : 0;
    if (ex + ew) {
        hipLaunchKernelGGL(k_rg_reduce, dim3((unsigned)((ex + ew + 255) / 256)), dim3(256), 0, s,
                           reinterpret_cast<const f4v*>(base + p.px), p.sx, ex, reinterpret_cast<f4v*>(dx), a.acc_x,
                           reinterpret_cast<const f4v*>(base + p.pw), p.sw, ew, reinterpret_cast<f4v*>(dWr), a.acc_w);
        r = hipGetLastError();
    }
    return r;
}

}  // namespace moe

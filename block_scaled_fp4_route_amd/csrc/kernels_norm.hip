// The norms around a block (gfx950): behind it, its output's RMS norm times the
// gate and the residual scale onto the residual stream, and the RMS norm of the
// sum for the next block, in one pass over memory; and the gradients of both.
//
//   q = y rs_y,  rs_y = 1 / sqrt(mean(y^2) + eps)
//   s = r + scale g (q post),  r' = s rounded to the stream's type
//   x = s rs_s pre,            rs_s = 1 / sqrt(mean(s^2) + eps)
// Backward, from r' as stored (n = r' rs, rs from r'):
//   a = dx pre,  d = dr' + rs (a - n mean(a n)),   dr = d
//   dpre = sum_t dx n;  u = scale g d;  dpost = sum_t u q
//   dgate = scale sum d q post over what the gate is broadcast along
//   b = u post,  dy = rs_y (b - q mean(b q))
//
// Memory bounds both: every row is held in registers between its sums and its
// outputs, so each value is read once and written once. A workgroup of 256
// threads takes a row at a time; the sums over the tokens are kept in registers
// by workgroups that run through rows, written out as one partial row for each
// and added in a fixed order by a second launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_rows.h"
#include "moe_serve.h"

namespace moe {
namespace {

// Loads and stores of eight elements in a type known at run time (uniform).
__device__ __forceinline__ void get8(int dt, const void* row, size_t at, float (&v)[8]) {
    if (dt == kActF32) unpack8<kActF32>(load8<kActF32>(row, at), v);
    else if (dt == kActBf16) unpack8<kActBf16>(load8<kActBf16>(row, at), v);
    else unpack8<kActF16>(load8<kActF16>(row, at), v);
}
__device__ __forceinline__ void put8(int dt, void* row, size_t at, const float (&v)[8]) {
    if (dt == kActF32) store8<kActF32>(row, at, pack8<kActF32>(v));
    else if (dt == kActBf16) store8<kActBf16>(row, at, pack8<kActBf16>(v));
    else store8<kActF16>(row, at, pack8<kActF16>(v));
}
__device__ __forceinline__ size_t es(int dt) { return dt == kActF32 ? 4 : 2; }

// Sum over the workgroup's 256 threads, in a fixed order, for everybody. The
// caller alternates between two places so that one barrier a sum is enough.
__device__ __forceinline__ float block_sum(float v, float* place) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) place[wave_id()] = v;
    __syncthreads();
    return (place[0] + place[1]) + (place[2] + place[3]);
}

// NI: pieces of 8 channels a thread, H <= 2048 NI.
template <int NI>
__global__ __launch_bounds__(256) void k_norm_fwd(NormArgs a) {
    __shared__ float red[2][4];
    const int t = blockIdx.x, tid = threadIdx.x, n8 = a.H / 8;
    if (a.mask && !a.mask[t]) return;
    const float inv = 1.0f / (float)a.H;
    const char* r = static_cast<const char*>(a.r) + (size_t)t * a.ldr * es(a.rt);
    float s[NI][8], y[NI][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = tid + 256 * i;
        if (c < n8) {
            get8(a.rt, r, 8 * (size_t)c, s[i]);
            if (a.y) {
                get8(a.yt, static_cast<const char*>(a.y) + (size_t)t * a.ldy * es(a.yt), 8 * (size_t)c, y[i]);
#pragma unroll
                for (int j = 0; j < 8; j++) sum = fmaf(y[i][j], y[i][j], sum);
            }
        }
    }
    if (a.y) {
        const float rs = a.post ? 1.0f / sqrtf(block_sum(sum, red[0]) * inv + a.eps) : 1.0f;
        const float gt = a.scale * (a.gate_kind == kGateToken ? a.gate[t] : 1.0f);
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int c = tid + 256 * i;
            if (c < n8) {
                float w[8], g[8];
                if (a.post) get8(kActF32, a.post, 8 * (size_t)c, w);
                if (a.gate_kind == kGateChannel) get8(kActF32, a.gate, 8 * (size_t)c, g);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    float v = y[i][j] * rs;
                    if (a.post) v *= w[j];
                    s[i][j] = fmaf(a.gate_kind == kGateChannel ? gt * g[j] : gt, v, s[i][j]);
                }
            }
        }
    }
    sum = 0.0f;
    char* ro = static_cast<char*>(a.r_out) + (size_t)t * a.ldro * es(a.rt);
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = tid + 256 * i;
        if (c < n8) {
            if (a.r_out) put8(a.rt, ro, 8 * (size_t)c, s[i]);
#pragma unroll
            for (int j = 0; j < 8; j++) sum = fmaf(s[i][j], s[i][j], sum);
        }
    }
    if (!a.pre) return;
    const float rs = 1.0f / sqrtf(block_sum(sum, red[1]) * inv + a.eps);
    char* x = static_cast<char*>(a.x) + (size_t)t * a.ldx * es(a.xt);
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = tid + 256 * i;
        if (c < n8) {
            float w[8];
            get8(kActF32, a.pre, 8 * (size_t)c, w);
#pragma unroll
            for (int j = 0; j < 8; j++) w[j] *= s[i][j] * rs;
            put8(a.xt, x, 8 * (size_t)c, w);
        }
    }
}

// Workgroups of the backward pass: each runs through the rows t, t + n, ...
int norm_groups(int T) { return T < 512 ? T : 512; }

// part: [3][groups][H] sums of dpost, dpre, dgate (channel).
template <int NI>
__global__ __launch_bounds__(256) void k_norm_bwd(NormArgs a, float* __restrict__ part) {
    __shared__ float red[4][4];
    const int tid = threadIdx.x, n8 = a.H / 8, groups = gridDim.x;
    const float inv = 1.0f / (float)a.H;
    float spost[NI][8], spre[NI][8], sgate[NI][8];
#pragma unroll
    for (int i = 0; i < NI; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) spost[i][j] = spre[i][j] = sgate[i][j] = 0.0f;
    for (int t = blockIdx.x; t < a.T; t += groups) {
        const bool on = !a.mask || a.mask[t];
        char* dr = a.dr ? static_cast<char*>(a.dr) + (size_t)t * a.lddr * es(a.rt) : nullptr;
        char* dy = a.dy ? static_cast<char*>(a.dy) + (size_t)t * a.lddy * es(a.yt) : nullptr;
        if (!on) {
            const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < NI; i++) {
                const int c = tid + 256 * i;
                if (c < n8) {
                    if (dr) put8(a.rt, dr, 8 * (size_t)c, z);
                    if (dy) put8(a.yt, dy, 8 * (size_t)c, z);
                }
            }
            if (a.gate_kind == kGateToken && a.dgate && tid == 0 && !a.accumulate) a.dgate[t] = 0.0f;
            continue;
        }
        float d[NI][8], y[NI][8];
        {
            float r[NI][8], av[NI][8];
            float sr = 0.0f, sar = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; i++) {
                const int c = tid + 256 * i;
                if (c < n8) {
                    if (a.dr_out) get8(a.rt, static_cast<const char*>(a.dr_out) + (size_t)t * a.lddro * es(a.rt), 8 * (size_t)c, d[i]);
                    else
#pragma unroll
                        for (int j = 0; j < 8; j++) d[i][j] = 0.0f;
                    if (a.dx) {
                        float w[8];
                        get8(a.rt, static_cast<const char*>(a.r) + (size_t)t * a.ldr * es(a.rt), 8 * (size_t)c, r[i]);
                        get8(a.xt, static_cast<const char*>(a.dx) + (size_t)t * a.lddx * es(a.xt), 8 * (size_t)c, av[i]);
                        get8(kActF32, a.pre, 8 * (size_t)c, w);
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            sr = fmaf(r[i][j], r[i][j], sr);
                            sar = fmaf(av[i][j] * w[j], r[i][j], sar);
                        }
                    }
                }
            }
            if (a.dx) {
                const float rs = 1.0f / sqrtf(block_sum(sr, red[0]) * inv + a.eps);
                const float m = block_sum(sar, red[1]) * rs * inv;
#pragma unroll
                for (int i = 0; i < NI; i++) {
                    const int c = tid + 256 * i;
                    if (c < n8) {
                        float w[8];
                        get8(kActF32, a.pre, 8 * (size_t)c, w);
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            const float n = r[i][j] * rs;
                            spre[i][j] = fmaf(av[i][j], n, spre[i][j]);
                            d[i][j] = fmaf(rs, fmaf(-n, m, av[i][j] * w[j]), d[i][j]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NI; i++)
            if (dr && tid + 256 * i < n8) put8(a.rt, dr, 8 * (size_t)(tid + 256 * i), d[i]);
        if (!a.y) {
            __syncthreads();  // red is free again
            continue;
        }
        float sy = 0.0f, sg = 0.0f, sby = 0.0f;
        const float gt = a.scale * (a.gate_kind == kGateToken ? a.gate[t] : 1.0f);
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int c = tid + 256 * i;
            if (c < n8) {
                get8(a.yt, static_cast<const char*>(a.y) + (size_t)t * a.ldy * es(a.yt), 8 * (size_t)c, y[i]);
                float w[8], g[8];
                if (a.post) get8(kActF32, a.post, 8 * (size_t)c, w);
                if (a.gate_kind == kGateChannel) get8(kActF32, a.gate, 8 * (size_t)c, g);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float p = a.post ? w[j] : 1.0f;
                    sy = fmaf(y[i][j], y[i][j], sy);
                    sg = fmaf(d[i][j] * p, y[i][j], sg);
                    sby = fmaf(d[i][j] * p * (a.gate_kind == kGateChannel ? g[j] : 1.0f), y[i][j], sby);
                }
            }
        }
        const float rs = a.post ? 1.0f / sqrtf(block_sum(sy, red[2]) * inv + a.eps) : 1.0f;
        const float m = a.post ? block_sum(sby, red[3]) * gt * rs * inv : 0.0f;
        if (a.gate_kind == kGateToken && a.dgate) {
            const float v = block_sum(sg, red[0]) * rs * a.scale;
            if (tid == 0) a.dgate[t] = a.accumulate ? a.dgate[t] + v : v;
        }
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int c = tid + 256 * i;
            if (c < n8) {
                float w[8], g[8], o[8];
                if (a.post) get8(kActF32, a.post, 8 * (size_t)c, w);
                if (a.gate_kind == kGateChannel) get8(kActF32, a.gate, 8 * (size_t)c, g);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float p = a.post ? w[j] : 1.0f, q = y[i][j] * rs;
                    const float u = (a.gate_kind == kGateChannel ? gt * g[j] : gt) * d[i][j];
                    spost[i][j] = fmaf(u, q, spost[i][j]);
                    if (a.gate_kind == kGateChannel) sgate[i][j] = fmaf(d[i][j] * p, q, sgate[i][j]);
                    o[j] = a.post ? rs * fmaf(-q, m, u * p) : u;
                }
                if (dy) put8(a.yt, dy, 8 * (size_t)c, o);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int c = tid + 256 * i;
        if (c < n8) {
            const size_t at = (size_t)blockIdx.x * a.H, all = (size_t)groups * a.H;
            put8(kActF32, part + at, 8 * (size_t)c, spost[i]);
            put8(kActF32, part + all + at, 8 * (size_t)c, spre[i]);
#pragma unroll
            for (int j = 0; j < 8; j++) sgate[i][j] *= a.scale;
            put8(kActF32, part + 2 * all + at, 8 * (size_t)c, sgate[i]);
        }
    }
}

// The partial rows of one output (blockIdx.y) added in order.
__global__ __launch_bounds__(256) void k_norm_sum(const float* __restrict__ part, int groups, int H, float* dpost,
                                                  float* dpre, float* dgate, int accumulate) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    float* out = blockIdx.y == 0 ? dpost : blockIdx.y == 1 ? dpre : dgate;
    if (c >= H || !out) return;
    const float* p = part + (size_t)blockIdx.y * groups * H + c;
    float v = 0.0f;
    for (int g = 0; g < groups; g++) v += p[(size_t)g * H];
    out[c] = accumulate ? out[c] + v : v;
}

}  // namespace

size_t norm_ws_bytes(int H, int gate_kind, int T) { return align256((size_t)3 * norm_groups(T) * H * sizeof(float)); }

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
    const int ni = (a.H + 2047) / 2048;
    const dim3 grid(a.T), block(256);
    if (ni <= 1) hipLaunchKernelGGL(k_norm_fwd<1>, grid, block, 0, s, a);
    else if (ni <= 2) hipLaunchKernelGGL(k_norm_fwd<2>, grid, block, 0, s, a);
    else if (ni <= 4) hipLaunchKernelGGL(k_norm_fwd<4>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_norm_fwd<8>, grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_block_norm_backward(const NormArgs& a, void* ws, hipStream_t s) {
    const int ni = (a.H + 2047) / 2048, groups = norm_groups(a.T);
    const dim3 grid(groups), block(256);
    float* part = static_cast<float*>(ws);
    if (groups) {
        if (ni <= 1) hipLaunchKernelGGL(k_norm_bwd<1>, grid, block, 0, s, a, part);
        else if (ni <= 2) hipLaunchKernelGGL(k_norm_bwd<2>, grid, block, 0, s, a, part);
        else if (ni <= 4) hipLaunchKernelGGL(k_norm_bwd<4>, grid, block, 0, s, a, part);
        else hipLaunchKernelGGL(k_norm_bwd<8>, grid, block, 0, s, a, part);
        const hipError_t r = hipGetLastError();
        if (r != hipSuccess) return r;
    }
    float* dg = a.gate_kind == kGateChannel ? a.dgate : nullptr;
    if (a.dpost || a.dpre || dg)
        hipLaunchKernelGGL(k_norm_sum, dim3((a.H + 255) / 256, 3), block, 0, s, part, groups, a.H, a.dpost, a.dpre, dg,
                           a.accumulate);
    return hipGetLastError();
}

}  // namespace moe

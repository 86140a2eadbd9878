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
// outputs, so each value is read once and written once. A workgroup takes a row
// at a time; the sums over the tokens are kept in registers by workgroups that
// run through rows, written out as one partial row for each and added in a
// fixed order by a second launch. 8191 x 4096 bf16: forward 61 us, 4.4 TB/s,
// backward 92-95 + 6, 4.2 TB/s (both slower with the next row's loads on their way
// while a row is worked through).
//
// In the backward pass that holds up to 4096 channels. Above, a workgroup has 1024
// threads of 128 registers: up to 8192 channels any fp32 side leaves 20 to 56
// bytes a lane in scratch memory, from there on all types 444 to 536. The same
// bytes as 8192 x 4096 bf16 (97 us) take 116 at 4096 x 8192 and 536 at 2048 x
// 16384; in fp32 4096 x 4096 takes 94, 2048 x 8192 133, 1024 x 16384 363.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_rows.h"
#include "moe_serve.h"

namespace moe {
namespace {

// Eight elements of a row whose type's size S is known at compile time (the
// loads of a row go out together and are waited for once) and whose kind, of
// the 16-bit ones, at run time.
template <int S>
struct Piece {
    u4w w[S / 2];
};
template <int S>
__device__ __forceinline__ void fetch(Piece<S>& p, const void* row, uint32_t c) {
    const u4w* q = reinterpret_cast<const u4w*>(row) + (size_t)c * (S / 2);
#pragma unroll
    for (int i = 0; i < S / 2; i++) p.w[i] = q[i];
}
template <int S>
__device__ __forceinline__ void widen(const Piece<S>& p, int dt, float (&v)[8]) {
    if constexpr (S == 4) {
        unpack8<kActF32>(Raw8<kActF32>{{p.w[0], p.w[1]}}, v);
    } else {
        if (dt == kActBf16) unpack8<kActBf16>(Raw8<kActBf16>{{p.w[0]}}, v);
        else unpack8<kActF16>(Raw8<kActF16>{{p.w[0]}}, v);
    }
}
template <int S>
__device__ __forceinline__ void put(int dt, void* row, uint32_t c, const float (&v)[8]) {
    if constexpr (S == 4) store8<kActF32>(row, 8 * (size_t)c, pack8<kActF32>(v));
    else store8<kActBf16>(row, 8 * (size_t)c, dt == kActBf16 ? pack8<kActBf16>(v) : Raw8<kActBf16>{{pack8<kActF16>(v).w[0]}});
}
template <int S>
__device__ __forceinline__ auto row_of(const void* p, size_t ld, size_t t) {
    return static_cast<const char*>(p) + t * ld * S;
}

// Sums over the workgroup's threads, in a fixed order, for everybody.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*place)[16]) {
#pragma unroll
    for (int n = 0; n < N; n++) v[n] = wave_sum(v[n]);
    const int waves = blockDim.x >> 6;
    if (waves == 1) return;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int n = 0; n < N; n++) place[n][wave_id()] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; n++) {
        float s = 0.0f;
        for (int w = 0; w < waves; w++) s += place[n][w];
        v[n] = s;
    }
}
__device__ __forceinline__ float rms_inv(float sum, const NormArgs& a) { return 1.0f / sqrtf(sum * (1.0f / (float)a.H) + a.eps); }

// A workgroup a row. NI: pieces of 8 channels a thread (H <= 8 NI threads).
template <int SR, int SY, int SX, int NI, int NT>
__global__ __launch_bounds__(NT) void k_norm_fwd(NormArgs a) {
    __shared__ float red[2][1][16];
    const uint32_t t = blockIdx.x, n8 = a.H / 8;
    if (a.mask && !a.mask[t]) return;
    uint32_t c[NI];
    Piece<SR> pr[NI];
    Piece<SY> py[NI];
    Piece<4> wpost[NI], wgate[NI], wpre[NI];
    const bool ch = a.gate_kind == kGateChannel && a.y;
#pragma unroll
    for (int i = 0; i < NI; i++) {
        c[i] = threadIdx.x + blockDim.x * i;
        const uint32_t l = min(c[i], n8 - 1);
        fetch<SR>(pr[i], row_of<SR>(a.r, a.ldr, t), l);
        if (a.y) fetch<SY>(py[i], row_of<SY>(a.y, a.ldy, t), l);
        if (a.post) fetch<4>(wpost[i], a.post, l);
        if (ch) fetch<4>(wgate[i], a.gate, l);
        if (a.pre) fetch<4>(wpre[i], a.pre, l);
    }
    const float gt = a.scale * (a.y && a.gate_kind == kGateToken ? a.gate[t] : 1.0f);
    float s[NI][8];
#pragma unroll
    for (int i = 0; i < NI; i++) widen<SR>(pr[i], a.rt, s[i]);
    if (a.y) {
        float y[NI][8], sum[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NI; i++) {
            widen<SY>(py[i], a.yt, y[i]);
            if (c[i] < n8)
#pragma unroll
                for (int j = 0; j < 8; j++) sum[0] = fmaf(y[i][j], y[i][j], sum[0]);
        }
        float rs = 1.0f;
        if (a.post) {
            block_sums(sum, red[0]);
            rs = rms_inv(sum[0], a);
        }
#pragma unroll
        for (int i = 0; i < NI; i++) {
            float w[8], g[8];
            if (a.post) widen<4>(wpost[i], kActF32, w);
            if (ch) widen<4>(wgate[i], kActF32, g);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                float v = y[i][j] * rs;
                if (a.post) v *= w[j];
                s[i][j] = fmaf(ch ? gt * g[j] : gt, v, s[i][j]);
            }
        }
    }
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NI; i++)
        if (c[i] < n8) {
            if (a.r_out) put<SR>(a.rt, const_cast<char*>(row_of<SR>(a.r_out, a.ldro, t)), c[i], s[i]);
#pragma unroll
            for (int j = 0; j < 8; j++) sum[0] = fmaf(s[i][j], s[i][j], sum[0]);
        }
    if (!a.pre) return;
    block_sums(sum, red[1]);
    const float rs = rms_inv(sum[0], a);
#pragma unroll
    for (int i = 0; i < NI; i++)
        if (c[i] < n8) {
            float w[8];
            widen<4>(wpre[i], kActF32, w);
#pragma unroll
            for (int j = 0; j < 8; j++) w[j] *= s[i][j] * rs;
            put<SX>(a.xt, const_cast<char*>(row_of<SX>(a.x, a.ldx, t)), c[i], w);
        }
}

// part: [3][groups][H] sums of dpost, dpre, dgate (channel).
template <int SR, int SY, int SX, int NI, int NT>
__global__ __launch_bounds__(NT) void k_norm_bwd(NormArgs a, float* __restrict__ part) {
    __shared__ float red[2][3][16];
    const uint32_t n8 = a.H / 8, groups = gridDim.x;
    const float inv = 1.0f / (float)a.H;
    const bool ch = a.gate_kind == kGateChannel && a.y, tok = a.gate_kind == kGateToken && a.y;
    uint32_t c[NI], l[NI];
    float spost[NI][8], spre[NI][8], sgate[NI][8];
    struct Row {
        Piece<SR> r[NI], dro[NI];
        Piece<SX> dx[NI];
        Piece<SY> y[NI];
        float gate;
        bool on;
    };
#pragma unroll
    for (int i = 0; i < NI; i++) {
        c[i] = threadIdx.x + blockDim.x * i;
        l[i] = min(c[i], n8 - 1);
#pragma unroll
        for (int j = 0; j < 8; j++) spost[i][j] = spre[i][j] = sgate[i][j] = 0.0f;
    }
    Piece<4> wpre[NI], wpost[NI], wgate[NI];
    auto weights = [&]() {
#pragma unroll
        for (int i = 0; i < NI; i++) {
            if (a.dx) fetch<4>(wpre[i], a.pre, l[i]);
            if (a.post) fetch<4>(wpost[i], a.post, l[i]);
            if (ch) fetch<4>(wgate[i], a.gate, l[i]);
        }
    };
    auto start = [&](uint32_t t, Row& q) {
        q.on = !a.mask || a.mask[t];
        q.gate = tok ? a.gate[t] : 1.0f;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            if (a.dx) {
                fetch<SR>(q.r[i], row_of<SR>(a.r, a.ldr, t), l[i]);
                fetch<SX>(q.dx[i], row_of<SX>(a.dx, a.lddx, t), l[i]);
            }
            if (a.dr_out) fetch<SR>(q.dro[i], row_of<SR>(a.dr_out, a.lddro, t), l[i]);
            if (a.y) fetch<SY>(q.y[i], row_of<SY>(a.y, a.ldy, t), l[i]);
        }
    };
    auto work = [&](uint32_t t, const Row& q) {
        void* dr = a.dr ? const_cast<char*>(row_of<SR>(a.dr, a.lddr, t)) : nullptr;
        void* dy = a.dy ? const_cast<char*>(row_of<SY>(a.dy, a.lddy, t)) : nullptr;
        if (!q.on) {
            const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < NI; i++)
                if (c[i] < n8) {
                    if (dr) put<SR>(a.rt, dr, c[i], z);
                    if (dy) put<SY>(a.yt, dy, c[i], z);
                }
            if (tok && a.dgate && threadIdx.x == 0 && !a.accumulate) a.dgate[t] = 0.0f;
            return;
        }
        if (NI > 1) weights();
        float s[3] = {0.0f, 0.0f, 0.0f};  // r^2, dx pre r, y^2
        float d[NI][8], y[NI][8], r[NI][8], av[NI][8];
#pragma unroll
        for (int i = 0; i < NI; i++) {
            if (a.dx) {
                float w[8];
                widen<SR>(q.r[i], a.rt, r[i]);
                widen<SX>(q.dx[i], a.xt, av[i]);
                widen<4>(wpre[i], kActF32, w);
                if (c[i] < n8)
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        s[0] = fmaf(r[i][j], r[i][j], s[0]);
                        s[1] = fmaf(av[i][j] * w[j], r[i][j], s[1]);
                    }
            }
            if (a.dr_out) widen<SR>(q.dro[i], a.rt, d[i]);
            else
#pragma unroll
                for (int j = 0; j < 8; j++) d[i][j] = 0.0f;
            if (a.y) {
                widen<SY>(q.y[i], a.yt, y[i]);
                if (c[i] < n8)
#pragma unroll
                    for (int j = 0; j < 8; j++) s[2] = fmaf(y[i][j], y[i][j], s[2]);
            }
        }
        block_sums(s, red[0]);
        if (a.dx) {
            const float rs = rms_inv(s[0], a), m = s[1] * rs * inv;
#pragma unroll
            for (int i = 0; i < NI; i++) {
                float w[8];
                widen<4>(wpre[i], kActF32, w);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float n = r[i][j] * rs;
                    spre[i][j] = fmaf(av[i][j], n, spre[i][j]);
                    d[i][j] = fmaf(rs, fmaf(-n, m, av[i][j] * w[j]), d[i][j]);
                }
            }
        }
        if (dr) {
#pragma unroll
            for (int i = 0; i < NI; i++)
                if (c[i] < n8) put<SR>(a.rt, dr, c[i], d[i]);
        }
        if (!a.y) return;
        const float rs = a.post ? rms_inv(s[2], a) : 1.0f, gt = a.scale * q.gate;
        float b[2] = {0.0f, 0.0f};  // d post y, and times the channel's gate
#pragma unroll
        for (int i = 0; i < NI; i++) {
            float w[8], g[8];
            if (a.post) widen<4>(wpost[i], kActF32, w);
            if (ch) widen<4>(wgate[i], kActF32, g);
            if (c[i] < n8)
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float v = a.post ? d[i][j] * w[j] : d[i][j];
                    b[0] = fmaf(v, y[i][j], b[0]);
                    if (ch) b[1] = fmaf(v * g[j], y[i][j], b[1]);
                }
        }
        if (a.post || tok) block_sums(b, red[1]);
        const float m = a.post ? (ch ? b[1] : b[0]) * gt * rs * inv : 0.0f;
        if (tok && a.dgate && threadIdx.x == 0) {
            const float v = b[0] * rs * a.scale;
            a.dgate[t] = a.accumulate ? a.dgate[t] + v : v;
        }
#pragma unroll
        for (int i = 0; i < NI; i++) {
            float w[8], g[8], o[8];
            if (a.post) widen<4>(wpost[i], kActF32, w);
            if (ch) widen<4>(wgate[i], kActF32, g);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float p = a.post ? w[j] : 1.0f, n = y[i][j] * rs;
                const float u = (ch ? gt * g[j] : gt) * d[i][j];
                spost[i][j] = fmaf(u, n, spost[i][j]);
                if (ch) sgate[i][j] = fmaf(d[i][j] * p, n, sgate[i][j]);
                o[j] = a.post ? rs * fmaf(-n, m, u * p) : u;
            }
            if (dy && c[i] < n8) put<SY>(a.yt, dy, c[i], o);
        }
    };
    if (NI == 1) weights();
    const uint32_t T = a.T;
    for (uint32_t t = blockIdx.x; t < T; t += groups) {
        Row q;
        start(t, q);
        work(t, q);
        __syncthreads();  // red is free again
    }
#pragma unroll
    for (int i = 0; i < NI; i++)
        if (c[i] < n8) {
            const size_t at = (size_t)blockIdx.x * a.H, all = (size_t)groups * a.H;
            if (a.dpost) store8<kActF32>(part + at, 8 * (size_t)c[i], pack8<kActF32>(spost[i]));
            if (a.dpre) store8<kActF32>(part + all + at, 8 * (size_t)c[i], pack8<kActF32>(spre[i]));
            if (ch && a.dgate) {
#pragma unroll
                for (int j = 0; j < 8; j++) sgate[i][j] *= a.scale;
                store8<kActF32>(part + 2 * all + at, 8 * (size_t)c[i], pack8<kActF32>(sgate[i]));
            }
        }
}

// The partial rows of one output (blockIdx.y), added in a fixed order: 16
// slices of consecutive rows, 16 quads of channels a workgroup, then the slices.
__global__ __launch_bounds__(256) void k_norm_sum(const float* __restrict__ part, int groups, int H, float* dpost,
                                                  float* dpre, float* dgate, int accumulate) {
    __shared__ f4v slice[16][16];
    float* out = blockIdx.y == 0 ? dpost : blockIdx.y == 1 ? dpre : dgate;
    if (!out) return;
    const int q = threadIdx.x & 15, sl = threadIdx.x >> 4, col = blockIdx.x * 16 + q, per = (groups + 15) / 16;
    const int g0 = min(groups, sl * per), g1 = min(groups, g0 + per);
    f4v v = {0.f, 0.f, 0.f, 0.f};
    if (col < H / 4) {
        const f4v* p = reinterpret_cast<const f4v*>(part + (size_t)blockIdx.y * groups * H) + col;
#pragma unroll 8
        for (int g = g0; g < g1; g++) v += p[(size_t)g * (H / 4)];
    }
    slice[sl][q] = v;
    __syncthreads();
    if (sl == 0 && col < H / 4) {
        for (int i = 1; i < 16; i++) v += slice[i][q];
        f4v* o = reinterpret_cast<f4v*>(out) + col;
        *o = accumulate ? *o + v : v;
    }
}

// Threads of a row and pieces of each: 64 to 1024 threads with one piece of 8
// channels (a short row leaves no lanes idle, the sums over tokens take 24
// registers a thread and the weights stay in as many), two above 8192 channels.
struct NormShape {
    int threads, ni;
};
NormShape norm_shape(int H) {
    int t = 64;
    while (t < 1024 && 8 * t < H) t *= 2;
    return {t, 8 * t < H ? 2 : 1};
}

// Workgroups of the backward pass: each runs through the rows t, t + n, ...
// Two of 512 threads a compute unit fill the chip; shorter rows take more
// workgroups, as long as each has 8 rows (a workgroup leaves three rows of fp32
// sums).
int norm_groups(int H, int T) {
    const int most = 512 * 512 / norm_shape(H).threads;
    int n = T / 8 < most ? T / 8 : most;
    n = n > 512 ? n : 512;
    return T < n ? T : n;
}

template <int SR, int SY, int SX>
hipError_t norm_launch(const NormArgs& a, float* part, hipStream_t s) {
    const NormShape n = norm_shape(a.H);
    const dim3 block(n.threads);
    if (!part) {
        const dim3 grid(a.T);
        if (n.ni == 2) hipLaunchKernelGGL((k_norm_fwd<SR, SY, SX, 2, 1024>), grid, block, 0, s, a);
        else if (n.threads == 1024) hipLaunchKernelGGL((k_norm_fwd<SR, SY, SX, 1, 1024>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_norm_fwd<SR, SY, SX, 1, 512>), grid, block, 0, s, a);
    } else {
        const dim3 grid(norm_groups(a.H, a.T));
        if (n.ni == 2) hipLaunchKernelGGL((k_norm_bwd<SR, SY, SX, 2, 1024>), grid, block, 0, s, a, part);
        else if (n.threads == 1024) hipLaunchKernelGGL((k_norm_bwd<SR, SY, SX, 1, 1024>), grid, block, 0, s, a, part);
        else hipLaunchKernelGGL((k_norm_bwd<SR, SY, SX, 1, 512>), grid, block, 0, s, a, part);
    }
    return hipGetLastError();
}
hipError_t norm_types(const NormArgs& a, float* part, hipStream_t s) {
    const int k = (a.rt == kActF32) * 4 + (a.yt == kActF32) * 2 + (a.xt == kActF32);
    switch (k) {
        case 0: return norm_launch<2, 2, 2>(a, part, s);
        case 1: return norm_launch<2, 2, 4>(a, part, s);
        case 2: return norm_launch<2, 4, 2>(a, part, s);
        case 3: return norm_launch<2, 4, 4>(a, part, s);
        case 4: return norm_launch<4, 2, 2>(a, part, s);
        case 5: return norm_launch<4, 2, 4>(a, part, s);
        case 6: return norm_launch<4, 4, 2>(a, part, s);
        default: return norm_launch<4, 4, 4>(a, part, s);
    }
}

}  // namespace

size_t norm_ws_bytes(int H, int T) { return kCounterBytes + align256((size_t)3 * norm_groups(H, T) * H * sizeof(float)); }

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) { return norm_types(a, nullptr, s); }

hipError_t launch_block_norm_backward(const NormArgs& a, void* ws, hipStream_t s) {
    const int groups = norm_groups(a.H, a.T);
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + kCounterBytes);
    if (groups) {
        const hipError_t r = norm_types(a, part, s);
        if (r != hipSuccess) return r;
    }
    float* dg = a.gate_kind == kGateChannel ? a.dgate : nullptr;
    if (a.dpost || a.dpre || dg)
        hipLaunchKernelGGL(k_norm_sum, dim3((a.H / 4 + 15) / 16, 3), dim3(256), 0, s, part, groups, a.H, a.dpost, a.dpre, dg,
                           a.accumulate);
    return hipGetLastError();
}

}  // namespace moe

// A whole mixture-of-experts layer for a few tokens (gfx950): T tokens routed,
// each through its k experts (SwiGLU over block-scaled FP4 weights) and the
// bf16 shared expert, in fp32 as the single-token decode has it.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_rows.h"
#include "moe_serve.h"

namespace moe {
namespace {

struct BatchArgs {
    int H, I, E, k, T, slots;  // slots: k, and one more for a shared expert
    const float* x;
    const uint8_t* mask;
    const void* const* ptrs;
    const uint16_t *sg, *su, *sd;
    const int32_t* idx;
    const float* w;
    float* h;  // [T][slots][I]
    float* y;
    int32_t* idx_out;
    float* w_out;
};

// One row of a stored matrix times v, over a wave.
template <int FMT>
__device__ __forceinline__ float row_dot(const uint8_t* codes, const uint8_t* scales, size_t row, int cols, const float* v) {
    const uint32_t* c = reinterpret_cast<const uint32_t*>(codes + row * (cols / 2));
    const uint8_t* s = scales + row * (cols / Fmt<FMT>::G);
    float sum = 0.0f;
    for (int i = threadIdx.x & 63; i < cols / 8; i += 64)
        sum = fmaf(dot8_fp4(c[i], v + 8 * i), scale_to_f32<FMT>(s[i / (Fmt<FMT>::G / 8)]), sum);
    return wave_sum(sum);
}
__device__ __forceinline__ float row_dot_bf16(const uint16_t* m, size_t row, int cols, const float* v) {
    float sum = 0.0f;
    for (int i = threadIdx.x & 63; i < cols / 8; i += 64) {
        float u[8];
        unpack8<kActBf16>(load8<kActBf16>(m, row * cols + 8 * i), u);
#pragma unroll
        for (int j = 0; j < 8; j++) sum = fmaf(u[j], v[8 * i + j], sum);
    }
    return wave_sum(sum);
}

template <int FMT>
__global__ __launch_bounds__(256) void k_batch_gateup(BatchArgs a) {
    const int t = blockIdx.y / a.slots, j = blockIdx.y % a.slots, row = blockIdx.x * 4 + wave_id();
    if (a.mask && !a.mask[t]) return;
    const float* x = a.x + (size_t)t * a.H;
    float g, u;
    if (j < a.k) {
        const uint8_t* b = static_cast<const uint8_t*>(a.ptrs[a.idx[t * a.k + j]]);
        const size_t n = (size_t)a.H * a.I, sc = n / Fmt<FMT>::G;
        g = row_dot<FMT>(b, b + 3 * n / 2, row, a.H, x);
        u = row_dot<FMT>(b + n / 2, b + 3 * n / 2 + sc, row, a.H, x);
    } else {
        g = row_dot_bf16(a.sg, row, a.H, x);
        u = row_dot_bf16(a.su, row, a.H, x);
    }
    if ((threadIdx.x & 63) == 0) a.h[((size_t)t * a.slots + j) * a.I + row] = silu_mul(g, u);
}

template <int FMT>
__global__ __launch_bounds__(256) void k_batch_down(BatchArgs a) {
    const int t = blockIdx.y, row = blockIdx.x * 4 + wave_id(), lane = threadIdx.x & 63;
    if (a.mask && !a.mask[t]) return;
    float y = 0.0f;
    for (int j = 0; j < a.slots; j++) {
        const float* h = a.h + ((size_t)t * a.slots + j) * a.I;
        if (j < a.k) {
            const uint8_t* b = static_cast<const uint8_t*>(a.ptrs[a.idx[t * a.k + j]]);
            const size_t n = (size_t)a.H * a.I, sc = n / Fmt<FMT>::G;
            y = fmaf(a.w[t * a.k + j], row_dot<FMT>(b + n, b + 3 * n / 2 + 2 * sc, row, a.I, h), y);
        } else {
            y += row_dot_bf16(a.sd, row, a.I, h);
        }
    }
    if (lane == 0) a.y[(size_t)t * a.H + row] = y;
    if (row == 0 && lane < a.k) {
        a.idx_out[t * a.k + lane] = a.idx[t * a.k + lane];
        a.w_out[t * a.k + lane] = a.w[t * a.k + lane];
    }
}

}  // namespace

size_t batch_ws_bytes(int fmt, int H, int I, int E, int k, int T) {
    return align256(route_ws_bytes(T, E)) + 2 * align256((size_t)T * k * 4) + align256((size_t)T * (k + 1) * I * 4);
}

hipError_t launch_layer_batch(int fmt, int H, int I, int E, int k, const float* x, int T, const uint8_t* mask,
                              const float* Wr, const void* const* expert_ptrs, const uint16_t* sh_gate,
                              const uint16_t* sh_up, const uint16_t* sh_down, float* y, int32_t* idx_out, float* w_out,
                              void* ws, hipStream_t s) {
    char* p = static_cast<char*>(ws) + align256(route_ws_bytes(T, E));
    int32_t* idx = reinterpret_cast<int32_t*>(p);
    p += align256((size_t)T * k * 4);
    float* w = reinterpret_cast<float*>(p);
    p += align256((size_t)T * k * 4);
    hipError_t r = launch_route(H, E, k, T, x, Wr, idx, w, nullptr, ws, s);
    if (r != hipSuccess) return r;
    const BatchArgs a = {H, I, E, k, T, k + (sh_gate ? 1 : 0), x, mask, expert_ptrs, sh_gate, sh_up, sh_down, idx, w,
                         reinterpret_cast<float*>(p), y, idx_out, w_out};
    const dim3 gu(I / 4, T * a.slots), down(H / 4, T), block(256);
    if (fmt == kFmtNvfp4) hipLaunchKernelGGL(k_batch_gateup<kFmtNvfp4>, gu, block, 0, s, a);
    else hipLaunchKernelGGL(k_batch_gateup<kFmtMxfp4>, gu, block, 0, s, a);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    if (fmt == kFmtNvfp4) hipLaunchKernelGGL(k_batch_down<kFmtNvfp4>, down, block, 0, s, a);
    else hipLaunchKernelGGL(k_batch_down<kFmtMxfp4>, down, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace moe

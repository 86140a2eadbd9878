// Host-side launch entry points of the kernels around a routed layer that
// serves a few tokens: 4-bit quantisation and products, the layer for a few
// tokens, the norms around a block (internal to the library). Each returns
// hipSuccess or the launch error; arguments were validated by the C-ABI layer
// (moe_api.cpp) before these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// ---- quantisation to block-scaled e2m1 ----
constexpr int kRuleNearest = 2;  // NVFP4: the E4M3 value nearest to amax / 6
hipError_t launch_fp4_quant(int dtype, int fmt, int rule, const void* x, size_t ldx, int rows, int cols,
                            int8_t* row_exp, uint8_t* codes, uint8_t* scales, void* values, size_t ldv, hipStream_t s);

// ---- products with a matrix stored in 4 bits ----
constexpr int kFp4MaxDim = 65536;            // K, N
constexpr int kFp4MaxT = 1 << 20;
constexpr int64_t kFp4MaxLd = 1 << 22;       // row strides, so that a tile's offsets fit 31 bits
struct Fp4Matrix {
    const uint8_t* codes;   // [N][K / 2]
    const uint8_t* scales;  // [N][K / G]
    const int8_t* row_exp;  // [N] or null
};
// Up to kGemvMaxT and kFewMaxT tokens (x of the second: the activations, their
// parts, or codes beside x_scales). The border stands for the types that would need
// parts: 4 tokens of 2560 x 8192 in fp32 take 9.1 (MXFP4) and 10.6 us (NVFP4) with
// the vector kernel, 12.8 and 13.6 with the other; fp16 beside MXFP4 9.4 and 10.7.
// Activations that are operands as they are would gain from 2 tokens on: bf16 takes
// 7.5 and 7.0 us at 2, 10.4 and 7.6 at 4, rounded ones 7.4 and 7.4, 10.9 and 7.6.
constexpr int kGemvMaxT = 4, kFewMaxT = 64;
hipError_t launch_fp4_gemv(int K, int N, int fmt, int dtype, const void* x, size_t ldx, int T, const Fp4Matrix& w,
                           bool round_x, const void* base, size_t ldbase, void* y, size_t ldy, hipStream_t s);
hipError_t launch_fp4_few(int K, int N, int fmt, int dtype, const void* x, size_t ldx_bytes, const uint8_t* x_scales, int T,
                          const Fp4Matrix& w, const void* base, size_t ldbase, void* y, size_t ldy, hipStream_t s);
size_t fp4_ws_bytes(int K, int N, int fmt, int dtype, int T, bool backward);
hipError_t launch_fp4_apply(int K, int N, int fmt, int dtype, const void* x, size_t ldx, int T, const Fp4Matrix& w,
                            bool round_x, const void* base, size_t ldbase, void* y, size_t ldy, void* ws,
                            hipStream_t s);
hipError_t launch_fp4_backward(int K, int N, int fmt, int dtype, const void* dy, size_t lddy, int T,
                               const Fp4Matrix& w, const void* dx_base, size_t lddxb, void* dx, size_t lddx, void* ws,
                               hipStream_t s);

// ---- the layer for a few tokens ----
constexpr int kBatchMaxT = 64;
size_t batch_ws_bytes(int fmt, int H, int I, int E, int k, int T);
hipError_t launch_layer_batch(int fmt, int H, int I, int E, int k, const float* x, int T, const uint8_t* mask,
                              const float* Wr, const void* const* expert_ptrs, const uint16_t* sh_gate,
                              const uint16_t* sh_up, const uint16_t* sh_down, float* y, int32_t* idx_out, float* w_out,
                              void* ws, hipStream_t s);

// ---- the norms around a block ----
constexpr int kNormMaxH = 16384;
constexpr int kNormMaxT = 1 << 20;
constexpr int kGateNone = 0, kGateChannel = 1, kGateToken = 2;
struct NormArgs {
    int H, T, rt, yt, xt, gate_kind;  // rt, yt, xt: kAct*
    float scale, eps;
    const void* r;     // forward: the residual stream; backward: the stored sum
    const void* y;
    const uint8_t* mask;
    const float *post, *gate, *pre;
    size_t ldr, ldy;
    void *r_out, *x;   // forward
    size_t ldro, ldx;
    const void *dr_out, *dx;  // backward
    void *dr, *dy;
    size_t lddro, lddx, lddr, lddy;
    float *dpost, *dgate, *dpre;
    int accumulate;
};
size_t norm_ws_bytes(int H, int T);
hipError_t launch_block_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_block_norm_backward(const NormArgs& a, void* ws, hipStream_t s);

}  // namespace moe

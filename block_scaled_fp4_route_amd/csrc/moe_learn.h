// Host-side launch entry points of the kernels that train a routed layer's
// router and carry low-rank adapters beside its projections (internal to the
// library). Each returns hipSuccess or the launch error; arguments were
// validated by the C-ABI layer (moe_api.cpp) before these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// ---- balance loss ----
size_t balance_ws_bytes(int T, int E, int S);
hipError_t launch_balance(int E, int k, const float* logits, int T, const int32_t* idx, const uint8_t* mask,
                          const int32_t* seq_off, int S, float cb, float cz, const float* dloss, float* loss,
                          int32_t* counts, float* probs, float* dlogits, void* ws, hipStream_t s);

// ---- routing gradient ----
size_t route_backward_ws_bytes(int H, int E, int T);
hipError_t launch_route_backward(int H, int E, int k, const float* x, int T, const float* Wr, const int32_t* idx,
                                 const float* w, const float* dw, const uint8_t* mask, const float* dlogits_in,
                                 float* dlogits_out, float* dx, float* dWr, int accumulate, void* ws, hipStream_t s);

// ---- low-rank adapters ----
constexpr int kActF32 = 0, kActBf16 = 1, kActF16 = 2;
constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxN = 1024;       // adapters
constexpr int kLoraMaxDim = 65536;    // K, N
constexpr int kLoraMaxT = 1 << 20;
struct LoraTable {
    const int32_t* ids;
    const void* const* a;
    const void* const* b;
    const int32_t* ranks;
    const float* scales;
};
size_t lora_ws_bytes(int K, int N, int n, int R, int T, bool backward);
hipError_t launch_lora_apply(int dtype, int K, int N, int n, int R, const void* x, size_t ldx, int T,
                             const LoraTable& tab, const void* base, size_t ldbase, void* y, size_t ldy, void* ws,
                             hipStream_t s);
hipError_t launch_lora_backward(int dtype, int K, int N, int n, int R, const void* x, size_t ldx, const void* dy,
                                size_t lddy, int T, const LoraTable& tab, const void* dx_base, size_t lddxb, void* dx,
                                size_t lddx, float* const* da, float* const* db, int accumulate, void* ws,
                                hipStream_t s);

}  // namespace moe

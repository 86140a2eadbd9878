// C ABI of the library (declared in include/moe_fp4.h): argument checks,
// workspace sizing and kernel launches on the caller's stream. No
// allocation, no synchronisation, no device reads on the host.
#include "../../include/moe_fp4.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "moe_internal.h"
#include "moe_learn.h"
#include "moe_serve.h"

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

int ok() {
    g_err[0] = 0;
    return MOE_OK;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int group_size(int fmt) { return fmt == MOE_FMT_NVFP4 ? 16 : (fmt == MOE_FMT_MXFP4 ? 32 : 0); }

int check_desc(const moe_desc* d) {
    if (!d) return fail(MOE_ERR_ARG, "desc is NULL");
    const int G = group_size(d->format);
    if (!G) return fail(MOE_ERR_ARG, "unknown format %d", d->format);
    if (d->H <= 0 || d->I <= 0 || d->E <= 0 || d->k <= 0)
        return fail(MOE_ERR_ARG, "H, I, E, k must be positive (H=%d I=%d E=%d k=%d)", d->H, d->I, d->E, d->k);
    if (d->k > d->E) return fail(MOE_ERR_ARG, "k=%d exceeds E=%d", d->k, d->E);
    if (d->H % G || d->I % G) return fail(MOE_ERR_ARG, "H=%d and I=%d must be multiples of the group size %d", d->H, d->I, G);
    return MOE_OK;
}

int check_ptr(const void* p, size_t align, const char* name) {
    if (!p) return fail(MOE_ERR_ARG, "%s is NULL", name);
    if (!aligned(p, align)) return fail(MOE_ERR_ARG, "%s is not %zu-byte aligned", name, align);
    return MOE_OK;
}

int check_ws(const void* ws, size_t have, size_t need) {
    if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", need);
    if (!aligned(ws, 256)) return fail(MOE_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    if (have < need) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
    return MOE_OK;
}

int hip_status(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
    return ok();
}

}  // namespace

extern "C" {

size_t moe_block_bytes(const moe_desc* d) {
    if (check_desc(d) != MOE_OK) return 0;
    const size_t n = (size_t)3 * d->H * d->I;
    return n / 2 + n / group_size(d->format);
}

int moe_block_layout(const moe_desc* d, int64_t off[7]) {
    int r = check_desc(d);
    if (r) return r;
    if (!off) return fail(MOE_ERR_ARG, "off is NULL");
    const int64_t codes = (int64_t)d->H * d->I / 2, scales = (int64_t)d->H * d->I / group_size(d->format);
    off[0] = 0;
    off[1] = codes;
    off[2] = 2 * codes;
    off[3] = 3 * codes;
    off[4] = 3 * codes + scales;
    off[5] = 3 * codes + 2 * scales;
    off[6] = 3 * codes + 3 * scales;
    return ok();
}

size_t moe_workspace_bytes(const moe_desc* d, int32_t T, int32_t mode) {
    if (check_desc(d) != MOE_OK || T < 0) return 0;
    switch (mode) {
        case MOE_MODE_ROUTE: return moe::route_ws_bytes(T, d->E);
        case MOE_MODE_DECODE: return moe::decode_ws_bytes(d->H, d->I, d->k, d->E);
        case MOE_MODE_PREFILL: return moe::prefill_ws_bytes(d->format, d->H, d->I, d->E, d->k, T);
        case MOE_MODE_DECODE_BATCH: return T > moe::kBatchMaxT ? 0 : moe::batch_ws_bytes(d->format, d->H, d->I, d->E, d->k, T);
        default: return 0;
    }
}

int moe_route(const moe_desc* d, const float* x, int32_t T, const float* Wr, int32_t* idx, float* w,
              float* logits_out, void* ws, size_t ws_bytes, void* stream) {
    int r;
    if ((r = check_desc(d))) return r;
    if (T < 1) return fail(MOE_ERR_ARG, "T=%d must be >= 1", T);
    if ((r = check_ptr(x, 16, "x")) || (r = check_ptr(Wr, 16, "Wr")) || (r = check_ptr(idx, 4, "idx")) ||
        (r = check_ptr(w, 4, "w")))
        return r;
    if (logits_out && !aligned(logits_out, 4)) return fail(MOE_ERR_ARG, "logits_out is not 4-byte aligned");
    if (!moe::route_supported(d->H, d->E, d->k))
        return fail(MOE_ERR_UNSUPPORTED, "router needs H %% 256 == 0, H <= 8192, E <= %d, k <= %d (H=%d E=%d k=%d)",
                    moe::kMaxE, moe::kMaxK, d->H, d->E, d->k);
    if ((r = check_ws(ws, ws_bytes, moe::route_ws_bytes(T, d->E)))) return r;
    return hip_status(moe::launch_route(d->H, d->E, d->k, T, x, Wr, idx, w, logits_out, ws,
                                        reinterpret_cast<hipStream_t>(stream)),
                      "router launch");
}

int moe_expert_decode(const moe_desc* d, const float* x, const void* const* expert_ptrs, const int32_t* idx,
                      const float* w, const moe_shared* shared, float* y, void* ws, size_t ws_bytes, void* stream) {
    int r;
    if ((r = check_desc(d))) return r;
    if ((r = check_ptr(x, 16, "x")) || (r = check_ptr(expert_ptrs, 8, "expert_ptrs")) ||
        (r = check_ptr(idx, 4, "idx")) || (r = check_ptr(w, 4, "w")) || (r = check_ptr(y, 4, "y")))
        return r;
    if (shared) {
        if ((r = check_ptr(shared->gate, 16, "shared->gate")) || (r = check_ptr(shared->up, 16, "shared->up")) ||
            (r = check_ptr(shared->down, 16, "shared->down")))
            return r;
    }
    if (d->k > moe::kMaxK) return fail(MOE_ERR_UNSUPPORTED, "k=%d exceeds %d", d->k, moe::kMaxK);
    if (d->E > moe::kMaxE) return fail(MOE_ERR_UNSUPPORTED, "E=%d exceeds %d", d->E, moe::kMaxE);
    moe::DecodePlan plan;
    if (!moe::plan_decode(d->format, d->H, d->I, &plan))
        return fail(MOE_ERR_UNSUPPORTED, "no decode kernel for H=%d I=%d (needs H %% 512 == 0, H <= 4096, I <= 4096)",
                    d->H, d->I);
    if ((r = check_ws(ws, ws_bytes, moe::decode_ws_bytes(d->H, d->I, d->k, d->E)))) return r;
    return hip_status(moe::launch_decode(d->format, plan, d->E, d->H, d->I, d->k, x, expert_ptrs, idx, w,
                                         shared ? shared->gate : nullptr, shared ? shared->up : nullptr,
                                         shared ? shared->down : nullptr, y, ws,
                                         reinterpret_cast<hipStream_t>(stream)),
                      "decode launch");
}

}  // extern "C"

namespace {

// Every argument check of moe_layer_decode except the workspace.
int layer_decode_checks(const moe_desc* d, const float* x, const float* Wr, const void* const* expert_ptrs,
                        const moe_shared* shared, float* y, int32_t* idx_out, float* w_out, moe::DecodePlan* plan) {
    int r;
    if ((r = check_desc(d))) return r;
    if ((r = check_ptr(x, 16, "x")) || (r = check_ptr(Wr, 16, "Wr")) || (r = check_ptr(expert_ptrs, 8, "expert_ptrs")) ||
        (r = check_ptr(y, 4, "y")) || (r = check_ptr(idx_out, 4, "idx_out")) || (r = check_ptr(w_out, 4, "w_out")))
        return r;
    if (shared) {
        if ((r = check_ptr(shared->gate, 16, "shared->gate")) || (r = check_ptr(shared->up, 16, "shared->up")) ||
            (r = check_ptr(shared->down, 16, "shared->down")))
            return r;
    }
    if (!moe::route_supported(d->H, d->E, d->k))
        return fail(MOE_ERR_UNSUPPORTED, "router needs H %% 256 == 0, H <= 8192, E <= %d, k <= %d (H=%d E=%d k=%d)",
                    moe::kMaxE, moe::kMaxK, d->H, d->E, d->k);
    if (!moe::plan_decode(d->format, d->H, d->I, plan))
        return fail(MOE_ERR_UNSUPPORTED, "no decode kernel for H=%d I=%d (needs H %% 512 == 0, H <= 4096, I <= 4096)",
                    d->H, d->I);
    return MOE_OK;
}

int layer_decode_launch(const moe_desc* d, const moe::DecodePlan& plan, const float* x, const float* Wr,
                        const void* const* expert_ptrs, const moe_shared* shared, float* y, int32_t* idx_out,
                        float* w_out, void* ws, void* stream) {
    return hip_status(moe::launch_layer_decode(d->format, plan, d->E, d->H, d->I, d->k, x, Wr, expert_ptrs,
                                               shared ? shared->gate : nullptr, shared ? shared->up : nullptr,
                                               shared ? shared->down : nullptr, y, idx_out, w_out, ws,
                                               reinterpret_cast<hipStream_t>(stream)),
                      "layer decode launch");
}

// ---- the allocation-free decode ----
// Its workspace: one copy of this array on every GPU the library runs on,
// loaded with the library's code object (zero-filled) and held until the
// process ends. In host code the name stands for a host-side shadow, not a
// device address: only the address hipGetSymbolAddress returns for the
// current device may reach a kernel.
constexpr size_t kScratchBytes = MOE_NOALLOC_SCRATCH_BYTES;
constexpr int kMaxDevices = 64;
static __device__ __align__(256) uint8_t scratch[kScratchBytes];
std::atomic<void*> g_scratch_addr[kMaxDevices];  // device address of scratch, per device, once looked up

// Device address of the current device's scratch (looked up on the first
// call on that device; a lookup by two threads at once stores the same value).
int scratch_address(void** out) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
    if (dev < 0 || dev >= kMaxDevices) return fail(MOE_ERR_UNSUPPORTED, "device %d: at most %d devices", dev, kMaxDevices);
    void* p = g_scratch_addr[dev].load(std::memory_order_acquire);
    if (!p) {
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess || !p)
            return fail(MOE_ERR_HIP, "hipGetSymbolAddress(scratch) on device %d: %s", dev, hipGetErrorString(e));
        g_scratch_addr[dev].store(p, std::memory_order_release);
    }
    *out = p;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_layer_decode(const moe_desc* d, const float* x, const float* Wr, const void* const* expert_ptrs,
                     const moe_shared* shared, float* y, int32_t* idx_out, float* w_out, void* ws, size_t ws_bytes,
                     void* stream) {
    int r;
    moe::DecodePlan plan;
    if ((r = layer_decode_checks(d, x, Wr, expert_ptrs, shared, y, idx_out, w_out, &plan))) return r;
    if ((r = check_ws(ws, ws_bytes, moe::decode_ws_bytes(d->H, d->I, d->k, d->E)))) return r;
    return layer_decode_launch(d, plan, x, Wr, expert_ptrs, shared, y, idx_out, w_out, ws, stream);
}

int moe_layer_decode_noalloc(const moe_desc* d, const float* x, const float* Wr, const void* const* expert_ptrs,
                             const moe_shared* shared, float* y, int32_t* idx_out, float* w_out, void* stream) {
    int r;
    moe::DecodePlan plan;
    if ((r = layer_decode_checks(d, x, Wr, expert_ptrs, shared, y, idx_out, w_out, &plan))) return r;
    const size_t need = moe::decode_ws_bytes(d->H, d->I, d->k, d->E);
    if (need > kScratchBytes)
        return fail(MOE_ERR_WORKSPACE, "this layer needs %zu bytes of scratch; the static scratch holds %zu", need,
                    kScratchBytes);
    void* ws = nullptr;
    if ((r = scratch_address(&ws))) return r;
    return layer_decode_launch(d, plan, x, Wr, expert_ptrs, shared, y, idx_out, w_out, ws, stream);
}

int moe_layer_decode_batch(const moe_desc* d, const float* x, int32_t T, const uint8_t* mask, const float* Wr,
                           const void* const* expert_ptrs, const moe_shared* shared, float* y, int32_t* idx_out,
                           float* w_out, void* ws, size_t ws_bytes, void* stream) {
    int r;
    moe::DecodePlan plan;
    if ((r = check_desc(d))) return r;
    if (T < 0) return fail(MOE_ERR_ARG, "T=%d is negative", T);
    if (T > moe::kBatchMaxT) return fail(MOE_ERR_UNSUPPORTED, "T=%d exceeds %d", T, moe::kBatchMaxT);
    if (T == 0) return ok();
    if ((r = layer_decode_checks(d, x, Wr, expert_ptrs, shared, y, idx_out, w_out, &plan))) return r;
    if (static_cast<const void*>(y) == x || y == w_out || static_cast<const void*>(y) == idx_out ||
        static_cast<const void*>(w_out) == idx_out || static_cast<const void*>(w_out) == x ||
        static_cast<const void*>(idx_out) == x)
        return fail(MOE_ERR_ARG, "an output is an input or another output");
    if ((r = check_ws(ws, ws_bytes, moe::batch_ws_bytes(d->format, d->H, d->I, d->E, d->k, T)))) return r;
    return hip_status(moe::launch_layer_batch(d->format, d->H, d->I, d->E, d->k, x, T, mask, Wr, expert_ptrs,
                                              shared ? shared->gate : nullptr, shared ? shared->up : nullptr,
                                              shared ? shared->down : nullptr, y, idx_out, w_out, ws,
                                              reinterpret_cast<hipStream_t>(stream)),
                      "batched decode launch");
}

int moe_expert_prefill(const moe_desc* d, const float* x, int32_t T, const void* const* expert_ptrs,
                       const int32_t* idx, const float* w, void* out, int32_t out_dtype, void* ws, size_t ws_bytes,
                       const moe_prefill_debug* dbg, void* stream) {
    int r;
    if ((r = check_desc(d))) return r;
    if (T < 1) return fail(MOE_ERR_ARG, "T=%d must be >= 1", T);
    if ((r = check_ptr(x, 16, "x")) || (r = check_ptr(expert_ptrs, 8, "expert_ptrs")) ||
        (r = check_ptr(idx, 4, "idx")) || (r = check_ptr(w, 4, "w")) || (r = check_ptr(out, 16, "out")))
        return r;
    if (out_dtype != MOE_OUT_F32 && out_dtype != MOE_OUT_BF16) return fail(MOE_ERR_ARG, "unknown out_dtype %d", out_dtype);
    if (!moe::prefill_supported(d->format, d->H, d->I, d->E, d->k))
        return fail(MOE_ERR_UNSUPPORTED, "no prefill kernel for format=%d H=%d I=%d E=%d k=%d", d->format, d->H, d->I,
                    d->E, d->k);
    if (!moe::prefill_tokens_supported(d->H, d->I, d->k, T))
        return fail(MOE_ERR_UNSUPPORTED, "T=%d: the rounded activations would exceed 2 GiB (H=%d I=%d k=%d)", T, d->H,
                    d->I, d->k);
    if ((r = check_ws(ws, ws_bytes, moe::prefill_ws_bytes(d->format, d->H, d->I, d->E, d->k, T)))) return r;
    moe::PrefillDebug pd = {};
    if (dbg) {
        pd.x_bf16 = dbg->x_bf16;
        pd.x_codes = dbg->x_codes;
        pd.x_scales = dbg->x_scales;
        pd.h_pre = dbg->h_pre;
        pd.h_q = dbg->h_q;
        pd.perm = dbg->perm;
        pd.off = dbg->off;
        pd.tile_wait_polls = dbg->tile_wait_polls;
        pd.tile_wait_unmet = dbg->tile_wait_unmet;
    }
    return hip_status(moe::launch_prefill(d->format, d->H, d->I, d->E, d->k, T, x, expert_ptrs, idx, w, out,
                                          out_dtype == MOE_OUT_BF16, ws, dbg ? &pd : nullptr,
                                          reinterpret_cast<hipStream_t>(stream)),
                      "prefill launch");
}

int moe_dequant_block(const moe_desc* d, const void* block, float* gate, float* up, float* down, void* stream) {
    int r;
    if ((r = check_desc(d))) return r;
    if ((r = check_ptr(block, 16, "block")) || (r = check_ptr(gate, 4, "gate")) || (r = check_ptr(up, 4, "up")) ||
        (r = check_ptr(down, 4, "down")))
        return r;
    return hip_status(moe::launch_dequant(d->format, d->H, d->I, block, gate, up, down,
                                          reinterpret_cast<hipStream_t>(stream)),
                      "dequant launch");
}

const char* moe_status_string(int status) {
    switch (status) {
        case MOE_OK: return "ok";
        case MOE_ERR_ARG: return "invalid argument";
        case MOE_ERR_UNSUPPORTED: return "unsupported shape (no tuned kernel)";
        case MOE_ERR_HIP: return "HIP launch error";
        case MOE_ERR_WORKSPACE: return "workspace missing or too small";
        default: return "unknown status";
    }
}

int moe_act_quant_fp8(const float* x, int32_t rows, int32_t cols, int32_t block, int32_t rule, uint8_t* codes,
                      uint8_t* scales, void* stream) {
    if (rows < 0) return fail(MOE_ERR_ARG, "rows=%d is negative", rows);
    if (block != 32 && block != 128) return fail(MOE_ERR_ARG, "block=%d (32 or 128)", block);
    if (cols <= 0 || cols % block) return fail(MOE_ERR_ARG, "cols=%d must be a positive multiple of block=%d", cols, block);
    if (rule != MOE_SCALE_FLOOR && rule != MOE_SCALE_CEIL) return fail(MOE_ERR_ARG, "unknown scale rule %d", rule);
    if ((size_t)rows * cols > ((size_t)1 << 34)) return fail(MOE_ERR_ARG, "rows*cols too large");
    if (rows == 0) return ok();
    int r;
    if ((r = check_ptr(x, 16, "x")) || (r = check_ptr(codes, 4, "codes")) || (r = check_ptr(scales, 1, "scales")))
        return r;
    return hip_status(moe::launch_act_quant_fp8(x, rows, cols, block, rule, codes, scales, (hipStream_t)stream),
                      "act_quant_fp8 launch");
}

int moe_gemv_fp8(const uint8_t* W, const float* row_scale, const float* x, int32_t rows, int32_t cols, float* y,
                 void* stream) {
    if (rows < 0) return fail(MOE_ERR_ARG, "rows=%d is negative", rows);
    if (cols <= 0) return fail(MOE_ERR_ARG, "cols=%d must be positive", cols);
    if (!moe::gemv_fp8_supported(cols))
        return fail(MOE_ERR_UNSUPPORTED, "cols=%d: no kernel (512*d, d in 1..8, 10, 12, 16)", cols);
    if ((size_t)rows * cols >= ((size_t)1 << 31)) return fail(MOE_ERR_UNSUPPORTED, "rows*cols too large");
    if (rows == 0) return ok();
    int r;
    if ((r = check_ptr(W, 16, "W")) || (r = check_ptr(row_scale, 4, "row_scale")) || (r = check_ptr(x, 16, "x")) ||
        (r = check_ptr(y, 4, "y")))
        return r;
    return hip_status(moe::launch_gemv_fp8(W, row_scale, x, y, rows, cols, (hipStream_t)stream), "gemv_fp8 launch");
}

}  // extern "C"

namespace {

int balance_checks(const moe_desc* d, int32_t T, int32_t S) {
    int r;
    if ((r = check_desc(d))) return r;
    if (T < 0) return fail(MOE_ERR_ARG, "T=%d is negative", T);
    if (S < 1) return fail(MOE_ERR_ARG, "S=%d must be >= 1", S);
    if (d->E > moe::kMaxE || d->k > moe::kMaxK || S > 65535 || T > (1 << 24))
        return fail(MOE_ERR_UNSUPPORTED, "balance loss needs E <= %d, k <= %d, S <= 65535, T <= 2^24 (E=%d k=%d S=%d T=%d)",
                    moe::kMaxE, moe::kMaxK, d->E, d->k, S, T);
    return MOE_OK;
}

int route_backward_checks(const moe_desc* d, int32_t T) {
    int r;
    if ((r = check_desc(d))) return r;
    if (T < 0) return fail(MOE_ERR_ARG, "T=%d is negative", T);
    if (!moe::route_supported(d->H, d->E, d->k))
        return fail(MOE_ERR_UNSUPPORTED, "router needs H %% 256 == 0, H <= 8192, E <= %d, k <= %d (H=%d E=%d k=%d)",
                    moe::kMaxE, moe::kMaxK, d->H, d->E, d->k);
    if (T > (1 << 20)) return fail(MOE_ERR_UNSUPPORTED, "T=%d exceeds 2^20", T);
    return MOE_OK;
}

int lora_checks(const moe_lora_desc* l, int32_t T) {
    if (!l) return fail(MOE_ERR_ARG, "lora desc is NULL");
    if (l->dtype != MOE_ACT_F32 && l->dtype != MOE_ACT_BF16 && l->dtype != MOE_ACT_F16)
        return fail(MOE_ERR_ARG, "unknown dtype %d", l->dtype);
    if (l->K <= 0 || l->N <= 0 || l->n <= 0 || l->max_rank <= 0)
        return fail(MOE_ERR_ARG, "K, N, n, max_rank must be positive (K=%d N=%d n=%d max_rank=%d)", l->K, l->N, l->n,
                    l->max_rank);
    if (l->K % 8 || l->N % 8) return fail(MOE_ERR_ARG, "K=%d and N=%d must be multiples of 8", l->K, l->N);
    if (T < 0) return fail(MOE_ERR_ARG, "T=%d is negative", T);
    if (l->K > moe::kLoraMaxDim || l->N > moe::kLoraMaxDim || l->n > moe::kLoraMaxN || l->max_rank > moe::kLoraMaxRank ||
        T > moe::kLoraMaxT)
        return fail(MOE_ERR_UNSUPPORTED, "adapters need K, N <= %d, n <= %d, max_rank <= %d, T <= %d (K=%d N=%d n=%d max_rank=%d T=%d)",
                    moe::kLoraMaxDim, moe::kLoraMaxN, moe::kLoraMaxRank, moe::kLoraMaxT, l->K, l->N, l->n, l->max_rank, T);
    return MOE_OK;
}

// A matrix of rows of `cols` elements with a stride.
int check_rows(const void* p, int64_t ld, int32_t cols, const char* name) {
    int r;
    if ((r = check_ptr(p, 16, name))) return r;
    if (ld < cols || ld % 8 || ld > ((int64_t)1 << 40))
        return fail(MOE_ERR_ARG, "%s: stride %lld must be a multiple of 8 and at least %d", name, (long long)ld, cols);
    return MOE_OK;
}

int lora_table_checks(const int32_t* ids, const void* const* a, const void* const* b, const int32_t* ranks,
                      const float* scales) {
    int r;
    if ((r = check_ptr(ids, 4, "ids")) || (r = check_ptr(a, 8, "a_ptrs")) || (r = check_ptr(b, 8, "b_ptrs")) ||
        (r = check_ptr(ranks, 4, "ranks")) || (r = check_ptr(scales, 4, "scales")))
        return r;
    return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_balance_workspace_bytes(const moe_desc* d, int32_t T, int32_t S) {
    return balance_checks(d, T, S) == MOE_OK ? moe::balance_ws_bytes(T, d->E, S) : 0;
}

int moe_balance_loss(const moe_desc* d, const float* logits, int32_t T, const int32_t* idx, const uint8_t* mask,
                     const int32_t* seq_off, int32_t S, float balance_coef, float z_coef, const float* dloss,
                     float* loss, int32_t* counts, float* probs, float* dlogits, void* ws, size_t ws_bytes,
                     void* stream) {
    int r;
    if ((r = balance_checks(d, T, S))) return r;
    if (T > 0 && ((r = check_ptr(logits, 16, "logits")) || (r = check_ptr(idx, 4, "idx")))) return r;
    if (!seq_off && S != 1) return fail(MOE_ERR_ARG, "S=%d without seq_off", S);
    if (seq_off && !aligned(seq_off, 4)) return fail(MOE_ERR_ARG, "seq_off is not 4-byte aligned");
    if (dloss && !aligned(dloss, 4)) return fail(MOE_ERR_ARG, "dloss is not 4-byte aligned");
    if (!std::isfinite(balance_coef) || !std::isfinite(z_coef)) return fail(MOE_ERR_ARG, "a coefficient is not finite");
    if ((r = check_ptr(loss, 4, "loss"))) return r;
    if (counts && !aligned(counts, 4)) return fail(MOE_ERR_ARG, "counts is not 4-byte aligned");
    if (probs && !aligned(probs, 4)) return fail(MOE_ERR_ARG, "probs is not 4-byte aligned");
    if (dlogits && !aligned(dlogits, 16)) return fail(MOE_ERR_ARG, "dlogits is not 16-byte aligned");
    if (dlogits && T > 0 && dlogits == logits) return fail(MOE_ERR_ARG, "dlogits is logits");
    if ((r = check_ws(ws, ws_bytes, moe::balance_ws_bytes(T, d->E, S)))) return r;
    return hip_status(moe::launch_balance(d->E, d->k, logits, T, idx, mask, seq_off, S, balance_coef, z_coef, dloss,
                                          loss, counts, probs, dlogits, ws, reinterpret_cast<hipStream_t>(stream)),
                      "balance loss launch");
}

size_t moe_route_backward_workspace_bytes(const moe_desc* d, int32_t T) {
    return route_backward_checks(d, T) == MOE_OK ? moe::route_backward_ws_bytes(d->H, d->E, T) : 0;
}

int moe_route_backward(const moe_desc* d, const float* x, int32_t T, const float* Wr, const int32_t* idx,
                       const float* w, const float* dw, const uint8_t* mask, const float* dlogits_in,
                       float* dlogits_out, float* dx, float* dWr, int32_t accumulate, void* ws, size_t ws_bytes,
                       void* stream) {
    int r;
    if ((r = route_backward_checks(d, T))) return r;
    if (accumulate & ~(MOE_ACC_DX | MOE_ACC_DWR | MOE_FP32_PRODUCTS)) return fail(MOE_ERR_ARG, "unknown accumulate bits %d", accumulate);
    if (T > 0) {
        if (!dw && !dlogits_in) return fail(MOE_ERR_ARG, "neither dw nor dlogits_in");
        if (!dlogits_out && !dx && !dWr) return fail(MOE_ERR_ARG, "no output");
        if (dw && ((r = check_ptr(idx, 4, "idx")) || (r = check_ptr(w, 4, "w")) || (r = check_ptr(dw, 4, "dw")))) return r;
        if (dlogits_in && (r = check_ptr(dlogits_in, 4, "dlogits_in"))) return r;
        if (dlogits_out && (r = check_ptr(dlogits_out, 4, "dlogits_out"))) return r;
        if (dx && ((r = check_ptr(dx, 16, "dx")) || (r = check_ptr(Wr, 16, "Wr")))) return r;
        if (dWr && (r = check_ptr(x, 16, "x"))) return r;
        // G, dx and dWr are written while the inputs are still read
        const float* in[] = {x, Wr, w, dw, dlogits_in};
        for (int i = 0; i < 5; i++)
            if (in[i] && (in[i] == dx || in[i] == dWr || (in[i] == dlogits_out && in[i] != dlogits_in)))
                return fail(MOE_ERR_ARG, "an output is an input");
        if ((dx && dx == dWr) || (dlogits_out && (dlogits_out == dx || dlogits_out == dWr)))
            return fail(MOE_ERR_ARG, "two outputs are the same");
    }
    if (dWr && (r = check_ptr(dWr, 16, "dWr"))) return r;
    if ((r = check_ws(ws, ws_bytes, moe::route_backward_ws_bytes(d->H, d->E, T)))) return r;
    return hip_status(moe::launch_route_backward(d->H, d->E, d->k, x, T, Wr, idx, w, dw, mask, dlogits_in, dlogits_out,
                                                 dx, dWr, accumulate, ws, reinterpret_cast<hipStream_t>(stream)),
                      "routing gradient launch");
}

size_t moe_lora_workspace_bytes(const moe_lora_desc* l, int32_t T, int32_t backward) {
    return lora_checks(l, T) == MOE_OK ? moe::lora_ws_bytes(l->K, l->N, l->n, l->max_rank, T, backward != 0) : 0;
}

int moe_lora_apply(const moe_lora_desc* l, const void* x, int64_t ldx, int32_t T, const int32_t* ids,
                   const void* const* a_ptrs, const void* const* b_ptrs, const int32_t* ranks, const float* scales,
                   const void* base, int64_t ldbase, void* y, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
    int r;
    if ((r = lora_checks(l, T))) return r;
    if (T == 0) return ok();
    if ((r = check_rows(x, ldx, l->K, "x")) || (r = lora_table_checks(ids, a_ptrs, b_ptrs, ranks, scales)) ||
        (r = check_rows(y, ldy, l->N, "y")) || (base && (r = check_rows(base, ldbase, l->N, "base"))))
        return r;
    if (base == y && ldbase != ldy) return fail(MOE_ERR_ARG, "base is y with another stride");
    if (x == y) return fail(MOE_ERR_ARG, "y is x");
    if ((r = check_ws(ws, ws_bytes, moe::lora_ws_bytes(l->K, l->N, l->n, l->max_rank, T, false)))) return r;
    const moe::LoraTable tab = {ids, a_ptrs, b_ptrs, ranks, scales};
    return hip_status(moe::launch_lora_apply(l->dtype, l->K, l->N, l->n, l->max_rank, x, (size_t)ldx, T, tab, base,
                                             (size_t)ldbase, y, (size_t)ldy, ws, reinterpret_cast<hipStream_t>(stream)),
                      "adapter launch");
}

int moe_lora_backward(const moe_lora_desc* l, const void* x, int64_t ldx, const void* dy, int64_t lddy, int32_t T,
                      const int32_t* ids, const void* const* a_ptrs, const void* const* b_ptrs, const int32_t* ranks,
                      const float* scales, const void* dx_base, int64_t lddx_base, void* dx, int64_t lddx,
                      float* const* da_ptrs, float* const* db_ptrs, int32_t accumulate, void* ws, size_t ws_bytes,
                      void* stream) {
    int r;
    if ((r = lora_checks(l, T))) return r;
    if (T > 0 && !dx && !da_ptrs && !db_ptrs) return fail(MOE_ERR_ARG, "no output");
    if (T == 0 && !da_ptrs && !db_ptrs) return ok();
    if (da_ptrs && (r = check_ptr(da_ptrs, 8, "da_ptrs"))) return r;
    if (db_ptrs && (r = check_ptr(db_ptrs, 8, "db_ptrs"))) return r;
    if (da_ptrs && da_ptrs == db_ptrs) return fail(MOE_ERR_ARG, "da_ptrs is db_ptrs");
    if (T > 0) {
        if ((r = check_rows(x, ldx, l->K, "x")) || (r = check_rows(dy, lddy, l->N, "dy")) ||
            (r = lora_table_checks(ids, a_ptrs, b_ptrs, ranks, scales)))
            return r;
        if (dx && (r = check_rows(dx, lddx, l->K, "dx"))) return r;
        if (dx && dx_base && (r = check_rows(dx_base, lddx_base, l->K, "dx_base"))) return r;
        if (dx && dx_base == dx && lddx_base != lddx) return fail(MOE_ERR_ARG, "dx_base is dx with another stride");
        if (dx && (dx == x || dx == dy)) return fail(MOE_ERR_ARG, "dx is an input");
    } else if ((r = check_ptr(ranks, 4, "ranks"))) {
        return r;
    }
    if ((r = check_ws(ws, ws_bytes, moe::lora_ws_bytes(l->K, l->N, l->n, l->max_rank, T, true)))) return r;
    const moe::LoraTable tab = {ids, a_ptrs, b_ptrs, ranks, scales};
    return hip_status(moe::launch_lora_backward(l->dtype, l->K, l->N, l->n, l->max_rank, x, (size_t)ldx, dy,
                                                (size_t)lddy, T, tab, dx_base, (size_t)lddx_base, dx, (size_t)lddx,
                                                da_ptrs, db_ptrs, accumulate, ws, reinterpret_cast<hipStream_t>(stream)),
                      "adapter gradient launch");
}

}  // extern "C"

namespace {

constexpr size_t kMaxQuant = (size_t)1 << 33;  // elements: the quantisation's pieces of 8 count in 32 bits

bool act_known(int32_t dtype) { return dtype == MOE_ACT_F32 || dtype == MOE_ACT_BF16 || dtype == MOE_ACT_F16; }

int fp4_checks(const moe_fp4_desc* f, int32_t T) {
    if (!f) return fail(MOE_ERR_ARG, "fp4 desc is NULL");
    if (!group_size(f->format)) return fail(MOE_ERR_ARG, "unknown format %d", f->format);
    if (!act_known(f->dtype)) return fail(MOE_ERR_ARG, "unknown dtype %d", f->dtype);
    if (f->K <= 0 || f->N <= 0 || f->K % 32 || f->N % 8)
        return fail(MOE_ERR_ARG, "K=%d must be a positive multiple of 32, N=%d of 8", f->K, f->N);
    if (T < 0) return fail(MOE_ERR_ARG, "T=%d is negative", T);
    if (f->K > moe::kFp4MaxDim || f->N > moe::kFp4MaxDim || T > moe::kFp4MaxT)
        return fail(MOE_ERR_UNSUPPORTED, "4-bit products need K, N <= %d, T <= %d (K=%d N=%d T=%d)", moe::kFp4MaxDim,
                    moe::kFp4MaxT, f->K, f->N, T);
    return MOE_OK;
}

int fp4_rows(const void* p, int64_t ld, int32_t cols, const char* name) {
    int r;
    if ((r = check_rows(p, ld, cols, name))) return r;
    if (ld > moe::kFp4MaxLd)
        return fail(MOE_ERR_UNSUPPORTED, "%s: stride %lld exceeds %lld", name, (long long)ld, (long long)moe::kFp4MaxLd);
    return MOE_OK;
}

int fp4_matrix(const moe_fp4_desc* f, const uint8_t* codes, const uint8_t* scales, const int8_t* row_exp) {
    int r;
    if ((r = check_ptr(codes, 16, "codes")) || (r = check_ptr(scales, 1, "scales"))) return r;
    if (row_exp && f->format != MOE_FMT_NVFP4) return fail(MOE_ERR_ARG, "row_exp beside a format without row exponents");
    return MOE_OK;
}

int norm_checks(const moe_norm_desc* n, int32_t T) {
    if (!n) return fail(MOE_ERR_ARG, "norm desc is NULL");
    if (n->H <= 0 || n->H % 8) return fail(MOE_ERR_ARG, "H=%d must be a positive multiple of 8", n->H);
    if (!act_known(n->r_dtype) || !act_known(n->y_dtype) || !act_known(n->x_dtype))
        return fail(MOE_ERR_ARG, "unknown dtype (r %d y %d x %d)", n->r_dtype, n->y_dtype, n->x_dtype);
    if (n->gate != MOE_GATE_NONE && n->gate != MOE_GATE_CHANNEL && n->gate != MOE_GATE_TOKEN)
        return fail(MOE_ERR_ARG, "unknown gate %d", n->gate);
    if (!(n->eps > 0.0f) || !std::isfinite(n->eps) || !std::isfinite(n->scale))
        return fail(MOE_ERR_ARG, "eps=%g must be above 0 and scale=%g finite", (double)n->eps, (double)n->scale);
    if (T < 0) return fail(MOE_ERR_ARG, "T=%d is negative", T);
    if (n->H > moe::kNormMaxH || T > moe::kNormMaxT)
        return fail(MOE_ERR_UNSUPPORTED, "norms need H <= %d, T <= %d (H=%d T=%d)", moe::kNormMaxH, moe::kNormMaxT, n->H, T);
    return MOE_OK;
}

// The vectors of a norm: post and gate only matter beside y. The rows of an
// empty batch may have no address.
int norm_vectors(const moe_norm_desc* n, int32_t T, const void* y, const float* post, const float* gate, const float* pre) {
    int r;
    if (post && (r = check_ptr(post, 16, "post"))) return r;
    if (pre && (r = check_ptr(pre, 16, "pre"))) return r;
    if (post && !y && T > 0) return fail(MOE_ERR_ARG, "post without y");
    if (n->gate == MOE_GATE_NONE && gate) return fail(MOE_ERR_ARG, "a gate beside MOE_GATE_NONE");
    if (n->gate != MOE_GATE_NONE && y && (r = check_ptr(gate, n->gate == MOE_GATE_CHANNEL ? 16 : 4, "gate"))) return r;
    return MOE_OK;
}

// Whether an output is an input or another output, but for the pairs that may be.
bool shared_memory(std::initializer_list<const void*> out, std::initializer_list<const void*> in, const void* ok_out,
                   const void* ok_in) {
    int i = 0;
    for (const void* o : out) {
        int j = 0;
        for (const void* p : out)
            if (j++ > i && o && o == p) return true;
        for (const void* p : in)
            if (o && o == p && !(o == ok_out && p == ok_in)) return true;
        i++;
    }
    return false;
}

}  // namespace

extern "C" {

int moe_fp4_quant(const void* x, int64_t ldx, int32_t rows, int32_t cols, int32_t dtype, int32_t format, int32_t rule,
                  int8_t* row_exp, uint8_t* codes, uint8_t* scales, void* values, int64_t ldv, void* stream) {
    const int G = group_size(format);
    int r;
    if (!G) return fail(MOE_ERR_ARG, "unknown format %d", format);
    if (!act_known(dtype)) return fail(MOE_ERR_ARG, "unknown dtype %d", dtype);
    if (rows < 0) return fail(MOE_ERR_ARG, "rows=%d is negative", rows);
    if (cols <= 0 || cols % G) return fail(MOE_ERR_ARG, "cols=%d must be a positive multiple of %d", cols, G);
    if (format == MOE_FMT_NVFP4 ? rule != MOE_SCALE_NEAREST : rule != MOE_SCALE_FLOOR && rule != MOE_SCALE_CEIL)
        return fail(MOE_ERR_ARG, "scale rule %d does not go with format %d", rule, format);
    if (row_exp && format != MOE_FMT_NVFP4) return fail(MOE_ERR_ARG, "row_exp beside a format without row exponents");
    if (!codes && !scales && !values && !row_exp) return fail(MOE_ERR_ARG, "no output");
    if ((size_t)rows * cols > kMaxQuant) return fail(MOE_ERR_UNSUPPORTED, "rows*cols exceeds 2^33");
    if (rows == 0) return ok();
    if ((r = check_rows(x, ldx, cols, "x"))) return r;
    if (codes && (r = check_ptr(codes, 4, "codes"))) return r;
    if (values && (r = check_rows(values, ldv, cols, "values"))) return r;
    if (values == x && ldv != ldx) return fail(MOE_ERR_ARG, "values is x with another stride");
    if (shared_memory({codes, scales, row_exp, values}, {x}, values, x))
        return fail(MOE_ERR_ARG, "an output is an input or another output");
    return hip_status(moe::launch_fp4_quant(dtype, format, rule, x, (size_t)ldx, rows, cols, row_exp, codes, scales, values,
                                            (size_t)ldv, reinterpret_cast<hipStream_t>(stream)),
                      "fp4 quantisation launch");
}

size_t moe_fp4_workspace_bytes(const moe_fp4_desc* f, int32_t T, int32_t backward) {
    return fp4_checks(f, T) == MOE_OK ? moe::fp4_ws_bytes(f->K, f->N, f->format, f->dtype, T, backward != 0) : 0;
}

int moe_fp4_apply(const moe_fp4_desc* f, const void* x, int64_t ldx, int32_t T, const uint8_t* codes,
                  const uint8_t* scales, const int8_t* row_exp, int32_t round_x, const void* base, int64_t ldbase,
                  void* y, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
    int r;
    if ((r = fp4_checks(f, T))) return r;
    if (round_x && f->format != MOE_FMT_MXFP4) return fail(MOE_ERR_ARG, "round_x needs an MXFP4 matrix");
    if (round_x && (size_t)T * f->K > kMaxQuant) return fail(MOE_ERR_UNSUPPORTED, "round_x: T*K exceeds 2^33");
    if (T == 0) return ok();
    if ((r = fp4_rows(x, ldx, f->K, "x")) || (r = fp4_matrix(f, codes, scales, row_exp)) ||
        (r = fp4_rows(y, ldy, f->N, "y")) || (base && (r = fp4_rows(base, ldbase, f->N, "base"))))
        return r;
    if (base == y && ldbase != ldy) return fail(MOE_ERR_ARG, "base is y with another stride");
    if (shared_memory({y}, {x, codes, scales, row_exp}, nullptr, nullptr)) return fail(MOE_ERR_ARG, "y is an input");
    if ((r = check_ws(ws, ws_bytes, moe::fp4_ws_bytes(f->K, f->N, f->format, f->dtype, T, false)))) return r;
    return hip_status(moe::launch_fp4_apply(f->K, f->N, f->format, f->dtype, x, (size_t)ldx, T, {codes, scales, row_exp},
                                            round_x != 0, base, (size_t)ldbase, y, (size_t)ldy, ws,
                                            reinterpret_cast<hipStream_t>(stream)),
                      "fp4 product launch");
}

int moe_fp4_backward(const moe_fp4_desc* f, const void* dy, int64_t lddy, int32_t T, const uint8_t* codes,
                     const uint8_t* scales, const int8_t* row_exp, const void* dx_base, int64_t lddx_base, void* dx,
                     int64_t lddx, void* ws, size_t ws_bytes, void* stream) {
    int r;
    if ((r = fp4_checks(f, T))) return r;
    if (T == 0) return ok();
    if ((r = fp4_rows(dy, lddy, f->N, "dy")) || (r = fp4_matrix(f, codes, scales, row_exp)) ||
        (r = fp4_rows(dx, lddx, f->K, "dx")) || (dx_base && (r = fp4_rows(dx_base, lddx_base, f->K, "dx_base"))))
        return r;
    if (dx_base == dx && lddx_base != lddx) return fail(MOE_ERR_ARG, "dx_base is dx with another stride");
    if (shared_memory({dx}, {dy, codes, scales, row_exp}, nullptr, nullptr)) return fail(MOE_ERR_ARG, "dx is an input");
    if ((r = check_ws(ws, ws_bytes, moe::fp4_ws_bytes(f->K, f->N, f->format, f->dtype, T, true)))) return r;
    return hip_status(moe::launch_fp4_backward(f->K, f->N, f->format, f->dtype, dy, (size_t)lddy, T,
                                               {codes, scales, row_exp}, dx_base, (size_t)lddx_base, dx, (size_t)lddx, ws,
                                               reinterpret_cast<hipStream_t>(stream)),
                      "fp4 gradient launch");
}

int moe_block_norm(const moe_norm_desc* n, const void* r, int64_t ldr, const void* y, int64_t ldy, int32_t T,
                   const uint8_t* mask, const float* post, const float* gate, const float* pre, void* r_out,
                   int64_t ldr_out, void* x, int64_t ldx, void* stream) {
    int e;
    if ((e = norm_checks(n, T))) return e;
    if ((e = norm_vectors(n, T, y, post, gate, pre))) return e;
    if (T == 0) return ok();
    if ((pre != nullptr) != (x != nullptr)) return fail(MOE_ERR_ARG, "x and pre go together");
    if (!r_out && !x) return fail(MOE_ERR_ARG, "no output");
    if ((e = check_rows(r, ldr, n->H, "r")) || (y && (e = check_rows(y, ldy, n->H, "y"))) ||
        (r_out && (e = check_rows(r_out, ldr_out, n->H, "r_out"))) || (x && (e = check_rows(x, ldx, n->H, "x"))))
        return e;
    if (r_out == r && ldr_out != ldr) return fail(MOE_ERR_ARG, "r_out is r with another stride");
    if (shared_memory({r_out, x}, {r, y, mask, post, gate, pre}, r_out, r))
        return fail(MOE_ERR_ARG, "an output is an input or another output");
    moe::NormArgs a = {};
    a.H = n->H; a.T = T; a.rt = n->r_dtype; a.yt = n->y_dtype; a.xt = n->x_dtype; a.gate_kind = n->gate;
    a.scale = n->scale; a.eps = n->eps;
    a.r = r; a.y = y; a.mask = mask; a.post = post; a.gate = gate; a.pre = pre;
    a.ldr = (size_t)ldr; a.ldy = (size_t)ldy; a.r_out = r_out; a.x = x; a.ldro = (size_t)ldr_out; a.ldx = (size_t)ldx;
    return hip_status(moe::launch_block_norm(a, reinterpret_cast<hipStream_t>(stream)), "norm launch");
}

size_t moe_block_norm_workspace_bytes(const moe_norm_desc* n, int32_t T) {
    return norm_checks(n, T) == MOE_OK ? moe::norm_ws_bytes(n->H, T) : 0;
}

int moe_block_norm_backward(const moe_norm_desc* n, const void* r_out, int64_t ldr_out, const void* y, int64_t ldy,
                            int32_t T, const uint8_t* mask, const float* post, const float* gate, const float* pre,
                            const void* dr_out, int64_t lddr_out, const void* dx, int64_t lddx, void* dr, int64_t lddr,
                            void* dy, int64_t lddy, float* dpost, float* dgate, float* dpre, int32_t accumulate,
                            void* ws, size_t ws_bytes, void* stream) {
    int e;
    if ((e = norm_checks(n, T))) return e;
    if ((e = norm_vectors(n, T, y, post, gate, pre))) return e;
    if (T > 0 && !dr && !dy && !dpost && !dgate && !dpre) return fail(MOE_ERR_ARG, "no output");
    if (T > 0 && !y && (dy || dgate)) return fail(MOE_ERR_ARG, "a gradient of y or its gate without y");
    if (dpost && !post) return fail(MOE_ERR_ARG, "dpost without post");
    if (dpre && !pre) return fail(MOE_ERR_ARG, "dpre without pre");
    if (dx && !pre) return fail(MOE_ERR_ARG, "dx without pre");
    if (dpre && !dx && T > 0) return fail(MOE_ERR_ARG, "dpre without dx");
    if (dgate && n->gate == MOE_GATE_NONE) return fail(MOE_ERR_ARG, "dgate beside MOE_GATE_NONE");
    if ((dpost && (e = check_ptr(dpost, 16, "dpost"))) || (dpre && (e = check_ptr(dpre, 16, "dpre"))) ||
        (dgate && (e = check_ptr(dgate, n->gate == MOE_GATE_CHANNEL ? 16 : 4, "dgate"))))
        return e;
    if (T > 0) {
        if ((dx && (e = check_rows(r_out, ldr_out, n->H, "r_out"))) || (y && (e = check_rows(y, ldy, n->H, "y"))) ||
            (dr_out && (e = check_rows(dr_out, lddr_out, n->H, "dr_out"))) ||
            (dx && (e = check_rows(dx, lddx, n->H, "dx"))) || (dr && (e = check_rows(dr, lddr, n->H, "dr"))) ||
            (dy && (e = check_rows(dy, lddy, n->H, "dy"))))
            return e;
        if (dr && dr == dr_out && lddr != lddr_out) return fail(MOE_ERR_ARG, "dr is dr_out with another stride");
        if (shared_memory({dr, dy, dpost, dgate, dpre}, {r_out, y, mask, post, gate, pre, dr_out, dx}, dr, dr_out))
            return fail(MOE_ERR_ARG, "an output is an input or another output");
    } else if (shared_memory({dpost, dgate, dpre}, {post, gate, pre}, nullptr, nullptr)) {
        return fail(MOE_ERR_ARG, "an output is an input or another output");
    }
    if ((e = check_ws(ws, ws_bytes, moe::norm_ws_bytes(n->H, T)))) return e;
    moe::NormArgs a = {};
    a.H = n->H; a.T = T; a.rt = n->r_dtype; a.yt = n->y_dtype; a.xt = n->x_dtype; a.gate_kind = n->gate;
    a.scale = n->scale; a.eps = n->eps;
    a.r = r_out; a.y = y; a.mask = mask; a.post = post; a.gate = gate; a.pre = pre;
    a.ldr = (size_t)ldr_out; a.ldy = (size_t)ldy;
    a.dr_out = dr_out; a.dx = dx; a.dr = dr; a.dy = dy;
    a.lddro = (size_t)lddr_out; a.lddx = (size_t)lddx; a.lddr = (size_t)lddr; a.lddy = (size_t)lddy;
    a.dpost = dpost; a.dgate = dgate; a.dpre = dpre; a.accumulate = accumulate != 0;
    return hip_status(moe::launch_block_norm_backward(a, ws, reinterpret_cast<hipStream_t>(stream)), "norm gradient launch");
}

size_t moe_prefetch_sink_bytes(const moe_desc* d, int32_t n) {
    const size_t bb = moe_block_bytes(d);
    if (!bb || n < 1 || n > 1024) return 0;
    return (size_t)n * moe::prefetch_chunks(bb) * sizeof(uint32_t);
}

int moe_expert_prefetch(const moe_desc* d, const void* const* expert_ptrs, const int32_t* idx, int32_t n,
                        uint32_t* sink, size_t sink_bytes, void* stream) {
    int r;
    if ((r = check_desc(d))) return r;
    if (n < 1 || n > 1024) return fail(MOE_ERR_ARG, "n=%d (1..1024)", n);
    if ((r = check_ptr(expert_ptrs, 8, "expert_ptrs")) || (r = check_ptr(idx, 4, "idx")) ||
        (r = check_ptr(sink, 4, "sink")))
        return r;
    const size_t need = moe_prefetch_sink_bytes(d, n);
    if (sink_bytes < need) return fail(MOE_ERR_ARG, "sink has %zu bytes, needs %zu", sink_bytes, need);
    return hip_status(moe::launch_prefetch(expert_ptrs, idx, n, d->E, moe_block_bytes(d), sink,
                                           reinterpret_cast<hipStream_t>(stream)),
                      "prefetch launch");
}

const char* moe_last_error(void) { return g_err; }

}  // extern "C"

// A whole mixture-of-experts layer for a few tokens (gfx950): T <= 64 tokens
// routed, each through its k experts (SwiGLU over block-scaled FP4 weights) and
// the bf16 shared expert, in fp32 as the single-token decode has it.
//
// What bounds it is the chosen experts' blocks, read once each: 4 tokens of 10
// experts choose about 39 of 512. Five launches:
//  1. front: the router's logits (fp32 matrix instructions over 16 experts x 16
//     tokens) and the activations as three bf16 parts each (x = p1 + p2 + p3
//     holds all 24 bits);
//  2. route: a workgroup a token takes its top-k, the last of them groups the
//     assignments by expert;
//  3. gate/up: 32 rows of both matrices of an expert for up to 5 or 15 of its
//     tokens (an item) a workgroup, codes decoded to bf16 in registers, where they are the matrix instruction's operand; its 16
//     columns are 5 tokens times their 3 parts, so that one or five tokens cost
//     one instruction; SiLU and product; the hidden values leave as parts again;
//  4. down: the same over 32 rows a wave, an output row for every assignment;
//  5. combine: the weighted sum over a token's assignments, in their order.
// An expert with more tokens than an item holds (5 or 15) is read again from the
// caches.
//
// 13 tokens of 6 out of 384 MXFP4 experts of 4096 x 2880 (1.35 GB): gate/up and
// down 304 us, 4.4 TB/s. 48 tokens of 10 out of 512 NVFP4 ones of 2560 x 640 (0.82
// GB): 227-232 us, 3.6 TB/s (fp16 decoding, half the instructions, gained 2%: not the
// arithmetic). 4 tokens: 44 of 61 us, 800 and 800 workgroups that each read for two or
// three blocks of the sum, so that their start and end count; the other three
// launches are chains of dependent loads. 2 tokens take 42 us in a graph, two calls of
// the single-token layer 32; 3 take 49 and 48.
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

constexpr int kTok = 5;          // tokens of a column group: their parts are columns 5 part + token
constexpr int kMaxGroups = 3;    // column groups of an item, at most
constexpr int kSlots = kTok * kMaxGroups;
constexpr int kRouterParts = 8;  // workgroups along the router's sums, at most

// All that a workgroup of an expert launch needs to begin, in one 64-byte scalar
// load: the expert's block, how many assignments (0: an item that is not used),
// which (t k + j; the shared expert's T k + t), two to a word.
constexpr uint32_t kRouted = 0, kSharedLow = 1, kSharedHigh = 2;  // the shared expert's: rows 0-15 or 16-31 of each 32
struct alignas(64) Item {
    const void* block;
    uint32_t n, kind;
    uint32_t slot[(kSlots + 1) / 2];
    uint32_t pad[4];
};
static_assert(sizeof(Item) == 64 && kBatchMaxT * (kMaxK + 1) <= 65536, "items");
__host__ __device__ inline int shared_items(bool shared, int T, int per) { return shared ? 2 * ((T + per - 1) / per) : 0; }

struct BatchArgs {
    int H, I, E, k, T, Ip, ks, per, items_n;  // Ip: I up to whole 32; ks: parts of the router's sums; per: assignments of an item; items_n: places for items
    const float *x, *Wr;
    const uint8_t* mask;
    const void* const* ptrs;
    const uint16_t *sg, *su, *sd;
    float* y;
    int32_t* idx_out;
    float* w_out;
    // workspace
    uint32_t* ticket;  // tokens routed
    Item* items;
    float* logits;     // [ks][T][E], parts of the sums
    uint16_t* xp;      // [T][3][H]
    int32_t* idx;      // [T][k], -1: a token left out
    float* w;          // [T][k]
    uint16_t* hp;      // [T k + T][3][Ip]
    float* out;        // [T k + T][H]
};

int max_items(int E, int k, int T, bool shared, int per) {
    const int a = T * k, n = E + a / per;
    return (a < n ? a : n) + shared_items(shared, T, per);
}

// The three bf16 parts of v, cut (all 24 bits down to 2^-133); those behind an
// infinity or a NaN are 0.
__device__ __forceinline__ void parts3(float v, uint32_t (&h)[3]) {
#pragma unroll
    for (int p = 0; p < 3; p++) {
        h[p] = v != v ? 0x7FC0u : __float_as_uint(v) >> 16;
        v = fabsf(v) < INFINITY ? v - __uint_as_float(h[p] << 16) : 0.0f;
    }
}

// ---------------------------------------------------------------------------
// 1. front: nr router tiles (16 experts x 16 tokens x a part of the sum, four
// waves along it; the parts are added when the top-k reads them), then
// workgroups for the activations' parts. All of a wave's loads go out at once.
constexpr int kFrontSteps = 8;  // of 16 in the sum a wave and round

__global__ __launch_bounds__(256) void k_batch_front(BatchArgs a, int et, int nr) {
    __shared__ f4v part[4][64];
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = wave_id();
    if (b >= nr) {
        if (b == nr && tid == 0) *a.ticket = 0;
        const int h8 = a.H / 8, i = (b - nr) * 256 + tid, t = i / h8, c = i - t * h8;
        if (t < a.T) {
            float v[8];
            unpack8<kActF32>(load8<kActF32>(a.x + (size_t)t * a.H, 8 * c), v);
            uint32_t h[8][3];
#pragma unroll
            for (int j = 0; j < 8; j++) parts3(v[j], h[j]);
#pragma unroll
            for (int p = 0; p < 3; p++)
                *reinterpret_cast<u4w*>(a.xp + ((size_t)t * 3 + p) * a.H + 8 * c) =
                    u4w{h[0][p] | h[1][p] << 16, h[2][p] | h[3][p] << 16, h[4][p] | h[5][p] << 16, h[6][p] | h[7][p] << 16};
        }
        return;
    }
    const int ks = b % a.ks, e0 = b / a.ks % et * 16, t0 = b / a.ks / et * 16, li = lane & 15, lg = lane >> 4;
    const rsrc_t rw = make_rsrc(a.Wr + (size_t)e0 * a.H, (uint32_t)min(16, a.E - e0) * a.H * 4u);
    const rsrc_t rx = make_rsrc(a.x + (size_t)t0 * a.H, (uint32_t)min(16, a.T - t0) * a.H * 4u);
    const uint32_t ow = e0 + li < a.E ? (uint32_t)li * a.H * 4u : kOOB, ox = t0 + li < a.T ? (uint32_t)li * a.H * 4u : kOOB;
    const int kw = a.H / (4 * a.ks), k0 = (4 * ks + wave) * kw;  // a multiple of 16
    f4v acc = {0.f, 0.f, 0.f, 0.f};
    for (int k = k0; k < k0 + kw; k += 16 * kFrontSteps) {
        f4v w[kFrontSteps], x[kFrontSteps];
#pragma unroll
        for (int i = 0; i < kFrontSteps; i++) {
            const bool on = k + 16 * i < k0 + kw;
            const uint32_t c = (uint32_t)(k + 16 * i + 4 * lg) * 4u;
            w[i] = __builtin_bit_cast(f4v, ld_b128(rw, on && ow != kOOB ? ow + c : kOOB));
            x[i] = __builtin_bit_cast(f4v, ld_b128(rx, on && ox != kOOB ? ox + c : kOOB));
        }
#pragma unroll
        for (int i = 0; i < kFrontSteps; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(w[i][j], x[i][j], acc, 0, 0, 0);
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int w = 1; w < 4; w++) acc += part[w][lane];
        const int t = t0 + li, e = e0 + 4 * lg;  // column: token, rows: experts
        if (t < a.T)
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (e + j < a.E) a.logits[((size_t)ks * a.T + t) * a.E + e + j] = acc[j];
    }
}

// ---------------------------------------------------------------------------
// 2. route: a workgroup a token, whose first wave takes the top-k. The last one
// to have done so (a ticket; the choices leave with device-coherent stores)
// groups the assignments by expert. (Left to the expert launches, where every
// workgroup looked through the T k choices for itself, it cost 65 us at 48
// tokens of 10 experts and saved 5 here.)
__global__ __launch_bounds__(256) void k_batch_route(BatchArgs a) {
    __shared__ int count[kMaxE], place[kMaxE], last, run[4][2];
    __shared__ uint16_t order[kBatchMaxT * (kMaxK + 1)];
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = wave_id(), A = a.T * a.k, is = shared_items(a.sg != nullptr, a.T, a.per);
    if (wave == 0) {
        const bool on = !a.mask || a.mask[t];
        int e = -1;
        float w = 0.0f;
        if (on) {
            const float* l = a.logits + (size_t)t * a.E;
            const size_t step = (size_t)a.T * a.E;
            if (a.ks == kRouterParts)
                topk_select([&](int i) { return ((l[i] + l[i + step]) + (l[i + 2 * step] + l[i + 3 * step])) +
                                                ((l[i + 4 * step] + l[i + 5 * step]) + (l[i + 6 * step] + l[i + 7 * step])); }, a.E, a.k, e, w);
            else
                topk_select([&](int i) { return l[i] + l[i + step]; }, a.E, a.k, e, w);
        }
        if (lane < a.k) {
            if (on) {
                a.idx_out[t * a.k + lane] = e;
                a.w_out[t * a.k + lane] = w;
                a.w[t * a.k + lane] = w;
            }
            __hip_atomic_store(a.idx + t * a.k + lane, on ? e : -1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if (lane == 0) last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)a.T - 1u;
    }
    for (int e = tid; e < kMaxE; e += 256) count[e] = 0;
    const void* block[4];  // of this thread's four experts
#pragma unroll
    for (int i = 0; i < 4; i++) block[i] = 4 * tid + i < a.E ? a.ptrs[4 * tid + i] : nullptr;
    __syncthreads();
    if (!last) return;
    constexpr int NA = kBatchMaxT * kMaxK / 256;
    int mine[NA];
#pragma unroll
    for (int i = 0; i < NA; i++) {
        const int q = tid + 256 * i;
        mine[i] = q < A ? __hip_atomic_load(a.idx + q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : -1;
    }
#pragma unroll
    for (int i = 0; i < NA; i++)
        if (mine[i] >= 0) atomicAdd(&count[mine[i]], 1);
    __syncthreads();
    int c[4], n = 0, m = 0;  // assignments and items of four experts
#pragma unroll
    for (int i = 0; i < 4; i++) {
        c[i] = count[4 * tid + i];
        n += c[i];
        m += (c[i] + a.per - 1) / a.per;
    }
    int ns = n, ms = m;  // inclusive over the wave
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int pn = __shfl_up(ns, o, 64), pm = __shfl_up(ms, o, 64);
        if (lane >= o) {
            ns += pn;
            ms += pm;
        }
    }
    if (lane == 63) {
        run[wave][0] = ns;
        run[wave][1] = ms;
    }
    __syncthreads();
    int n0 = ns - n, m0 = is + ms - m;  // the shared expert's items come first: they have the most bytes
    for (int w = 0; w < wave; w++) {
        n0 += run[w][0];
        m0 += run[w][1];
    }
    const int all = run[0][0] + run[1][0] + run[2][0] + run[3][0], items = is + run[0][1] + run[1][1] + run[2][1] + run[3][1];
    int first = n0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        place[4 * tid + i] = first;
        first += c[i];
    }
    __syncthreads();
    // the order within an expert is free: a column's sum does not depend on its neighbours
#pragma unroll
    for (int i = 0; i < NA; i++)
        if (mine[i] >= 0) order[atomicAdd(&place[mine[i]], 1)] = (uint16_t)(tid + 256 * i);
    int live = 0;  // tokens for the shared expert
    if (is) {
        const bool on = lane < a.T && (!a.mask || a.mask[lane]);
        const unsigned long long b = __ballot(on);
        live = (int)__popcll(b);
        if (on && wave == 0) order[all + (int)__popcll(b & ((1ull << lane) - 1))] = (uint16_t)(A + lane);
    }
    __syncthreads();
    auto put = [&](int at, const void* blk, uint32_t kind, int from, int len) {
        Item it;
        it.block = blk;
        it.n = (uint32_t)len;
        it.kind = kind;
#pragma unroll
        for (int u = 0; u < kSlots; u += 2) {
            const uint32_t lo = order[from + (u < len ? u : 0)], hi = u + 1 < len ? order[from + u + 1] : 0u;
            it.slot[u / 2] = lo | hi << 16;
        }
        a.items[at] = it;
    };
    first = n0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        for (int o = 0; o < c[i]; o += a.per) put(m0++, block[i], kRouted, first + o, c[i] - o < a.per ? c[i] - o : a.per);
        first += c[i];
    }
    if (tid < is) {  // each of the two halves of 32 rows has an item of its own
        const int from = tid / 2 * a.per, left = live - from;
        if (left > 0) put(tid, nullptr, kSharedLow + (tid & 1), all + from, left < a.per ? left : a.per);
        else a.items[tid].n = 0;
    }
    for (int i = items + tid; i < a.items_n; i += 256) a.items[i].n = 0;
}

// ---------------------------------------------------------------------------
// Blocks of 256 of the sum. A lane holds 64 values of row l % 16 (sum index 64
// (l / 16) ..) and the same 64 of its column: the two 16-byte loads of a row's
// 32 bytes of codes go out together, so that a row's 128 bytes are one cache
// line's.

template <int FMT>
struct Wide {  // a block of 4-bit rows
    u4w c[2];
    uint32_t s;  // NVFP4: four scale bytes; MXFP4: two
};
// A lane's offsets stay in registers (kOOB: a row that is not there) and the
// block's go into the scalar offset, so that a load costs no arithmetic.
__device__ __forceinline__ u4w at_b128(rsrc_t r, uint32_t v, uint32_t s) {
    return __builtin_bit_cast(u4w, __builtin_amdgcn_raw_buffer_load_b128(r, v, s, 0));
}
// k: the lane's first of the block, s: the block's first. WHOLE: the block is
// all there; otherwise what is behind K becomes zeros. AL: rows of scales are
// aligned for one load (K a multiple of 64).
template <int FMT, bool AL, bool WHOLE>
__device__ __forceinline__ Wide<FMT> fetch_w(rsrc_t r, uint32_t codes, uint32_t scales, uint32_t k, uint32_t s, uint32_t K) {
    constexpr uint32_t G = Fmt<FMT>::G;
    Wide<FMT> q;
    const bool o0 = WHOLE || k + s < K, o1 = WHOLE || k + s + 32 < K;
    q.c[0] = at_b128(r, o0 ? codes : kOOB, s / 2);
    q.c[1] = at_b128(r, o1 && codes != kOOB ? codes + 16 : kOOB, s / 2);
    if constexpr (FMT == kFmtNvfp4) {
        if constexpr (AL) {
            q.s = __builtin_amdgcn_raw_buffer_load_b32(r, o0 ? scales : kOOB, s / G, 0);
        } else {
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; i++)
                b[i] = __builtin_amdgcn_raw_buffer_load_b8(r, (WHOLE || k + s + 16 * i < K) && scales != kOOB ? scales + i : kOOB, s / G, 0);
            q.s = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
            if (!WHOLE) {  // the next row's
                if (k + s + 16 >= K) q.c[0][2] = q.c[0][3] = 0u;
                if (k + s + 48 >= K) q.c[1][2] = q.c[1][3] = 0u;
            }
        }
    } else {
        if constexpr (AL)
            q.s = __builtin_amdgcn_raw_buffer_load_b16(r, o0 ? scales : kOOB, s / G, 0);
        else
            q.s = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(r, o0 ? scales : kOOB, s / G, 0) |
                  (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(r, o1 && scales != kOOB ? scales + 1 : kOOB, s / G, 0) << 8;
    }
    return q;
}
template <int FMT>
__device__ __forceinline__ void widen_w(const Wide<FMT>& q, int h, u4w (&w)[4]) {
    constexpr int M = FMT == kFmtNvfp4 ? kNvBf16 : kMxBf16;
#pragma unroll
    for (int s = 0; s < 4; s++) w[s] = decode_op<M>(q.c[h][s], scale_op<M>(q.s >> (FMT == kFmtNvfp4 ? 16 * h + 8 * (s / 2) : 8 * h)));
}

// The columns of an item: lane l's row of the parts in each group (byte
// offset). div: slots of one row (gate/up: the k of a token), sub: the first
// slot's number (the shared expert's in gate/up).
__device__ __forceinline__ int slot_of(const Item* it, int u) { return (int)(it->slot[u / 2] >> (16 * (u & 1)) & 0xFFFFu); }
// Slot 5 g + j, j this lane's (0 .. 4).
__device__ __forceinline__ int lane_slot(const Item* it, int g, int j) {
    int s = slot_of(it, g * kTok);
#pragma unroll
    for (int u = 1; u < kTok; u++) {
        const int v = slot_of(it, g * kTok + u);
        s = j == u ? v : s;
    }
    return s;
}
template <int NG>
__device__ __forceinline__ void columns(const Item* it, int sub, int div, int rowlen, uint32_t (&col)[NG]) {
    const int li = threadIdx.x & 15, j = li % kTok, p = li / kTok;
#pragma unroll
    for (int g = 0; g < NG; g++)
        col[g] = p < 3 && g * kTok + j < (int)it->n ? ((uint32_t)((lane_slot(it, g, j) - sub) / div) * 3u + p) * (uint32_t)rowlen * 2u : kOOB;
}

// Half h (32 values a lane) of block s; col: with the lane's first value.
template <int NG, bool WHOLE>
__device__ __forceinline__ void fetch_x(rsrc_t rx, uint32_t const (&col)[NG], int ng, uint32_t k, uint32_t s, uint32_t K, u4w (&x)[NG][4]) {
#pragma unroll
    for (int g = 0; g < NG; g++)
        if (NG == 1 || g < ng)
#pragma unroll
            for (int i = 0; i < 4; i++) x[g][i] = at_b128(rx, (WHOLE || k + s < K) && col[g] != kOOB ? col[g] + 16 * i : kOOB, 2 * s);
}
template <int NG>
__device__ __forceinline__ void multiply(const u4w (&w)[4], const u4w (&x)[NG][4], int ng, f4v (&acc)[NG]) {
#pragma unroll
    for (int g = 0; g < NG; g++)
        if (NG == 1 || g < ng)
#pragma unroll
            for (int s = 0; s < 4; s++) acc[g] = mma16<false>(w[s], x[g][s], acc[g]);
}

// acc[m][i][g] += rows x columns over the whole blocks b0 .. b1 - 1 (TAIL: and
// what lies behind them up to K): M matrices of two row blocks. AHEAD: the next
// block's codes and column values are on their way while a block is multiplied;
// without it a block's column values go out before its codes, and other waves'
// loads are on their way.
template <int FMT, bool AL, bool TAIL, int M, int NG, bool AHEAD>
__device__ __forceinline__ void sums(rsrc_t const (&r)[M], uint32_t const (&codes)[M][2], uint32_t const (&scales)[M][2], rsrc_t rx,
                                     uint32_t const (&col)[NG], int ng, uint32_t K, int b0, int b1, f4v (&acc)[M][2][NG]) {
    const uint32_t lg = (threadIdx.x & 63) >> 4;
    struct Set {
        Wide<FMT> w[M][2];
    };
    struct Cols {
        u4w x[2][NG][4];
    };
    uint32_t c2[NG];  // of a lane's second half
#pragma unroll
    for (int g = 0; g < NG; g++) c2[g] = col[g] == kOOB ? kOOB : col[g] + 64;
    auto fetch = [&](int b, Set& q) {
#pragma unroll
        for (int m = 0; m < M; m++)
#pragma unroll
            for (int i = 0; i < 2; i++) q.w[m][i] = fetch_w<FMT, AL, true>(r[m], codes[m][i], scales[m][i], 0, 256u * b, K);
    };
    auto fetch_c = [&](int b, Cols& c) {
        fetch_x<NG, true>(rx, col, ng, 0, 256u * b, K, c.x[0]);
        fetch_x<NG, true>(rx, c2, ng, 0, 256u * b, K, c.x[1]);
    };
    auto products = [&](const Cols& c, const Set& q) {
        __builtin_amdgcn_sched_barrier(0);  // the loads go out before the products
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int m = 0; m < M; m++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    u4w w[4];
                    widen_w<FMT>(q.w[m][i], h, w);
                    multiply<NG>(w, c.x[h], ng, acc[m][i]);
                }
        __builtin_amdgcn_sched_barrier(0);
    };
    Set q0, q1;
    Cols c0, c1;
    const uint32_t rest = 256u * b1, k = 64 * lg;
    if (TAIL && rest < K) {  // the block that is not all there, first
#pragma unroll
        for (int m = 0; m < M; m++)
#pragma unroll
            for (int i = 0; i < 2; i++) q1.w[m][i] = fetch_w<FMT, AL, false>(r[m], codes[m][i], scales[m][i], k, rest, K);
        fetch_x<NG, false>(rx, col, ng, k, rest, K, c1.x[0]);
        fetch_x<NG, false>(rx, c2, ng, k + 32, rest, K, c1.x[1]);
        if (AHEAD && b0 < b1) fetch(b0, q0);
        if (AHEAD && b0 < b1) fetch_c(b0, c0);
        products(c1, q1);
    } else if (AHEAD && b0 < b1) {
        fetch(b0, q0);
        if (AHEAD) fetch_c(b0, c0);
    }
    for (int b = b0; b < b1; b += 2) {
        if constexpr (!AHEAD) {
            fetch_c(b, c0);
            fetch(b, q0);
            products(c0, q0);
            if (b + 1 < b1) {
                fetch_c(b + 1, c0);
                fetch(b + 1, q0);
                products(c0, q0);
            }
        } else {
            if (b + 1 < b1) {
                fetch(b + 1, q1);
                fetch_c(b + 1, c1);
            }
            products(c0, q0);
            if (b + 2 < b1) {
                fetch(b + 2, q0);
                fetch_c(b + 2, c0);
            }
            if (b + 1 < b1) products(c1, q1);
        }
    }
}

// The same for one row block of bf16 matrices, four times the bytes of 4-bit
// ones: a wave asks for U pieces of 128 of the sum at once and then works
// through them.
template <int M, int NG>
__device__ __forceinline__ void shared_sums(rsrc_t const (&r)[M], uint32_t row, rsrc_t rx, uint32_t const (&col)[NG], int ng, uint32_t K, int b0,
                                            int b1, f4v (&acc)[M][NG]) {
    constexpr int U = M == 1 ? 4 : 3;
    const uint32_t lg = (threadIdx.x & 63) >> 4, at = row == kOOB ? kOOB : row + 64 * lg;
    uint32_t cl[NG];
#pragma unroll
    for (int g = 0; g < NG; g++) cl[g] = col[g] == kOOB ? kOOB : col[g] + 64 * lg;
    for (int b = 2 * b0; b < 2 * b1; b += U) {
        u4w w[U][M][4];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t s = 128u * (b + u);
#pragma unroll
            for (int m = 0; m < M; m++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    w[u][m][j] = at_b128(r[m], at != kOOB && b + u < 2 * b1 && s + 32 * lg + 8 * j < K ? at + 16 * j : kOOB, 2 * s);
        }
#pragma unroll
        for (int u = 0; u < U; u++)
            if (b + u < 2 * b1) {
                u4w x[NG][4];
                fetch_x<NG, false>(rx, cl, ng, 32 * lg, 128u * (b + u), K, x);
#pragma unroll
                for (int m = 0; m < M; m++) multiply<NG>(w[u][m], x, ng, acc[m]);
            }
    }
}

// The sum of a token's three columns: lanes li < 5.
__device__ __forceinline__ float token_sum(float v, int lane) {
    return v + (__shfl(v, lane + kTok, 64) + __shfl(v, lane + 2 * kTok, 64));
}

// ---------------------------------------------------------------------------
// 3. gate/up: grid (row blocks of 32, items), four waves along the sum, whose
// parts meet in LDS.
template <int FMT, int NG, bool AHEAD>
__global__ __launch_bounds__(256) void k_batch_gateup(BatchArgs a, const Item* __restrict__ items) {
    __shared__ f4v part[4][2][2][64];
    const Item* it = items + blockIdx.y;
    const int n_it = (int)it->n;
    if (n_it == 0) return;
    const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4, wave = wave_id(), r0 = blockIdx.x * 32;
    const int ng = (n_it + kTok - 1) / kTok;
    const uint32_t kind = it->kind;
    f4v acc[2][2][NG];
#pragma unroll
    for (int m = 0; m < 2; m++)
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int g = 0; g < NG; g++) acc[m][i][g] = f4v{0.f, 0.f, 0.f, 0.f};
    uint32_t col[NG];
    columns<NG>(it, kind == kRouted ? 0 : a.T * a.k, kind == kRouted ? a.k : 1, a.H, col);
    const rsrc_t rx = make_rsrc(a.xp, (uint32_t)a.T * 3u * a.H * 2u);
    const uint32_t H = a.H, n = (uint32_t)a.H * a.I;
    const int nb = a.H / 256, b0 = wave * nb / 4, b1 = (wave + 1) * nb / 4;
    if (kind == kRouted) {
        constexpr uint32_t G = Fmt<FMT>::G;
        const rsrc_t rw = make_rsrc(it->block, 3 * n / 2 + 3 * n / G);
        const rsrc_t r[2] = {rw, rw};
        uint32_t codes[2][2], scales[2][2], cl[NG];
#pragma unroll
        for (int m = 0; m < 2; m++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const uint32_t row = r0 + 16 * i + li;
                codes[m][i] = (int)row < a.I ? m * (n / 2) + row * (H / 2) + 32 * lg : kOOB;
                scales[m][i] = (int)row < a.I ? 3 * n / 2 + m * (n / G) + row * (H / G) + 64 / G * lg : kOOB;
            }
#pragma unroll
        for (int g = 0; g < NG; g++) cl[g] = col[g] == kOOB ? kOOB : col[g] + 128 * lg;
        sums<FMT, true, false, 2, NG, AHEAD>(r, codes, scales, rx, cl, ng, H, b0, b1, acc);
    } else {
        const rsrc_t r[2] = {make_rsrc(a.sg, 2 * n), make_rsrc(a.su, 2 * n)};
        const int row = r0 + (kind == kSharedHigh ? 16 : 0) + li;
        f4v one[2][NG];
#pragma unroll
        for (int m = 0; m < 2; m++)
#pragma unroll
            for (int g = 0; g < NG; g++) one[m][g] = f4v{0.f, 0.f, 0.f, 0.f};
        shared_sums<2, NG>(r, row < a.I ? (uint32_t)row * H * 2u : kOOB, rx, col, ng, H, b0, b1, one);
#pragma unroll
        for (int m = 0; m < 2; m++)
#pragma unroll
            for (int g = 0; g < NG; g++) {
                if (kind == kSharedLow) acc[m][0][g] = one[m][g];
                else acc[m][1][g] = one[m][g];
            }
    }
#pragma unroll
    for (int g = 0; g < NG; g++) {
        if (NG > 1 && g >= ng) break;
        if (g) __syncthreads();
#pragma unroll
        for (int m = 0; m < 2; m++)
#pragma unroll
            for (int i = 0; i < 2; i++) part[wave][m][i][lane] = acc[m][i][g];
        __syncthreads();
        const int q = threadIdx.x, j = q / 32, row = q % 32, i = row >> 4;  // a token's 32 rows
        if (j < kTok && g * kTok + j < n_it && (kind == kRouted || (kind == kSharedHigh) == (i == 1))) {
            float v[2] = {0.0f, 0.0f};
            const int l = (row & 15) >> 2, c = row & 3;
#pragma unroll
            for (int m = 0; m < 2; m++)
#pragma unroll
                for (int p = 2; p >= 0; p--)
#pragma unroll
                    for (int w = 0; w < 4; w++) v[m] += reinterpret_cast<const float*>(&part[w][m][i][16 * l + kTok * p + j])[c];
            uint32_t h[3];
            parts3(silu_mul(v[0], v[1]), h);
            uint16_t* to = a.hp + (size_t)lane_slot(it, g, j) * 3 * a.Ip + r0 + row;
#pragma unroll
            for (int p = 0; p < 3; p++) to[(size_t)p * a.Ip] = (uint16_t)h[p];  // rows behind the last one: zeros, up to Ip
        }
    }
}

// ---------------------------------------------------------------------------
// 4. down: grid (row blocks of 128, items), 32 rows a wave.
template <int FMT, bool AL, int NG>
__global__ __launch_bounds__(256) void k_batch_down(BatchArgs a, const Item* __restrict__ items) {
    const Item* it = items + blockIdx.y;
    const int n_it = (int)it->n;
    if (n_it == 0) return;
    const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4, r0 = blockIdx.x * 128 + wave_id() * 32;
    const int ng = (n_it + kTok - 1) / kTok;
    const uint32_t kind = it->kind;
    f4v acc[1][2][NG];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int g = 0; g < NG; g++) acc[0][i][g] = f4v{0.f, 0.f, 0.f, 0.f};
    uint32_t col[NG];
    columns<NG>(it, 0, 1, a.Ip, col);
    const rsrc_t rx = make_rsrc(a.hp, (uint32_t)(a.T * a.k + a.T) * 3u * a.Ip * 2u);
    const uint32_t I = a.I, n = (uint32_t)a.H * a.I;
    if (kind == kRouted) {
        constexpr uint32_t G = Fmt<FMT>::G;
        const rsrc_t r[1] = {make_rsrc(it->block, 3 * n / 2 + 3 * n / G)};
        uint32_t codes[1][2], scales[1][2], cl[NG];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t row = r0 + 16 * i + li;
            codes[0][i] = n + row * (I / 2) + 32 * lg;
            scales[0][i] = 3 * n / 2 + 2 * (n / G) + row * (I / G) + 64 / G * lg;
        }
#pragma unroll
        for (int g = 0; g < NG; g++) cl[g] = col[g] == kOOB ? kOOB : col[g] + 128 * lg;
        sums<FMT, AL, true, 1, NG, NG == 1>(r, codes, scales, rx, cl, ng, I, 0, a.I / 256, acc);
    } else {
        const rsrc_t r[1] = {make_rsrc(a.sd, 2 * n)};
        f4v one[1][NG];
#pragma unroll
        for (int g = 0; g < NG; g++) one[0][g] = f4v{0.f, 0.f, 0.f, 0.f};
        shared_sums<1, NG>(r, (uint32_t)(r0 + (kind == kSharedHigh ? 16 : 0) + li) * I * 2u, rx, col, ng, I, 0, (a.I + 255) / 256, one);
#pragma unroll
        for (int g = 0; g < NG; g++) {
            if (kind == kSharedLow) acc[0][0][g] = one[0][g];
            else acc[0][1][g] = one[0][g];
        }
    }
#pragma unroll
    for (int g = 0; g < NG; g++)
        if (NG == 1 || g < ng) {
            const bool in = li < kTok && g * kTok + li < n_it;
            float* to = a.out + (in ? (size_t)lane_slot(it, g, li) * a.H + r0 + 4 * lg : 0);
#pragma unroll
            for (int i = 0; i < 2; i++) {
                f4v v = acc[0][i][g];
#pragma unroll
                for (int c = 0; c < 4; c++) v[c] = token_sum(acc[0][i][g][c], lane);
                if (in && (kind == kRouted || (kind == kSharedHigh) == (i == 1))) *reinterpret_cast<f4v*>(to + 16 * i) = v;
            }
        }
}

// ---------------------------------------------------------------------------
// 5. combine: grid (H / 1024 up, T)
__global__ __launch_bounds__(256) void k_batch_combine(BatchArgs a, int shared) {
    const int t = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
    if ((a.mask && !a.mask[t]) || 4 * c >= a.H) return;
    f4v y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int j = 0; j < a.k; j++) {
        const f4v v = reinterpret_cast<const f4v*>(a.out + (size_t)(t * a.k + j) * a.H)[c];
        const float w = a.w[t * a.k + j];
#pragma unroll
        for (int i = 0; i < 4; i++) y[i] = fmaf(w, v[i], y[i]);
    }
    if (shared) y += reinterpret_cast<const f4v*>(a.out + (size_t)(a.T * a.k + t) * a.H)[c];
    float* o = a.y + (size_t)t * a.H + 4 * c;  // y is 4-byte aligned
#pragma unroll
    for (int i = 0; i < 4; i++) o[i] = y[i];
}

template <int NG>
hipError_t experts(int fmt, const BatchArgs& a, hipStream_t s) {
    const dim3 gu((a.I + 31) / 32, a.items_n), down(a.H / 128, a.items_n), block(256);
    const Item* items = a.items;
    // With more workgroups than two rounds of the chip (two a compute unit, of
    // 195 registers a thread) four a compute unit without a block ahead: 48 tokens
    // 163 -> 151 us, while 4 tokens with 800 workgroups take 30 and 32. Three
    // column groups never look ahead: one workgroup a compute unit then (64 tokens
    // of 8 out of 128 experts of 2560 x 640: 117 us, without 81).
    const bool crowd = (size_t)gu.x * gu.y > 1024;
    auto gateup = [&](auto F) {
        constexpr int FMT = decltype(F)::value;
        if constexpr (NG == 1)
            if (!crowd) {
                hipLaunchKernelGGL((k_batch_gateup<FMT, NG, true>), gu, block, 0, s, a, items);
                return;
            }
        hipLaunchKernelGGL((k_batch_gateup<FMT, NG, false>), gu, block, 0, s, a, items);
    };
    if (fmt == kFmtNvfp4) gateup(std::integral_constant<int, kFmtNvfp4>{});
    else gateup(std::integral_constant<int, kFmtMxfp4>{});
    const hipError_t r = hipGetLastError();
    if (r != hipSuccess) return r;
    const bool al = a.I % 64 == 0;
    if (fmt == kFmtNvfp4) {
        if (al) hipLaunchKernelGGL((k_batch_down<kFmtNvfp4, true, NG>), down, block, 0, s, a, items);
        else hipLaunchKernelGGL((k_batch_down<kFmtNvfp4, false, NG>), down, block, 0, s, a, items);
    } else {
        if (al) hipLaunchKernelGGL((k_batch_down<kFmtMxfp4, true, NG>), down, block, 0, s, a, items);
        else hipLaunchKernelGGL((k_batch_down<kFmtMxfp4, false, NG>), down, block, 0, s, a, items);
    }
    return hipGetLastError();
}

struct BatchWs {
    size_t ticket, items, logits, xp, idx, w, hp, out, total;
};
BatchWs batch_plan(int H, int I, int E, int k, int T) {
    BatchWs b;
    size_t at = kCounterBytes;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += align256(n);
        return o;
    };
    const size_t A = (size_t)T * k, S = A + T, Ip = (I + 31) / 32 * 32;
    b.ticket = take(4);
    b.items = take((size_t)max_items(E, k, T, true, kTok) * sizeof(Item));
    b.logits = take((size_t)kRouterParts * T * E * 4);
    b.xp = take((size_t)T * 3 * H * 2);
    b.idx = take(A * 4);
    b.w = take(A * 4);
    b.hp = take(S * 3 * Ip * 2);
    b.out = take(S * H * 4);
    b.total = at;
    return b;
}

}  // namespace

size_t batch_ws_bytes(int fmt, int H, int I, int E, int k, int T) {
    const size_t one = decode_ws_bytes(H, I, k, E), n = batch_plan(H, I, E, k, T).total;  // one token may take the decode kernels
    return one > n ? one : n;
}

hipError_t launch_layer_batch(int fmt, int H, int I, int E, int k, const float* x, int T, const uint8_t* mask,
                              const float* Wr, const void* const* expert_ptrs, const uint16_t* sh_gate,
                              const uint16_t* sh_up, const uint16_t* sh_down, float* y, int32_t* idx_out, float* w_out,
                              void* ws, hipStream_t s) {
    if (T == 1 && !mask) {
        DecodePlan p;
        if (!plan_decode(fmt, H, I, &p)) return hipErrorInvalidValue;
        return launch_layer_decode(fmt, p, E, H, I, k, x, Wr, expert_ptrs, sh_gate, sh_up, sh_down, y, idx_out, w_out, ws, s);
    }
    const BatchWs b = batch_plan(H, I, E, k, T);
    char* p = static_cast<char*>(ws);
    BatchArgs a = {};
    a.H = H; a.I = I; a.E = E; a.k = k; a.T = T; a.Ip = (I + 31) / 32 * 32;
    a.x = x; a.Wr = Wr; a.mask = mask; a.ptrs = expert_ptrs; a.sg = sh_gate; a.su = sh_up; a.sd = sh_down;
    a.y = y; a.idx_out = idx_out; a.w_out = w_out;
    a.ticket = reinterpret_cast<uint32_t*>(p + b.ticket);
    a.items = reinterpret_cast<Item*>(p + b.items);
    a.logits = reinterpret_cast<float*>(p + b.logits);
    a.xp = reinterpret_cast<uint16_t*>(p + b.xp);
    a.idx = reinterpret_cast<int32_t*>(p + b.idx);
    a.w = reinterpret_cast<float*>(p + b.w);
    a.hp = reinterpret_cast<uint16_t*>(p + b.hp);
    a.out = reinterpret_cast<float*>(p + b.out);
    a.ks = T <= 32 ? kRouterParts : 2;  // workgroups for the whole chip, up to two groups of tokens
    const int et = (E + 15) / 16, nr = et * ((T + 15) / 16) * a.ks, shared = sh_gate ? 1 : 0;
    // experts with more tokens than an item are read again: few where the
    // assignments are fewer than two an expert (items of 5 against 15: 48 tokens of 10
    // out of 512 experts of 2560 x 640 255 and 286 us, 64 of 4 out of 128 109 and 122), while
    // items of 15 win from 8 to 16 an expert on (64 of 4 out of 16: 73 and 68; of 8 out of
    // 8: 120 and 104; of 2 out of 16 MXFP4 ones of 4096 x 2880: 194 and 173). In between
    // the border is early: 64 of 8 out of 128 142 and 150, 64 of 4 out of 64 89 and 97, out
    // of 32 77 and 79.
    const int groups = T * k <= 2 * E ? 1 : kMaxGroups;
    a.per = kTok * groups;
    a.items_n = max_items(E, k, T, shared, a.per);
    hipError_t r;
    hipLaunchKernelGGL(k_batch_front, dim3(nr + (T * (H / 8) + 255) / 256), dim3(256), 0, s, a, et, nr);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    hipLaunchKernelGGL(k_batch_route, dim3(T), dim3(256), 0, s, a);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    if ((r = groups == 1 ? experts<1>(fmt, a, s) : experts<kMaxGroups>(fmt, a, s)) != hipSuccess) return r;
    hipLaunchKernelGGL(k_batch_combine, dim3((H / 4 + 255) / 256, T), dim3(256), 0, s, a, shared);
    return hipGetLastError();
}

}  // namespace moe

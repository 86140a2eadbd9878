// Low-rank adapters of many requests at once beside a shared projection, and
// their gradients, for gfx950. Token t uses adapter a = ids[t] (a < 0: none)
// with factors A_a [r][K] and B_a [r][N] (both rank-major, so that each
// streams along its long axis whatever the rank) and scale s_a:
//   u_t = s_a A_a x_t          y_t  = base_t + B_a^T u_t
//   v_t = s_a B_a dy_t         dx_t = dx_base_t + A_a^T v_t
//   dA_a = sum_t v_t x_t^T     dB_a = sum_t u_t dy_t^T
// So there are three kinds of product, all with a factor of r rows: "down"
// (long axis to rank), "up" (rank to long axis, added to a base) and "grad"
// (an outer product summed over an adapter's tokens). u, v and every sum are
// fp32. The products run on the 16-bit matrix instructions: 16-bit operands
// as they are, and fp32 ones as three bf16 parts, each the truncation of what
// the ones before left, which hold all 24 bits over the whole fp32 range (the
// fp32 instructions run at a sixteenth of the rate; against fp32 u and v an
// fp16 operand enters as two bf16 parts, exactly).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_learn.h"

namespace moe {

namespace {

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef _Float16 h8v __attribute__((ext_vector_type(8)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef uint32_t u2v __attribute__((ext_vector_type(2)));

constexpr int kTile = 64;        // tokens of a tile of one adapter
constexpr int kDirectMaxT = 64;  // tokens up to which no grouping is done
constexpr int kUpCols = 256;     // columns of a workgroup of "up" and "grad"

// ---- element types ----
template <int ACT>
struct Act;
template <>
struct Act<kActF32> {
    typedef float T;
};
template <>
struct Act<kActBf16> {
    typedef uint16_t T;
};
template <>
struct Act<kActF16> {
    typedef uint16_t T;
};

__device__ __forceinline__ float f16_bits(uint32_t lo16) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)lo16);
}
// Two 16-bit factor elements -> fp32 (bf16 for fp32 and bf16 activations).
template <int ACT>
__device__ __forceinline__ void cvt2(uint32_t w, float& a, float& b) {
    if constexpr (ACT == kActF16) {
        a = f16_bits(w & 0xFFFFu);
        b = f16_bits(w >> 16);
    } else {
        a = bf16_lo(w);
        b = bf16_hi(w);
    }
}
// fp32 -> bf16 bits, round to nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t to_bf16(float f) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);
}
// Four consecutive activations as fp32, and back (one rounding).
template <int ACT>
__device__ __forceinline__ f4v ld4(const typename Act<ACT>::T* p) {
    if constexpr (ACT == kActF32) {
        return *reinterpret_cast<const f4v*>(p);
    } else {
        const u2v w = *reinterpret_cast<const u2v*>(p);
        f4v v;
        float a, b;
        cvt2<ACT>(w.x, a, b); v.x = a; v.y = b;
        cvt2<ACT>(w.y, a, b); v.z = a; v.w = b;
        return v;
    }
}
template <int ACT>
__device__ __forceinline__ void st4(typename Act<ACT>::T* p, f4v v) {
    if constexpr (ACT == kActF32) {
        *reinterpret_cast<f4v*>(p) = v;
    } else if constexpr (ACT == kActBf16) {
        *reinterpret_cast<u2v*>(p) = u2v{to_bf16(v.x) | to_bf16(v.y) << 16, to_bf16(v.z) | to_bf16(v.w) << 16};
    } else {
        auto h = [](float f) { return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f); };
        *reinterpret_cast<u2v*>(p) = u2v{h(v.x) | h(v.y) << 16, h(v.z) | h(v.w) << 16};
    }
}

// Eight consecutive activations and eight factor elements, multiplied into
// fp32 by fma.
template <int ACT>
__device__ __forceinline__ float dot8(const typename Act<ACT>::T* x, u4v w, float acc) {
    const f4v x0 = ld4<ACT>(x), x1 = ld4<ACT>(x + 4);
    float a, b;
    cvt2<ACT>(w.x, a, b); acc = fmaf(a, x0.x, acc); acc = fmaf(b, x0.y, acc);
    cvt2<ACT>(w.y, a, b); acc = fmaf(a, x0.z, acc); acc = fmaf(b, x0.w, acc);
    cvt2<ACT>(w.z, a, b); acc = fmaf(a, x1.x, acc); acc = fmaf(b, x1.y, acc);
    cvt2<ACT>(w.w, a, b); acc = fmaf(a, x1.z, acc); acc = fmaf(b, x1.w, acc);
    return acc;
}

// The rank of adapter a, or -1 where the table's rank is not in [0, R].
__device__ __forceinline__ int rank_of(const int32_t* __restrict__ ranks, int a, int R) {
    const int r = ranks[a];
    return r < 0 || r > R ? -1 : r;
}

// ---------------------------------------------------------------------------
// Few tokens: no grouping, every token on its own.

// grid (T, ceil(R / 4)), 256 threads: a wave makes one value of u.
template <int ACT>
__global__ __launch_bounds__(256) void k_lora_down_tok(const typename Act<ACT>::T* __restrict__ x, size_t ldx, int K,
                                                       int n, int R, LoraTable tab, float* __restrict__ u) {
    const int lane = threadIdx.x & 63, t = blockIdx.x, i = blockIdx.y * 4 + wave_id();
    const int a = tab.ids[t];
    if (a < 0 || a >= n) return;
    const int r = rank_of(tab.ranks, a, R);
    if (i >= r) return;
    const uint16_t* row = reinterpret_cast<const uint16_t*>(tab.a[a]) + (size_t)i * K;
    const typename Act<ACT>::T* xt = x + (size_t)t * ldx;
    float acc = 0.0f;
#pragma unroll 4
    for (int p = lane * 8; p < K; p += 512) acc = dot8<ACT>(xt + p, *reinterpret_cast<const u4v*>(row + p), acc);
    acc = wave_sum(acc);
    if (lane == 0) u[(size_t)t * R + i] = tab.scales[a] * acc;
}

// grid (T, ceil(N / 1024)), 256 threads: four columns of y a thread.
template <int ACT>
__global__ __launch_bounds__(256) void k_lora_up_tok(const float* __restrict__ u, int N, int n, int R, LoraTable tab,
                                                     const typename Act<ACT>::T* base, size_t ldb,
                                                     typename Act<ACT>::T* y, size_t ldy) {
    const int t = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 4;
    if (c >= N) return;
    const int a = tab.ids[t];
    f4v v = {0.f, 0.f, 0.f, 0.f};
    if (base) v = ld4<ACT>(base + (size_t)t * ldb + c);
    if (a >= 0) {
        const int r = a < n ? rank_of(tab.ranks, a, R) : -1;
        if (r < 0) {
            v.x = v.y = v.z = v.w = __builtin_nanf("");
        } else {
            const uint16_t* B = reinterpret_cast<const uint16_t*>(tab.b[a]) + c;
            const float* ut = u + (size_t)t * R;
            f4v s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
            for (int i = 0; i < r; i++) {
                const u2v w = *reinterpret_cast<const u2v*>(B + (size_t)i * N);
                float p, q;
                cvt2<ACT>(w.x, p, q); s.x = fmaf(p, ut[i], s.x); s.y = fmaf(q, ut[i], s.y);
                cvt2<ACT>(w.y, p, q); s.z = fmaf(p, ut[i], s.z); s.w = fmaf(q, ut[i], s.w);
            }
            v += s;
        }
    }
    st4<ACT>(y + (size_t)t * ldy + c, v);
}

// ---------------------------------------------------------------------------
// Many tokens: grouped by adapter.

// A tile (or piece) of a group: group g, grouped rows row .. row + rows - 1.
// Groups 0 .. n-1 are the adapters, n the tokens whose id is not below n,
// n + 1 those without an adapter. The j-th tile of a group that starts at
// grouped row f has the slot f / 64 + g + j: later tiles have higher slots
// and no two share one. Slots without a tile have rows 0.
struct Slot {
    int32_t g, row, rows, pad;
};
struct Group {
    int32_t row, rows;
};

// The low values u and v, as "down" leaves them for what follows, in bf16
// parts (chunks of 8 values of one part):
//   by token  [3][T][R32 / 8]             grouped rows, for "up" (R32: at least 32)
//   by rank   [tile slot][3][R16][8]      chunk c (tokens 8 c .. of the tile) of
//             rank k at place c ^ (k & 7), so that neighbouring ranks' reads
//             from LDS fall on different banks, for "grad"
struct LoraWs {
    int R16, R32, slots, piece, pslots, ks;
    size_t perm, groups, tiles, pieces, tickets, part, ut, vt, ur, vr, grad, total;
};

int col_blocks(int cols) { return (cols + kUpCols - 1) / kUpCols; }

LoraWs lora_ws(int K, int N, int n, int R, int T, bool backward) {
    LoraWs w = {};
    w.R16 = R <= 16 ? 16 : (R <= 32 ? 32 : (R <= 64 ? 64 : 128));
    w.R32 = w.R16 < 32 ? 32 : w.R16;
    w.slots = T / kTile + n + 3;
    // tokens of a piece of the gradient: about 512 workgroups, so that the
    // parts that k_lora_grad_reduce adds stay few
    const int64_t piece = ((int64_t)T * (col_blocks(K) + col_blocks(N)) / 512 + kTile - 1) / kTile * kTile;
    w.piece = (int)(piece < 2 * kTile ? 2 * kTile : (piece > 4096 ? 4096 : piece));
    w.pslots = T / w.piece + n + 3;
    // parts of the long axis of "down", so that short batches fill the chip
    // (about 512 workgroups), at most 8 and at least four steps of 64 a wave
    const int tiles = T / kTile + 1 + (n < T ? n : T) / 2;
    const int steps = ((backward && N < K ? N : K) + 63) / 64;
    int ks = (512 + tiles - 1) / tiles;
    if (ks > 8) ks = 8;
    while (ks > 1 && steps / ks < 16) ks--;
    w.ks = ks;
    size_t o = kCounterBytes;
    auto take = [&o](size_t bytes) {
        const size_t at = o;
        o += align256(bytes);
        return at;
    };
    if (!backward && T <= kDirectMaxT) {
        w.ut = take((size_t)T * R * 4);
        w.total = o;
        return w;
    }
    const int sides = backward ? 2 : 1;
    w.perm = take((size_t)T * 4);
    w.groups = take((size_t)(n + 2) * sizeof(Group));
    w.tiles = take((size_t)w.slots * sizeof(Slot));
    w.pieces = take(backward ? (size_t)w.pslots * sizeof(Slot) : 0);
    w.tickets = take((size_t)w.slots * 2 * 4);
    w.part = take(ks > 1 ? (size_t)sides * ks * T * w.R16 * 4 : 0);
    const size_t by_token = (size_t)T * w.R32 * 6, by_rank = (size_t)w.slots * w.R16 * kTile * 6;
    w.ut = take(backward ? 0 : by_token);
    w.vt = take(backward ? by_token : 0);
    w.ur = take(backward ? by_rank : 0);
    w.vr = take(backward ? by_rank : 0);
    w.grad = take(backward ? (size_t)w.pslots * w.R16 * ((size_t)K + N) * 4 : 0);
    w.total = o;
    return w;
}

// grid n + 2, 1024 threads: group g counts the tokens before it and its own,
// lists its own in increasing t, and writes its tiles and pieces. Eight ids a
// thread are loaded at once (batches of up to 8192 tokens are read once), and
// a wave's places among 8192 tokens come from one table of counts in LDS.
constexpr int kPlanIds = 8;
__global__ __launch_bounds__(1024) void k_lora_plan(const int32_t* __restrict__ ids, int T, int n,
                                                    int32_t* __restrict__ perm, Group* __restrict__ groups,
                                                    Slot* __restrict__ tiles, Slot* __restrict__ pieces, int piece,
                                                    uint32_t* __restrict__ tickets, int slots) {
    __shared__ int acc[2];
    __shared__ int wsum[kPlanIds * 16];  // own tokens of each wave's 64 ids, then the places of their first
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = blockIdx.x;
    constexpr int SPAN = 1024 * kPlanIds;
    int key[kPlanIds];  // -1 behind the end
    auto load = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kPlanIds; i++) {
            const int t = t0 + 1024 * i + tid;
            const int a = ids[min(t, T - 1)];
            key[i] = t < T ? (a < 0 ? n + 1 : min(a, n)) : -1;
        }
    };
    if (tid < 2) acc[tid] = 0;
    __syncthreads();
    int less = 0, own = 0;
    for (int t0 = 0; t0 < T; t0 += SPAN) {
        load(t0);
#pragma unroll
        for (int i = 0; i < kPlanIds; i++) {
            less += key[i] >= 0 && key[i] < g;
            own += key[i] == g;
        }
    }
    if (less) atomicAdd(&acc[0], less);
    if (own) atomicAdd(&acc[1], own);
    __syncthreads();
    const int first = acc[0], count = acc[1];
    int at = first;
    for (int t0 = 0; count && t0 < T; t0 += SPAN) {
        if (T > SPAN) load(t0);
        unsigned long long mine[kPlanIds];
#pragma unroll
        for (int i = 0; i < kPlanIds; i++) {
            mine[i] = __ballot(key[i] == g);
            if (lane == 0) wsum[16 * i + wave] = __popcll(mine[i]);
        }
        __syncthreads();
        int all = 0;
        if (wave == 0) {  // exclusive sums of the 128 counts, two a lane
            const int a = wsum[2 * lane], b = wsum[2 * lane + 1];
            int v = a + b;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int w = __shfl_up(v, o, 64);
                if (lane >= o) v += w;
            }
            wsum[2 * lane] = v - a - b;
            wsum[2 * lane + 1] = v - b;
            if (lane == 63) acc[0] = v;
        }
        __syncthreads();
        all = acc[0];
#pragma unroll
        for (int i = 0; i < kPlanIds; i++)
            if (key[i] == g)
                perm[at + wsum[16 * i + wave] + __popcll(mine[i] & ((1ull << lane) - 1))] = t0 + 1024 * i + tid;
        at += all;
        __syncthreads();
    }
    if (tid == 0) groups[g] = Group{first, count};
    auto list = [&](Slot* out, int size) {
        const int b0 = first / size + g, b1 = (first + count) / size + g + 1;
        const int end = g == n + 1 ? T / size + n + 3 : b1;
        for (int i = b0 + tid; i < end; i += 1024) {
            const int j = (i - b0) * size;
            out[i] = Slot{g, first + j, j < count ? min(size, count - j) : 0, 0};
        }
    };
    list(tiles, kTile);
    if (pieces) list(pieces, piece);
    // the tickets of "down"
    for (int i = g * 1024 + tid; i < 2 * slots; i += (n + 2) * 1024) tickets[i] = 0;
}

// ---- bf16 parts of fp32 ----
__device__ __forceinline__ uint32_t hi16(float f) { return __float_as_uint(f) & 0xFFFF0000u; }
// What truncation to bf16 leaves (0 behind an infinity).
__device__ __forceinline__ float rest(float f) {
    const uint32_t h = hi16(f);
    return __float_as_uint(f) == h ? 0.0f : f - __uint_as_float(h);
}
// The bf16 truncations of a (low half) and b.
__device__ __forceinline__ uint32_t pack_hi(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302);
}
// Eight values as P chunks of bf16 parts.
template <int P>
__device__ __forceinline__ void parts8(const float (&v)[8], u4v (&p)[P]) {
#pragma unroll
    for (int q = 0; q < 4; q++) {
        float a = v[2 * q], b = v[2 * q + 1];
#pragma unroll
        for (int i = 0; i < P; i++) {
            p[i][q] = pack_hi(a, b);
            a = rest(a);
            b = rest(b);
        }
    }
}
__device__ __forceinline__ f4v mma_bf16(u4v a, u4v b, f4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// "down": the two sides of a pass (x with A; dy with B) in one launch.
struct DownJob {
    const void* x;
    size_t ldx;
    int K;
    const void* const* fac;
    float* part;    // [parts][T][R16]
    u4v* by_token;  // either may be null
    u4v* by_rank;
};

// Sixteen consecutive activations of a row, as loaded.
template <int ACT>
struct Raw {
    static constexpr int W = ACT == kActF32 ? 4 : 2;
    u4v w[W];
};
// c += the product of half h (eight values) of x rows and w rows.
template <int ACT>
__device__ __forceinline__ f4v down_mma(const Raw<ACT>& x, int h, u4v w, f4v c) {
    if constexpr (ACT == kActF32) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = __uint_as_float(x.w[2 * h + i / 4][i % 4]);
        u4v p[3];
        parts8<3>(v, p);
#pragma unroll
        for (int i = 2; i >= 0; i--) c = mma_bf16(p[i], w, c);
        return c;
    } else if constexpr (ACT == kActBf16) {
        return mma_bf16(x.w[h], w, c);
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, x.w[h]), __builtin_bit_cast(h8v, w), c, 0, 0, 0);
    }
}
__device__ __forceinline__ u4v ld_b128(rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u4v, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// Steps s0 .. s1 - 1 of 64 of the long axis for NB x 16 tokens and RW x 16
// ranks: lane (i = lane % 16, q = lane / 16) holds the elements 64 s + 16 q ..
// + 15 of rows i, so a row's 128 bytes (16-bit types) arrive by neighbouring
// lanes; which elements a matrix instruction pairs does not matter as long as
// both operands agree. The loads of step s + 1 are under way during step s.
// The elements of the last step that lie behind K are set to 0.
template <int ACT, int NB, int RW>
__device__ __forceinline__ void down_steps(f4v (&acc)[4][RW], const typename Act<ACT>::T* const (&xr)[4], int b0,
                                           rsrc_t rf, const uint32_t (&wo)[RW], int s0, int s1, int K) {
    const int lq = (threadIdx.x & 63) >> 4;
    struct Set {
        Raw<ACT> x[NB];
        u4v w[RW][2];
    } p, q;
    auto load = [&](int s, Set& t) {
        // pieces of eight behind K read the row's first ones
        const int k = 64 * s + 16 * lq;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int o = k + 8 * h < K ? 64 * s + 8 * h : -16 * lq;
#pragma unroll
            for (int b = 0; b < NB; b++)
#pragma unroll
                for (int i = 0; i < Raw<ACT>::W / 2; i++)
                    t.x[b].w[h * Raw<ACT>::W / 2 + i] = reinterpret_cast<const u4v*>(xr[b0 + b] + o)[i];
#pragma unroll
            for (int j = 0; j < RW; j++) t.w[j][h] = ld_b128(rf, wo[j] + (uint32_t)o * 2u);
        }
    };
    auto multiply = [&](int s, Set& t) {
        if (64 * s + 64 > K) {  // uniform: the last step only
            const int k = 64 * s + 16 * lq;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const bool in = k + 8 * h < K;
#pragma unroll
                for (int e = 0; e < 4; e++) {
#pragma unroll
                    for (int b = 0; b < NB; b++)
#pragma unroll
                        for (int i = 0; i < Raw<ACT>::W / 2; i++)
                            t.x[b].w[h * Raw<ACT>::W / 2 + i][e] = in ? t.x[b].w[h * Raw<ACT>::W / 2 + i][e] : 0u;
#pragma unroll
                    for (int j = 0; j < RW; j++) t.w[j][h][e] = in ? t.w[j][h][e] : 0u;
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int b = 0; b < NB; b++)
#pragma unroll
                for (int j = 0; j < RW; j++) acc[b0 + b][j] = down_mma<ACT>(t.x[b], h, t.w[j][h], acc[b0 + b][j]);
    };
    if (s0 >= s1) return;
    load(s0, p);
    for (int s = s0; s < s1; s += 2) {
        load(min(s + 1, s1 - 1), q);
        __builtin_amdgcn_sched_barrier(0);  // the loads stay before the products
        multiply(s, p);
        if (s + 1 >= s1) break;
        load(min(s + 2, s1 - 1), p);
        __builtin_amdgcn_sched_barrier(0);
        multiply(s + 1, q);
    }
}

// grid (slots, parts of the long axis, sides): the low values of one tile over
// one part. Four waves: each takes a quarter of the part's steps and all
// ranks, or above 64 ranks a half of the steps and 64 ranks; operands go from
// memory to registers, and the waves' sums are added in order through LDS.
// Where the axis is in several parts, every workgroup leaves its own with
// device-coherent stores, and the last one of a tile to finish (by a ticket)
// adds them in order. Out go the bf16 parts of the scaled values.
template <int ACT, int RB>
__global__ __launch_bounds__(256) void k_lora_down(DownJob ja, DownJob jb, int n, int R,
                                                   const int32_t* __restrict__ ranks, const float* __restrict__ scales,
                                                   const int32_t* __restrict__ perm, const Slot* __restrict__ tiles,
                                                   int T, uint32_t* __restrict__ tickets) {
    constexpr int RW = RB > 4 ? 4 : RB, KW = 4 * RW / RB;  // rank blocks of a wave, waves along the long axis
    constexpr int R16 = RB * 16, CH = (R16 < 32 ? 32 : R16) / 8;
    __shared__ float red[kTile][R16 + 1];
    __shared__ uint32_t ticket;
    const Slot sl = tiles[blockIdx.x];
    if (sl.rows == 0 || sl.g >= n) return;
    const DownJob j = blockIdx.z ? jb : ja;
    const int r = rank_of(ranks, sl.g, R);
    if (r < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), li = lane & 15, lq = lane >> 4;
    const int kw = wave % KW, r0 = wave / KW * RW;
    const typename Act<ACT>::T* xr[4];
    // rows behind the tile's tokens repeat the last one; their sums are not used
#pragma unroll
    for (int b = 0; b < 4; b++)
        xr[b] = reinterpret_cast<const typename Act<ACT>::T*>(j.x) +
                (size_t)perm[sl.row + min(16 * b + li, sl.rows - 1)] * j.ldx + 16 * lq;
    const rsrc_t rf = make_rsrc(j.fac[sl.g], (uint32_t)r * (uint32_t)j.K * 2u);  // rows behind the rank read 0
    uint32_t wo[RW];
#pragma unroll
    for (int i = 0; i < RW; i++) wo[i] = ((uint32_t)(16 * (r0 + i) + li) * (uint32_t)j.K + (uint32_t)(16 * lq)) * 2u;
    f4v acc[4][RW];
#pragma unroll
    for (int b = 0; b < 4; b++)
#pragma unroll
        for (int i = 0; i < RW; i++) acc[b][i] = f4v{0.f, 0.f, 0.f, 0.f};
    const int steps = (j.K + 63) / 64, parts = gridDim.y * KW, part = blockIdx.y * KW + kw;
    const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
    if (16 * r0 < r) {
        if (sl.rows <= 16) {
            down_steps<ACT, 1, RW>(acc, xr, 0, rf, wo, s0, s1, j.K);
        } else if (sl.rows <= 32) {
            down_steps<ACT, 2, RW>(acc, xr, 0, rf, wo, s0, s1, j.K);
        } else if constexpr (ACT == kActF32) {  // fp32 rows take twice the registers
            down_steps<ACT, 2, RW>(acc, xr, 0, rf, wo, s0, s1, j.K);
            down_steps<ACT, 2, RW>(acc, xr, 2, rf, wo, s0, s1, j.K);
        } else {
            down_steps<ACT, 4, RW>(acc, xr, 0, rf, wo, s0, s1, j.K);
        }
    }
    for (int w = 0; w < KW; w++) {
        if (kw == w)
#pragma unroll
            for (int b = 0; b < 4; b++)
#pragma unroll
                for (int i = 0; i < RW; i++)
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        float* p = &red[16 * b + 4 * lq + q][16 * (r0 + i) + li];
                        *p = w ? *p + acc[b][i][q] : acc[b][i][q];
                    }
        __syncthreads();
    }
    const int ks = gridDim.y, cells = sl.rows * R16;
    if (ks > 1) {
        float* mine = j.part + ((size_t)blockIdx.y * T + sl.row) * R16;
        for (int i = tid; i < cells; i += 256)
            __hip_atomic_store(mine + i, red[i / R16][i % R16], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        // each wave waits for its own stores, then one ticket for all of them
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (tid == 0)
            ticket = __hip_atomic_fetch_add(tickets + blockIdx.z * gridDim.x + blockIdx.x, 1u, __ATOMIC_RELAXED,
                                            __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (ticket + 1 != (uint32_t)ks) return;
        for (int i = tid; i < cells; i += 256) {
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; q++)
                v[q] = __hip_atomic_load(j.part + ((size_t)min(q, ks - 1) * T + sl.row) * R16 + i, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
            float a = v[0];
#pragma unroll
            for (int q = 1; q < 8; q++) a += q < ks ? v[q] : 0.0f;
            red[i / R16][i % R16] = a;
        }
        __syncthreads();
    }
    const float sc = scales[sl.g];
    if (j.by_token)
        for (int i = tid; i < sl.rows * CH; i += 256) {
            const int p = i / CH, c = i % CH;
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; q++) v[q] = 8 * c + q < r ? sc * red[p][min(8 * c + q, R16 - 1)] : 0.0f;
            u4v o[3];
            parts8<3>(v, o);
#pragma unroll
            for (int h = 0; h < 3; h++) j.by_token[((size_t)h * T + sl.row + p) * CH + c] = o[h];
        }
    if (j.by_rank)
        for (int i = tid; i < R16 * 8; i += 256) {
            const int k = i % R16, c = i / R16;
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; q++) v[q] = 8 * c + q < sl.rows && k < r ? sc * red[8 * c + q][k] : 0.0f;
            u4v o[3];
            parts8<3>(v, o);
#pragma unroll
            for (int h = 0; h < 3; h++) j.by_rank[(((size_t)blockIdx.x * 3 + h) * R16 + k) * 8 + (c ^ (k & 7))] = o[h];
        }
}

// Eight rows of four neighbouring 16-bit columns -> for each column a chunk
// of its eight rows.
__device__ __forceinline__ void transpose8x4(const u2v (&w)[8], u4v (&c)[4]) {
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int q = 0; q < 4; q++)
            c[j][q] = __builtin_amdgcn_perm(w[2 * q + 1][j / 2], w[2 * q][j / 2], j % 2 ? 0x07060302 : 0x05040100);
}
// Two fp16 -> the bf16 parts of both: 8 and the last 3 bits, exact.
__device__ __forceinline__ void f16_parts(uint32_t w, uint32_t& hi, uint32_t& lo) {
    const float a = f16_bits(w & 0xFFFFu), b = f16_bits(w >> 16);
    hi = pack_hi(a, b);
    lo = pack_hi(rest(a), rest(b));
}
// Parts of eight rows of four neighbouring values of a 16-bit type, by column.
template <bool F16>
struct Cols16 {
    static constexpr int P = F16 ? 2 : 1;
    u4v c[P][4];
};
template <bool F16>
__device__ __forceinline__ void cols16(const u2v (&w)[8], Cols16<F16>& o) {
    if constexpr (F16) {
        u2v h[8], l[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int d = 0; d < 2; d++) {
                uint32_t a, b;
                f16_parts(w[i][d], a, b);
                h[i][d] = a;
                l[i][d] = b;
            }
        transpose8x4(h, o.c[0]);
        transpose8x4(l, o.c[1]);
    } else {
        transpose8x4(w, o.c[0]);
    }
}
// c += (a's three parts) (b's PB parts), the smallest products first. Part i
// of a value is below 2^(1 - 8 i) of it; the product of two third parts, below
// 2^-30, is left out.
template <int PB>
__device__ __forceinline__ f4v mma_parts(const u4v (&a)[3], const u4v (&b)[PB], f4v c) {
#pragma unroll
    for (int t = 3; t >= 0; t--)
#pragma unroll
        for (int i = 2; i >= 0; i--)
            if (i <= t && t - i < PB) c = mma_bf16(a[i], b[t - i], c);
    return c;
}

// ---------------------------------------------------------------------------
// "up": grid (slots, ceil(N / 256)): y of one tile and 256 columns, 64 a wave,
// everything from memory to registers. The base rows are requested first. Of
// the factor, lane (i, q) loads ranks 8 q .. + 7 of 4 neighbouring columns
// 4 i + j and turns them into one operand for each column, so that a lane ends
// with 4 neighbouring columns of its rows.
template <int ACT, int RB>
__global__ __launch_bounds__(256) void k_lora_up(const u4v* __restrict__ u, int T, int N, int n, int R,
                                                 const void* const* __restrict__ fac,
                                                 const int32_t* __restrict__ ranks, const int32_t* __restrict__ perm,
                                                 const Slot* __restrict__ tiles, const typename Act<ACT>::T* base,
                                                 size_t ldb, typename Act<ACT>::T* y, size_t ldy) {
    constexpr int R16 = RB * 16, R32 = R16 < 32 ? 32 : R16, CH = R32 / 8;
    constexpr bool F16 = ACT == kActF16;
    const Slot sl = tiles[blockIdx.x];
    if (sl.rows == 0) return;
    const bool none = sl.g == n + 1;
    if (none && base == y) return;
    const int lane = threadIdx.x & 63, wave = wave_id(), li = lane & 15, lq = lane >> 4;
    const int c0 = blockIdx.y * kUpCols + wave * 64 + 4 * li, cl = min(c0, N - 4);
    const int mine = perm[sl.row + min(lane, sl.rows - 1)];
    int t[4][4];  // tokens of the lane's rows; rows behind the tile repeat the last one and are not written
#pragma unroll
    for (int b = 0; b < 4; b++)
#pragma unroll
        for (int q = 0; q < 4; q++) t[b][q] = __shfl(mine, 16 * b + 4 * lq + q, 64);
    constexpr int WB = ACT == kActF32 ? 4 : 2;
    typedef uint32_t wv __attribute__((ext_vector_type(WB)));
    wv old[4][4];
    if (base) {
#pragma unroll
        for (int b = 0; b < 4; b++)
#pragma unroll
            for (int q = 0; q < 4; q++) old[b][q] = *reinterpret_cast<const wv*>(base + (size_t)t[b][q] * ldb + cl);
    }
    const int r = none ? 0 : (sl.g == n ? -1 : rank_of(ranks, sl.g, R));
    f4v acc[4][4];
#pragma unroll
    for (int b = 0; b < 4; b++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[b][j] = f4v{0.f, 0.f, 0.f, 0.f};
    if (r > 0) {
        const rsrc_t rf = make_rsrc(fac[sl.g], (uint32_t)r * (uint32_t)N * 2u);  // rows behind the rank read 0
        const int nb = (sl.rows + 15) / 16;
#pragma unroll
        for (int g = 0; g < R32 / 32; g++) {
            if (32 * g >= r) break;
            u2v w[8];
            u4v a[4][3];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint2 x = ld_b64(rf, ((uint32_t)(32 * g + 8 * lq + i) * (uint32_t)N + (uint32_t)cl) * 2u);
                w[i] = u2v{x.x, x.y};
            }
#pragma unroll
            for (int b = 0; b < 4; b++)
#pragma unroll
                for (int h = 0; h < 3; h++)
                    a[b][h] = u[((size_t)h * T + sl.row + min(16 * b + li, sl.rows - 1)) * CH + 4 * g + lq];
            Cols16<F16> f;
            cols16<F16>(w, f);
#pragma unroll
            for (int b = 0; b < 4; b++) {
                if (b >= nb) break;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    u4v p[Cols16<F16>::P];
#pragma unroll
                    for (int h = 0; h < Cols16<F16>::P; h++) p[h] = f.c[h][j];
                    acc[b][j] = mma_parts<Cols16<F16>::P>(a[b], p, acc[b][j]);
                }
            }
        }
    }
    if (c0 >= N) return;
#pragma unroll
    for (int b = 0; b < 4; b++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            f4v v = {acc[b][0][q], acc[b][1][q], acc[b][2][q], acc[b][3][q]};
            if (base) {
                if constexpr (ACT == kActF32) {
                    v += __builtin_bit_cast(f4v, old[b][q]);
                } else {
                    float e, f;
                    cvt2<ACT>(old[b][q][0], e, f); v.x += e; v.y += f;
                    cvt2<ACT>(old[b][q][1], e, f); v.z += e; v.w += f;
                }
            }
            if (r < 0) v.x = v.y = v.z = v.w = __builtin_nanf("");
            if (16 * b + 4 * lq + q < sl.rows) st4<ACT>(y + (size_t)t[b][q] * ldy + c0, v);
        }
}

// ---------------------------------------------------------------------------
// One side of the gradient: D [r][cols] = sum over a piece's tokens of
// low[t][.] row[t][.].
struct GradSide {
    const u4v* low;          // u or v by rank
    const void* row;         // dy or x
    size_t ld;
    int cols;
    float* const* out;       // per adapter, or null
};

// grid (piece slots, column blocks of A then of B): 256 columns, 64 a wave,
// over one piece, a tile of 64 tokens at a time: low's parts go from memory
// straight into LDS, the rows' values into registers, by lane (i, q) as tokens
// 8 q .. + 7 (and 32 more) of 4 neighbouring columns, both a tile ahead; the
// values are turned into an operand for each column. An adapter of one piece
// writes its gradient, others the piece's part for k_lora_grad_reduce.
template <int ACT, int RB>
__global__ __launch_bounds__(256) void k_lora_grad(GradSide ga, GradSide gb, int n, int R, int piece,
                                                   const int32_t* __restrict__ ranks, const int32_t* __restrict__ perm,
                                                   const Group* __restrict__ groups, const Slot* __restrict__ pieces,
                                                   int accumulate, float* __restrict__ part) {
    constexpr int R16 = RB * 16, TILE = 3 * R16 * 8;  // chunks of a tile's low values
    constexpr int WB = ACT == kActF32 ? 4 : 2, PX = ACT == kActF32 ? 3 : (ACT == kActF16 ? 2 : 1);
    typedef uint32_t wv __attribute__((ext_vector_type(WB)));
    __shared__ u4v us[2 * TILE];
    const Slot sl = pieces[blockIdx.x];
    if (sl.rows == 0 || sl.g >= n) return;
    const int r = rank_of(ranks, sl.g, R);
    if (r <= 0) return;
    const int nba = (ga.cols + kUpCols - 1) / kUpCols;
    const bool second = (int)blockIdx.y >= nba;
    const GradSide side = second ? gb : ga;
    float* out = side.out ? side.out[sl.g] : nullptr;
    if (!out) return;
    const int lane = threadIdx.x & 63, wave = wave_id(), li = lane & 15, lq = lane >> 4;
    const int cols = side.cols, c0 = ((int)blockIdx.y - (second ? nba : 0)) * kUpCols + wave * 64 + 4 * li;
    const typename Act<ACT>::T* X = reinterpret_cast<const typename Act<ACT>::T*>(side.row) + min(c0, cols - 4);
    const Group grp = groups[sl.g];
    // the piece's tiles follow one another from this slot
    const u4v* low = side.low + (size_t)(grp.row / kTile + sl.g + (sl.row - grp.row) / kTile) * TILE;
    const rsrc_t rl = make_rsrc(low, (uint32_t)((sl.rows + kTile - 1) / kTile) * (uint32_t)(TILE * 16));
    const int tiles = (sl.rows + kTile - 1) / kTile;
    f4v acc[RB][4];
#pragma unroll
    for (int b = 0; b < RB; b++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[b][j] = f4v{0.f, 0.f, 0.f, 0.f};
    wv x[2][8];
    auto token = [&](int k) { return perm[sl.row + min(64 * k + lane, sl.rows - 1)]; };
    auto fetch = [&](int k, int tok) {
#pragma unroll
        for (int i = 0; i < TILE / 256 + (TILE % 256 ? 1 : 0); i++) {
            const int c = 256 * i + 64 * wave;  // TILE is a multiple of 64: whole waves are in or out
            if (TILE % 256 == 0 || c < TILE)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rl, (__attribute__((address_space(3))) void*)(us + (k & 1) * TILE + c), 16,
                    (uint32_t)(k * TILE + c + lane) * 16u, 0, 0, 0);
        }
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int i = 0; i < 8; i++)
                x[h][i] = *reinterpret_cast<const wv*>(X + (size_t)__shfl(tok, 32 * h + 8 * lq + i, 64) * side.ld);
    };
    int tok = token(0);
    fetch(0, tok);
    tok = token(1);
    for (int k = 0; k < tiles; k++) {
        // tile k is there, and every wave is done with tile k - 1
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        // values of tokens behind the piece are set to 0: they may be NaN
        wv w[2][8];
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int i = 0; i < 8; i++)
#pragma unroll
                for (int d = 0; d < WB; d++) w[h][i][d] = 64 * k + 32 * h + 8 * lq + i < sl.rows ? x[h][i][d] : 0u;
        if (k + 1 < tiles) {
            fetch(k + 1, tok);
            tok = token(k + 2);
        }
        __builtin_amdgcn_sched_barrier(0);  // the next tile's loads stay before this one's products
        const u4v* us_k = us + (k & 1) * TILE;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            if (64 * k + 32 * h >= sl.rows) break;
            u4v f[PX][4];
            if constexpr (ACT == kActF32) {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) v[i] = __uint_as_float(w[h][i][j]);
                    u4v o[3];
                    parts8<3>(v, o);
#pragma unroll
                    for (int q = 0; q < 3; q++) f[q][j] = o[q];
                }
            } else {
                Cols16<ACT == kActF16> c;
                cols16<ACT == kActF16>(w[h], c);
#pragma unroll
                for (int q = 0; q < PX; q++)
#pragma unroll
                    for (int j = 0; j < 4; j++) f[q][j] = c.c[q][j];
            }
#pragma unroll
            for (int b = 0; b < RB; b++) {
                u4v a[3];
#pragma unroll
                for (int q = 0; q < 3; q++) a[q] = us_k[(q * R16 + 16 * b + li) * 8 + ((4 * h + lq) ^ (li & 7))];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    u4v o[PX];
#pragma unroll
                    for (int q = 0; q < PX; q++) o[q] = f[q][j];
                    acc[b][j] = mma_parts<PX>(a, o, acc[b][j]);
                }
            }
        }
    }
    if (c0 >= cols) return;
    const bool whole = grp.rows <= piece;
    typedef __attribute__((address_space(1))) f4v* gp;  // the table's pointers are to global memory
    float* to = whole ? out : part + (size_t)blockIdx.x * R16 * ((size_t)ga.cols + gb.cols) +
                                  (second ? (size_t)R16 * ga.cols : 0);
#pragma unroll
    for (int b = 0; b < RB; b++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int m = 16 * b + 4 * lq + q;
            if (m >= r) continue;
            gp p = (gp)(uintptr_t)(to + (size_t)m * cols + c0);
            f4v v = {acc[b][0][q], acc[b][1][q], acc[b][2][q], acc[b][3][q]};
            if (whole && accumulate) v += *p;
            *p = v;
        }
}

// grid (column blocks of 1024, R, n): gradients of adapters with no token
// (zeros) and with several pieces (the parts, in increasing order); an
// adapter whose rank is not usable gets nothing.
__global__ __launch_bounds__(256) void k_lora_grad_reduce(int ca, int cb, float* const* da, float* const* db, int n,
                                                          int R, int R16, int piece, const int32_t* __restrict__ ranks,
                                                          const Group* __restrict__ groups, int accumulate,
                                                          const float* __restrict__ part) {
    const int a = blockIdx.z, m = blockIdx.y;
    const Group g = groups[a];
    const int r = rank_of(ranks, a, R);
    if (m >= r) return;
    if (g.rows == 0 ? accumulate != 0 : g.rows <= piece) return;
    const int nba = (ca + 1023) / 1024;
    const bool second = (int)blockIdx.x >= nba;
    float* out = second ? (db ? db[a] : nullptr) : (da ? da[a] : nullptr);
    const int cols = second ? cb : ca, c = (((int)blockIdx.x - (second ? nba : 0)) * 256 + (int)threadIdx.x) * 4;
    if (!out || c >= cols) return;
    f4v v = {0.f, 0.f, 0.f, 0.f};
    const int s0 = g.row / piece + a, np = (g.rows + piece - 1) / piece;
    const size_t stride = (size_t)R16 * ((size_t)ca + cb);
    const float* p = part + (size_t)s0 * stride + (second ? (size_t)R16 * ca : 0) + (size_t)m * cols + c;
#pragma unroll 4
    for (int i = 0; i < np; i++) v += *reinterpret_cast<const f4v*>(p + (size_t)i * stride);
    f4v* o = reinterpret_cast<f4v*>(out + (size_t)m * cols + c);
    if (accumulate) v += *o;
    *o = v;
}

// ---- launches ----

template <int ACT>
hipError_t down(const LoraWs& w, int sides, hipStream_t s, const DownJob& a, const DownJob& b, int n, int R,
                const LoraTable& tab, const int32_t* perm, const Slot* tiles, int T, uint32_t* tickets) {
    const dim3 grid(w.slots, w.ks, sides);
#define DN(B)                                                                                                       \
    hipLaunchKernelGGL((k_lora_down<ACT, B>), grid, dim3(256), 0, s, a, b, n, R, tab.ranks, tab.scales, perm, tiles, T, \
                       tickets)
    if (w.R16 == 16) DN(1); else if (w.R16 == 32) DN(2); else if (w.R16 == 64) DN(4); else DN(8);
#undef DN
    return hipGetLastError();
}

template <int ACT>
hipError_t up(const LoraWs& w, hipStream_t s, const u4v* u, int T, int N, int n, int R, const void* const* fac,
              const LoraTable& tab, const int32_t* perm, const Slot* tiles, const void* base, size_t ldb, void* y,
              size_t ldy) {
    typedef typename Act<ACT>::T E;
    const dim3 grid(w.slots, col_blocks(N));
#define UP(B)                                                                                                      \
    hipLaunchKernelGGL((k_lora_up<ACT, B>), grid, dim3(256), 0, s, u, T, N, n, R, fac, tab.ranks, perm, tiles, (const E*)base, \
                       ldb, (E*)y, ldy)
    if (w.R16 == 16) UP(1); else if (w.R16 == 32) UP(2); else if (w.R16 == 64) UP(4); else UP(8);
#undef UP
    return hipGetLastError();
}

// The workspace's regions.
struct LoraMem {
    int32_t* perm;
    Group* groups;
    Slot *tiles, *pieces;
    uint32_t* tickets;
    float *part, *grad;
    u4v *ut, *vt, *ur, *vr;
    LoraMem(const LoraWs& w, void* ws) {
        char* b = reinterpret_cast<char*>(ws);
        perm = reinterpret_cast<int32_t*>(b + w.perm);
        groups = reinterpret_cast<Group*>(b + w.groups);
        tiles = reinterpret_cast<Slot*>(b + w.tiles);
        pieces = reinterpret_cast<Slot*>(b + w.pieces);
        tickets = reinterpret_cast<uint32_t*>(b + w.tickets);
        part = reinterpret_cast<float*>(b + w.part);
        grad = reinterpret_cast<float*>(b + w.grad);
        ut = reinterpret_cast<u4v*>(b + w.ut);
        vt = reinterpret_cast<u4v*>(b + w.vt);
        ur = reinterpret_cast<u4v*>(b + w.ur);
        vr = reinterpret_cast<u4v*>(b + w.vr);
    }
};

template <int ACT>
hipError_t apply(int K, int N, int n, int R, const void* x, size_t ldx, int T, const LoraTable& tab, const void* base,
                 size_t ldb, void* y, size_t ldy, void* ws, hipStream_t s) {
    typedef typename Act<ACT>::T E;
    const LoraWs w = lora_ws(K, N, n, R, T, false);
    const LoraMem m(w, ws);
    hipError_t r;
    if (T <= kDirectMaxT) {
        float* u = reinterpret_cast<float*>(m.ut);
        hipLaunchKernelGGL((k_lora_down_tok<ACT>), dim3(T, (R + 3) / 4), dim3(256), 0, s, (const E*)x, ldx, K, n, R, tab, u);
        if ((r = hipGetLastError()) != hipSuccess) return r;
        hipLaunchKernelGGL((k_lora_up_tok<ACT>), dim3(T, (N + 1023) / 1024), dim3(256), 0, s, u, N, n, R, tab,
                           (const E*)base, ldb, (E*)y, ldy);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(k_lora_plan, dim3(n + 2), dim3(1024), 0, s, tab.ids, T, n, m.perm, m.groups, m.tiles,
                       (Slot*)nullptr, w.piece, m.tickets, w.slots);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    const DownJob j = {x, ldx, K, tab.a, m.part, m.ut, nullptr};
    if ((r = down<ACT>(w, 1, s, j, j, n, R, tab, m.perm, m.tiles, T, m.tickets)) != hipSuccess) return r;
    return up<ACT>(w, s, m.ut, T, N, n, R, tab.b, tab, m.perm, m.tiles, base, ldb, y, ldy);
}

template <int ACT>
hipError_t backward(int K, int N, int n, int R, const void* x, size_t ldx, const void* dy, size_t lddy, int T,
                    const LoraTable& tab, const void* dxb, size_t lddxb, void* dx, size_t lddx, float* const* da,
                    float* const* db, int accumulate, void* ws, hipStream_t s) {
    const LoraWs w = lora_ws(K, N, n, R, T, true);
    const LoraMem m(w, ws);
    hipError_t r;
    hipLaunchKernelGGL(k_lora_plan, dim3(n + 2), dim3(1024), 0, s, tab.ids, T, n, m.perm, m.groups, m.tiles, m.pieces,
                       w.piece, m.tickets, w.slots);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    if (T > 0) {
        const DownJob jv = {dy, lddy, N, tab.b, m.part, dx ? m.vt : nullptr, da ? m.vr : nullptr};
        const DownJob ju = {x, ldx, K, tab.a, m.part + (size_t)w.ks * T * w.R16, nullptr, m.ur};
        const bool nv = dx || da;  // v: for dx and dA; u: for dB
        r = down<ACT>(w, nv && db ? 2 : 1, s, nv ? jv : ju, ju, n, R, tab, m.perm, m.tiles, T, m.tickets);
        if (r != hipSuccess) return r;
        if (dx) {
            r = up<ACT>(w, s, m.vt, T, K, n, R, tab.a, tab, m.perm, m.tiles, dxb, lddxb, dx, lddx);
            if (r != hipSuccess) return r;
        }
    }
    if (!da && !db) return hipSuccess;
    if (T > 0) {
        const GradSide ga = {m.vr, x, ldx, K, da}, gb = {m.ur, dy, lddy, N, db};
        const dim3 grid(w.pslots, col_blocks(K) + col_blocks(N));
#define GR(B)                                                                                                       \
    hipLaunchKernelGGL((k_lora_grad<ACT, B>), grid, dim3(256), 0, s, ga, gb, n, R, w.piece, tab.ranks, m.perm, m.groups, \
                       m.pieces, accumulate, m.grad)
        if (w.R16 == 16) GR(1); else if (w.R16 == 32) GR(2); else if (w.R16 == 64) GR(4); else GR(8);
#undef GR
        if ((r = hipGetLastError()) != hipSuccess) return r;
    }
    hipLaunchKernelGGL(k_lora_grad_reduce, dim3((K + 1023) / 1024 + (N + 1023) / 1024, R, n), dim3(256), 0, s, K, N, da,
                       db, n, R, w.R16, w.piece, tab.ranks, m.groups, accumulate, m.grad);
    return hipGetLastError();
}

}  // namespace

size_t lora_ws_bytes(int K, int N, int n, int R, int T, bool back) { return lora_ws(K, N, n, R, T, back).total; }

hipError_t launch_lora_apply(int dtype, int K, int N, int n, int R, const void* x, size_t ldx, int T,
                             const LoraTable& tab, const void* base, size_t ldbase, void* y, size_t ldy, void* ws,
                             hipStream_t s) {
    if (T == 0) return hipSuccess;
    switch (dtype) {
        case kActF32: return apply<kActF32>(K, N, n, R, x, ldx, T, tab, base, ldbase, y, ldy, ws, s);
        case kActBf16: return apply<kActBf16>(K, N, n, R, x, ldx, T, tab, base, ldbase, y, ldy, ws, s);
        case kActF16: return apply<kActF16>(K, N, n, R, x, ldx, T, tab, base, ldbase, y, ldy, ws, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_lora_backward(int dtype, int K, int N, int n, int R, const void* x, size_t ldx, const void* dy,
                                size_t lddy, int T, const LoraTable& tab, const void* dx_base, size_t lddxb, void* dx,
                                size_t lddx, float* const* da, float* const* db, int accumulate, void* ws,
                                hipStream_t s) {
    switch (dtype) {
        case kActF32: return backward<kActF32>(K, N, n, R, x, ldx, dy, lddy, T, tab, dx_base, lddxb, dx, lddx, da, db, accumulate, ws, s);
        case kActBf16: return backward<kActBf16>(K, N, n, R, x, ldx, dy, lddy, T, tab, dx_base, lddxb, dx, lddx, da, db, accumulate, ws, s);
        case kActF16: return backward<kActF16>(K, N, n, R, x, ldx, dy, lddy, T, tab, dx_base, lddxb, dx, lddx, da, db, accumulate, ws, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace moe

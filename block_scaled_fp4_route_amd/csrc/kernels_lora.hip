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

struct LoraWs {
    int R16, slots, piece, pslots, ks;
    size_t perm, groups, tiles, pieces, u, v, grad, total;
};

int col_blocks(int cols) { return (cols + kUpCols - 1) / kUpCols; }

LoraWs lora_ws(int K, int N, int n, int R, int T, bool backward) {
    LoraWs w = {};
    w.R16 = R <= 16 ? 16 : (R <= 32 ? 32 : (R <= 64 ? 64 : 128));
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
        w.u = take((size_t)T * R * 4);
        w.total = o;
        return w;
    }
    w.perm = take((size_t)T * 4);
    w.groups = take((size_t)(n + 2) * sizeof(Group));
    w.tiles = take((size_t)w.slots * sizeof(Slot));
    w.pieces = take(backward ? (size_t)w.pslots * sizeof(Slot) : 0);
    w.u = take((size_t)w.ks * T * w.R16 * 4);
    w.v = take(backward ? (size_t)w.ks * T * w.R16 * 4 : 0);
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
                                                    Slot* __restrict__ tiles, Slot* __restrict__ pieces, int piece) {
    __shared__ int acc[2];
    __shared__ int wsum[kPlanIds][16];
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
            if (lane == 0) wsum[i][wave] = __popcll(mine[i]);
        }
        __syncthreads();
        int before = 0;  // own tokens of this span before place (i, wave)
#pragma unroll
        for (int i = 0; i < kPlanIds; i++)
#pragma unroll
            for (int v = 0; v < 16; v++) {
                if (v == wave && key[i] == g)
                    perm[at + before + __popcll(mine[i] & ((1ull << lane) - 1))] = t0 + 1024 * i + tid;
                before += wsum[i][v];
            }
        at += before;
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
    float* u;
};

// Sixteen consecutive activations of a row, as loaded.
template <int ACT>
struct Raw {
    static constexpr int W = ACT == kActF32 ? 4 : 2;
    u4v w[W];
};
template <int ACT>
__device__ __forceinline__ Raw<ACT> raw_load(const typename Act<ACT>::T* x) {
    Raw<ACT> r;
#pragma unroll
    for (int i = 0; i < Raw<ACT>::W; i++) r.w[i] = reinterpret_cast<const u4v*>(x)[i];
    return r;
}
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

// Steps s0 .. s1 - 1 of 64 of the long axis for NB x 16 tokens and RW x 16
// ranks: lane (i = lane % 16, q = lane / 16) holds the elements 64 s + 16 q ..
// + 15 of rows i, so a row's 128 bytes (16-bit types) arrive by neighbouring
// lanes; which elements a matrix instruction pairs does not matter as long as
// both operands agree. The loads of step s + 1 are under way during step s.
// A last step behind K's end (tail) has its missing elements set to 0.
template <int ACT, int NB, int RW>
__device__ __forceinline__ void down_steps(f4v (&acc)[4][RW], const typename Act<ACT>::T* const (&xr)[4], int b0,
                                           const uint16_t* const (&wr)[RW], int s0, int s1, int K) {
    const int lq = (threadIdx.x & 63) >> 4, full = min(s1, K / 64);
    if (s0 < full) {
        Raw<ACT> x[NB];
        u4v w[RW][2];
        auto load = [&](int s) {
#pragma unroll
            for (int b = 0; b < NB; b++) x[b] = raw_load<ACT>(xr[b0 + b] + 64 * s);
#pragma unroll
            for (int j = 0; j < RW; j++) {
                w[j][0] = *reinterpret_cast<const u4v*>(wr[j] + 64 * s);
                w[j][1] = *reinterpret_cast<const u4v*>(wr[j] + 64 * s + 8);
            }
        };
        load(s0);
        for (int s = s0; s < full; s++) {
            Raw<ACT> y[NB];
            u4v z[RW][2];
#pragma unroll
            for (int b = 0; b < NB; b++) y[b] = x[b];
#pragma unroll
            for (int j = 0; j < RW; j++) {
                z[j][0] = w[j][0];
                z[j][1] = w[j][1];
            }
            load(min(s + 1, full - 1));
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int b = 0; b < NB; b++)
#pragma unroll
                    for (int j = 0; j < RW; j++) acc[b0 + b][j] = down_mma<ACT>(y[b], h, z[j][h], acc[b0 + b][j]);
        }
    }
    if (s1 > K / 64) {  // the elements behind the last whole step (K is a multiple of 8)
        const int k0 = K / 64 * 64;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const bool in = k0 + 16 * lq + 8 * h < K;
            const int o = in ? k0 + 8 * h : 0;
#pragma unroll
            for (int b = 0; b < NB; b++) {
                Raw<ACT> x = {};
                if (in) {
#pragma unroll
                    for (int i = 0; i < Raw<ACT>::W / 2; i++)
                        x.w[h * Raw<ACT>::W / 2 + i] = reinterpret_cast<const u4v*>(xr[b0 + b] + o)[i];
                }
#pragma unroll
                for (int j = 0; j < RW; j++) {
                    const u4v w = in ? *reinterpret_cast<const u4v*>(wr[j] + o) : u4v{0, 0, 0, 0};
                    acc[b0 + b][j] = down_mma<ACT>(x, h, w, acc[b0 + b][j]);
                }
            }
        }
    }
}

// grid (slots, parts of the long axis, sides): u of one tile over one part.
// Four waves: each takes a quarter of the part's steps and all ranks, or
// above 64 ranks a half of the steps and 64 ranks; operands go from memory to
// registers, and the waves' sums are added in order through LDS.
template <int ACT, int RB>
__global__ __launch_bounds__(256) void k_lora_down(DownJob ja, DownJob jb, int n, int R,
                                                   const int32_t* __restrict__ ranks, const float* __restrict__ scales,
                                                   const int32_t* __restrict__ perm, const Slot* __restrict__ tiles,
                                                   int T) {
    constexpr int RW = RB > 4 ? 4 : RB, KW = 4 * RW / RB;  // rank blocks of a wave, waves along the long axis
    __shared__ float red[kTile][RB * 16 + 1];
    const Slot sl = tiles[blockIdx.x];
    if (sl.rows == 0 || sl.g >= n) return;
    const DownJob j = blockIdx.z ? jb : ja;
    const int r = rank_of(ranks, sl.g, R);
    if (r < 0) return;
    const int lane = threadIdx.x & 63, wave = wave_id(), li = lane & 15, lq = lane >> 4;
    const int kw = wave % KW, r0 = wave / KW * RW;
    const uint16_t* F = reinterpret_cast<const uint16_t*>(uniform_ptr(j.fac[sl.g]));
    const typename Act<ACT>::T* xr[4];
    const uint16_t* wr[RW];
    // rows behind the tile's tokens and behind the rank repeat the last one;
    // their sums are not written
#pragma unroll
    for (int b = 0; b < 4; b++)
        xr[b] = reinterpret_cast<const typename Act<ACT>::T*>(j.x) +
                (size_t)perm[sl.row + min(16 * b + li, sl.rows - 1)] * j.ldx + 16 * lq;
#pragma unroll
    for (int i = 0; i < RW; i++) wr[i] = F + (size_t)max(min(16 * (r0 + i) + li, r - 1), 0) * j.K + 16 * lq;
    f4v acc[4][RW];
#pragma unroll
    for (int b = 0; b < 4; b++)
#pragma unroll
        for (int i = 0; i < RW; i++) acc[b][i] = f4v{0.f, 0.f, 0.f, 0.f};
    const int steps = (j.K + 63) / 64, parts = gridDim.y * KW, part = blockIdx.y * KW + kw;
    const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
    if (r > 0 && 16 * r0 < r) {
        if (sl.rows <= 16) {
            down_steps<ACT, 1, RW>(acc, xr, 0, wr, s0, s1, j.K);
        } else if (sl.rows <= 32) {
            down_steps<ACT, 2, RW>(acc, xr, 0, wr, s0, s1, j.K);
        } else if constexpr (ACT == kActF32) {  // fp32 rows take twice the registers
            down_steps<ACT, 2, RW>(acc, xr, 0, wr, s0, s1, j.K);
            down_steps<ACT, 2, RW>(acc, xr, 2, wr, s0, s1, j.K);
        } else {
            down_steps<ACT, 4, RW>(acc, xr, 0, wr, s0, s1, j.K);
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
    const float sc = scales[sl.g];
    float* out = j.u + ((size_t)blockIdx.y * T + sl.row) * (RB * 16);
    for (int i = threadIdx.x; i < sl.rows * RB * 16; i += 256) {
        const int c = i % (RB * 16);
        out[i] = c < r ? sc * red[i / (RB * 16)][c] : 0.0f;
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
// "up": grid (slots, ceil(N / 256)): y of one tile and 256 columns, 64 a wave.
// The base rows are requested before anything else is waited for. u's parts
// go through LDS ([3][64 tokens][ranks], a row padded by a chunk); of the
// factor, lane (i, q) loads ranks 8 q .. + 7 of 4 neighbouring columns 4 i + j
// and turns them into one operand for each column, so that a lane ends with 4
// neighbouring columns of its rows.
template <int ACT, int RB>
__global__ __launch_bounds__(256) void k_lora_up(const float* __restrict__ u, int T, int ks, int N, int n, int R,
                                                 const void* const* __restrict__ fac,
                                                 const int32_t* __restrict__ ranks, const int32_t* __restrict__ perm,
                                                 const Slot* __restrict__ tiles, const typename Act<ACT>::T* base,
                                                 size_t ldb, typename Act<ACT>::T* y, size_t ldy) {
    constexpr int R16 = RB * 16, R32 = R16 < 32 ? 32 : R16, CH = R32 / 8, ROW = CH + 1;  // chunks of a row
    constexpr bool F16 = ACT == kActF16;
    __shared__ u4v us[3][kTile][ROW];
    const Slot sl = tiles[blockIdx.x];
    if (sl.rows == 0) return;
    const bool none = sl.g == n + 1;
    if (none && base == y) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), li = lane & 15, lq = lane >> 4;
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
        const uint16_t* F = reinterpret_cast<const uint16_t*>(uniform_ptr(fac[sl.g])) + cl;
        u2v w[R32 / 32][8];
#pragma unroll
        for (int g = 0; g < R32 / 32; g++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const int k = 32 * g + 8 * lq + i;
                w[g][i] = *reinterpret_cast<const u2v*>(F + (size_t)min(k, r - 1) * N);
                if (k >= r) w[g][i] = u2v{0, 0};
            }
        for (int i = tid; i < kTile * CH; i += 256) {
            const int p = i / CH, c = i % CH;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (p < sl.rows && 8 * c < R16)
                for (int q = 0; q < ks; q++) {
                    const f4v* s = reinterpret_cast<const f4v*>(u + ((size_t)q * T + sl.row + p) * R16 + 8 * c);
                    const f4v a = s[0], b = s[1];
#pragma unroll
                    for (int h = 0; h < 4; h++) {
                        v[h] += a[h];
                        v[4 + h] += b[h];
                    }
                }
            u4v o[3];
            parts8<3>(v, o);
#pragma unroll
            for (int h = 0; h < 3; h++) us[h][p][c] = o[h];
        }
        __syncthreads();
#pragma unroll
        for (int g = 0; g < R32 / 32; g++) {
            if (32 * g >= r) break;
            Cols16<F16> f;
            cols16<F16>(w[g], f);
#pragma unroll
            for (int b = 0; b < 4; b++) {
                u4v a[3];
#pragma unroll
                for (int h = 0; h < 3; h++) a[h] = us[h][16 * b + li][4 * g + lq];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    u4v p[Cols16<F16>::P];
#pragma unroll
                    for (int h = 0; h < Cols16<F16>::P; h++) p[h] = f.c[h][j];
                    acc[b][j] = mma_parts<Cols16<F16>::P>(a, p, acc[b][j]);
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
    const float* low;        // u or v, grouped order, parts [ks][T][R16]
    const void* row;         // dy or x
    size_t ld;
    int cols;
    float* const* out;       // per adapter, or null
};

// grid (piece slots, column blocks of A then of B): 256 columns, 64 a wave,
// over one piece, 64 tokens at a time: low's parts in LDS as [3][ranks][64
// tokens] (two sets, the next one made while one is multiplied), the rows'
// values by lane (i, q) as tokens 8 q .. + 7 of 4 neighbouring columns, turned
// into an operand for each column, the next 32 tokens' under way. An adapter
// of one piece writes its gradient, others the piece's part for
// k_lora_grad_reduce.
template <int ACT, int RB>
__global__ __launch_bounds__(256) void k_lora_grad(GradSide ga, GradSide gb, int T, int ks, int n, int R, int piece,
                                                   const int32_t* __restrict__ ranks, const int32_t* __restrict__ perm,
                                                   const Group* __restrict__ groups, const Slot* __restrict__ pieces,
                                                   int accumulate, float* __restrict__ part) {
    constexpr int R16 = RB * 16, JOBS = (R16 * 8 + 255) / 256;  // a job: 8 tokens of one rank
    constexpr int WB = ACT == kActF32 ? 4 : 2;
    typedef uint32_t wv __attribute__((ext_vector_type(WB)));
    __shared__ u4v us[2][3][R16][9];
    const Slot sl = pieces[blockIdx.x];
    if (sl.rows == 0 || sl.g >= n) return;
    const int r = rank_of(ranks, sl.g, R);
    if (r <= 0) return;
    const int nba = (ga.cols + kUpCols - 1) / kUpCols;
    const bool second = (int)blockIdx.y >= nba;
    const GradSide side = second ? gb : ga;
    float* out = side.out ? side.out[sl.g] : nullptr;
    if (!out) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), li = lane & 15, lq = lane >> 4;
    const int cols = side.cols, c0 = ((int)blockIdx.y - (second ? nba : 0)) * kUpCols + wave * 64 + 4 * li;
    const typename Act<ACT>::T* X = reinterpret_cast<const typename Act<ACT>::T*>(side.row) + min(c0, cols - 4);
    f4v acc[RB][4];
#pragma unroll
    for (int b = 0; b < RB; b++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[b][j] = f4v{0.f, 0.f, 0.f, 0.f};
    float low[JOBS][8];
    // low of the 64 tokens from p0; tokens behind the piece are 0
    auto fetch_low = [&](int p0) {
#pragma unroll
        for (int j = 0; j < JOBS; j++) {
            const int job = tid + 256 * j, rk = job % R16, c = job / R16 % 8;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const int p = p0 + 8 * c + i;
                const float* s = side.low + (size_t)(sl.row + min(p, sl.rows - 1)) * R16 + rk;
                float v = s[0];
                for (int q = 1; q < ks; q++) v += s[(size_t)q * T * R16];
                low[j][i] = p < sl.rows ? v : 0.0f;
            }
        }
    };
    auto put_low = [&](int set) {
#pragma unroll
        for (int j = 0; j < JOBS; j++) {
            const int job = tid + 256 * j;
            u4v o[3];
            parts8<3>(low[j], o);
            if (R16 * 8 >= 256 || job < R16 * 8)
#pragma unroll
                for (int h = 0; h < 3; h++) us[set][h][job % R16][job / R16 % 8] = o[h];
        }
    };
    wv x[8];
    int tok = 0;  // token of grouped row (64-token block) + lane
    auto fetch_tok = [&](int p0) { tok = perm[sl.row + min(p0 + lane, sl.rows - 1)]; };
    auto fetch_x = [&](int h) {  // rows 32 h + 8 lq + i of the block that `tok` holds
#pragma unroll
        for (int i = 0; i < 8; i++)
            x[i] = *reinterpret_cast<const wv*>(X + (size_t)__shfl(tok, 32 * h + 8 * lq + i, 64) * side.ld);
    };
    fetch_tok(0);
    fetch_low(0);
    fetch_x(0);
    put_low(0);
    int set = 0;
    for (int p0 = 0; p0 < sl.rows; p0 += kTile, set ^= 1) {
        __syncthreads();
        const bool more = p0 + kTile < sl.rows;
        if (more) fetch_low(p0 + kTile);
#pragma unroll
        for (int h = 0; h < 2; h++) {
            if (p0 + 32 * h >= sl.rows) break;
            // values of tokens behind the piece are set to 0: they may be NaN
            wv w[8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                w[i] = x[i];
                if (p0 + 32 * h + 8 * lq + i >= sl.rows)
#pragma unroll
                    for (int d = 0; d < WB; d++) w[i][d] = 0;
            }
            if (h == 0)
                fetch_x(1);
            else if (more) {
                fetch_tok(p0 + kTile);
                fetch_x(0);
            }
            constexpr int PX = ACT == kActF32 ? 3 : (ACT == kActF16 ? 2 : 1);
            u4v f[PX][4];
            if constexpr (ACT == kActF32) {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) v[i] = __uint_as_float(w[i][j]);
                    u4v o[3];
                    parts8<3>(v, o);
#pragma unroll
                    for (int q = 0; q < 3; q++) f[q][j] = o[q];
                }
            } else {
                Cols16<ACT == kActF16> c;
                cols16<ACT == kActF16>(w, c);
#pragma unroll
                for (int q = 0; q < PX; q++)
#pragma unroll
                    for (int j = 0; j < 4; j++) f[q][j] = c.c[q][j];
            }
#pragma unroll
            for (int b = 0; b < RB; b++) {
                u4v a[3];
#pragma unroll
                for (int q = 0; q < 3; q++) a[q] = us[set][q][16 * b + li][4 * h + lq];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    u4v o[PX];
#pragma unroll
                    for (int q = 0; q < PX; q++) o[q] = f[q][j];
                    acc[b][j] = mma_parts<PX>(a, o, acc[b][j]);
                }
            }
        }
        if (more) put_low(set ^ 1);
    }
    if (c0 >= cols) return;
    const bool whole = groups[sl.g].rows <= piece;
    float* to = whole ? out : part + (size_t)blockIdx.x * R16 * ((size_t)ga.cols + gb.cols) +
                                  (second ? (size_t)R16 * ga.cols : 0);
#pragma unroll
    for (int b = 0; b < RB; b++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int m = 16 * b + 4 * lq + q;
            if (m >= r) continue;
            f4v* p = reinterpret_cast<f4v*>(to + (size_t)m * cols + c0);
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
hipError_t down(int RB, dim3 grid, hipStream_t s, const DownJob& a, const DownJob& b, int n, int R,
                const LoraTable& tab, const int32_t* perm, const Slot* tiles, int T) {
#define DN(B) \
    hipLaunchKernelGGL((k_lora_down<ACT, B>), grid, dim3(256), 0, s, a, b, n, R, tab.ranks, tab.scales, perm, tiles, T)
    if (RB == 1) DN(1); else if (RB == 2) DN(2); else if (RB == 4) DN(4); else DN(8);
#undef DN
    return hipGetLastError();
}

template <int ACT>
hipError_t up(int RB, dim3 grid, hipStream_t s, const float* u, int T, int ks, int N, int n, int R,
              const void* const* fac, const LoraTable& tab, const int32_t* perm, const Slot* tiles, const void* base,
              size_t ldb, void* y, size_t ldy) {
    typedef typename Act<ACT>::T E;
#define UP(B)                                                                                                    \
    hipLaunchKernelGGL((k_lora_up<ACT, B>), grid, dim3(256), 0, s, u, T, ks, N, n, R, fac, tab.ranks, perm, tiles, \
                       (const E*)base, ldb, (E*)y, ldy)
    if (RB == 1) UP(1); else if (RB == 2) UP(2); else if (RB == 4) UP(4); else UP(8);
#undef UP
    return hipGetLastError();
}

template <int ACT>
hipError_t apply(int K, int N, int n, int R, const void* x, size_t ldx, int T, const LoraTable& tab, const void* base,
                 size_t ldb, void* y, size_t ldy, void* ws, hipStream_t s) {
    typedef typename Act<ACT>::T E;
    const LoraWs w = lora_ws(K, N, n, R, T, false);
    char* b = reinterpret_cast<char*>(ws);
    float* u = reinterpret_cast<float*>(b + w.u);
    hipError_t r;
    if (T <= kDirectMaxT) {
        hipLaunchKernelGGL((k_lora_down_tok<ACT>), dim3(T, (R + 3) / 4), dim3(256), 0, s, (const E*)x, ldx, K, n, R, tab, u);
        if ((r = hipGetLastError()) != hipSuccess) return r;
        hipLaunchKernelGGL((k_lora_up_tok<ACT>), dim3(T, (N + 1023) / 1024), dim3(256), 0, s, u, N, n, R, tab,
                           (const E*)base, ldb, (E*)y, ldy);
        return hipGetLastError();
    }
    int32_t* perm = reinterpret_cast<int32_t*>(b + w.perm);
    Slot* tiles = reinterpret_cast<Slot*>(b + w.tiles);
    hipLaunchKernelGGL(k_lora_plan, dim3(n + 2), dim3(1024), 0, s, tab.ids, T, n, perm,
                       reinterpret_cast<Group*>(b + w.groups), tiles, (Slot*)nullptr, w.piece);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    const DownJob j = {x, ldx, K, tab.a, u};
    r = down<ACT>(w.R16 / 16, dim3(w.slots, w.ks), s, j, j, n, R, tab, perm, tiles, T);
    if (r != hipSuccess) return r;
    return up<ACT>(w.R16 / 16, dim3(w.slots, (N + kUpCols - 1) / kUpCols), s, u, T, w.ks, N, n, R, tab.b, tab, perm,
                   tiles, base, ldb, y, ldy);
}

template <int ACT>
hipError_t backward(int K, int N, int n, int R, const void* x, size_t ldx, const void* dy, size_t lddy, int T,
                    const LoraTable& tab, const void* dxb, size_t lddxb, void* dx, size_t lddx, float* const* da,
                    float* const* db, int accumulate, void* ws, hipStream_t s) {
    const LoraWs w = lora_ws(K, N, n, R, T, true);
    char* b = reinterpret_cast<char*>(ws);
    float* u = reinterpret_cast<float*>(b + w.u);
    float* v = reinterpret_cast<float*>(b + w.v);
    int32_t* perm = reinterpret_cast<int32_t*>(b + w.perm);
    Group* groups = reinterpret_cast<Group*>(b + w.groups);
    Slot* tiles = reinterpret_cast<Slot*>(b + w.tiles);
    Slot* pieces = reinterpret_cast<Slot*>(b + w.pieces);
    float* part = reinterpret_cast<float*>(b + w.grad);
    const int RB = w.R16 / 16;
    hipError_t r;
    hipLaunchKernelGGL(k_lora_plan, dim3(n + 2), dim3(1024), 0, s, tab.ids, T, n, perm, groups, tiles, pieces, w.piece);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    if (T > 0) {
        const DownJob jv = {dy, lddy, N, tab.b, v}, ju = {x, ldx, K, tab.a, u};  // the larger side first
        const bool both = db != nullptr;
        r = down<ACT>(RB, dim3(w.slots, w.ks, both ? 2 : 1), s, jv, ju, n, R, tab, perm, tiles, T);
        if (r != hipSuccess) return r;
        if (dx) {
            r = up<ACT>(RB, dim3(w.slots, (K + kUpCols - 1) / kUpCols), s, v, T, w.ks, K, n, R, tab.a, tab, perm,
                        tiles, dxb, lddxb, dx, lddx);
            if (r != hipSuccess) return r;
        }
    }
    if (!da && !db) return hipSuccess;
    if (T > 0) {
        const GradSide ga = {v, x, ldx, K, da}, gb = {u, dy, lddy, N, db};
        const dim3 grid(w.pslots, (K + kUpCols - 1) / kUpCols + (N + kUpCols - 1) / kUpCols);
#define GR(B)                                                                                                     \
    hipLaunchKernelGGL((k_lora_grad<ACT, B>), grid, dim3(256), 0, s, ga, gb, T, w.ks, n, R, w.piece, tab.ranks, perm, \
                       groups, pieces, accumulate, part)
        if (RB == 1) GR(1); else if (RB == 2) GR(2); else if (RB == 4) GR(4); else GR(8);
#undef GR
        if ((r = hipGetLastError()) != hipSuccess) return r;
    }
    hipLaunchKernelGGL(k_lora_grad_reduce, dim3((K + 1023) / 1024 + (N + 1023) / 1024, R, n), dim3(256), 0, s, K, N, da,
                       db, n, R, w.R16, w.piece, tab.ranks, groups, accumulate, part);
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

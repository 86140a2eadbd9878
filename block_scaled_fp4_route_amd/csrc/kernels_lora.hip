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
// fp32; products of 16-bit operands are exact in the matrix instructions, and
// an fp32 activation enters them as three bf16 parts (its 24 bits, exactly).
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
constexpr int kPiece = 256;      // tokens of a piece of one adapter's gradient
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
    int R16, slots, pslots, ks;
    size_t perm, groups, tiles, pieces, u, v, grad, total;
};

LoraWs lora_ws(int K, int N, int n, int R, int T, bool backward) {
    LoraWs w;
    w.R16 = (R + 15) / 16 * 16;
    if (w.R16 == 48) w.R16 = 64;
    if (w.R16 > 64) w.R16 = 128;
    w.slots = T / kTile + n + 3;
    w.pslots = T / kPiece + n + 3;
    // parts of the long axis of "down", so that short batches fill the chip
    // (about 512 workgroups), at most 8 and at least 4 x 4 steps of 32 each
    const int tiles = T / kTile + 1 + (n < T ? n : T) / 2;
    const int steps = ((K > N && backward ? K : (backward ? N : K)) + 31) / 32;
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
    w.pieces = take((size_t)w.pslots * sizeof(Slot));
    w.u = take((size_t)w.ks * T * w.R16 * 4);
    w.v = take(backward ? (size_t)w.ks * T * w.R16 * 4 : 0);
    w.grad = take(backward ? (size_t)w.pslots * w.R16 * ((size_t)K + N) * 4 : 0);
    w.total = o;
    return w;
}

// grid n + 2, 1024 threads: group g counts the tokens before it and its own,
// lists its own in increasing t, and writes its tiles and pieces.
__global__ __launch_bounds__(1024) void k_lora_plan(const int32_t* __restrict__ ids, int T, int n,
                                                    int32_t* __restrict__ perm, Group* __restrict__ groups,
                                                    Slot* __restrict__ tiles, Slot* __restrict__ pieces) {
    __shared__ int acc[2];
    __shared__ int wsum[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = blockIdx.x;
    auto key = [&](int t) {
        const int a = ids[t];
        return a < 0 ? n + 1 : (a >= n ? n : a);
    };
    if (tid < 2) acc[tid] = 0;
    __syncthreads();
    int less = 0, own = 0;
    for (int t = tid; t < T; t += 1024) {
        const int q = key(t);
        less += q < g;
        own += q == g;
    }
    if (less) atomicAdd(&acc[0], less);
    if (own) atomicAdd(&acc[1], own);
    __syncthreads();
    const int first = acc[0], count = acc[1];
    if (count) {
        int at = first;
        for (int t0 = 0; t0 < T; t0 += 1024) {
            const int t = t0 + tid;
            const bool mine = t < T && key(t) == g;
            const unsigned long long b = __ballot(mine);
            if (lane == 0) wsum[wave] = __popcll(b);
            __syncthreads();
            int before = 0, all = 0;
#pragma unroll
            for (int i = 0; i < 16; i++) {
                before += i < wave ? wsum[i] : 0;
                all += wsum[i];
            }
            if (mine) perm[at + before + __popcll(b & ((1ull << lane) - 1))] = t;
            at += all;
            __syncthreads();
        }
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
    if (pieces) list(pieces, kPiece);
}

// Eight consecutive activations of a row as MFMA operands: one for 16-bit
// types, three bf16 parts for fp32 (each the truncation of what the ones
// before left: 8 + 8 + 8 bits, exact; the parts behind an infinity are 0).
template <int ACT>
struct Frag {
    static constexpr int P = ACT == kActF32 ? 3 : 1;
    u4v p[P];
};
template <int ACT>
__device__ __forceinline__ void frag_zero(Frag<ACT>& f) {
#pragma unroll
    for (int i = 0; i < Frag<ACT>::P; i++) f.p[i] = u4v{0, 0, 0, 0};
}
__device__ __forceinline__ uint32_t hi16(float f) { return __float_as_uint(f) & 0xFFFF0000u; }
__device__ __forceinline__ float rest(float f, uint32_t h) {
    return __float_as_uint(f) == h ? 0.0f : f - __uint_as_float(h);
}
template <int ACT>
__device__ __forceinline__ void frag_load(Frag<ACT>& f, const typename Act<ACT>::T* x) {
    if constexpr (ACT == kActF32) {
        const f4v a = *reinterpret_cast<const f4v*>(x), b = *reinterpret_cast<const f4v*>(x + 4);
        float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float e = v[2 * i], o = v[2 * i + 1];
#pragma unroll
            for (int q = 0; q < 3; q++) {
                const uint32_t he = hi16(e), ho = hi16(o);
                f.p[q][i] = he >> 16 | ho;
                e = rest(e, he);
                o = rest(o, ho);
            }
        }
    } else {
        f.p[0] = *reinterpret_cast<const u4v*>(x);
    }
}
template <int ACT>
__device__ __forceinline__ f4v mma(const Frag<ACT>& x, u4v w, f4v c) {
    if constexpr (ACT == kActF16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, x.p[0]), __builtin_bit_cast(h8v, w), c, 0, 0, 0);
    } else {
#pragma unroll
        for (int i = Frag<ACT>::P - 1; i >= 0; i--)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, x.p[i]), __builtin_bit_cast(bf8v, w), c, 0, 0, 0);
        return c;
    }
}

// grid (slots, parts): u of one tile over one part of the long axis. The
// four waves take quarters of the part's steps of 32; operands go from
// memory to registers (x rows once, the factor's rows once per 64 tokens),
// and the waves' sums are added in order through LDS.
template <int ACT, int RB>
__global__ __launch_bounds__(256) void k_lora_down(const typename Act<ACT>::T* __restrict__ x, size_t ldx, int K,
                                                   int n, int R, const void* const* __restrict__ fac,
                                                   const int32_t* __restrict__ ranks, const float* __restrict__ scales,
                                                   const int32_t* __restrict__ perm, const Slot* __restrict__ tiles,
                                                   int T, float* __restrict__ u) {
    __shared__ float red[kTile][RB * 16 + 1];
    const Slot sl = tiles[blockIdx.x];
    if (sl.rows == 0 || sl.g >= n) return;
    const int r = rank_of(ranks, sl.g, R);
    if (r < 0) return;
    const int lane = threadIdx.x & 63, wave = wave_id(), li = lane & 15, lq = lane >> 4;
    const uint16_t* F = reinterpret_cast<const uint16_t*>(uniform_ptr(fac[sl.g]));
    const typename Act<ACT>::T* xr[4];
#pragma unroll
    for (int b = 0; b < 4; b++) {
        const int p = 16 * b + li;
        xr[b] = x + (size_t)perm[sl.row + (p < sl.rows ? p : 0)] * ldx + 8 * lq;
    }
    f4v acc[4][RB];
#pragma unroll
    for (int b = 0; b < 4; b++)
#pragma unroll
        for (int j = 0; j < RB; j++) acc[b][j] = f4v{0.f, 0.f, 0.f, 0.f};
    const int steps = (K + 31) / 32, parts = gridDim.y * 4, part = blockIdx.y * 4 + wave;
    const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
    const int nb = (sl.rows + 15) / 16;
    for (int s = s0; s < s1; s++) {
        const int kk = 32 * s + 8 * lq;
        Frag<ACT> f[4];
        u4v w[RB];
#pragma unroll
        for (int j = 0; j < RB; j++) {
            w[j] = u4v{0, 0, 0, 0};
            if (16 * j + li < r && kk < K) w[j] = *reinterpret_cast<const u4v*>(F + (size_t)(16 * j + li) * K + kk);
        }
#pragma unroll
        for (int b = 0; b < 4; b++) {
            frag_zero<ACT>(f[b]);
            if (b < nb && kk < K) frag_load<ACT>(f[b], xr[b] + 32 * s);
        }
#pragma unroll
        for (int b = 0; b < 4; b++)
            if (b < nb)
#pragma unroll
                for (int j = 0; j < RB; j++) acc[b][j] = mma<ACT>(f[b], w[j], acc[b][j]);
    }
    for (int w = 0; w < 4; w++) {
        if (wave == w)
#pragma unroll
            for (int b = 0; b < 4; b++)
#pragma unroll
                for (int j = 0; j < RB; j++)
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        float* p = &red[16 * b + 4 * lq + q][16 * j + li];
                        *p = w ? *p + acc[b][j][q] : acc[b][j][q];
                    }
        __syncthreads();
    }
    const float sc = scales[sl.g];
    float* out = u + ((size_t)blockIdx.y * T + sl.row) * (RB * 16);
    for (int i = threadIdx.x; i < sl.rows * RB * 16; i += 256) out[i] = sc * red[i / (RB * 16)][i % (RB * 16)];
}

// Stages grouped rows row .. row + rows - 1 of u (the parts added in order)
// in LDS, zero up to `upto` rows.
template <int RB>
__device__ __forceinline__ void stage_u(const float* __restrict__ u, int T, int ks, int row, int rows, int upto,
                                        float (*out)[RB * 16 + 4]) {
    for (int i = threadIdx.x; i < upto * RB * 4; i += 256) {
        const int p = i / (RB * 4), c = i % (RB * 4) * 4;
        f4v v = {0.f, 0.f, 0.f, 0.f};
        if (p < rows)
            for (int q = 0; q < ks; q++)
                v += *reinterpret_cast<const f4v*>(u + ((size_t)q * T + row + p) * (RB * 16) + c);
        *reinterpret_cast<f4v*>(&out[p][c]) = v;
    }
}

// grid (slots, ceil(N / 256)): y of one tile and 256 columns, 64 a wave.
// fp32 matrix instructions over the rank: lane (i = lane % 16, q = lane / 16)
// reads rank rows 4 q + s of the factor, 4 consecutive columns 4 i + j each,
// so MFMA j of step s has the columns 4 i + j and the lane ends with 4
// consecutive columns of its rows.
template <int ACT, int RB>
__global__ __launch_bounds__(256) void k_lora_up(const float* __restrict__ u, int T, int ks, int N, int n, int R,
                                                 const void* const* __restrict__ fac,
                                                 const int32_t* __restrict__ ranks, const int32_t* __restrict__ perm,
                                                 const Slot* __restrict__ tiles, const typename Act<ACT>::T* base,
                                                 size_t ldb, typename Act<ACT>::T* y, size_t ldy) {
    __shared__ __align__(16) float us[kTile][RB * 16 + 4];
    __shared__ int rows[kTile];
    const Slot sl = tiles[blockIdx.x];
    if (sl.rows == 0) return;
    const bool none = sl.g == n + 1;
    if (none && base == y) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), li = lane & 15, lq = lane >> 4;
    const int r = none ? 0 : (sl.g == n ? -1 : rank_of(ranks, sl.g, R));
    if (tid < kTile) rows[tid] = tid < sl.rows ? perm[sl.row + tid] : -1;
    if (r > 0) stage_u<RB>(u, T, ks, sl.row, sl.rows, kTile, us);
    __syncthreads();
    const int c0 = blockIdx.y * kUpCols + wave * 64 + 4 * li;
    f4v acc[4][4];
#pragma unroll
    for (int b = 0; b < 4; b++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[b][j] = f4v{0.f, 0.f, 0.f, 0.f};
    if (r > 0) {
        const uint16_t* F = reinterpret_cast<const uint16_t*>(uniform_ptr(fac[sl.g]));
#pragma unroll
        for (int g = 0; g < RB; g++) {
            if (16 * g >= r) break;
            float w[4][4];
#pragma unroll
            for (int s = 0; s < 4; s++) {
                const int k = 16 * g + 4 * lq + s;
                u2v q = {0, 0};
                if (k < r && c0 < N) q = *reinterpret_cast<const u2v*>(F + (size_t)k * N + c0);
                cvt2<ACT>(q.x, w[s][0], w[s][1]);
                cvt2<ACT>(q.y, w[s][2], w[s][3]);
            }
#pragma unroll
            for (int b = 0; b < 4; b++) {
                const f4v a = *reinterpret_cast<const f4v*>(&us[16 * b + li][16 * g + 4 * lq]);
#pragma unroll
                for (int s = 0; s < 4; s++)
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        acc[b][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], w[s][j], acc[b][j], 0, 0, 0);
            }
        }
    }
    if (c0 >= N) return;
#pragma unroll
    for (int b = 0; b < 4; b++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int t = rows[16 * b + 4 * lq + q];
            if (t < 0) continue;
            f4v v = {acc[b][0][q], acc[b][1][q], acc[b][2][q], acc[b][3][q]};
            if (base) v += ld4<ACT>(base + (size_t)t * ldb + c0);
            if (r < 0) v.x = v.y = v.z = v.w = __builtin_nanf("");
            st4<ACT>(y + (size_t)t * ldy + c0, v);
        }
}

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
// over one piece of 256 tokens; an adapter of one piece writes its gradient,
// others write the piece's part for k_lora_grad_reduce.
template <int ACT, int RB>
__global__ __launch_bounds__(256) void k_lora_grad(GradSide ga, GradSide gb, int T, int ks, int n, int R,
                                                   const int32_t* __restrict__ ranks, const int32_t* __restrict__ perm,
                                                   const Group* __restrict__ groups, const Slot* __restrict__ pieces,
                                                   int accumulate, float* __restrict__ part) {
    __shared__ __align__(16) float us[kTile][RB * 16 + 4];
    __shared__ int rows[kTile];
    const Slot sl = pieces[blockIdx.x];
    if (sl.rows == 0 || sl.g >= n) return;
    const int r = rank_of(ranks, sl.g, R);
    if (r <= 0) return;
    const int nba = (ga.cols + kUpCols - 1) / kUpCols;
    const bool second = (int)blockIdx.y >= nba;
    const GradSide& side = second ? gb : ga;
    float* out = side.out ? side.out[sl.g] : nullptr;
    if (!out) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), li = lane & 15, lq = lane >> 4;
    const int cols = side.cols, c0 = ((int)blockIdx.y - (second ? nba : 0)) * kUpCols + wave * 64 + 4 * li;
    const typename Act<ACT>::T* X = reinterpret_cast<const typename Act<ACT>::T*>(side.row);
    f4v acc[RB][4];
#pragma unroll
    for (int b = 0; b < RB; b++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[b][j] = f4v{0.f, 0.f, 0.f, 0.f};
    for (int p0 = 0; p0 < sl.rows; p0 += kTile) {
        const int cnt = min(kTile, sl.rows - p0);
        __syncthreads();
        stage_u<RB>(side.low, T, ks, sl.row + p0, cnt, kTile, us);
        if (tid < kTile) rows[tid] = tid < cnt ? perm[sl.row + p0 + tid] : -1;
        __syncthreads();
#pragma unroll
        for (int g = 0; g < kTile / 16; g++) {
            if (16 * g >= cnt) break;
            f4v w[4];
#pragma unroll
            for (int s = 0; s < 4; s++) {
                const int t = rows[16 * g + 4 * lq + s];
                w[s] = f4v{0.f, 0.f, 0.f, 0.f};
                if (t >= 0 && c0 < cols) w[s] = ld4<ACT>(X + (size_t)t * side.ld + c0);
            }
#pragma unroll
            for (int b = 0; b < RB; b++)
#pragma unroll
                for (int s = 0; s < 4; s++) {
                    const float a = us[16 * g + 4 * lq + s][16 * b + li];
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        acc[b][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, w[s][j], acc[b][j], 0, 0, 0);
                }
        }
    }
    if (c0 >= cols) return;
    const bool whole = groups[sl.g].rows <= kPiece;
    float* to = whole ? out : part + (size_t)blockIdx.x * (RB * 16) * ((size_t)ga.cols + gb.cols) +
                                  (second ? (size_t)(RB * 16) * ga.cols : 0);
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
                                                          int R, int R16, const int32_t* __restrict__ ranks,
                                                          const Group* __restrict__ groups, int accumulate,
                                                          const float* __restrict__ part) {
    const int a = blockIdx.z, m = blockIdx.y;
    const Group g = groups[a];
    const int r = rank_of(ranks, a, R);
    if (m >= r) return;
    if (g.rows == 0 ? accumulate != 0 : g.rows <= kPiece) return;
    const int nba = (ca + 1023) / 1024;
    const bool second = (int)blockIdx.x >= nba;
    float* out = second ? (db ? db[a] : nullptr) : (da ? da[a] : nullptr);
    const int cols = second ? cb : ca, c = (((int)blockIdx.x - (second ? nba : 0)) * 256 + (int)threadIdx.x) * 4;
    if (!out || c >= cols) return;
    f4v v = {0.f, 0.f, 0.f, 0.f};
    const int s0 = g.row / kPiece + a, np = (g.rows + kPiece - 1) / kPiece;
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
hipError_t down(int RB, dim3 grid, hipStream_t s, const void* x, size_t ldx, int K, int n, int R,
                const void* const* fac, const LoraTable& tab, const int32_t* perm, const Slot* tiles, int T, float* u) {
    typedef const typename Act<ACT>::T* P;
#define DN(B)                                                                                                     \
    hipLaunchKernelGGL((k_lora_down<ACT, B>), grid, dim3(256), 0, s, (P)x, ldx, K, n, R, fac, tab.ranks, tab.scales, \
                       perm, tiles, T, u)
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
                       reinterpret_cast<Group*>(b + w.groups), tiles, (Slot*)nullptr);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    r = down<ACT>(w.R16 / 16, dim3(w.slots, w.ks), s, x, ldx, K, n, R, tab.a, tab, perm, tiles, T, u);
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
    hipLaunchKernelGGL(k_lora_plan, dim3(n + 2), dim3(1024), 0, s, tab.ids, T, n, perm, groups, tiles, pieces);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    if (T > 0) {
        const dim3 gd(w.slots, w.ks);
        if (db && (r = down<ACT>(RB, gd, s, x, ldx, K, n, R, tab.a, tab, perm, tiles, T, u)) != hipSuccess) return r;
        if ((r = down<ACT>(RB, gd, s, dy, lddy, N, n, R, tab.b, tab, perm, tiles, T, v)) != hipSuccess) return r;
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
    hipLaunchKernelGGL((k_lora_grad<ACT, B>), grid, dim3(256), 0, s, ga, gb, T, w.ks, n, R, tab.ranks, perm, groups, \
                       pieces, accumulate, part)
        if (RB == 1) GR(1); else if (RB == 2) GR(2); else if (RB == 4) GR(4); else GR(8);
#undef GR
        if ((r = hipGetLastError()) != hipSuccess) return r;
    }
    hipLaunchKernelGGL(k_lora_grad_reduce, dim3((K + 1023) / 1024 + (N + 1023) / 1024, R, n), dim3(256), 0, s, K, N, da,
                       db, n, R, w.R16, tab.ranks, groups, accumulate, part);
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

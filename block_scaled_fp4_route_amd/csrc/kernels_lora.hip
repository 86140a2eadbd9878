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
// the ones before left, which hold all 24 bits of values above 2^-110 (bits
// below 2^-133, bf16's smallest step, are cut off; the fp32 instructions run at
// a sixteenth of the rate; against fp32 u and v an fp16 operand enters as two
// bf16 parts, exactly).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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
// No grouping up to so many tokens and tokens x max_rank: every token then
// reads its factors for itself (rank 16, K 2560, N 8192, 32 adapters: 13.4 us
// against 21.7 at 256 tokens, 19 against 23 at 512; rank 64, 8 adapters: 18.5
// against 25 at 128, 30 against 28 at 256).
constexpr int kDirectMaxT = 512, kDirectWork = 8192;
bool direct(int T, int R) { return T <= kDirectMaxT && (int64_t)T * R <= kDirectWork; }
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
__device__ __forceinline__ int table_rank(const LoraTable& tab, int a, int R) {
    const int r = tab.ranks[a];
    return r < 0 || r > R ? -1 : r;
}
// The same, -1 also where a factor that it needs is NULL.
__device__ __forceinline__ int rank_of(const LoraTable& tab, int a, int R) {
    const int r = table_rank(tab, a, R);
    const bool none = (tab.a[a] == nullptr) | (tab.b[a] == nullptr);
    return r > 0 && none ? -1 : r;
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
    const int r = rank_of(tab, a, R);
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
        const int r = a < n ? rank_of(tab, a, R) : -1;
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

// One launch for both: grid (T, ceil(N / 512)), 1024 threads. Every workgroup
// makes all of its token's u itself (a wave one value at a time), while its
// factor rows for 512 columns are on their way: thread (g = tid / 128, c = tid
// % 128) has the ranks g, g + 8, ... and the columns 4 c .. + 3, and the eight
// sums of a column are added through LDS. The factor A is read once per column
// block, so this form is for small factors and for as many workgroups as run
// at once: 5.2 us against 6.2 and a launch at one token, rank 16, 2560 to
// 8192; 9.0 against 8.4 at rank 64; 13 against 7.3 at 64 tokens.
constexpr int kTokFused = 65536;  // elements of A (max_rank K)
template <int ACT>
__global__ __launch_bounds__(1024) void k_lora_tok(const typename Act<ACT>::T* __restrict__ x, size_t ldx, int K,
                                                   int N, int n, int R, LoraTable tab,
                                                   const typename Act<ACT>::T* base, size_t ldb,
                                                   typename Act<ACT>::T* y, size_t ldy) {
    __shared__ float us[kLoraMaxRank];
    __shared__ f4v red[8][128];
    const int tid = threadIdx.x, lane = tid & 63, t = blockIdx.x, g = tid >> 7, c = blockIdx.y * 512 + (tid & 127) * 4;
    const bool mine = g == 0 && c < N;
    const int a = tab.ids[t];
    f4v v = {0.f, 0.f, 0.f, 0.f};
    if (mine && base) v = ld4<ACT>(base + (size_t)t * ldb + c);
    const int r = a < 0 ? 0 : (a < n ? rank_of(tab, a, R) : -1);
    if (r > 0) {
        const rsrc_t rb = make_rsrc(tab.b[a], (uint32_t)r * (uint32_t)N * 2u);  // rows behind the rank read 0
        const rsrc_t ra = make_rsrc(tab.a[a], (uint32_t)r * (uint32_t)K * 2u);
        const uint32_t oc = c < N ? (uint32_t)c * 2u : kOOB;
        uint2 w[4];
#pragma unroll
        for (int m = 0; m < 4; m++) w[m] = ld_b64(rb, (uint32_t)(g + 8 * m) * (uint32_t)N * 2u + oc);
        const typename Act<ACT>::T* xt = x + (size_t)t * ldx;
        const float sc = tab.scales[a];
        for (int i = wave_id(); i < r; i += 16) {
            float acc = 0.0f;
#pragma unroll 4
            for (int p = lane * 8; p < K; p += 512) {
                const auto q = __builtin_amdgcn_raw_buffer_load_b128(ra, ((uint32_t)i * (uint32_t)K + (uint32_t)p) * 2u, 0, 0);
                acc = dot8<ACT>(xt + p, u4v{q[0], q[1], q[2], q[3]}, acc);
            }
            acc = wave_sum(acc);
            if (lane == 0) us[i] = sc * acc;
        }
        __syncthreads();
        f4v s = {0.f, 0.f, 0.f, 0.f};
        for (int m0 = 0; 8 * m0 < r; m0 += 4) {
            if (m0)
#pragma unroll
                for (int m = 0; m < 4; m++) w[m] = ld_b64(rb, (uint32_t)(g + 8 * (m0 + m)) * (uint32_t)N * 2u + oc);
#pragma unroll
            for (int m = 0; m < 4; m++) {
                const int i = g + 8 * (m0 + m);
                const float ui = i < r ? us[i] : 0.0f;
                float p, q;
                cvt2<ACT>(w[m].x, p, q); s.x = fmaf(p, ui, s.x); s.y = fmaf(q, ui, s.y);
                cvt2<ACT>(w[m].y, p, q); s.z = fmaf(p, ui, s.z); s.w = fmaf(q, ui, s.w);
            }
        }
        red[g][tid & 127] = s;
        __syncthreads();
        if (g == 0) {
            s = red[0][tid];
#pragma unroll
            for (int i = 1; i < 8; i++) s += red[i][tid];
            v += s;
        }
    }
    if (r < 0) v.x = v.y = v.z = v.w = __builtin_nanf("");
    if (mine) st4<ACT>(y + (size_t)t * ldy + c, v);
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
//             rank k at place c ^ (k / 2 % 8), so that neighbouring ranks' reads
//             from LDS fall on different banks, for "grad"
struct LoraWs {
    int R16, R32, slots, piece, pslots;
    int ku, kv;  // parts of the long axis of "down": x with A, dy with B
    size_t perm, groups, tiles, pieces, tickets, part, ut, vt, ur, vr, grad, total;
};

int col_blocks(int cols) { return (cols + kUpCols - 1) / kUpCols; }

LoraWs lora_ws(int K, int N, int n, int R, int T, bool backward, bool f32) {
    LoraWs w = {};
    w.R16 = R <= 16 ? 16 : (R <= 32 ? 32 : (R <= 64 ? 64 : 128));
    w.R32 = w.R16 < 32 ? 32 : w.R16;
    w.slots = T / kTile + n + 3;
    // tokens of a piece of the gradient: about 512 workgroups, so that the
    // parts that k_lora_grad_reduce adds stay few
    const int64_t piece = ((int64_t)T * (col_blocks(K) + col_blocks(N)) / 512 + kTile - 1) / kTile * kTile;
    w.piece = (int)(piece < 2 * kTile ? 2 * kTile : (piece > 4096 ? 4096 : piece));
    w.pslots = T / w.piece + n + 3;
    // T / piece at most (512 / 128 (128 + 1) because the quotient is rounded
    // down), growing with T: fewer tokens never need more workspace
    const int in128 = T / 128, in512 = 516 / (col_blocks(K) + col_blocks(N)), least = in128 < in512 ? in128 : in512;
    const size_t pslots = (size_t)(T / 4096 > least ? T / 4096 : least) + n + 3;
    // parts of the long axes of "down": one workgroup per compute unit, or two
    // (what runs at once) for two sides, whose lengths share them out; at most 8
    // parts of a side, of four steps at least. One side, one against two a unit:
    // 16000 x 1024 12 us against 15, 4000 x 4096 14 against 16; two sides: 8192 x
    // (2560 + 8192), rank 64, 81 against 64 (bf16). Four steps against two: 2451 x
    // 2560 fp16 14 us against 16, against eight: 22 at 300 x (2560 + 640) fp32,
    // where four take 12.
    const int tiles = T / kTile + 1 + (n < T ? n : T) / 2;
    auto parts = [=](int len, int all) {
        int64_t k = ((backward ? 512 : 256) / tiles * (int64_t)len + (all - 1) / 2) / all;
        if (k > 8) k = 8;
        const int step = f32 ? 64 : 128;
        if (k > len / (4 * step)) k = len / (4 * step);
        return (int)(k < 1 ? 1 : k);
    };
    w.ku = parts(K, backward ? K + N : K);
    w.kv = backward ? parts(N, K + N) : 0;
    size_t o = kCounterBytes;
    auto take = [&o](size_t bytes) {
        const size_t at = o;
        o += align256(bytes);
        return at;
    };
    if (!backward && direct(T, R)) {
        w.ut = take((size_t)T * R * 4);
        w.total = o;
        return w;
    }
    w.perm = take((size_t)T * 4);
    w.groups = take((size_t)(n + 2) * sizeof(Group));
    w.tiles = take((size_t)w.slots * sizeof(Slot));
    w.pieces = take(backward ? pslots * sizeof(Slot) : 0);
    w.tickets = take((size_t)w.slots * 2 * 4);
    // parts x tokens: 8 of a side at most, and 512 / (T / 64) in all
    const size_t rows = (size_t)T * (backward ? 16 : 8), most = 512 * kTile;
    w.part = take((rows < most ? rows : most) * w.R16 * 4);
    const size_t by_token = (size_t)T * w.R32 * 6, by_rank = (size_t)w.slots * w.R16 * kTile * 6;
    w.ut = take(backward ? 0 : by_token);
    w.vt = take(backward ? by_token : 0);
    w.ur = take(backward ? by_rank : 0);
    w.vr = take(backward ? by_rank : 0);
    w.grad = take(backward ? pslots * w.R16 * ((size_t)K + N) * 4 : 0);
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
    int less = 0, own = 0;  // of the wave
    for (int t0 = 0; t0 < T; t0 += SPAN) {
        load(t0);
#pragma unroll
        for (int i = 0; i < kPlanIds; i++) {
            less += __popcll(__ballot(key[i] >= 0 && key[i] < g));
            own += __popcll(__ballot(key[i] == g));
        }
    }
    if (lane == 0) {
        atomicAdd(&acc[0], less);
        atomicAdd(&acc[1], own);
    }
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
// Infinities. An infinity has the parts (inf, 0, 0), and a finite value of few
// bits has low parts of 0 too, so an infinite product of two values becomes NaN
// where the infinity meets such a part. The product of the two first parts
// alone has the class of the whole product (infinite with its sign, NaN or
// finite; values below 2^-133 have no parts and count as 0). So a sum that
// comes out as NaN is formed once more from the first parts, and is infinite
// if that one is. Other sums cost a comparison each.
__device__ __forceinline__ bool is_nan(float v) { return v != v; }
__device__ __forceinline__ int has_nan(f4v v) {
    return __builtin_isunordered(v.x, v.y) | __builtin_isunordered(v.z, v.w);
}
// What a NaN among the sums is, from the sum of the first parts.
__device__ __forceinline__ float nan_or_inf(float first) {
    return fabsf(first) == INFINITY ? first : __builtin_nanf("");
}
// The bf16 truncations of a and b, NaN also where the truncation cuts off all
// bits that make one.
__device__ __forceinline__ uint32_t pack_first(float a, float b) {
    return pack_hi(is_nan(a) ? __builtin_nanf("") : a, is_nan(b) ? __builtin_nanf("") : b);
}
// Infinities taken out. "down", where only the activations are in parts and
// there are many steps, runs all of them again instead, with the low parts
// beside a factor without its infinities.
__device__ __forceinline__ u4v without_inf(u4v p) {
#pragma unroll
    for (int q = 0; q < 4; q++) {
        if ((p[q] & 0x7FFFu) == 0x7F80u) p[q] &= 0xFFFF0000u;
        if ((p[q] & 0x7FFF0000u) == 0x7F800000u) p[q] &= 0xFFFFu;
    }
    return p;
}

// ---------------------------------------------------------------------------
// "down": the two sides of a pass (x with A; dy with B) in one launch.
struct DownJob {
    const void* x;
    size_t ldx;
    int K;
    const void* const* fac;
    int ks;         // parts of the long axis
    float* part;    // [ks][T][R16]
    u4v* by_token;  // either may be null
    u4v* by_rank;
};

// A step of the long axis: 256 bytes of every activation row (128 above 32
// ranks) and as many elements of every factor row. LDS holds a ring of RING
// steps in at most 80 KB (two workgroups a compute unit), each as 16-byte
// chunks, [64 tokens][XC] of activations and [ranks][FC] of the factor; chunk
// c of row p is at place c ^ swizzle(p), so that the 16 rows that a matrix
// operand reads at once lie on different banks.
template <int ACT, int RB>
struct DownStep {
    static constexpr int XC = RB >= 4 ? 8 : 16;                  // chunks of an activation row
    static constexpr int KE = XC * (ACT == kActF32 ? 4 : 8);     // elements
    static constexpr int FC = KE / 8;                            // chunks of a factor row
    static constexpr int XI = XC / 4;                            // 1 KB loads of a wave: its 16 tokens
    static constexpr int FI = RB * 16 * FC / 64;                 // of the factor, all waves
    static constexpr int FW = (FI + 3) / 4;                      // a wave's (each one twice where there are two)
    static constexpr int CHUNKS = kTile * XC + RB * 16 * FC;
    static constexpr int FIT = 81920 / (16 * CHUNKS), RING = FIT > 6 ? 6 : FIT;
    static_assert(RING >= 3, "a step being read, one arriving, one to come");
};
// Rows of C chunks: 16 / C of them span the banks, the next ones are shifted.
template <int C>
__device__ __forceinline__ int swizzle(int row) {
    return row / (16 / C) % C;
}

// Cache policy of loads and stores that other XCDs' workgroups take part in
// (sc1: device scope).
constexpr int kCoherent = 16;

// A load of 16 bytes a lane from p straight into LDS: lane l writes lds + l.
__device__ __forceinline__ void load_lds(const void* p, u4v* lds) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(uintptr_t)p,
                                     (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}
// Wait until at most N vector memory operations of this wave are outstanding
// (they complete in issue order) and its LDS accesses are done, then a
// workgroup barrier.
template <int N>
__device__ __forceinline__ void ring_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// grid (slots, parts of side a, then of side b): the low values of one tile
// over one part of one side's long axis. Wave w has the tokens 16 w .. + 15
// and all ranks; the step after next is on its way from memory while one is
// multiplied. (Operands loaded straight into registers kept too little in
// flight: the backward pass of 8192 tokens, 2560 and 8192 wide, rank 64 took
// 214 us with them and 187 with the ring.) Where the axis is in several parts,
// every workgroup leaves its own with device-coherent stores, and the last one
// of a tile to finish (by a ticket) adds them in order. Out go the bf16 parts
// of the scaled values. One side of 8192 x 2560 bf16, rank 16: 17 us (42 MB, 2.5
// TB/s). Both sides of 8192 x (2560 + 8192), rank 64: 64 us; 176 MB come from
// memory, as much again of the factors from L2 (64 tokens stand against 64
// ranks), and 384 workgroups of 40 or 64 steps share 256 compute units, where a
// kernel that only reads the 134 MB side in such row pieces takes 26 to 33 us.
// Few tokens: one round of loads and the join, 12 us at 300 x (2560 + 640) fp32.
template <int ACT, int RB>
__global__ __launch_bounds__(256) void k_lora_down(DownJob ja, DownJob jb, int n, int R,
                                                   LoraTable tab,
                                                   const int32_t* __restrict__ perm, const Slot* __restrict__ tiles,
                                                   int T, uint32_t* __restrict__ tickets) {
    typedef DownStep<ACT, RB> S;
    typedef typename Act<ACT>::T E;
    constexpr int R16 = RB * 16, CH = (R16 < 32 ? 32 : R16) / 8, RING = S::RING;
    // one array for everything (with several the compiler waits for every load
    // in flight before each LDS read): the ring, later the tile's sums and a ticket
    constexpr int SUMS = (kTile * (R16 + 1) * 4 + 15) / 16;
    static_assert(RING * S::CHUNKS > SUMS, "the sums take the ring's place");
    __shared__ u4v lds[RING * S::CHUNKS];
    const Slot sl = tiles[blockIdx.x];
    if (sl.rows == 0 || sl.g >= n) return;
    const bool second = (int)blockIdx.y >= ja.ks;
    const DownJob j = second ? jb : ja;
    const int ks = j.ks, ky = (int)blockIdx.y - (second ? ja.ks : 0);
    const int r = rank_of(tab, sl.g, R);
    if (r < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), li = lane & 15, lq = lane >> 4;
    const int steps = (j.K + S::KE - 1) / S::KE;
    const int s0 = (int)((int64_t)steps * ky / ks), s1 = (int)((int64_t)steps * (ky + 1) / ks);
    // activations: load i of wave w has 64 / XC rows from 16 w + 64 i / XC;
    // rows behind the tile's tokens repeat the last one, their sums are not used
    const E* xp[S::XI];
    int xk[S::XI];
#pragma unroll
    for (int i = 0; i < S::XI; i++) {
        const int row = 16 * wave + (64 * i + lane) / S::XC, c = lane % S::XC ^ swizzle<S::XC>(row);
        xk[i] = c * (S::KE / S::XC);
        xp[i] = reinterpret_cast<const E*>(j.x) + (size_t)perm[sl.row + min(row, sl.rows - 1)] * j.ldx + xk[i];
    }
    // factor: load i of wave w has the chunks 64 (w + 4 i) .. + 63; rows behind
    // the rank repeat the last one, their sums are replaced by 0
    const uint16_t* F = reinterpret_cast<const uint16_t*>(uniform_ptr(j.fac[sl.g]));
    const uint16_t* fp[S::FW];
    int fk[S::FW], fd[S::FW];
#pragma unroll
    for (int i = 0; i < S::FW; i++) {
        fd[i] = (wave + 4 * i) % S::FI * 64;
        const int q = fd[i] + lane, row = q / S::FC, c = q % S::FC ^ swizzle<S::FC>(row);
        fk[i] = c * 8;
        fp[i] = F + (size_t)max(min(row, r - 1), 0) * j.K + fk[i];
    }
    // elements behind K read the row's first ones and are set to 0 when used
    auto issue = [&](int s, u4v* to) {
        const int k = min(s, s1 - 1) * S::KE;
#pragma unroll
        for (int i = 0; i < S::XI; i++) load_lds(xp[i] + (k + xk[i] < j.K ? k : -xk[i]), to + 64 * (S::XI * wave + i));
#pragma unroll
        for (int i = 0; i < S::FW; i++) load_lds(fp[i] + (k + fk[i] < j.K ? k : -fk[i]), to + kTile * S::XC + fd[i]);
    };
    f4v acc[RB];
    auto sums = [&](auto INF) {
#pragma unroll
        for (int i = 0; i < RB; i++) acc[i] = f4v{0.f, 0.f, 0.f, 0.f};
        if (r > 0 && s0 < s1) {
            constexpr int NI = S::XI + S::FW;
#pragma unroll
            for (int i = 0; i < RING - 1; i++) issue(s0 + i, lds + i * S::CHUNKS);
            int cur = 0, put = RING - 1;
            const bool rows = 16 * wave < sl.rows;  // of this wave
            for (int s = s0; s < s1; s++) {
                ring_barrier<(RING - 2) * NI>();  // step s is there, and every wave is done with step s - 1
                issue(s + RING - 1, lds + put * S::CHUNKS);
                const u4v* x = lds + cur * S::CHUNKS + S::XC * (16 * wave + li);
                const u4v* f = lds + cur * S::CHUNKS + kTile * S::XC + li * S::FC;
                const int sx = swizzle<S::XC>(li), sf = swizzle<S::FC>(li);  // (rows 16 further have the same)
                cur = cur + 1 == RING ? 0 : cur + 1;
                put = put + 1 == RING ? 0 : put + 1;
                // TAIL: the axis's last step, whose missing elements count as 0
                auto multiply = [&](auto TAIL) {
#pragma unroll
                    for (int m = 0; m < S::KE / 32; m++) {
                        const int c = 4 * m + lq;  // the chunk of eight elements
                        const bool in = !TAIL || s * S::KE + 8 * c < j.K;
                        u4v a[ACT == kActF32 ? 3 : 1];
                        if constexpr (ACT == kActF32) {
                            const u4v u = x[(2 * c) ^ sx], v = x[(2 * c + 1) ^ sx];
                            float e[8];
#pragma unroll
                            for (int q = 0; q < 4; q++) {
                                e[q] = in ? __uint_as_float(u[q]) : 0.0f;
                                e[4 + q] = in ? __uint_as_float(v[q]) : 0.0f;
                            }
                            parts8<3>(e, a);
                        } else {
                            a[0] = x[c ^ sx];
#pragma unroll
                            for (int q = 0; q < 4; q++) a[0][q] = in ? a[0][q] : 0u;
                        }
#pragma unroll
                        for (int i = 0; i < RB; i++) {
                            u4v w = f[16 * i * S::FC + (c ^ sf)];
#pragma unroll
                            for (int q = 0; q < 4; q++) w[q] = in ? w[q] : 0u;
                            if constexpr (ACT == kActF32) {
#pragma unroll
                                for (int q = 2; q >= 0; q--) acc[i] = mma_bf16(a[q], INF && q ? without_inf(w) : w, acc[i]);
                            } else if constexpr (ACT == kActBf16) {
                                acc[i] = mma_bf16(a[0], w, acc[i]);
                            } else {
                                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, a[0]),
                                                                                __builtin_bit_cast(h8v, w), acc[i], 0, 0, 0);
                            }
                        }
                    }
                };
                if (rows && (s + 1) * S::KE <= j.K) multiply(std::false_type());
                else if (rows) multiply(std::true_type());
            }
            ring_barrier<0>();  // nothing is on its way into LDS any more, nobody reads the ring
        }
    };
    sums(std::false_type());
    float(*red)[R16 + 1] = reinterpret_cast<float(*)[R16 + 1]>(lds);
    uint32_t* ticket = reinterpret_cast<uint32_t*>(lds + SUMS);
    if constexpr (ACT == kActF32) {  // operands in parts: all waves once more, by one's NaN
        int nan = 0;
#pragma unroll
        for (int i = 0; i < RB; i++) nan |= has_nan(acc[i]);
        const bool any = __ballot(nan) != 0;
        if (lane == 0) ticket[wave] = any;
        __syncthreads();
        const bool again = ticket[0] | ticket[1] | ticket[2] | ticket[3];
        __syncthreads();
        if (again) sums(std::true_type());
    }
#pragma unroll
    for (int i = 0; i < RB; i++)
#pragma unroll
        for (int q = 0; q < 4; q++) red[16 * wave + 4 * lq + q][16 * i + li] = acc[i][q];
    __syncthreads();
    if (ks > 1) {
        // 16 bytes a thread at a time, kCoherent: past this XCD's L2
        constexpr int PER = R16 / 16;  // of a thread: 64 tokens x R16 / 4 / 256
        const rsrc_t rp = make_rsrc(j.part + (size_t)sl.row * R16, (uint32_t)sl.rows * (uint32_t)(R16 * 4));
        auto cell = [&](int i) { return (tid + 256 * i) * 4; };  // rows behind the tile's store nothing, read 0
        const size_t stride = (size_t)T * R16;
        const rsrc_t mine = make_rsrc(j.part + ky * stride + (size_t)sl.row * R16, (uint32_t)sl.rows * (uint32_t)(R16 * 4));
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int c = cell(i);
            const float* q = &red[c / R16][c % R16];
            const u4v v = {__float_as_uint(q[0]), __float_as_uint(q[1]), __float_as_uint(q[2]), __float_as_uint(q[3])};
            __builtin_amdgcn_raw_buffer_store_b128(v, mine, (uint32_t)c * 4u, 0, kCoherent);
        }
        // each wave waits for its own stores, then one ticket for all of them
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (tid == 0)
            *ticket = __hip_atomic_fetch_add(tickets + (second ? gridDim.x : 0) + blockIdx.x, 1u, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (*ticket + 1 != (uint32_t)ks) return;
        f4v sum[PER];
#pragma unroll
        for (int i = 0; i < PER; i++)
            sum[i] = __builtin_bit_cast(f4v, __builtin_amdgcn_raw_buffer_load_b128(rp, (uint32_t)cell(i) * 4u, 0, kCoherent));
        for (int q = 1; q < ks; q++) {
            const rsrc_t rq = make_rsrc(j.part + q * stride + (size_t)sl.row * R16, (uint32_t)sl.rows * (uint32_t)(R16 * 4));
            f4v v[PER];
#pragma unroll
            for (int i = 0; i < PER; i++)
                v[i] = __builtin_bit_cast(f4v, __builtin_amdgcn_raw_buffer_load_b128(rq, (uint32_t)cell(i) * 4u, 0, kCoherent));
#pragma unroll
            for (int i = 0; i < PER; i++) sum[i] += v[i];
        }
#pragma unroll
        for (int i = 0; i < PER; i++)
#pragma unroll
            for (int q = 0; q < 4; q++) red[cell(i) / R16][cell(i) % R16 + q] = sum[i][q];
        __syncthreads();
    }
    const float sc = tab.scales[sl.g];
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
            for (int h = 0; h < 3; h++) j.by_rank[(((size_t)blockIdx.x * 3 + h) * R16 + k) * 8 + (c ^ swizzle<8>(k))] = o[h];
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
// "up": grid (ceil(N / 256), slots): y of one tile and 256 columns, 64 a wave,
// everything from memory to registers. Workgroups that run together write whole
// rows (the tiles first: 68 us against 59 at 8192 x 8192, rank 16). The base
// rows are requested first. Of the factor, lane (i, q) loads ranks 8 q .. + 7
// of 4 neighbouring columns 4 i + j and turns them into one operand for each
// column, so that a lane ends with 4 neighbouring columns of its rows. Bound by
// memory: base read and y written, 268 MB at 8192 x 8192 bf16 in 59 us, 4.5
// TB/s (a large copy: 5.1); 2451 x 2560 fp16, rank 64: 16 us, 1.6 TB/s, where
// the launch, the factor's loads and their turning count.
template <int ACT, int RB>
__global__ __launch_bounds__(256) void k_lora_up(const u4v* __restrict__ u, int T, int N, int n, int R,
                                                 const void* const* __restrict__ fac,
                                                 LoraTable tab, const int32_t* __restrict__ perm,
                                                 const Slot* __restrict__ tiles, const typename Act<ACT>::T* base,
                                                 size_t ldb, typename Act<ACT>::T* y, size_t ldy) {
    constexpr int R32 = RB < 2 ? 32 : RB * 16, CH = R32 / 8;
    constexpr bool F16 = ACT == kActF16;
    const Slot sl = tiles[blockIdx.y];
    if (sl.rows == 0) return;
    const bool none = sl.g == n + 1;
    if (none && base == y) return;
    const int lane = threadIdx.x & 63, wave = wave_id(), li = lane & 15, lq = lane >> 4;
    const int c0 = blockIdx.x * kUpCols + wave * 64 + 4 * li, cl = min(c0, N - 4);
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
    const int r = none ? 0 : (sl.g == n ? -1 : rank_of(tab, sl.g, R));
    constexpr int NG = R32 / 32, P = Cols16<F16>::P;
    u4v f[NG][P][4];
    u4v a[NG][3];
    const u4v* ub = u + (size_t)(sl.row + li) * CH + lq;
    auto load_u = [&](int b) {  // rows behind the tile repeat the last one
        const int back = max(16 * b + li - (sl.rows - 1), 0);
#pragma unroll
        for (int g = 0; g < NG; g++)
#pragma unroll
            for (int h = 0; h < 3; h++) a[g][h] = ub[((size_t)h * T + 16 * b - back) * CH + 4 * g];
    };
    if (r > 0) {
        const rsrc_t rf = make_rsrc(fac[sl.g], (uint32_t)r * (uint32_t)N * 2u);  // rows behind the rank read 0
        u2v w[NG][8];
#pragma unroll
        for (int g = 0; g < NG; g++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint2 x = ld_b64(rf, ((uint32_t)(32 * g + 8 * lq + i) * (uint32_t)N + (uint32_t)cl) * 2u);
                w[g][i] = u2v{x.x, x.y};
            }
        load_u(0);
#pragma unroll
        for (int g = 0; g < NG; g++) {
            Cols16<F16> c;
            cols16<F16>(w[g], c);
#pragma unroll
            for (int h = 0; h < P; h++)
#pragma unroll
                for (int j = 0; j < 4; j++) f[g][h][j] = c.c[h][j];
        }
    }
    f4v acc[4];
    auto value = [&](int q, wv o4) {  // of row q of acc
        f4v v = {acc[0][q], acc[1][q], acc[2][q], acc[3][q]};
        if (base) {
            if constexpr (ACT == kActF32) {
                v += __builtin_bit_cast(f4v, o4);
            } else {
                float e, o;
                cvt2<ACT>(o4[0], e, o); v.x += e; v.y += o;
                cvt2<ACT>(o4[1], e, o); v.z += e; v.w += o;
            }
        }
        return v;
    };
    uint32_t todo = 0;  // blocks of 16 rows, not written yet for a NaN
#pragma unroll
    for (int b = 0; b < 4; b++) {
        if (16 * b >= sl.rows) break;
#pragma unroll
        for (int j = 0; j < 4; j++) acc[j] = f4v{0.f, 0.f, 0.f, 0.f};
        if (r > 0) {
#pragma unroll
            for (int g = 0; g < NG; g++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    u4v p[P];
#pragma unroll
                    for (int h = 0; h < P; h++) p[h] = f[g][h][j];
                    acc[j] = mma_parts<P>(a[g], p, acc[j]);
                }
            if (b < 3 && 16 * (b + 1) < sl.rows) load_u(b + 1);
            if (__ballot(has_nan(acc[0]) | has_nan(acc[1]) | has_nan(acc[2]) | has_nan(acc[3]))) {
                todo |= 1u << b;
                continue;
            }
        }
        if (c0 < N)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                f4v v = value(q, old[b][q]);
                if (r < 0) v.x = v.y = v.z = v.w = __builtin_nanf("");
                if (16 * b + 4 * lq + q < sl.rows) st4<ACT>(y + (size_t)t[b][q] * ldy + c0, v);
            }
    }
    if (!todo) return;
    // See nan_or_inf. Everything is loaded again, from places that the compiler
    // does not know to be the same: kept for this, they take the registers of a
    // workgroup above.
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int i2 = ln & 15, q2 = ln >> 4, c2 = blockIdx.x * kUpCols + wave * 64 + 4 * i2, cl2 = min(c2, N - 4);
    const int tok = perm[sl.row + min(ln, sl.rows - 1)];
    const rsrc_t rf = make_rsrc(fac[sl.g], (uint32_t)r * (uint32_t)N * 2u);
#pragma unroll 1
    for (int b = 0; b < 4; b++) {
        if (!(todo >> b & 1u)) continue;
        f4v first[4];
#pragma unroll
        for (int j = 0; j < 4; j++) acc[j] = first[j] = f4v{0.f, 0.f, 0.f, 0.f};
        const int row = sl.row + min(16 * b + i2, sl.rows - 1);
#pragma unroll 1
        for (int g = 0; g < NG; g++) {
            u2v w[8];
            u4v au[3];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint2 x = ld_b64(rf, ((uint32_t)(32 * g + 8 * q2 + i) * (uint32_t)N + (uint32_t)cl2) * 2u);
                w[i] = u2v{x.x, x.y};
            }
#pragma unroll
            for (int h = 0; h < 3; h++) au[h] = u[((size_t)h * T + row) * CH + 4 * g + q2];
            Cols16<F16> c;
            cols16<F16>(w, c);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                u4v p[P];
#pragma unroll
                for (int h = 0; h < P; h++) p[h] = c.c[h][j];
                acc[j] = mma_parts<P>(au, p, acc[j]);
                first[j] = mma_bf16(au[0], p[0], first[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int q = 0; q < 4; q++) acc[j][q] = is_nan(acc[j][q]) ? nan_or_inf(first[j][q]) : acc[j][q];
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int tq = __shfl(tok, 16 * b + 4 * q2 + q, 64);
            if (16 * b + 4 * q2 + q >= sl.rows || c2 >= N) continue;
            wv o = {};
            if (base) o = *reinterpret_cast<const wv*>(base + (size_t)tq * ldb + c2);
            st4<ACT>(y + (size_t)tq * ldy + c2, value(q, o));
        }
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

// grid (column blocks of A then of B, piece slots; the pieces first: 62 us
// against 46 at 8192 tokens, rank 64: 3.8 TB/s of x and dy read): 256 columns,
// 64 a wave, over one piece, a tile of 64 tokens at a time. One workgroup
// reads each row piece once for all ranks, so the rows pass by once and the
// sums stay in registers. low's parts go from memory straight into LDS, the
// rows' values into registers, by lane (i, q) as tokens 8 q .. + 7 (and 32
// more) of 4 neighbouring columns, both a tile ahead; the values are turned
// into an operand for each column. An adapter of one piece
// writes its gradient, others the piece's part for k_lora_grad_reduce.
template <int ACT, int RB>
__global__ __launch_bounds__(256) void k_lora_grad(GradSide ga, GradSide gb, int n, int R, int piece,
                                                   LoraTable tab, const int32_t* __restrict__ perm,
                                                   const Group* __restrict__ groups, const Slot* __restrict__ pieces,
                                                   int accumulate, float* __restrict__ part) {
    constexpr int R16 = RB * 16, TILE = 3 * R16 * 8;  // chunks of a tile's low values
    constexpr int WB = ACT == kActF32 ? 4 : 2, PX = ACT == kActF32 ? 3 : (ACT == kActF16 ? 2 : 1);
    typedef uint32_t wv __attribute__((ext_vector_type(WB)));
    __shared__ u4v us[2 * TILE];
    const Slot sl = pieces[blockIdx.y];
    if (sl.rows == 0 || sl.g >= n) return;
    const int r = rank_of(tab, sl.g, R);
    if (r <= 0) return;
    const int nba = (ga.cols + kUpCols - 1) / kUpCols;
    const bool second = (int)blockIdx.x >= nba;
    const GradSide side = second ? gb : ga;
    float* out = side.out ? side.out[sl.g] : nullptr;
    if (!out) return;
    const int lane = threadIdx.x & 63, wave = wave_id(), li = lane & 15, lq = lane >> 4;
    const int cols = side.cols, c0 = ((int)blockIdx.x - (second ? nba : 0)) * kUpCols + wave * 64 + 4 * li;
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
                for (int q = 0; q < 3; q++) a[q] = us_k[(q * R16 + 16 * b + li) * 8 + ((4 * h + lq) ^ swizzle<8>(li))];
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
    const bool whole = grp.rows <= piece;
    typedef __attribute__((address_space(1))) f4v* gp;  // the table's pointers are to global memory
    float* to = whole ? out : part + (size_t)blockIdx.y * R16 * ((size_t)ga.cols + gb.cols) +
                                  (second ? (size_t)R16 * ga.cols : 0);
    int nan = 0;
#pragma unroll
    for (int b = 0; b < RB; b++)
#pragma unroll
        for (int j = 0; j < 4; j++) nan |= has_nan(acc[b][j]);
    if (!__ballot(nan)) {
        if (c0 >= cols) return;
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
        return;
    }
    // see nan_or_inf: the other sums are written as they are
    uint32_t todo[4] = {0, 0, 0, 0};  // of column j: bit 4 b + q
    auto place = [&](int b, int q, int j) { return to + (size_t)(16 * b + 4 * lq + q) * cols + c0 + j; };
    auto write = [&](float* p, float v) { *p = whole && accumulate ? *p + v : v; };
#pragma unroll
    for (int b = 0; b < RB; b++)
#pragma unroll
        for (int q = 0; q < 4; q++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (c0 >= cols || 16 * b + 4 * lq + q >= r) continue;
                if (is_nan(acc[b][j][q])) todo[j] |= 1u << (4 * b + q);
                else write(place(b, q, j), acc[b][j][q]);
            }
#pragma unroll 1
    for (int b = 0; b < RB; b++) {
        if (!__ballot((todo[0] | todo[1] | todo[2] | todo[3]) >> (4 * b) & 15u)) continue;
        f4v first[4];
#pragma unroll
        for (int j = 0; j < 4; j++) first[j] = f4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int k = 0; k < 2 * tiles; k++) {  // 32 tokens
            const int tk = perm[sl.row + min(32 * k + (lane & 31), sl.rows - 1)];
            const u4v a = low[(k / 2) * TILE + (16 * b + li) * 8 + ((4 * (k % 2) + lq) ^ swizzle<8>(li))];
            wv w[8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const wv v = *reinterpret_cast<const wv*>(X + (size_t)__shfl(tk, 8 * lq + i, 64) * side.ld);
#pragma unroll
                for (int d = 0; d < WB; d++) w[i][d] = 32 * k + 8 * lq + i < sl.rows ? v[d] : 0u;
            }
            u4v f[4];
            if constexpr (ACT == kActF32) {
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        f[j][q] = pack_first(__uint_as_float(w[2 * q][j]), __uint_as_float(w[2 * q + 1][j]));
            } else {
                Cols16<ACT == kActF16> c;
                cols16<ACT == kActF16>(w, c);
#pragma unroll
                for (int j = 0; j < 4; j++) f[j] = c.c[0][j];
            }
#pragma unroll
            for (int j = 0; j < 4; j++) first[j] = mma_bf16(a, f[j], first[j]);
        }
#pragma unroll
        for (int q = 0; q < 4; q++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (todo[j] >> (4 * b + q) & 1u) write(place(b, q, j), nan_or_inf(first[j][q]));
    }
}

// grid (column blocks of 1024, R, n): gradients of adapters with no token
// (zeros) and with several pieces (the parts, in increasing order); an
// adapter whose rank is not usable gets nothing.
__global__ __launch_bounds__(256) void k_lora_grad_reduce(int ca, int cb, float* const* da, float* const* db, int n,
                                                          int R, int R16, int piece, LoraTable tab,
                                                          const Group* __restrict__ groups, int accumulate,
                                                          const float* __restrict__ part) {
    const int a = blockIdx.z, m = blockIdx.y;
    const Group g = groups[a];
    const int r = g.rows ? rank_of(tab, a, R) : table_rank(tab, a, R);  // without tokens there may be no factors
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
    const dim3 grid(w.slots, a.ks + (sides > 1 ? b.ks : 0));
#define DN(B)                                                                                                       \
    hipLaunchKernelGGL((k_lora_down<ACT, B>), grid, dim3(256), 0, s, a, b, n, R, tab, perm, tiles, T, \
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
    const dim3 grid(col_blocks(N), w.slots);
#define UP(B)                                                                                                      \
    hipLaunchKernelGGL((k_lora_up<ACT, B>), grid, dim3(256), 0, s, u, T, N, n, R, fac, tab, perm, tiles, (const E*)base, \
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
    const LoraWs w = lora_ws(K, N, n, R, T, false, ACT == kActF32);
    const LoraMem m(w, ws);
    hipError_t r;
    if (direct(T, R)) {
        if (R * K <= kTokFused && (int64_t)T * ((N + 511) / 512) <= 256) {
            hipLaunchKernelGGL((k_lora_tok<ACT>), dim3(T, (N + 511) / 512), dim3(1024), 0, s, (const E*)x, ldx, K, N, n, R,
                               tab, (const E*)base, ldb, (E*)y, ldy);
            return hipGetLastError();
        }
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
    const DownJob j = {x, ldx, K, tab.a, w.ku, m.part, m.ut, nullptr};
    if ((r = down<ACT>(w, 1, s, j, j, n, R, tab, m.perm, m.tiles, T, m.tickets)) != hipSuccess) return r;
    return up<ACT>(w, s, m.ut, T, N, n, R, tab.b, tab, m.perm, m.tiles, base, ldb, y, ldy);
}

template <int ACT>
hipError_t backward(int K, int N, int n, int R, const void* x, size_t ldx, const void* dy, size_t lddy, int T,
                    const LoraTable& tab, const void* dxb, size_t lddxb, void* dx, size_t lddx, float* const* da,
                    float* const* db, int accumulate, void* ws, hipStream_t s) {
    const LoraWs w = lora_ws(K, N, n, R, T, true, ACT == kActF32);
    const LoraMem m(w, ws);
    hipError_t r;
    hipLaunchKernelGGL(k_lora_plan, dim3(n + 2), dim3(1024), 0, s, tab.ids, T, n, m.perm, m.groups, m.tiles, m.pieces,
                       w.piece, m.tickets, w.slots);
    if ((r = hipGetLastError()) != hipSuccess) return r;
    if (T > 0) {
        const DownJob jv = {dy, lddy, N, tab.b, w.kv, m.part, dx ? m.vt : nullptr, da ? m.vr : nullptr};
        const DownJob ju = {x, ldx, K, tab.a, w.ku, m.part + (w.kv > 1 ? (size_t)w.kv * T * w.R16 : 0), nullptr, m.ur};
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
        const dim3 grid(col_blocks(K) + col_blocks(N), w.pslots);
#define GR(B)                                                                                                       \
    hipLaunchKernelGGL((k_lora_grad<ACT, B>), grid, dim3(256), 0, s, ga, gb, n, R, w.piece, tab, m.perm, m.groups, \
                       m.pieces, accumulate, m.grad)
        if (w.R16 == 16) GR(1); else if (w.R16 == 32) GR(2); else if (w.R16 == 64) GR(4); else GR(8);
#undef GR
        if ((r = hipGetLastError()) != hipSuccess) return r;
    }
    hipLaunchKernelGGL(k_lora_grad_reduce, dim3((K + 1023) / 1024 + (N + 1023) / 1024, R, n), dim3(256), 0, s, K, N, da,
                       db, n, R, w.R16, w.piece, tab, m.groups, accumulate, m.grad);
    return hipGetLastError();
}

}  // namespace

size_t lora_ws_bytes(int K, int N, int n, int R, int T, bool back) { return lora_ws(K, N, n, R, T, back, false).total; }

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

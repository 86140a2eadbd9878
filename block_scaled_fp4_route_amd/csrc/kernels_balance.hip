// The router's balance loss, its z loss, the per-expert counts and the
// gradient of the logits, for gfx950.
//
// Over the counted tokens C_s of sequence s (n_s of them; live sequences have
// n_s > 0; N counted tokens in all), with p_t = softmax(l_t):
//   counts[s][e] = #{(t, j): t in C_s, idx[t][j] = e}
//   probs[s][e]  = (1 / n_s) sum_t p[t][e]
//   balance      = (1 / live) sum_s E sum_e counts[s][e] / (n_s k) probs[s][e]
//   z            = (1 / N) sum_t lse_t^2
// The counts are constants of the gradient, so with
//   c[s][e] = E counts[s][e] / (live k n_s^2)
// the logits' gradient needs nothing that other tokens' logits decide:
//   dl[t][e] = up p[t][e] (cb (c[s][e] - sum_e' c[s][e'] p[t][e']) + cz (2 / N) lse_t)
// and one pass over the logits gives the loss and the gradient. Order:
//   k_bal_count  counts per sequence from idx alone (LDS histograms, J parts
//                per sequence; k_bal_merge adds the parts when J > 1)
//   k_bal_main   softmax, gradient and each chunk's sums of p and lse^2
//   k_bal_reduce the chunks' sums in fixed order, the probabilities, the loss
// No float atomics: results are bit-identical from run to run.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_internal.h"
#include "moe_learn.h"

namespace moe {

namespace {

constexpr int kMaxParts = 4;  // parts of a sequence's counts that k_bal_main adds
constexpr int kBadSeq = -1;  // n_s of a sequence with a bad offset or a bad expert index

// T * k up to which k_bal_main counts by itself (with the counting launch of 2.2
// to 3.2 us beside it, or not: 10 indices 6.3 against 4.7 us, 1866 8.2 against
// 5.6, 8000 8.5 against 7.6, 13000 10.0 against 10.2, 24510 11.5 against 16.8).
constexpr int kSelfCount = 8192;

// Workspace regions (all 256-byte aligned).
struct BalWs {
    int J;           // parts per sequence of the counting launch
    int JM;          // parts that k_bal_main finds (1 behind k_bal_merge)
    int TB;          // tokens per chunk of the main launch
    int chunks;
    size_t part, cnt, n, ticket, psum, zsum, q, total;
};

BalWs bal_ws(int T, int E, int S) {
    BalWs b;
    // about 1024 tokens per counting workgroup, 64 parts at most; several
    // sequences, which may be of unlike lengths, get 4 parts where that still
    // leaves 128 tokens each; the main launch adds up to kMaxParts itself
    const int64_t per = ((int64_t)T + S - 1) / S;
    b.J = (int)((per + 1023) / 1024);
    if (S > 1 && b.J < kMaxParts) b.J = (int)(per / 128 < kMaxParts ? per / 128 : kMaxParts);
    b.J = b.J < 1 ? 1 : (b.J > 64 ? 64 : b.J);
    b.JM = b.J <= kMaxParts ? b.J : 1;
    // about 1024 chunks (four workgroups per compute unit) of whole rounds of
    // the four waves
    b.TB = (int)(((int64_t)T + 1023) / 1024);
    b.TB = (b.TB + 3) / 4 * 4;
    if (b.TB < 4) b.TB = 4;
    b.chunks = (int)(((int64_t)T + b.TB - 1) / b.TB);
    size_t o = kCounterBytes;
    auto take = [&o](size_t bytes) {
        const size_t at = o;
        o += align256(bytes);
        return at;
    };
    const size_t row = (size_t)E * 4;
    // Sized so that fewer tokens never need more: JM and chunks fall where the
    // parts or the tokens of a chunk grow.
    const size_t jm = b.J < kMaxParts ? b.J : kMaxParts, most = T < 4096 ? ((size_t)T + 3) / 4 : 1024;
    b.part = take(b.J > b.JM ? (size_t)S * b.J * (row + 4) : 0);
    b.cnt = take((size_t)S * jm * row);
    b.n = take((size_t)S * jm * 4);
    b.ticket = take(4);
    b.psum = take((most + S) * row);
    b.zsum = take((most + S) * 4);
    b.q = take((size_t)S * (((size_t)E + 15) / 16 + 1) * 4);
    b.total = o;
    return b;
}

// Bounds of sequence s; false if the list is not usable there.
__device__ __forceinline__ bool seq_bounds(const int32_t* __restrict__ off, int s, int T, int& lo, int& hi) {
    lo = off ? off[s] : 0;
    hi = off ? off[s + 1] : T;
    return lo >= 0 && lo <= hi && hi <= T;
}

// Adds the routing of tokens a .. b - 1 to hist (LDS) by NT threads; returns
// whether this thread saw a bad index, and its share of the counted tokens in
// `mine`. Without a mask the indices are one list, eight loads a thread at
// once; with one a thread takes a token, its mask byte beside its indices
// (finding the token of each index of the list and then its mask: 12 us
// against 9 at 32768 tokens; token by token without a mask: 8 against 4 at
// 2451).
template <int NT>
__device__ __forceinline__ bool bal_hist(const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask, int a,
                                         int b, int E, int k, int* hist, int& mine) {
    bool bad = false;
    mine = 0;
    if (!mask) {
        if (threadIdx.x == 0) mine = b - a;
        const int i1 = b * k;  // T k <= 2^29
        for (int i = a * k + (int)threadIdx.x; i < i1; i += 8 * NT) {
            int e[8];
#pragma unroll
            for (int u = 0; u < 8; u++) e[u] = i + u * NT < i1 ? idx[i + u * NT] : 0;
#pragma unroll
            for (int u = 0; u < 8; u++) {
                const bool in = (unsigned)e[u] < (unsigned)E, use = i + u * NT < i1;
                if (use && in) atomicAdd(&hist[e[u]], 1);
                bad |= use && !in;
            }
        }
        return bad;
    }
    for (int t = a + (int)threadIdx.x; t < b; t += NT) {
        const bool on = mask[t] != 0;
        const int32_t* it = idx + (size_t)t * k;
        for (int i = 0; i < k; i += 8) {
            int e[8];
#pragma unroll
            for (int u = 0; u < 8; u++) e[u] = it[min(i + u, k - 1)];
#pragma unroll
            for (int u = 0; u < 8; u++) {
                const bool in = (unsigned)e[u] < (unsigned)E, use = on && i + u < k;
                if (use && in) atomicAdd(&hist[e[u]], 1);
                bad |= use && !in;
            }
        }
        mine += on;
    }
    return bad;
}

// grid (J, S), 1024 threads: counts of the tokens of part j of sequence s.
__global__ __launch_bounds__(1024) void k_bal_count(const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
                                                    const int32_t* __restrict__ off, int T, int E, int k, int J,
                                                    int32_t* __restrict__ cnt, int32_t* __restrict__ n,
                                                    uint32_t* __restrict__ ticket) {
    __shared__ int hist[kMaxE];
    __shared__ int tot[2];
    const int j = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
    if (tid < E) hist[tid] = 0;
    if (tid < 2) tot[tid] = 0;
    if (tid == 0 && j == 0 && s == 0) *ticket = 0;
    int lo, hi;
    const bool fine = seq_bounds(off, s, T, lo, hi);
    __syncthreads();
    int mine = 0;
    bool bad = !fine;
    if (fine) {
        const int per = (hi - lo + J - 1) / J;
        const int a = (int)min((int64_t)hi, lo + (int64_t)j * per), b = (int)min((int64_t)hi, (int64_t)a + per);
        bad = bal_hist<1024>(idx, mask, a, b, E, k, hist, mine);
    }
    if (mine) atomicAdd(&tot[0], mine);
    if (bad) atomicOr(&tot[1], 1);
    __syncthreads();
    const size_t p = (size_t)s * J + j;
    if (tid < E) cnt[p * E + tid] = hist[tid];
    if (tid == 0) n[p] = tot[1] ? kBadSeq : tot[0];
}

// grid (ceil(E / 256), S): adds the J parts of each sequence.
__global__ __launch_bounds__(256) void k_bal_merge(const int32_t* __restrict__ pc, const int32_t* __restrict__ pn,
                                                   int E, int J, int32_t* __restrict__ cnt, int32_t* __restrict__ n) {
    const int e = blockIdx.x * 256 + threadIdx.x, s = blockIdx.y;
    if (e < E) {
        int a = 0;
#pragma unroll 8
        for (int j = 0; j < J; j++) a += pc[((size_t)s * J + j) * E + e];
        cnt[(size_t)s * E + e] = a;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        int a = 0;
        bool bad = false;
        for (int j = 0; j < J; j++) {
            const int v = pn[(size_t)s * J + j];
            bad |= v < 0;
            a += v;
        }
        n[s] = bad ? kBadSeq : a;
    }
}

// Counted tokens of sequence s from its J <= kMaxParts parts, loaded together;
// kBadSeq if one of them is bad.
__device__ __forceinline__ int seq_n(const int32_t* __restrict__ n, int s, int J) {
    int v[kMaxParts], a = 0;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < kMaxParts; j++) v[j] = n[(size_t)s * J + min(j, J - 1)];
#pragma unroll
    for (int j = 0; j < kMaxParts; j++) {
        bad |= v[j] < 0;
        a += j < J ? v[j] : 0;
    }
    return bad ? kBadSeq : a;
}

// What a workgroup has to know of all sequences: the live ones, the counted
// tokens, the first one that ends behind token t0 (the offsets do not decrease
// where all are fine), and whether all are fine. One round of loads; the first
// kSeqLds sequences' numbers stay in LDS for what follows.
constexpr int kSeqLds = 256;
struct Seqs {
    int live, total, first;
    bool fine;
};
template <int NT>
__device__ __forceinline__ Seqs bal_totals(const int32_t* __restrict__ n, const int32_t* __restrict__ off, int T,
                                           int t0, int S, int J, int* sn, int* so) {
    __shared__ int acc[4];
    if (threadIdx.x < 4) acc[threadIdx.x] = 0;
    __syncthreads();
    int l = 0, t = 0, b = 0, f = 0;
    for (int s = threadIdx.x; s < S; s += NT) {
        const int v = seq_n(n, s, J), lo = off ? off[s] : 0, hi = off ? off[s + 1] : T;
        if (s < kSeqLds) {
            sn[s] = v;
            so[2 * s] = lo;
            so[2 * s + 1] = hi;
        }
        f += hi <= t0;
        l += v > 0;
        t += max(v, 0);
        b |= v < 0;
    }
    if (l) {
        atomicAdd(&acc[0], l);
        atomicAdd(&acc[1], t);
    }
    if (b) atomicOr(&acc[2], 1);
    if (f) atomicAdd(&acc[3], f);
    __syncthreads();
    return Seqs{acc[0], acc[1], acc[3], acc[2] == 0};
}

// Column i (< NV) of this lane: vector form 4 lane + 256 (i / 4) + i % 4,
// scalar form lane + 64 i. Both cover 64 NV columns.
template <bool VEC>
__device__ __forceinline__ int bal_col(int lane, int i) {
    return VEC ? 4 * lane + 256 * (i / 4) + i % 4 : lane + 64 * i;
}

template <int NV, bool VEC>
__device__ __forceinline__ void row_load(const float* __restrict__ row, int E, int lane, float fill, float (&v)[NV]) {
    if constexpr (VEC) {
#pragma unroll
        for (int c = 0; c < NV / 4; c++) {
            const int e = 4 * lane + 256 * c;
            f4v q = {fill, fill, fill, fill};
            if (e < E) q = *reinterpret_cast<const f4v*>(row + e);
            v[4 * c] = q.x; v[4 * c + 1] = q.y; v[4 * c + 2] = q.z; v[4 * c + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int e = lane + 64 * i;
            v[i] = e < E ? row[e] : fill;
        }
    }
}

template <int NV, bool VEC>
__device__ __forceinline__ void row_store(float* __restrict__ row, int E, int lane, const float (&v)[NV]) {
    if constexpr (VEC) {
#pragma unroll
        for (int c = 0; c < NV / 4; c++) {
            const int e = 4 * lane + 256 * c;
            const f4v q = {v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]};
            if (e < E) *reinterpret_cast<f4v*>(row + e) = q;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int e = lane + 64 * i;
            if (e < E) row[e] = v[i];
        }
    }
}

// grid chunks, 256 threads. A chunk's tokens are cut at the sequences'
// bounds; the piece of sequence s in chunk c writes its sums at row c + s
// (pieces follow one another with c or s growing, so no two share a row).
// Each wave takes every fourth token of a piece, a lane NV columns, the next
// token's row in flight while one is worked on.
// SELF (one sequence, few tokens): every workgroup counts the whole routing
// itself, the first one also for k_bal_reduce, and no counting launch runs
// (see kSelfCount). Bound by memory at length: logits read and gradient written
// once, 134 MB of 32768 x 512 in 34 us, 4.0 TB/s.
template <int NV, bool VEC, bool SELF>
__global__ __launch_bounds__(256) void k_bal_main(const float* __restrict__ logits, const uint8_t* __restrict__ mask,
                                                  const int32_t* __restrict__ off, int T, int E, int k, int S, int TB,
                                                  const int32_t* __restrict__ idx, int J, int32_t* __restrict__ cnt,
                                                  int32_t* __restrict__ n, uint32_t* __restrict__ ticket,
                                                  float cb, float cz, const float* __restrict__ dloss,
                                                  float* __restrict__ dlogits, float* __restrict__ psum,
                                                  float* __restrict__ zsum) {
    __shared__ float red[4][64 * NV];
    __shared__ float zred[4];
    const int lane = threadIdx.x & 63, wave = wave_id(), c = blockIdx.x;
    const int t0 = c * TB, t1 = min(T, t0 + TB);
    __shared__ int sn[kSeqLds], so[2 * kSeqLds];  // counted tokens and bounds of the sequences
    Seqs all;
    const float up = dloss ? *dloss : 1.0f;
    __shared__ int hist[SELF ? 64 * NV : 1];
    __shared__ int tot[2];
    if constexpr (SELF) {
        const int tid = threadIdx.x;
        for (int e = tid; e < E; e += 256) hist[e] = 0;
        if (tid < 2) tot[tid] = 0;
        int lo, hi, mine = 0;
        bool bad = !seq_bounds(off, 0, T, lo, hi);
        __syncthreads();
        if (!bad) bad = bal_hist<256>(idx, mask, lo, hi, E, k, hist, mine);
        if (mine) atomicAdd(&tot[0], mine);
        if (bad) atomicOr(&tot[1], 1);
        if (tid == 0) {
            so[0] = lo;
            so[1] = hi;
        }
        __syncthreads();
        all = Seqs{tot[0] > 0, tot[0], hi <= t0, tot[1] == 0};
        if (tid == 0) sn[0] = all.total;
        if (c == 0) {
            for (int e = tid; e < E; e += 256) cnt[e] = hist[e];
            if (tid == 0) {
                *n = all.fine ? all.total : kBadSeq;
                *ticket = 0;
            }
        }
        __syncthreads();
    } else {
        all = bal_totals<256>(n, off, T, t0, S, J, sn, so);
    }
    if (!all.fine) {
        if (dlogits) {
            float q[NV];
#pragma unroll
            for (int i = 0; i < NV; i++) q[i] = __builtin_nanf("");
            for (int t = t0 + wave; t < t1; t += 4) row_store<NV, VEC>(dlogits + (size_t)t * E, E, lane, q);
        }
        return;
    }
    const int live = all.live, total = all.total;
    float zero[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) zero[i] = 0.0f;
    int t = t0, s = all.first;
    while (t < t1) {
        int lo = t1, hi = t1, ns = 0;
        if (s < kSeqLds) {
            if (s < S) {
                lo = so[2 * s];
                hi = so[2 * s + 1];
                ns = sn[s];
            }
        } else if (s < S) {
            lo = off[s];
            hi = off[s + 1];
            ns = seq_n(n, s, J);
        }
        const int a = __builtin_amdgcn_readfirstlane(max(t, min(t1, lo)));
        const int b = __builtin_amdgcn_readfirstlane(max(a, min(t1, hi)));
        if (dlogits)
            for (int u = t + wave; u < a; u += 4) row_store<NV, VEC>(dlogits + (size_t)u * E, E, lane, zero);
        if (a < b) {
            const float cf = ns > 0 ? cb * (float)E / ((float)live * (float)k * (float)ns * (float)ns) : 0.0f;
            const float zf = cz != 0.0f && total > 0 ? cz * 2.0f / (float)total : 0.0f;
            float co[NV], ps[NV], nx[2][NV];
            uint32_t on[2];
            // Rows go through buffer resources over the piece: rows behind it
            // and columns behind E read 0 and store nothing, and nothing in
            // the loop branches. (A load or store behind a branch makes the
            // compiler wait for every store in flight before the next row is
            // used.) Masked rows are
            // loaded too and left out.
            const uint32_t rowb = (uint32_t)E * 4u, bytes = (uint32_t)(b - a) * rowb;
            const rsrc_t rl = make_rsrc(logits + (size_t)a * E, bytes);
            const rsrc_t rd = make_rsrc(dlogits ? dlogits + (size_t)a * E : nullptr, dlogits ? bytes : 0u);
            const rsrc_t rm = make_rsrc(mask ? mask + a : nullptr, mask ? (uint32_t)(b - a) : 0u);
            uint32_t colo[VEC ? NV / 4 : NV];
#pragma unroll
            for (int q = 0; q < (VEC ? NV / 4 : NV); q++) {
                const int e = VEC ? 4 * lane + 256 * q : lane + 64 * q;
                colo[q] = e < E ? (uint32_t)e * 4u : kOOB;
            }
            auto fetch = [&](int u) {
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const uint32_t row = (uint32_t)(u + 4 * r);  // of the piece
                    on[r] = mask ? ld_b8(rm, row) : (uint32_t)((int)row < b - a);
#pragma unroll
                    for (int q = 0; q < (VEC ? NV / 4 : NV); q++) {
                        if constexpr (VEC) {
                            const auto x = __builtin_amdgcn_raw_buffer_load_b128(rl, row * rowb + colo[q], 0, 0);
#pragma unroll
                            for (int h = 0; h < 4; h++) nx[r][4 * q + h] = __uint_as_float(x[h]);
                        } else {
                            nx[r][q] = __uint_as_float(ld_b32(rl, row * rowb + colo[q]));
                        }
                    }
                }
            };
            fetch(wave);
#pragma unroll
            for (int i = 0; i < NV; i++) ps[i] = 0.0f;
            if constexpr (SELF) {
#pragma unroll
                for (int i = 0; i < NV; i++) {
                    const int e = bal_col<VEC>(lane, i);
                    co[i] = e < E ? cf * (float)hist[e] : 0.0f;
                }
            } else {
                // the parts' counts, all loads together (those past part J read 0)
                const rsrc_t rc = make_rsrc(cnt + (size_t)s * J * E, (uint32_t)J * rowb);
                uint32_t h[kMaxParts][NV];
#pragma unroll
                for (int j = 0; j < kMaxParts; j++)
#pragma unroll
                    for (int q = 0; q < (VEC ? NV / 4 : NV); q++) {
                        if constexpr (VEC) {
                            const auto x = __builtin_amdgcn_raw_buffer_load_b128(rc, (uint32_t)j * rowb + colo[q], 0, 0);
#pragma unroll
                            for (int g = 0; g < 4; g++) h[j][4 * q + g] = x[g];
                        } else {
                            h[j][q] = ld_b32(rc, (uint32_t)j * rowb + colo[q]);
                        }
                    }
#pragma unroll
                for (int i = 0; i < NV; i++) co[i] = cf * (float)(int)((h[0][i] + h[1][i]) + (h[2][i] + h[3][i]));
                static_assert(kMaxParts == 4, "four parts are added");
            }
            float zs = 0.0f;
            for (int u = wave; u < b - a; u += 8) {
                float v[2][NV], m[2], z[2], dot[2];
                bool mine[2];
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    mine[r] = on[r] != 0;
#pragma unroll
                    for (int i = 0; i < NV; i++) v[r][i] = bal_col<VEC>(lane, i) < E ? nx[r][i] : -INFINITY;
                }
                fetch(u + 8);
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    m[r] = v[r][0];
#pragma unroll
                    for (int i = 1; i < NV; i++) m[r] = fmaxf(m[r], v[r][i]);
                    m[r] = wave_max(m[r]);
                    m[r] = m[r] == -INFINITY ? 0.0f : m[r];  // nothing finite: every e^v is 0 (or NaN)
                }
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    z[r] = dot[r] = 0.0f;
#pragma unroll
                    for (int i = 0; i < NV; i++) {
                        // e^d by the hardware's 2^x: rounding d log2(e) adds |d| 2^-24
                        // relative, as much as rounding v - m did
                        v[r][i] = __builtin_amdgcn_exp2f((v[r][i] - m[r]) * 1.44269504f);
                        z[r] += v[r][i];
                        dot[r] = fmaf(co[i], v[r][i], dot[r]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    z[r] = wave_sum(z[r]);
                    dot[r] = wave_sum(dot[r]);
                }
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const float inv = z[r] == 0.0f ? 0.0f : 1.0f / z[r];
                    const float lse = z[r] == 0.0f ? 0.0f : m[r] + logf(z[r]);
                    zs += mine[r] ? lse * lse : 0.0f;
                    const float sh = (zf != 0.0f ? zf * lse : 0.0f) - dot[r] * inv, ui = up * inv;
#pragma unroll
                    for (int i = 0; i < NV; i++) {
                        ps[i] += mine[r] ? v[r][i] * inv : 0.0f;
                        v[r][i] = mine[r] ? ui * (v[r][i] * (co[i] + sh)) : 0.0f;
                    }
                    const uint32_t ro = (uint32_t)(u + 4 * r) * rowb;
#pragma unroll
                    for (int q = 0; q < (VEC ? NV / 4 : NV); q++) {
                        if constexpr (VEC) {
                            typedef uint32_t w4 __attribute__((ext_vector_type(4)));
                            const w4 x = {__float_as_uint(v[r][4 * q]), __float_as_uint(v[r][4 * q + 1]),
                                          __float_as_uint(v[r][4 * q + 2]), __float_as_uint(v[r][4 * q + 3])};
                            __builtin_amdgcn_raw_buffer_store_b128(x, rd, ro + colo[q], 0, 0);
                        } else {
                            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[r][q]), rd, ro + colo[q], 0, 0);
                        }
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; i++) red[wave][64 * i + lane] = ps[i];
            if (lane == 0) zred[wave] = zs;
            __syncthreads();
            const size_t row = (size_t)c + s;
            if (wave == 0) {
#pragma unroll
                for (int i = 0; i < NV; i++)
                    ps[i] = (red[0][64 * i + lane] + red[1][64 * i + lane]) +
                            (red[2][64 * i + lane] + red[3][64 * i + lane]);
                row_store<NV, VEC>(psum + row * E, E, lane, ps);
                if (lane == 0) zsum[row] = (zred[0] + zred[1]) + (zred[2] + zred[3]);
            }
        }
        t = b;
        s++;
    }
}

// grid (ceil(E / CB), rows), 1024 threads: CB columns x 1024 / CB row groups
// over the pieces of a sequence, every gridDim.y-th sequence; the last
// workgroup to finish adds the sequences up. Every workgroup takes a ticket
// from one counter, about 15 ns each, and looks at all sequences' numbers, so
// up to kFewSeqs sequences get narrow blocks, many pieces at a time, and more
// get wide ones, about kReduceGroups of them in all. Whole calls, narrow
// against wide: 2451 x 512 in 1 sequence 18 against 23 us, in 4 19 against 21,
// in 8 21 against 21, in 16 27 against 21; 32768 x 512 in 1 45 against 54, in 4
// 44 against 48, in 8 45 against 47, in 16 49 against 43, in 37 70 against 45;
// 32768 x 64 in 8 28 against 31. (This launch alone, 32768 x 512 in 200
// sequences: 17 us against 35 with a workgroup for each sequence and block, in
// 1000: 42 against 164, 99 with 2048 in all.) Bound by latency: 6 to 7 us for
// one sequence of 311 or 2451 tokens, of which the ticket and the last
// workgroup's part are about 2. Very many sequences stay slow, since each
// chunk and each workgroup here looks at all of them: calls of 32768 x 512
// take 58 us in 200, 94 in 1000, 364 in 8000, 2357 in 65535.
constexpr int kNarrow = 16, kWide = 128, kFewSeqs = 8, kReduceGroups = 256;
template <int CB>
__global__ __launch_bounds__(1024) void k_bal_reduce(const int32_t* __restrict__ off, int T, int E, int k, int S,
                                                     int TB, int J, const int32_t* __restrict__ cnt,
                                                     const int32_t* __restrict__ n, float cb, float cz,
                                                     const float* __restrict__ psum, const float* __restrict__ zsum,
                                                     float* __restrict__ q, uint32_t* __restrict__ ticket,
                                                     float* __restrict__ loss, int32_t* __restrict__ counts,
                                                     float* __restrict__ probs) {
    constexpr int NT = 1024, NW = 16, RG = NT / CB;
    __shared__ float red[RG][CB + 1];
    __shared__ float wr[2][NW];
    __shared__ uint32_t last;
    const int tid = threadIdx.x, col = tid % CB, g = tid / CB;
    const int EB = gridDim.x, e = blockIdx.x * CB + col;
    __shared__ int sn[kSeqLds], so[2 * kSeqLds];
    Seqs all;
    for (int s = blockIdx.y; s < S; s += gridDim.y) {
        const int ns = seq_n(n, s, J);
        int lo, hi, c = 0;
        const bool mine = seq_bounds(off, s, T, lo, hi);
        if (tid < CB && e < E) {
            int h[kMaxParts];
#pragma unroll
            for (int j = 0; j < kMaxParts; j++) h[j] = cnt[((size_t)s * J + min(j, J - 1)) * E + e];
#pragma unroll
            for (int j = 0; j < kMaxParts; j++) c += j < J ? h[j] : 0;
        }
        if (s == (int)blockIdx.y) all = bal_totals<NT>(n, off, T, 0, S, J, sn, so);
        const bool any = all.fine && mine && hi > lo;
        const int r0 = any ? lo / TB + s : 0, r1 = any ? (hi - 1) / TB + s + 1 : 0;
        float a = 0.0f;
        if (e < E)
#pragma unroll 4
            for (int r = r0 + g; r < r1; r += RG) a += psum[(size_t)r * E + e];
        float z = 0.0f;  // this sequence's sum of lse^2, by the first column block
        if (blockIdx.x == 0)
            for (int r = r0 + tid; r < r1; r += NT) z += zsum[r];
        red[g][col] = a;
        __syncthreads();
#pragma unroll
        for (int h = RG / 2; h >= 1; h >>= 1) {
            if (g < h) red[g][col] += red[g + h][col];
            __syncthreads();
        }
        float v = 0.0f;
        if (tid < CB && e < E) {
            float p = ns > 0 ? red[0][col] / (float)ns : 0.0f;
            if (!all.fine) p = __builtin_nanf("");
            if (probs) probs[(size_t)s * E + e] = p;
            if (counts) counts[(size_t)s * E + e] = all.fine ? c : -1;
            v = (float)c * p;
        }
        v = wave_sum(v);
        z = wave_sum(z);
        if ((tid & 63) == 0) {
            wr[0][tid >> 6] = v;
            wr[1][tid >> 6] = z;
        }
        __syncthreads();
        if (tid == 0) {
            v = z = 0.0f;
            for (int i = 0; i < NW; i++) {
                v += wr[0][i];
                z += wr[1][i];
            }
            if (ns > 0) v *= (float)E / ((float)all.live * (float)k * (float)ns);
            __hip_atomic_store(&q[(size_t)s * (EB + 1) + blockIdx.x], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (blockIdx.x == 0)
                __hip_atomic_store(&q[(size_t)s * (EB + 1) + EB], z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        if constexpr (CB == kNarrow) break;  // a workgroup for each of the few sequences
        // (wr is written again only behind the next sequence's barriers)
    }
    const int total = all.total;
    const bool fine = all.fine;
    // Thread 0 made this workgroup's stores of q itself, with
    // device-coherent stores: it waits for them, then takes the ticket. (A
    // release fence would write back the XCD's whole L2, here full of the
    // gradient just written: 65 us against 7 at 32768 x 512 in 37 sequences.)
    if (tid == 0) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u ==
               (uint32_t)EB * gridDim.y;
    }
    __syncthreads();
    if (!last) return;
    float bal = 0.0f, z = 0.0f;
    const size_t cells = (size_t)S * (EB + 1);
    for (size_t i = tid; i < cells; i += NT) {
        const float x = __hip_atomic_load(&q[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (i % (EB + 1) == (size_t)EB) z += x; else bal += x;
    }
    bal = wave_sum(bal);
    z = wave_sum(z);
    if ((tid & 63) == 0) {
        wr[0][tid >> 6] = bal;
        wr[1][tid >> 6] = z;
    }
    __syncthreads();
    if (tid == 0) {
        bal = z = 0.0f;
        for (int i = 0; i < NW; i++) {
            bal += wr[0][i];
            z += wr[1][i];
        }
        z = total > 0 ? z / (float)total : 0.0f;
        if (!fine) bal = z = __builtin_nanf("");
        // a term with a zero coefficient does not enter (its value may be infinite)
        loss[0] = (cb != 0.0f ? cb * bal : 0.0f) + (cz != 0.0f ? cz * z : 0.0f);
        if (!fine) loss[0] = __builtin_nanf("");
        loss[1] = bal;
        loss[2] = z;
    }
}

}  // namespace

size_t balance_ws_bytes(int T, int E, int S) { return bal_ws(T, E, S).total; }

hipError_t launch_balance(int E, int k, const float* logits, int T, const int32_t* idx, const uint8_t* mask,
                          const int32_t* seq_off, int S, float cb, float cz, const float* dloss, float* loss,
                          int32_t* counts, float* probs, float* dlogits, void* ws, hipStream_t s) {
    const BalWs b = bal_ws(T, E, S);
    const bool self = S == 1 && T > 0 && (int64_t)T * k <= kSelfCount;
    char* base = reinterpret_cast<char*>(ws);
    int32_t* cnt = reinterpret_cast<int32_t*>(base + b.cnt);
    int32_t* n = reinterpret_cast<int32_t*>(base + b.n);
    uint32_t* ticket = reinterpret_cast<uint32_t*>(base + b.ticket);
    float* psum = reinterpret_cast<float*>(base + b.psum);
    float* zsum = reinterpret_cast<float*>(base + b.zsum);
    float* q = reinterpret_cast<float*>(base + b.q);
    const int J = self ? 1 : b.JM;  // parts of each sequence in cnt and n
    hipError_t r;
    if (!self) {
        int32_t* pc = b.J > b.JM ? reinterpret_cast<int32_t*>(base + b.part) : cnt;
        int32_t* pn = b.J > b.JM ? pc + (size_t)S * b.J * E : n;
        hipLaunchKernelGGL(k_bal_count, dim3(b.J, S), dim3(1024), 0, s, idx, mask, seq_off, T, E, k, b.J, pc, pn, ticket);
        if ((r = hipGetLastError()) != hipSuccess) return r;
        if (b.J > b.JM) {
            hipLaunchKernelGGL(k_bal_merge, dim3((E + 255) / 256, S), dim3(256), 0, s, pc, pn, E, b.J, cnt, n);
            if ((r = hipGetLastError()) != hipSuccess) return r;
        }
    }
    if (b.chunks > 0) {
        const bool vec = E % 4 == 0;
#define BM(NV, VEC, SELF)                                                                                              hipLaunchKernelGGL((k_bal_main<NV, VEC, SELF>), dim3(b.chunks), dim3(256), 0, s, logits, mask, seq_off, T, E, k, S,                        b.TB, idx, J, cnt, n, ticket, cb, cz, dloss, dlogits, psum, zsum)
#define BMV(NV)     if (vec) { if (self) BM(NV, true, true); else BM(NV, true, false); } else { if (self) BM(NV, false, true); else BM(NV, false, false); }
        if (E <= 256) {
            BMV(4)
        } else if (E <= 512) {
            BMV(8)
        } else {
            BMV(16)
        }
#undef BMV
#undef BM
        if ((r = hipGetLastError()) != hipSuccess) return r;
    }
#define BR(CB)                                                                                                         \
    hipLaunchKernelGGL((k_bal_reduce<CB>), dim3((E + CB - 1) / CB, rows), dim3(1024), 0, s, seq_off, T, E, k, S, b.TB, J, cnt, \
                       n, cb, cz, psum, zsum, q, ticket, loss, counts, probs)
    const int most = kReduceGroups / ((E + kWide - 1) / kWide), rows = S <= kFewSeqs || S < most ? S : most;
    if (S <= kFewSeqs) BR(kNarrow); else BR(kWide);
#undef BR
    return hipGetLastError();
}

}  // namespace moe

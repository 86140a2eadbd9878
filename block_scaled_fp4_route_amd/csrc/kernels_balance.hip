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

constexpr int kBadSeq = -1;  // n_s of a sequence with a bad offset or a bad expert index

// Workspace regions (all 256-byte aligned).
struct BalWs {
    int J;           // parts per sequence of the counting launch
    int TB;          // tokens per chunk of the main launch
    int chunks;
    size_t part, cnt, n, ticket, psum, zsum, q, total;
};

BalWs bal_ws(int T, int E, int S) {
    BalWs b;
    // about 512 tokens per counting workgroup, 64 parts at most
    const int64_t per = ((int64_t)T + S - 1) / S;
    b.J = (int)((per + 511) / 512);
    b.J = b.J < 1 ? 1 : (b.J > 64 ? 64 : b.J);
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
    b.part = take(b.J > 1 ? (size_t)S * b.J * (row + 4) : 0);
    b.cnt = take((size_t)S * row);
    b.n = take((size_t)S * 4);
    b.ticket = take(4);
    b.psum = take(((size_t)b.chunks + S) * row);
    b.zsum = take(((size_t)b.chunks + S) * 4);
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

// grid (J, S), 256 threads: counts of the tokens of part j of sequence s.
__global__ __launch_bounds__(256) void k_bal_count(const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
                                                   const int32_t* __restrict__ off, int T, int E, int k, int J,
                                                   int32_t* __restrict__ cnt, int32_t* __restrict__ n,
                                                   uint32_t* __restrict__ ticket) {
    __shared__ int hist[kMaxE];
    __shared__ int tot[2];
    const int j = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
    for (int e = tid; e < E; e += 256) hist[e] = 0;
    if (tid < 2) tot[tid] = 0;
    if (tid == 0 && j == 0 && s == 0) *ticket = 0;
    __syncthreads();
    int lo, hi;
    const bool fine = seq_bounds(off, s, T, lo, hi);
    int mine = 0, bad = fine ? 0 : 1;
    if (fine) {
        const int per = (hi - lo + J - 1) / J;
        const int a = (int)min((int64_t)hi, lo + (int64_t)j * per), b = (int)min((int64_t)hi, (int64_t)a + per);
        for (int t = a + tid; t < b; t += 256) {
            if (mask && !mask[t]) continue;
            mine++;
            const int32_t* it = idx + (size_t)t * k;
            for (int i = 0; i < k; i++) {
                const int e = it[i];
                if ((unsigned)e < (unsigned)E)
                    atomicAdd(&hist[e], 1);
                else
                    bad = 1;
            }
        }
    }
    if (mine) atomicAdd(&tot[0], mine);
    if (bad) atomicOr(&tot[1], 1);
    __syncthreads();
    const size_t p = (size_t)s * J + j;
    for (int e = tid; e < E; e += 256) cnt[p * E + e] = hist[e];
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

// Live sequences and counted tokens over all S (every thread of a workgroup
// of NT threads gets them); false if any sequence is bad.
template <int NT>
__device__ __forceinline__ bool bal_totals(const int32_t* __restrict__ n, int S, int& live, int& total) {
    if (S == 1) {
        const int v = n[0];
        live = v > 0;
        total = v;
        return v >= 0;
    }
    __shared__ int acc[3];
    if (threadIdx.x < 3) acc[threadIdx.x] = 0;
    __syncthreads();
    int l = 0, t = 0, b = 0;
    for (int s = threadIdx.x; s < S; s += NT) {
        const int v = n[s];
        l += v > 0;
        t += max(v, 0);
        b |= v < 0;
    }
    if (l) {
        atomicAdd(&acc[0], l);
        atomicAdd(&acc[1], t);
    }
    if (b) atomicOr(&acc[2], 1);
    __syncthreads();
    live = acc[0];
    total = acc[1];
    return acc[2] == 0;
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
// Each wave takes every fourth token of a piece, a lane 64 NV / 64 columns.
template <int NV, bool VEC>
__global__ __launch_bounds__(256) void k_bal_main(const float* __restrict__ logits, const uint8_t* __restrict__ mask,
                                                  const int32_t* __restrict__ off, int T, int E, int k, int S, int TB,
                                                  const int32_t* __restrict__ cnt, const int32_t* __restrict__ n,
                                                  float cb, float cz, const float* __restrict__ dloss,
                                                  float* __restrict__ dlogits, float* __restrict__ psum,
                                                  float* __restrict__ zsum) {
    __shared__ float red[4][64 * NV];
    __shared__ float zred[4];
    const int lane = threadIdx.x & 63, wave = wave_id(), c = blockIdx.x;
    const int t0 = c * TB, t1 = min(T, t0 + TB);
    int live, total;
    const bool fine = bal_totals<256>(n, S, live, total);
    if (!fine) {
        if (dlogits) {
            float q[NV];
#pragma unroll
            for (int i = 0; i < NV; i++) q[i] = __builtin_nanf("");
            for (int t = t0 + wave; t < t1; t += 4) row_store<NV, VEC>(dlogits + (size_t)t * E, E, lane, q);
        }
        return;
    }
    const float up = dloss ? *dloss : 1.0f;
    float zero[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) zero[i] = 0.0f;
    // the first sequence that ends behind t0 (the offsets do not decrease: fine)
    int s = 0;
    if (off) {
        int lo = 0, hi = S;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (off[mid + 1] > t0) hi = mid; else lo = mid + 1;
        }
        s = lo;
    }
    int t = t0;
    while (t < t1) {
        const int a = s < S ? max(t, min(t1, off ? off[s] : 0)) : t1;
        const int b = s < S ? max(a, min(t1, off ? off[s + 1] : T)) : t1;
        if (dlogits)
            for (int u = t + wave; u < a; u += 4) row_store<NV, VEC>(dlogits + (size_t)u * E, E, lane, zero);
        if (a < b) {
            const int ns = n[s];
            const float cf = ns > 0 ? cb * (float)E / ((float)live * (float)k * (float)ns * (float)ns) : 0.0f;
            const float zf = cz != 0.0f && total > 0 ? cz * 2.0f / (float)total : 0.0f;
            float co[NV], ps[NV], v[NV];
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int e = bal_col<VEC>(lane, i);
                co[i] = e < E ? cf * (float)cnt[(size_t)s * E + e] : 0.0f;
                ps[i] = 0.0f;
            }
            float zs = 0.0f;
            for (int u = a + wave; u < b; u += 4) {
                if (mask && !mask[u]) {
                    if (dlogits) row_store<NV, VEC>(dlogits + (size_t)u * E, E, lane, zero);
                    continue;
                }
                row_load<NV, VEC>(logits + (size_t)u * E, E, lane, -INFINITY, v);
                float m = v[0];
#pragma unroll
                for (int i = 1; i < NV; i++) m = fmaxf(m, v[i]);
                m = wave_max(m);
                if (m == -INFINITY) m = 0.0f;  // nothing finite: every e^v is 0 (or NaN)
                float z = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; i++) {
                    v[i] = expf(v[i] - m);
                    z += v[i];
                }
                z = wave_sum(z);
                const float inv = z == 0.0f ? 0.0f : 1.0f / z;
                const float lse = z == 0.0f ? 0.0f : m + logf(z);
                zs += lse * lse;
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; i++) {
                    v[i] *= inv;
                    ps[i] += v[i];
                    dot = fmaf(co[i], v[i], dot);
                }
                if (dlogits) {
                    dot = wave_sum(dot);
                    const float sh = (zf != 0.0f ? zf * lse : 0.0f) - dot;
#pragma unroll
                    for (int i = 0; i < NV; i++) v[i] = up * (v[i] * (co[i] + sh));
                    row_store<NV, VEC>(dlogits + (size_t)u * E, E, lane, v);
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

// grid (ceil(E / 16), S), 1024 threads: 16 columns x 64 row groups over the
// pieces of sequence s; the last workgroup to finish adds the sequences up.
__global__ __launch_bounds__(1024) void k_bal_reduce(const int32_t* __restrict__ off, int T, int E, int k, int S,
                                                     int TB, const int32_t* __restrict__ cnt,
                                                     const int32_t* __restrict__ n, float cb, float cz,
                                                     const float* __restrict__ psum, const float* __restrict__ zsum,
                                                     float* __restrict__ q, uint32_t* __restrict__ ticket,
                                                     float* __restrict__ loss, int32_t* __restrict__ counts,
                                                     float* __restrict__ probs) {
    __shared__ float red[64][17];
    __shared__ float zr[16];
    __shared__ uint32_t last;
    const int tid = threadIdx.x, col = tid & 15, g = tid >> 4, s = blockIdx.y;
    const int EB = gridDim.x, e = blockIdx.x * 16 + col;
    int live, total;
    const bool fine = bal_totals<1024>(n, S, live, total);
    int lo = 0, hi = 0;
    if (fine) seq_bounds(off, s, T, lo, hi);
    const int ns = n[s];
    const bool any = fine && hi > lo;
    const int r0 = any ? lo / TB + s : 0, r1 = any ? (hi - 1) / TB + s + 1 : 0;
    float a = 0.0f;
    if (e < E)
#pragma unroll 4
        for (int r = r0 + g; r < r1; r += 64) a += psum[(size_t)r * E + e];
    red[g][col] = a;
    __syncthreads();
#pragma unroll
    for (int h = 32; h >= 1; h >>= 1) {
        if (g < h) red[g][col] += red[g + h][col];
        __syncthreads();
    }
    if (tid < 16) {
        float p = ns > 0 ? red[0][col] / (float)ns : 0.0f;
        if (!fine) p = __builtin_nanf("");
        const int c = e < E ? cnt[(size_t)s * E + e] : 0;
        if (e < E) {
            if (probs) probs[(size_t)s * E + e] = p;
            if (counts) counts[(size_t)s * E + e] = fine ? c : -1;
        }
        float v = e < E ? (float)c * p : 0.0f;
        v = row16_sum(v);
        if (ns > 0) v *= (float)E / ((float)live * (float)k * (float)ns);
        if (col == 0)
            __hip_atomic_store(&q[(size_t)s * (EB + 1) + blockIdx.x], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (blockIdx.x == 0) {  // this sequence's sum of lse^2
        float z = 0.0f;
        for (int r = r0 + tid; r < r1; r += 1024) z += zsum[r];
        z = wave_sum(z);
        if ((tid & 63) == 0) zr[tid >> 6] = z;
        __syncthreads();
        if (tid == 0) {
            z = 0.0f;
            for (int i = 0; i < 16; i++) z += zr[i];
            __hip_atomic_store(&q[(size_t)s * (EB + 1) + EB], z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    // the workgroup's stores are out before its ticket is taken
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1u ==
               (uint32_t)EB * (uint32_t)S;
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
    float bal = 0.0f, z = 0.0f;
    const size_t cells = (size_t)S * (EB + 1);
    for (size_t i = tid; i < cells; i += 1024) {
        const float v = __hip_atomic_load(&q[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (i % (EB + 1) == (size_t)EB) z += v; else bal += v;
    }
    bal = wave_sum(bal);
    z = wave_sum(z);
    if ((tid & 63) == 0) {
        red[tid >> 6][0] = bal;
        red[tid >> 6][1] = z;
    }
    __syncthreads();
    if (tid == 0) {
        bal = z = 0.0f;
        for (int i = 0; i < 16; i++) {
            bal += red[i][0];
            z += red[i][1];
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

template <int NV, bool VEC>
void bal_main(const float* logits, const uint8_t* mask, const int32_t* off, int T, int E, int k, int S, const BalWs& b,
              const int32_t* cnt, const int32_t* n, float cb, float cz, const float* dloss, float* dlogits,
              float* psum, float* zsum, hipStream_t s) {
    hipLaunchKernelGGL((k_bal_main<NV, VEC>), dim3(b.chunks), dim3(256), 0, s, logits, mask, off, T, E, k, S, b.TB,
                       cnt, n, cb, cz, dloss, dlogits, psum, zsum);
}

}  // namespace

size_t balance_ws_bytes(int T, int E, int S) { return bal_ws(T, E, S).total; }

hipError_t launch_balance(int E, int k, const float* logits, int T, const int32_t* idx, const uint8_t* mask,
                          const int32_t* seq_off, int S, float cb, float cz, const float* dloss, float* loss,
                          int32_t* counts, float* probs, float* dlogits, void* ws, hipStream_t s) {
    const BalWs b = bal_ws(T, E, S);
    char* base = reinterpret_cast<char*>(ws);
    int32_t* cnt = reinterpret_cast<int32_t*>(base + b.cnt);
    int32_t* n = reinterpret_cast<int32_t*>(base + b.n);
    int32_t* pc = b.J > 1 ? reinterpret_cast<int32_t*>(base + b.part) : cnt;
    int32_t* pn = b.J > 1 ? pc + (size_t)S * b.J * E : n;
    uint32_t* ticket = reinterpret_cast<uint32_t*>(base + b.ticket);
    float* psum = reinterpret_cast<float*>(base + b.psum);
    float* zsum = reinterpret_cast<float*>(base + b.zsum);
    float* q = reinterpret_cast<float*>(base + b.q);
    hipLaunchKernelGGL(k_bal_count, dim3(b.J, S), dim3(256), 0, s, idx, mask, seq_off, T, E, k, b.J, pc, pn, ticket);
    hipError_t r = hipGetLastError();
    if (r != hipSuccess) return r;
    if (b.J > 1) {
        hipLaunchKernelGGL(k_bal_merge, dim3((E + 255) / 256, S), dim3(256), 0, s, pc, pn, E, b.J, cnt, n);
        if ((r = hipGetLastError()) != hipSuccess) return r;
    }
    if (b.chunks > 0) {
        const bool vec = E % 4 == 0;
#define BM(NV, VEC) \
    bal_main<NV, VEC>(logits, mask, seq_off, T, E, k, S, b, cnt, n, cb, cz, dloss, dlogits, psum, zsum, s)
        if (E <= 256) {
            if (vec) BM(4, true); else BM(4, false);
        } else if (E <= 512) {
            if (vec) BM(8, true); else BM(8, false);
        } else {
            if (vec) BM(16, true); else BM(16, false);
        }
#undef BM
        if ((r = hipGetLastError()) != hipSuccess) return r;
    }
    hipLaunchKernelGGL(k_bal_reduce, dim3((E + 15) / 16, S), dim3(1024), 0, s, seq_off, T, E, k, S, b.TB, cnt, n, cb,
                       cz, psum, zsum, q, ticket, loss, counts, probs);
    return hipGetLastError();
}

}  // namespace moe

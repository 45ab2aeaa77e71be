// Losses that keep a router's experts in use, and the gradient of its logits.
//
// For a sequence s of T tokens, c[s, e] the pairs (token, pick) of expert e, and
// p[t, e] the token's normalised scores -- softmax(l), or sigma(l) over their sum
// -- with k picks a token and E experts:
//   balance[s] = E sum_e (c[s, e] / (k T)) (sum_t p[t, e] / T)
//              = E / (k T^2) sum_t q[t],  q[t] = sum_e c[s, e] p[t, e]
//   z[s] = 1 / T sum_t lse(l[t])^2,  lse the logarithm of the sum of exponentials
// The second form of balance needs the counts first and then one number of each
// token, so that no sums over tokens are kept per expert.  The counts come from the
// ids alone, 4 k bytes a token; the logits are read once.
// Gradients, with G[e] = dbalance[s] E / (k T^2) (c[s, e] - k T / E) -- the constant
// changes nothing, the p of a token add up to one, and takes out of the difference
// below what all experts have in common --
//   softmax: p (G - sum p G)     sigmoid: p (1 - sigma) (G - sum p G)
//   z: dz[s] / T 2 lse softmax(l)
// and of the routing weights w[t, j] of the picks, given dw:
//   softmax over the picks: w_j (dw_j - sum w dw)
//   sigmoid, renormalised: with u = sigma_j / sum sigma, scale u_j (1 - sigma_j) (dw_j - sum u dw)
//   sigmoid alone: scale sigma_j (1 - sigma_j) dw_j
// Picks that name the same expert add up, in their order.  A token whose logits are
// all -inf has p = 0 and no part in z.
//
// A token belongs to G lanes of a warp, which hold its E logits in registers.
// Deterministic: integer counts, and sums in the order of the tokens of a chunk,
// then of the chunks; whichever block finishes a sequence last adds its chunks up.
//
// 16384 tokens of 256 experts, 4 sequences, sigmoid: losses 14.3 us (counts some 5 of
// it, the last sequence's sum 2), gradient 13.5 us for 34 MB, logits in L2.  It is
// bound by its chains of loads, exponentials and sums over lanes (a token's lanes execute
// some 280 and 600 instructions), which the warps that fit (42 and 31% of an SM's)
// hide in part: 53 and 61% of the issue slots are taken, 14% of DRAM's rate.  So are fewer
// tokens, with the hand-over of counts between two kernels: 333 tokens of 8 experts 5.7 and
// 3.4 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ops.h"
#include "pairs.cuh"
#include "sm100.cuh"
#include "tmap.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxChunk = 128;   // tokens of a block
constexpr int kMinChunk = 8;     // ... at least: what one round of 32-lane groups takes
constexpr int kCountThreads = 512;  // 131072 ids in 4 sequences: losses 15.7 us, with 256 16.8
constexpr int kIdsAhead = 8;     // ids that a counting thread has on their way
constexpr int kPartsAhead = 2;   // chunks' sums that a lane has on their way
constexpr int kOffsShared = 512; // sequences whose offsets a block keeps in shared memory

// The tokens of sequence s, within [0, m] whatever the offsets hold.
__device__ __forceinline__ void span(const RouterArgs& a, int s, int& t0, int& t1) {
    t0 = 0;
    t1 = a.m;
    if (a.off) {
        t0 = min(max(a.off[s], 0), a.m);
        t1 = min(max(a.off[s + 1], t0), a.m);
    }
}

// Counts of a sequence's pairs: a cluster per sequence (or a block alone, where
// sequences are many), a histogram in each block's shared memory, added up through
// distributed shared memory.  Nothing has to be zeroed before and no atomics reach
// global memory.  It also opens the losses' tickets.
template <int cluster>
__global__ void __launch_bounds__(kCountThreads) count_pairs(const RouterArgs a) {
    __shared__ int hist[kMaxExperts];
    const int s = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    for (int e = threadIdx.x; e < a.E; e += kCountThreads) hist[e] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    int t0, t1;
    span(a, s, t0, t1);
    const int64_t end = (int64_t)t1 * a.k, step = (int64_t)cluster * kCountThreads;
    int64_t p = (int64_t)t0 * a.k + rank * kCountThreads + threadIdx.x;
    for (; p < end; p += kIdsAhead * step) {
        int id[kIdsAhead];
#pragma unroll
        for (int i = 0; i < kIdsAhead; ++i) id[i] = p + i * step < end ? a.ids[p + i * step] : -1;
#pragma unroll
        for (int i = 0; i < kIdsAhead; ++i)
            if ((unsigned)id[i] < (unsigned)a.E) atomicAdd(&hist[id[i]], 1);
    }
    if (rank == 0 && threadIdx.x == 0) {
        a.ticket[s] = 0;
        if (t0 == t1) a.balance[s] = a.z[s] = 0.f;
    }
    __syncthreads();
    if (cluster > 1) sm100::cluster_sync();
    const uint32_t h = sm100::smem_u32(hist);
    for (int e = rank * kCountThreads + threadIdx.x; e < a.E; e += cluster * kCountThreads) {
        int n = 0;
        if (cluster > 1) {
            int v[cluster];
#pragma unroll
            for (int c = 0; c < cluster; ++c)
                asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v[c]) : "r"(sm100::mapa(h + 4 * e, c)) : "memory");
#pragma unroll
            for (int c = 0; c < cluster; ++c) n += v[c];
        } else {
            n = hist[e];
        }
        a.counts[(size_t)s * a.E + e] = n;
    }
    if (cluster > 1) sm100::cluster_sync();  // the others may still read this block's histogram
}

// Sums and maxima over the G lanes of a token, of several values at once.
template <int G, int M>
__device__ __forceinline__ void group_sum(float (&v)[M]) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < M; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}
template <int G, int M>
__device__ __forceinline__ void group_max(float (&v)[M]) {
    if constexpr (G == 32) {
#pragma unroll
        for (int k = 0; k < M; ++k) asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v[k]));
    } else {
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < M; ++k) v[k] = fmaxf(v[k], __shfl_xor_sync(0xffffffffu, v[k], o));
    }
}

// exp(v) of v <= 0, as 2^(v log2 e): off by 2^-22 and by the product's rounding, |v| 2^-24,
// of a number that counts for exp(v) (below 2^-126 for nothing).
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float exp_neg(float v) { return exp2_approx(v * kLog2e); }
// 1 / v of a normal v up to 2^126, within 2^-23; 0 of 0.
__device__ __forceinline__ float inverse(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return v == 0.f ? 0.f : r;
}

__device__ __forceinline__ float min_or_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// ... of a v that is not 0.
__device__ __forceinline__ float inverse_of_some(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Over the N values of a lane, two an instruction where there are two.
template <int N>
__device__ __forceinline__ Pair two(const float (&v)[N], int n) { return Pair{v[n], v[n + 1]}; }
template <int N>
__device__ __forceinline__ void put(float (&v)[N], int n, Pair p) {
    v[n] = p.x;
    v[n + 1] = p.y;
}
template <int N>
__device__ __forceinline__ float dot(const float (&x)[N], const float (&y)[N]) {
    if constexpr (N == 1) {
        return x[0] * y[0];
    } else {
        Pair s{0.f, 0.f};
#pragma unroll
        for (int n = 0; n < N; n += 2) s = fma2(two(x, n), two(y, n), s);
        return s.x + s.y;
    }
}
template <int N>
__device__ __forceinline__ float total(const float (&x)[N]) {
    if constexpr (N == 1) {
        return x[0];
    } else {
        Pair s = two(x, 0);
#pragma unroll
        for (int n = 2; n < N; n += 2) s = add2(s, two(x, n));
        return s.x + s.y;
    }
}
// e = exp(l - at), l <= at; their sum
template <int N>
__device__ __forceinline__ float exps(const float (&l)[N], float at, float (&e)[N]) {
    if constexpr (N == 1) e[0] = exp_neg(l[0] - at);
#pragma unroll
    for (int n = 0; n + 1 < N; n += 2) {
        const Pair v = mul2(add2(two(l, n), Pair{-at, -at}), Pair{kLog2e, kLog2e});
        e[n] = exp2_approx(v.x);
        e[n + 1] = exp2_approx(v.y);
    }
    return total(e);
}

// sigma(l) / exp(shift) and 1 - sigma(l), neither by a difference, shift = min(0, the largest l): sums of the first do not
// underflow where all l are far below zero.  low: shift < 0, for any lane of the warp.
__device__ __forceinline__ float shifted_logistic(float l, float shift, bool low, float& rest) {
    const float e = exp_neg(-fabsf(l)), big = inverse_of_some(1.0f + e);
    rest = l >= 0.f ? e * big : big;
    if (low) return (l >= 0.f ? 1.0f : exp_neg(l - shift)) * big;
    return l >= 0.f ? big : e * big;
}

// A token's values over its lanes: value n * VEC + j of lane i is that of expert
// (i + G n) VEC + j.
template <int G, int VEC, int NV>
struct Row {
    float v[NV * VEC];
    // PAST_L1: global memory, read before this kernel waits for the one ahead of it
    template <bool PAST_L1 = false>
    __device__ __forceinline__ void load(const float* row, int i, int E, bool live, float none) {
        const auto get = [](const auto* p) { return PAST_L1 ? __ldcg(p) : *p; };
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int e = (i + G * n) * VEC;
            if (VEC == 4) {
                const float4 q = live && e < E ? get(reinterpret_cast<const float4*>(row + e)) : make_float4(none, none, none, none);
                v[n * VEC] = q.x;
                v[n * VEC + VEC / 4] = q.y;
                v[n * VEC + VEC / 2] = q.z;
                v[n * VEC + VEC - 1] = q.w;
            } else {
                v[n * VEC] = live && e < E ? get(row + e) : none;
            }
        }
    }
    __device__ __forceinline__ void load_counts(const int32_t* row, int i, int E, bool live) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int e = (i + G * n) * VEC;
            if (VEC == 4) {
                const int4 q = live && e < E ? *reinterpret_cast<const int4*>(row + e) : make_int4(0, 0, 0, 0);
                v[n * VEC] = (float)q.x;
                v[n * VEC + VEC / 4] = (float)q.y;
                v[n * VEC + VEC / 2] = (float)q.z;
                v[n * VEC + VEC - 1] = (float)q.w;
            } else {
                v[n * VEC] = live && e < E ? (float)row[e] : 0.f;
            }
        }
    }
    __device__ __forceinline__ void store(float* row, int i, int E) const {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int e = (i + G * n) * VEC;
            if (e >= E) continue;
            if (VEC == 4)
                *reinterpret_cast<float4*>(row + e) =
                    make_float4(v[n * VEC], v[n * VEC + VEC / 4], v[n * VEC + VEC / 2], v[n * VEC + VEC - 1]);
            else
                row[e] = v[n * VEC];
        }
    }
};

// The scores of a token's logits, and their complements (of scores that are not 0; p times them is what is asked for).
template <int N>
__device__ __forceinline__ void scores(const float (&l)[N], float shift, bool low, float (&p)[N], float (&rest)[N]) {
    if (low || N == 1) {
#pragma unroll
        for (int n = 0; n < N; ++n) p[n] = shifted_logistic(l[n], shift, low, rest[n]);
        return;
    }
    // 1 / (1 + e), e = exp(-l) up to 2^127.97: from 2^126 on, what counts for 0 (and -inf), the inverse is 0
#pragma unroll
    for (int n = 0; n + 1 < N; n += 2) {
        const Pair v = mul2(two(l, n), Pair{-kLog2e, -kLog2e});
        const Pair e{exp2_approx(min_or_nan(v.x, 127.97f)), exp2_approx(min_or_nan(v.y, 127.97f))};
        const Pair b = add2(e, Pair{1.0f, 1.0f});
        const Pair s{inverse_of_some(b.x), inverse_of_some(b.y)};
        put(p, n, s);
        put(rest, n, mul2(e, s));
    }
}

// The sequence of each token of the block's chunk, -1 outside of all.
struct Chunk {
    int seq[kMaxChunk];
    int off[kOffsShared + 1];
};
__device__ __forceinline__ void find_sequences(const RouterArgs& a, int first, Chunk& ch) {
    const bool kept = a.off && a.S <= kOffsShared;
    if (kept)
        for (int i = threadIdx.x; i <= a.S; i += kThreads) ch.off[i] = __ldcg(a.off + i);
    __syncthreads();
    if ((int)threadIdx.x < a.chunk) {
        const int t = first + threadIdx.x;
        int s = t < a.m ? 0 : -1;
        if (a.off && t < a.m) {
            const auto off = [&](int i) { return kept ? ch.off[i] : __ldcg(a.off + i); };
            int lo = 0, hi = a.S;  // the first s whose end is past t, S: none
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (off(mid + 1) > t)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            s = lo < a.S && off(lo) <= t ? lo : -1;
        }
        ch.seq[threadIdx.x] = s;
    }
    __syncthreads();
}

// The losses.  A block takes a chunk of tokens; then a warp for each sequence that
// the chunk holds tokens of adds up theirs, and the warp that is the sequence's last
// adds up the chunks.  Chunk c and sequence s meet at slot c + s, which no other
// meeting has: along them c or s rises from one to the next and neither falls.
template <bool SIGMOID, int G, int VEC, int NV>
__global__ void __launch_bounds__(kThreads) balance_loss(const RouterArgs a) {
    __shared__ Chunk ch;
    __shared__ float2 each[kMaxChunk];
    const int first = blockIdx.x * a.chunk, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = threadIdx.x % G, group = threadIdx.x / G;
    constexpr int GROUPS = kThreads / G;
    constexpr bool kAhead = NV * VEC <= 8;  // registers for the next token's logits
    auto load = [&](int r) {
        Row<G, VEC, NV> l;
        const int j = r + group;
        l.template load<true>(a.logits + (size_t)(first + j) * a.E, i, a.E, j < a.chunk && first + j < a.m, -INFINITY);
        return l;
    };
    // logits and offsets are older than the counting kernel, whose counts alone are waited for
    Row<G, VEC, NV> next;
    if (kAhead) next = load(0);
    find_sequences(a, first, ch);
    Row<G, VEC, NV> c;  // counts of sequence `of`
    int of = -1;
    const auto load_counts = [&](int s) {
        c.load_counts(a.counts + (size_t)max(s, 0) * a.E, i, a.E, s >= 0);
        of = s;
    };
    for (int r = 0; r < a.chunk; r += GROUPS) {  // warps stay together
        const int j = r + group, s = j < a.chunk ? ch.seq[j] : -1;
        Row<G, VEC, NV> l;
        if (kAhead) {
            l = next;
            next = load(r + GROUPS);
        } else {
            l = load(r);
        }
        if (s != of && r > 0) load_counts(s);
        float top[1] = {-INFINITY};
#pragma unroll
        for (int n = 0; n < NV * VEC; ++n) top[0] = fmaxf(top[0], l.v[n]);
        group_max<G>(top);
        const float at = top[0] == -INFINITY ? 0.f : top[0], shift = fminf(at, 0.f);
        const bool low = SIGMOID && __any_sync(0xffffffffu, shift < 0.f);
        float sum[3] = {};  // of exp(l - at), of the scores, of the scores times their counts
        Row<G, VEC, NV> p, rest;
        sum[0] = exps(l.v, at, p.v);
        if (SIGMOID) {
            scores(l.v, shift, low, p.v, rest.v);
            sum[1] = total(p.v);
        }
        if (r == 0) {  // the first tokens' scores do without the counts
            pdl_wait();
            pdl_trigger();
            load_counts(s);
        }
        sum[2] = dot(p.v, c.v);
        group_sum<G>(sum);
        const float lse = at + logf(sum[0]);
        if (i == 0 && j < a.chunk)
            each[j] = s < 0 ? make_float2(0.f, 0.f)
                            : make_float2(sum[2] * inverse(SIGMOID ? sum[1] : sum[0]), sum[0] == 0.f ? 0.f : lse * lse);
    }
    __syncthreads();
    const int last = min(first + a.chunk, a.m);
    // the sequences of the chunk's first and last tokens that are in any
    int s0 = a.S, s1 = -1;
    for (int j = lane; j < last - first; j += 32) {
        const int s = ch.seq[j];
        if (s >= 0) {
            s0 = min(s0, s);
            s1 = max(s1, s);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s0 = min(s0, __shfl_xor_sync(0xffffffffu, s0, o));
        s1 = max(s1, __shfl_xor_sync(0xffffffffu, s1, o));
    }
    for (int s = s0 + warp; s <= s1; s += kThreads / 32) {
        int t0, t1;
        span(a, s, t0, t1);
        const int from = max(t0, first), to = min(t1, last);
        if (from >= to) continue;
        float q = 0.f, z = 0.f;
        for (int t = from + lane; t < to; t += 32) {
            q += each[t - first].x;
            z += each[t - first].y;
        }
        q = warp_sum(q);
        z = warp_sum(z);
        const int c0 = t0 / a.chunk, c1 = (t1 - 1) / a.chunk;
        int done = 0;
        if (lane == 0) {
            a.part[blockIdx.x + s] = make_float2(q, z);
            int before;  // after this block's sums, before the others' are read
            asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(a.ticket + s) : "memory");
            done = before == c1 - c0;
        }
        if (!__shfl_sync(0xffffffffu, done, 0)) continue;
        __syncwarp();  // the other lanes' reads come after lane 0's
        double qs = 0.0, zs = 0.0;
        for (int c = c0 + lane; c <= c1; c += 32 * kPartsAhead) {
            float2 v[kPartsAhead];
#pragma unroll
            for (int n = 0; n < kPartsAhead; ++n)
                v[n] = c + 32 * n <= c1 ? __ldcg(&a.part[c + 32 * n + s]) : make_float2(0.f, 0.f);
#pragma unroll
            for (int n = 0; n < kPartsAhead; ++n) {
                qs += (double)v[n].x;
                zs += (double)v[n].y;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            qs += __shfl_xor_sync(0xffffffffu, qs, o);
            zs += __shfl_xor_sync(0xffffffffu, zs, o);
        }
        if (lane == 0) {
            const double T = (double)(t1 - t0);
            a.balance[s] = (float)(qs * a.E / ((double)a.k * T * T));
            a.z[s] = (float)(zs / T);
        }
    }
}

// The gradient of the logits: of the routing weights, and of the losses for tokens
// of sequences.  Pick j of a token is lane j % G's, its number j / G there.
// Up to 64 experts (4 picks a lane) 4 to 92 bytes spill at the 80 registers that three
// blocks an SM leave.
template <bool SIGMOID, int G, int VEC, int NV>
__global__ void __launch_bounds__(kThreads, NV * VEC <= 8 ? 3 : 1) route_backward(const RouterArgs a) {
    constexpr int N = NV * VEC;
    __shared__ Chunk ch;
    extern __shared__ float4 row_mem[];  // [GROUPS, E], zero between tokens
    float* row_of = reinterpret_cast<float*>(row_mem);
    const int i = threadIdx.x % G, group = threadIdx.x / G;
    constexpr int GROUPS = kThreads / G;
    if (a.dtopk_w)
        for (int e = i; e < a.E; e += G) row_of[group * a.E + e] = 0.f;
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    const int first = blockIdx.x * a.chunk;
    const bool losses = a.dbalance || a.dz;
    if (losses) find_sequences(a, first, ch);
    constexpr int PICKS = G == 32 ? 1 : 4;  // k <= min(E, 32), and G < 32 only where E <= 4 G
    constexpr bool kAhead = NV * VEC <= 8;  // registers for the next token's logits
    struct Picks {
        int id[PICKS];
        float dk[PICKS];
    };
    auto load_picks = [&](int r) {
        Picks x;
        const int j = r + group, t = first + j;
#pragma unroll
        for (int n = 0; n < PICKS; ++n) {
            const int pick = n * G + i;
            const bool in = a.dtopk_w && j < a.chunk && t < a.m && pick < a.k;
            x.id[n] = in ? a.ids[(size_t)t * a.k + pick] : -1;
            x.dk[n] = in ? a.dtopk_w[(size_t)t * a.k + pick] : 0.f;
        }
        return x;
    };
    struct Token {
        Row<G, VEC, NV> l;
        int id[PICKS];
        float dk[PICKS], lk[PICKS];
    };
    auto load = [&](int r, const Picks& picks) {
        Token x;
        const int j = r + group, t = first + j;
        const float* row = a.logits + (size_t)t * a.E;
        if (losses) x.l.load(row, i, a.E, j < a.chunk && t < a.m, -INFINITY);
#pragma unroll
        for (int n = 0; n < PICKS; ++n) {
            x.id[n] = (unsigned)picks.id[n] < (unsigned)a.E ? picks.id[n] : -1;
            x.dk[n] = picks.dk[n];
            x.lk[n] = x.id[n] >= 0 ? row[x.id[n]] : -INFINITY;
        }
        return x;
    };
    // terms of sequence `of`: its counts less what an even share would be, factors of the two losses
    Row<G, VEC, NV> c;
    float db = 0.f, dz = 0.f;
    int of = -2;
    // the picks' logits are found through their ids: these are loaded a token earlier still
    Picks later = load_picks(0);
    Token next;
    if (kAhead) {
        next = load(0, later);
        later = load_picks(GROUPS);
    }
    for (int r = 0; r < a.chunk; r += GROUPS) {
        const int j = r + group, t = first + j;
        const bool live = j < a.chunk && t < a.m;
        const int s = losses && live ? ch.seq[j] : -1;
        Token x;
        if (kAhead) {
            x = next;
            next = load(r + GROUPS, later);
            later = load_picks(r + 2 * GROUPS);
        } else {
            x = load(r, later);
            later = load_picks(r + GROUPS);
        }
        if (losses && s != of) {
            int t0 = 0, t1 = 1;
            if (s >= 0) span(a, s, t0, t1);
            const float T = (float)max(t1 - t0, 1);
            dz = s >= 0 && a.dz ? a.dz[s] / T * 2.f : 0.f;
            db = 0.f;
            if (a.dbalance) {
                if (s >= 0) db = a.dbalance[s] * (float)a.E / ((float)a.k * T) / T;
                c.load_counts(a.counts + (size_t)max(s, 0) * a.E, i, a.E, s >= 0);
                const float even = (float)a.k * T / (float)a.E;
#pragma unroll
                for (int n = 0; n < NV * VEC; ++n) c.v[n] -= even;
            }
            of = s;
        }
        float top[2] = {-INFINITY, -INFINITY};  // of the row, of the picks
        if (losses) {
#pragma unroll
            for (int n = 0; n < NV * VEC; ++n) top[0] = fmaxf(top[0], x.l.v[n]);
        }
        if (a.dtopk_w) {
#pragma unroll
            for (int n = 0; n < PICKS; ++n) top[1] = fmaxf(top[1], x.lk[n]);
        }
        group_max<G>(top);
        const float at = top[0] == -INFINITY ? 0.f : top[0], shift = fminf(at, 0.f);
        const float pick_at = top[1] == -INFINITY ? 0.f : top[1], pick_shift = fminf(pick_at, 0.f);
        const bool low = SIGMOID && __any_sync(0xffffffffu, shift < 0.f || pick_shift < 0.f);
        // sums of: exp(l - at); the scores; the scores times c; the picks' scores; these times dw
        float sum[5] = {};
        Row<G, VEC, NV> e, p, rest;
        float wk[PICKS], rest_k[PICKS];
        if (losses) {
            if (!SIGMOID || a.dz) sum[0] = exps(x.l.v, at, e.v);
            if (a.dbalance) {
                if (SIGMOID) {
                    scores(x.l.v, shift, low, p.v, rest.v);
                    sum[1] = total(p.v);
                }
                sum[2] = SIGMOID ? dot(p.v, c.v) : dot(e.v, c.v);
            }
        }
        if (a.dtopk_w) {
#pragma unroll
            for (int n = 0; n < PICKS; ++n) {
                if (x.id[n] < 0) x.dk[n] = 0.f;
                wk[n] = SIGMOID ? shifted_logistic(x.lk[n], pick_shift, low, rest_k[n]) : exp_neg(x.lk[n] - pick_at);
                sum[3] += wk[n];
                sum[4] = fmaf(wk[n], x.dk[n], sum[4]);
            }
        }
        group_sum<G>(sum);
        Row<G, VEC, NV> d;
#pragma unroll
        for (int n = 0; n < NV * VEC; ++n) d.v[n] = 0.f;
        if (losses && s >= 0) {  // padding gets nothing, whatever its logits hold
            if (a.dz) {
                const float f = sum[0] == 0.f ? 0.f : dz * (at + logf(sum[0])) * inverse_of_some(sum[0]);
                if constexpr (N == 1) d.v[0] = f * e.v[0];
#pragma unroll
                for (int n = 0; n + 1 < N; n += 2) put(d.v, n, mul2(Pair{f, f}, two(e.v, n)));
            }
            if (a.dbalance) {
                const float inv = inverse(SIGMOID ? sum[1] : sum[0]), mean = sum[2] * inv, f = db * inv;
                if constexpr (N == 1) {
                    const float g = f * (SIGMOID ? p.v[0] : e.v[0]);
                    d.v[0] = fmaf(SIGMOID ? g * rest.v[0] : g, c.v[0] - mean, d.v[0]);
                }
#pragma unroll
                for (int n = 0; n + 1 < N; n += 2) {
                    Pair g = mul2(Pair{f, f}, SIGMOID ? two(p.v, n) : two(e.v, n));
                    if (SIGMOID) g = mul2(g, two(rest.v, n));
                    put(d.v, n, fma2(g, add2(two(c.v, n), Pair{-mean, -mean}), two(d.v, n)));
                }
            }
        }
        int id[PICKS];
        float dk[PICKS];
        if (a.dtopk_w) {
            const float inv = inverse(sum[3]), mean = sum[4] * inv;
#pragma unroll
            for (int n = 0; n < PICKS; ++n) {
                id[n] = x.id[n];
                const float w = wk[n] * inv;
                if (!SIGMOID)
                    dk[n] = w * (x.dk[n] - mean);
                else if (a.norm)
                    dk[n] = a.scale * rest_k[n] * w * (x.dk[n] - mean);
                else
                    dk[n] = a.scale * rest_k[n] * (wk[n] * exp_neg(pick_shift)) * x.dk[n];
            }
        }
        // The picks' gradients go to their experts' lanes through the group's row in shared memory,
        // where each first leaves its number: one that is not found there shares its expert.
        bool twice = false;
        float* own = row_of + group * a.E;
        if (a.dtopk_w) {
#pragma unroll
            for (int n = 0; n < PICKS; ++n)
                if (id[n] >= 0) own[id[n]] = __int_as_float(n * G + i);
            __syncwarp();
#pragma unroll
            for (int n = 0; n < PICKS; ++n) twice |= id[n] >= 0 && __float_as_int(own[id[n]]) != n * G + i;
            twice = __any_sync(0xffffffffu, twice);
#pragma unroll
            for (int n = 0; n < PICKS; ++n)
                if (id[n] >= 0) own[id[n]] = twice ? 0.f : dk[n];
            __syncwarp();
            if (!twice) {
                Row<G, VEC, NV> k;
                k.load(own, i, a.E, true, 0.f);
                if constexpr (N == 1) d.v[0] += k.v[0];
#pragma unroll
                for (int n = 0; n + 1 < N; n += 2) put(d.v, n, add2(two(d.v, n), two(k.v, n)));
                __syncwarp();
#pragma unroll
                for (int n = 0; n < PICKS; ++n)
                    if (id[n] >= 0) own[id[n]] = 0.f;
            }
            __syncwarp();
        }
        if (twice) {  // one after another, in their order
#pragma unroll
            for (int n = 0; n < PICKS; ++n) {
                for (int q = 0; q < G && n * G + q < a.k; ++q) {
                    const int e = __shfl_sync(0xffffffffu, id[n], q, G);
                    const float g = __shfl_sync(0xffffffffu, dk[n], q, G);
                    const int piece = e / VEC;
                    const int pos = e >= 0 && piece % G == i ? piece / G * VEC + e % VEC : -1;
#pragma unroll
                    for (int v = 0; v < NV * VEC; ++v)
                        if (v == pos) d.v[v] += g;
                }
            }
        }
        if (live) d.store(a.dlogits + (size_t)t * a.E, i, a.E);
    }
}

int sms() {
    static int n = device_sm_count();
    return n;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int N>
using Int = std::integral_constant<int, N>;

// Lanes and registers by E: the fewest lanes (of 2 to 32) whose one piece of 4
// experts each cover E, then more pieces a lane.  Rows that are not all 16-byte
// aligned go by single values, a warp each (8 lanes up to 8 experts).
template <class F>
cudaError_t by_width(int E, bool wide, F&& f) {
    if (wide) {
        if (E <= 8) return f(Int<2>(), Int<4>(), Int<1>());
        if (E <= 16) return f(Int<4>(), Int<4>(), Int<1>());
        if (E <= 32) return f(Int<8>(), Int<4>(), Int<1>());
        if (E <= 64) return f(Int<16>(), Int<4>(), Int<1>());
        if (E <= 128) return f(Int<32>(), Int<4>(), Int<1>());
        if (E <= 256) return f(Int<32>(), Int<4>(), Int<2>());
        if (E <= 512) return f(Int<32>(), Int<4>(), Int<4>());
        return f(Int<32>(), Int<4>(), Int<8>());
    }
    if (E <= 8) return f(Int<8>(), Int<1>(), Int<1>());
    if (E <= 32) return f(Int<32>(), Int<1>(), Int<1>());
    if (E <= 64) return f(Int<32>(), Int<1>(), Int<2>());
    if (E <= 128) return f(Int<32>(), Int<1>(), Int<4>());
    if (E <= 256) return f(Int<32>(), Int<1>(), Int<8>());
    if (E <= 512) return f(Int<32>(), Int<1>(), Int<16>());
    return f(Int<32>(), Int<1>(), Int<32>());
}

// Tokens of a block: what spreads them over the device so many blocks to an SM, in
// whole rounds of the block's groups.
int chunk_for(int m, int groups, int per_sm) {
    const int even = ceil_div(m, per_sm * sms());
    return std::min(kMaxChunk, std::max(kMinChunk, ceil_div(even, groups) * groups));
}

}  // namespace

// Chunks of the losses and their meetings with sequences, at most.
int64_t balance_slots(int64_t m, int64_t S) { return (m + kMinChunk - 1) / kMinChunk + S; }

cudaError_t launch_balance_loss(RouterArgs a, cudaStream_t st) {
    // A block counts kCountThreads x kIdsAhead ids in a step; sequences that fill the device by
    // themselves have one block each.  That goes by their number, not their lengths: 500000 tokens
    // with k = 8 among 200 short sequences take 964 us, alone 185, as 201 even ones 52.
    const int cluster = a.S >= sms() || (int64_t)a.m * a.k <= (int64_t)a.S * 1024 ? 1 : 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.S * cluster);
    cfg.blockDim = dim3(kCountThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, cluster == 1 ? count_pairs<1> : count_pairs<8>, a);
    if (e != cudaSuccess) return e;
    return by_width(a.E, a.E % 4 == 0 && aligned16(a.logits) && aligned16(a.counts), [&](auto g, auto vec, auto nv) {
        a.chunk = chunk_for(a.m, kThreads / g, 6);
        return launch_pdl(a.sigmoid ? balance_loss<true, g, vec, nv> : balance_loss<false, g, vec, nv>, dim3(ceil_div(a.m, a.chunk)), dim3(kThreads), 0, st, (const RouterArgs)a);
    });
}

cudaError_t launch_route_backward(RouterArgs a, cudaStream_t st) {
    const bool wide = a.E % 4 == 0 && aligned16(a.logits) && aligned16(a.dlogits) && (!a.counts || aligned16(a.counts));
    return by_width(a.E, wide, [&](auto g, auto vec, auto nv) {
        a.chunk = chunk_for(a.m, kThreads / g, 3);
        const size_t smem = a.dtopk_w ? (size_t)(kThreads / g) * a.E * 4 : 0;  // at most 32 KB
        return launch_pdl(a.sigmoid ? route_backward<true, g, vec, nv> : route_backward<false, g, vec, nv>, dim3(ceil_div(a.m, a.chunk)), dim3(kThreads), smem, st, (const RouterArgs)a);
    });
}

}  // namespace moe

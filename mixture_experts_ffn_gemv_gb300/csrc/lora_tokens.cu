// Low-rank adapters for few tokens: out[t] = y[t] + scale B (A x[t]), the
// adapter of each token its own.
//
// A token belongs to a cluster of 8, 4 or 2 blocks (as many as let all clusters run
// at once, two blocks an SM) and one launch does all of it: each block takes its
// share of K of A x, the blocks add their r partial sums up through distributed
// shared memory (in the order of the blocks), and each takes its share of the rows
// of B.  The first rows of B are on their way before the sums are done.
// What it reads is the token's A and B, 2 r (K + N) bytes; tokens that share an
// adapter read it from L2.  Bound by that for many tokens (128 of rank 16, 7168 ->
// 7168: 59 MB in 12.5 us), by the chain of loads, sums and loads for one (4.8 us).
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "launch.cuh"
#include "ops.h"
#include "sm100.cuh"
#include "tmap.h"

namespace moe {

namespace {

using namespace sm100;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPieces = 4;  // pieces of 8 inputs that a lane holds of x at a time
constexpr int kAhead = 4;   // rows of B that a lane has on their way at a time

__device__ __forceinline__ void unpack8(const uint4& a, float (&v)[8]) {
    v[0] = bf16lo(a.x); v[1] = bf16hi(a.x); v[2] = bf16lo(a.y); v[3] = bf16hi(a.y);
    v[4] = bf16lo(a.z); v[5] = bf16hi(a.z); v[6] = bf16lo(a.w); v[7] = bf16hi(a.w);
}

// LPR lanes hold a row of B, 8 of its r values each (LPR the power of two from r / 8 on).
template <int LPR, int kCluster>
__global__ void __launch_bounds__(kThreads) lora_tokens(const LoraArgs a) {
    __shared__ float part[kLoraMaxRank], low[kLoraMaxRank];
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x / kCluster, rank = (int)cluster_ctarank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t* y = a.y + (size_t)t * a.ldy;
    uint16_t* out = a.out + (size_t)t * a.ldo;
    // this block's rows of B
    const int rows = (a.N + kCluster - 1) / kCluster, n0 = rank * rows, n1 = min(a.N, n0 + rows);
    const int id = a.ids[t];
    if (id < 0 || id >= a.n) {  // no adapter: the whole cluster leaves
        if (id != -1 && rank == 0 && threadIdx.x == 0) note_error(a.hdr, DEV_ERR_BAD_ID, t);
        if (a.y != a.out)
            for (int j = n0 + threadIdx.x; j < n1; j += kThreads) out[j] = y[j];
        return;
    }
    const uint16_t* A = a.a + (size_t)id * a.r * a.K;
    const uint16_t* B = a.b + (size_t)id * a.N * a.r;

    constexpr int kRowsPerStep = kThreads / LPR;
    const int q = threadIdx.x % LPR, row0 = n0 + threadIdx.x / LPR;
    const bool mine = 8 * q < a.r;
    uint4 bv[kAhead];
    auto load_b = [&](int j) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int row = j + i * kRowsPerStep;
            bv[i] = mine && row < n1 ? ld_stream_v4(B + (size_t)row * a.r + 8 * q) : make_uint4(0, 0, 0, 0);
        }
    };

    // A x over this block's share of K
    const int pieces = a.K / 8, each = (pieces + kCluster - 1) / kCluster;
    const int p1 = min(pieces, (rank + 1) * each);
    const uint16_t* x = a.x + (size_t)t * a.ldx;
    for (int j = threadIdx.x; j < a.r; j += kThreads) part[j] = 0.f;
    load_b(row0);
    __syncthreads();
    for (int p0 = rank * each; p0 < p1; p0 += 32 * kPieces) {
        float xv[kPieces][8];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int p = p0 + 32 * i + lane;
            unpack8(p < p1 ? *reinterpret_cast<const uint4*>(x + 8 * p) : make_uint4(0, 0, 0, 0), xv[i]);
        }
        for (int j = warp; j < a.r; j += 2 * kWarps) {  // two rows of A at a time, one for r = 8
            const int j2 = j + kWarps;
            uint4 av[2][kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int p = p0 + 32 * i + lane;
                av[0][i] = p < p1 ? ld_stream_v4(A + (size_t)j * a.K + 8 * p) : make_uint4(0, 0, 0, 0);
                av[1][i] = p < p1 && j2 < a.r ? ld_stream_v4(A + (size_t)j2 * a.K + 8 * p) : make_uint4(0, 0, 0, 0);
            }
            float s[2] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    float v[8];
                    unpack8(av[h][i], v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[h] = fmaf(v[e], xv[i][e], s[h]);
                }
            s[0] = warp_sum(s[0]);
            s[1] = warp_sum(s[1]);
            if (lane == 0) {
                part[j] += s[0];
                if (j2 < a.r) part[j2] += s[1];
            }
        }
    }
    __syncthreads();
    cluster_sync();
    if ((int)threadIdx.x < a.r) {
        const uint32_t p = smem_u32(part + threadIdx.x);
        float v[kCluster], s = 0.f;
#pragma unroll
        for (int c = 0; c < kCluster; ++c)
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[c]) : "r"(mapa(p, c)) : "memory");
#pragma unroll
        for (int c = 0; c < kCluster; ++c) s += v[c];
        low[threadIdx.x] = a.scale ? s * a.scale[id] : s;
    }
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // has read the others' sums
    float lv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) lv[e] = mine ? low[8 * q + e] : 0.f;
    for (int base = n0; base < n1; base += kAhead * kRowsPerStep) {  // the block's warps stay together
        const int j = base + threadIdx.x / LPR;
        uint4 cur[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) cur[i] = bv[i];
        if (base + kAhead * kRowsPerStep < n1) load_b(j + kAhead * kRowsPerStep);
        float yv[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int row = j + i * kRowsPerStep;
            yv[i] = q == 0 && row < n1 ? bf16_to_f32(y[row]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            float v[8], s = 0.f;
            unpack8(cur[i], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(v[e], lv[e], s);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            const int row = j + i * kRowsPerStep;
            if (q == 0 && row < n1) out[row] = f32_to_bf16(yv[i] + s);
        }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the others have read this block's
}

template <int LPR, int kCluster>
cudaError_t launch(const LoraArgs& a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.m * kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = kCluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, lora_tokens<LPR, kCluster>, a);
}

int sms() {
    static int n = device_sm_count();
    return n;
}

template <int LPR>
cudaError_t launch_by_tokens(const LoraArgs& a, cudaStream_t st) {
    const int room = 2 * sms();
    return a.m * 8 <= room ? launch<LPR, 8>(a, st) : a.m * 4 <= room ? launch<LPR, 4>(a, st) : launch<LPR, 2>(a, st);
}

}  // namespace

// Clusters by token, or tiles of 128 tokens?  Tiles read a shared adapter once, but each
// adapter that occurs costs a tile its products and an accumulator's way through the
// epilogue; by token it makes no difference who shares what.  In us, by token / by tiles,
// tokens of all adapters mixed and (one for all):
//   2048 -> 7168, r = 16, 32 adapters: 128 tokens 8.6 / 18 (8.3 / 9.7), 256 tokens 15 / 26
//     (15 / 9.5), 384 tokens 21 / 38 (21 / 10)
//   7168 -> 2048, r = 32, 32 adapters: 128 tokens 14 / 17 (14 / 12), 192 tokens 24 / 21 (23 / 13)
//   7168 -> 2048, r = 64, 32 adapters: 65 tokens 14 / 19 (14 / 14), 96 tokens 22 / 20 (23 / 15)
//   4096 -> 4096, r = 16, 3 adapters: 128 tokens 7.9 / 13 (7.9 / 10), 192 tokens 13 / 13 (13 / 10)
// So few tokens, weighed by their rank, go by token, and twice as many where there are
// adapters to mix.
bool lora_by_token(int m, int n, int r) {
    return m <= kLoraByToken || (int64_t)m * std::max(r, 16) <= (n >= 4 ? 4096 : 2048);
}

cudaError_t launch_lora_tokens(const LoraArgs& a, cudaStream_t st) {
    if (a.r <= 8) return launch_by_tokens<1>(a, st);
    if (a.r <= 16) return launch_by_tokens<2>(a, st);
    if (a.r <= 32) return launch_by_tokens<4>(a, st);
    if (a.r <= 64) return launch_by_tokens<8>(a, st);
    return launch_by_tokens<16>(a, st);
}

}  // namespace moe

// RMSNorm with the residual's addition, to bf16 and to e4m3 with a scale per
// 128 columns, and its backward pass.
//
//   r = bf16(x + res)   n = r rstd, rstd = 1 / sqrt(sum r^2 / H + eps)   out = n w
//   s = max |out| / 448 of a block of 128 (1 where that is 0), code = e4m3(out / s)
//
// The norm is taken of the rounded r, which is what the residual stream goes on
// with; out is rounded once, to bf16 and (from the same fp32 values) to e4m3.
// Every element is read once and every result written once: a row stays in
// registers, as the bf16 pairs it was rounded to, between its sum and its
// scaling.  Bound by HBM for many rows: 16384 x 7168 with residual and both outputs
// (1061 MB) in 158 us, 6.7 TB/s; by one row's way through a block for few: 2.9 us for
// one row of 7168.
//
// A row belongs to a warp (H up to 1024) or to a block; a thread holds V pieces
// of 8 columns, piece v at v * threads + thread, so that 16 neighbouring lanes
// hold one block of 128 and its maximum takes four shuffles.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "launch.cuh"
#include "ops.h"
#include "pairs.cuh"
#include "tmap.h"

namespace moe {

namespace {

constexpr int kWarpRows = 8;       // rows of a block whose warps take a row each
constexpr int kWarpMaxH = 1024;    // widest of them: 32 lanes x 4 x 8 columns

// 16 bytes that are read once (not through the read-only path: out may be x and
// res_out may be res).
__device__ __forceinline__ uint4 ld_once(const uint16_t* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
__device__ __forceinline__ void unpack8(const uint4& a, float (&v)[8]) {
    v[0] = bf16lo(a.x); v[1] = bf16hi(a.x); v[2] = bf16lo(a.y); v[3] = bf16hi(a.y);
    v[4] = bf16lo(a.z); v[5] = bf16hi(a.z); v[6] = bf16lo(a.w); v[7] = bf16hi(a.w);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void load_w8(const float* p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p + 4));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// The sum of v over a row's threads, in a fixed order: a warp's butterfly, then
// every warp's over the block's warps.  buf: a float per warp.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* buf) {
    v = warp_sum(v);
    if (WARP) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < (int)(blockDim.x >> 5) ? buf[lane] : 0.f);
}

// A block's rows have two pieces a thread (three above 16384 columns): with one, 16384 x
// 7168 take 203 us instead of 161.
template <int V, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) add_rmsnorm(const NormArgs a) {
    __shared__ float buf[32];
    pdl_wait();
    pdl_trigger();
    const int n = WARP ? 32 : (int)blockDim.x, i = WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int t = WARP ? (int)blockIdx.x * kWarpRows + (int)(threadIdx.x >> 5) : (int)blockIdx.x;
    if (WARP && t >= a.m) return;  // whole warps, and no block-wide barrier on this path
    const int pieces = a.H >> 3;
    const uint16_t* x = a.x + (size_t)t * a.ldx;
    const uint16_t* res = a.res ? a.res + (size_t)t * a.ldr : nullptr;
    uint4 r[V];
    if (res) {
        uint4 q[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * n + i;
            r[v] = c < pieces ? ld_once(x + 8 * c) : make_uint4(0, 0, 0, 0);
            q[v] = c < pieces ? ld_once(res + 8 * c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f[8], g[8];
            unpack8(r[v], f);
            unpack8(q[v], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += g[j];
            r[v] = pack8(f);
            const int c = v * n + i;
            if (c < pieces) *reinterpret_cast<uint4*>(a.res_out + (size_t)t * a.ldo + 8 * c) = r[v];
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * n + i;
            r[v] = c < pieces ? ld_once(x + 8 * c) : make_uint4(0, 0, 0, 0);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float f[8];
        unpack8(r[v], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
    }
    const float inv = 1.0f / sqrtf(row_sum<WARP>(ss, buf) / (float)a.H + a.eps);
    const int blocks = (a.H + 127) >> 7;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = v * n + i;
        const bool in = c < pieces;
        float f[8], w[8];
        unpack8(r[v], f);
        if (in) {
            load_w8(a.w + 8 * c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] * inv * w[j];
            if (a.out) *reinterpret_cast<uint4*>(a.out + (size_t)t * a.H + 8 * c) = pack8(f);
        }
        if (a.codes) {
            float top = 0.f;
            if (in) {
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[j]));
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            // a block of zeros, or too small for a scale: 1, and codes 0 of either sign (NaN stays)
            const float q = __fdiv_rn(top, 448.0f), s = q > 0.f ? q : 1.0f;
            const uint32_t keep = q > 0.f ? 0xffffffffu : 0x7f7f7f7fu;
            const QuotientBracket b = quotient_bracket(s);
            if (in) {
                *reinterpret_cast<uint2*>(a.codes + (size_t)t * a.H + 8 * c) =
                    make_uint2(e4m3x4_quotient(f, s, b) & keep, e4m3x4_quotient(f + 4, s, b) & keep);
                if ((c & 15) == 0) a.scales[(size_t)t * blocks + (c >> 4)] = s;
            }
        }
    }
}

__device__ __forceinline__ Pair unpack2(uint32_t w) { return Pair{bf16lo(w), bf16hi(w)}; }
__device__ __forceinline__ void load_w4(const float* p, Pair (&v)[4]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p + 4));
    v[0] = Pair{a.x, a.y}; v[1] = Pair{a.z, a.w}; v[2] = Pair{b.x, b.y}; v[3] = Pair{b.z, b.w};
}
// Waits for the T threads of group g of the block.
__device__ __forceinline__ void group_sync(int g, int T) { asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(T) : "memory"); }

// Backward: with g = dout w and n = r rstd, both of a row's sums (r^2 and g r)
// in one pass,
//   dx = rstd (g - n sum(g n) / H) + dres
// and dw = sum over rows of dout n: a thread adds up its own columns over the
// rows of its group (T threads take a row, a block has several groups), the
// groups of a block are added in shared memory and the blocks' sums [blocks, H]
// by column_sums, each in its order.
// 16384 x 2048 (268 MB) in 49 us, 5.5 TB/s, some 5 of it the sums of dw.  Registers
// leave 1024 threads to an SM, whose loads, sums and stores hide each other only so
// far: rows wider than 8192 columns, a block to an SM, reach 0.5 to 0.75 of the copy
// rate.  (Copying the next row to shared memory meanwhile cost more than it hid:
// 16384 x 2048 53 -> 59 us at the time, 4096 x 16384 126 -> 141.)  Three pieces a
// thread (rows wider than 16384 columns) spill 92 bytes: 2048 x 24576 in 108 us.
template <int V>
__global__ void __launch_bounds__(1024) add_rmsnorm_backward(const NormGradArgs a, int T) {
    __shared__ float2 buf[2][32];
    extern __shared__ float sum[];  // [H] where the block has more than one group
    pdl_wait();
    pdl_trigger();
    const int g = threadIdx.x / T, i = threadIdx.x % T, groups = blockDim.x / T;
    const int pieces = a.H >> 3, warp = threadIdx.x >> 5, warps = T >> 5;
    constexpr bool kEarly = V <= 2;  // registers for dres from the start
    Pair dw[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[v][j] = Pair{0.f, 0.f};
    int turn = 0;
    for (int t = blockIdx.x * groups + g; t < a.m; t += gridDim.x * groups, turn ^= 1) {
        const uint16_t *dout = a.dout + (size_t)t * a.ldd, *row = a.r + (size_t)t * a.ldr;
        const uint16_t* dres = a.dres ? a.dres + (size_t)t * a.ldq : nullptr;
        uint4 r[V], d[V], q[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * T + i;
            const uint4 none = make_uint4(0, 0, 0, 0);
            r[v] = c < pieces ? ld_once(row + 8 * c) : none;
            d[v] = c < pieces ? ld_once(dout + 8 * c) : none;
            if (kEarly) q[v] = dres && c < pieces ? ld_once(dres + 8 * c) : none;
        }
        Pair s2{0.f, 0.f}, g2{0.f, 0.f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * T + i;
            if (c < pieces) {
                const uint32_t rw[4] = {r[v].x, r[v].y, r[v].z, r[v].w}, ew[4] = {d[v].x, d[v].y, d[v].z, d[v].w};
                Pair w[4];
                load_w4(a.w + 8 * c, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Pair f = unpack2(rw[j]);
                    s2 = fma2(f, f, s2);
                    g2 = fma2(mul2(unpack2(ew[j]), w[j]), f, g2);
                }
            }
        }
        float ss = warp_sum(s2.x + s2.y), gr = warp_sum(g2.x + g2.y);
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) buf[turn][warp] = make_float2(ss, gr);
            group_sync(g, T);
            const float2 b = (int)(threadIdx.x & 31) < warps ? buf[turn][g * warps + (threadIdx.x & 31)] : make_float2(0.f, 0.f);
            ss = warp_sum(b.x);
            gr = warp_sum(b.y);
        }
        const float inv = 1.0f / sqrtf(ss / (float)a.H + a.eps);
        const float mean = gr / (float)a.H * inv;  // of g n
        const Pair inv2{inv, inv};
        const Pair back{-mean * inv, -mean * inv};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * T + i;
            if (c < pieces) {
                if (!kEarly) q[v] = dres ? ld_once(dres + 8 * c) : make_uint4(0, 0, 0, 0);
                const uint32_t rw[4] = {r[v].x, r[v].y, r[v].z, r[v].w}, ew[4] = {d[v].x, d[v].y, d[v].z, d[v].w},
                               qw[4] = {q[v].x, q[v].y, q[v].z, q[v].w};
                Pair w[4];
                load_w4(a.w + 8 * c, w);
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Pair f = unpack2(rw[j]), e = unpack2(ew[j]);
                    const Pair nj = mul2(f, inv2);
                    dw[v][j] = fma2(e, nj, dw[v][j]);
                    const Pair x = fma2(mul2(e, w[j]), inv2, fma2(nj, back, unpack2(qw[j])));
                    o[j] = pack_bf16x2(x.x, x.y);
                }
                *reinterpret_cast<uint4*>(a.dx + (size_t)t * a.H + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
    if (!a.dw) return;
    float* part = a.part + (size_t)blockIdx.x * a.H;
    for (int k = 0; k < groups; ++k) {  // the last group's turn writes the block's sum out
        if (k == g) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = v * T + i;
                if (c < pieces)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float4 f = make_float4(dw[v][2 * h].x, dw[v][2 * h].y, dw[v][2 * h + 1].x, dw[v][2 * h + 1].y);
                        float4* s4 = reinterpret_cast<float4*>(sum + 8 * c + 4 * h);
                        if (k) {
                            const float4 q = *s4;
                            f = make_float4(f.x + q.x, f.y + q.y, f.z + q.z, f.w + q.w);
                        }
                        *(k == groups - 1 ? reinterpret_cast<float4*>(part + 8 * c + 4 * h) : s4) = f;
                    }
            }
        }
        __syncthreads();
    }
}

// out[c] = sum over p of part[p, c]: a block takes 32 columns, its warps every
// 16th row, then the warps in order.
__global__ void __launch_bounds__(512) column_sums(const float* __restrict__ part, int P, int H, float* __restrict__ out) {
    __shared__ float s[16][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < H) {
#pragma unroll 10
        for (int p = warp; p < P; p += 16) v += __ldcg(part + (size_t)p * H + c);
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < H) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) t += s[k][lane];
        out[c] = t;
    }
}

int sms() {
    static int n = device_sm_count();
    return n;
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t st) {
    if (a.H <= kWarpMaxH) {
        const dim3 grid(ceil_div(a.m, kWarpRows)), block(32 * kWarpRows);
        switch (ceil_div(a.H, 256)) {
            case 1: return launch_pdl(add_rmsnorm<1, true>, grid, block, 0, st, a);
            case 2: return launch_pdl(add_rmsnorm<2, true>, grid, block, 0, st, a);
            case 3: return launch_pdl(add_rmsnorm<3, true>, grid, block, 0, st, a);
            default: return launch_pdl(add_rmsnorm<4, true>, grid, block, 0, st, a);
        }
    }
    const int v = a.H <= 16384 ? 2 : 3;
    const dim3 grid(a.m), block(ceil_div(ceil_div(a.H / 8, v), 32) * 32);
    return v == 2 ? launch_pdl(add_rmsnorm<2, false>, grid, block, 0, st, a) : launch_pdl(add_rmsnorm<3, false>, grid, block, 0, st, a);
}

namespace {

// Pieces of a thread, threads of a row, rows of a block at a time, blocks: 1024
// threads to an SM, which the registers allow; few rows go to as many SMs.
struct GradShape {
    int v, T, most, groups, blocks;
};
GradShape grad_shape(int m, int H) {
    GradShape s;
    s.v = H <= 256 ? 1 : H <= 16384 ? 2 : 3;
    s.T = ceil_div(ceil_div(H / 8, s.v), 32) * 32;
    s.most = std::max(1, 512 / s.T);
    s.groups = std::min(s.most, std::max(1, ceil_div(m, 2 * sms())));
    s.blocks = std::min(ceil_div(m, s.groups), sms() * (1024 / (s.T * s.groups)));
    return s;
}

}  // namespace

// Blocks, at most, of m rows and of fewer: below s.most groups they are at most two an SM.
int norm_grad_blocks(int m, int H) {
    const GradShape s = grad_shape(m, H);
    return std::min(m, sms() * std::max(2, 1024 / (s.T * s.most)));
}

cudaError_t launch_add_rmsnorm_backward(const NormGradArgs& a, cudaStream_t st) {
    const GradShape s = grad_shape(a.m, a.H);
    const dim3 grid(s.blocks), block(s.T * s.groups);
    const size_t smem = a.dw && s.groups > 1 ? (size_t)a.H * 4 : 0;  // at most 16 KB
    cudaError_t e;
    switch (s.v) {
        case 1: e = launch_pdl(add_rmsnorm_backward<1>, grid, block, smem, st, a, s.T); break;
        case 2: e = launch_pdl(add_rmsnorm_backward<2>, grid, block, smem, st, a, s.T); break;
        default: e = launch_pdl(add_rmsnorm_backward<3>, grid, block, smem, st, a, s.T); break;
    }
    if (e != cudaSuccess || !a.dw) return e;
    return launch_pdl(column_sums, dim3(ceil_div(a.H, 32)), dim3(512), 0, st, (const float*)a.part, s.blocks, a.H, a.dw);
}

}  // namespace moe

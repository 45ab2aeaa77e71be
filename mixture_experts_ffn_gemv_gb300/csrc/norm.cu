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
// scaling.  Bound by HBM for many rows, by one row's latency for few.
//
// A row belongs to a warp (H up to 1024) or to a block; a thread holds V pieces
// of 8 columns, piece v at v * threads + thread, so that 16 neighbouring lanes
// hold one block of 128 and its maximum takes four shuffles.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "launch.cuh"
#include "ops.h"
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
// the block's warps one after another.  buf: a float per warp, two of them used
// in turn by callers that loop.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* buf) {
    v = warp_sum(v);
    if (WARP) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) t += buf[i];
    return t;
}

// Threads up to 512 for up to 4 pieces each; wider rows have 1024 threads.
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
            const float s = top > 0.f ? __fdiv_rn(top, 448.0f) : 1.0f;
            const QuotientBracket b = quotient_bracket(s);
            if (in) {
                const uint32_t keep = top > 0.f ? 0xffffffffu : 0x7f7f7f7fu;  // a block of zeros: codes 0, of either sign
                *reinterpret_cast<uint2*>(a.codes + (size_t)t * a.H + 8 * c) =
                    make_uint2(e4m3x4_quotient(f, s, b) & keep, e4m3x4_quotient(f + 4, s, b) & keep);
                if ((c & 15) == 0) a.scales[(size_t)t * blocks + (c >> 4)] = s;
            }
        }
    }
}

// Backward: with g = dout w and n = r rstd, both of a row's sums (r^2 and g r)
// in one pass,
//   dx = rstd (g - n sum(g n) / H) + dres
// and dw = sum over rows of dout n: a thread adds up its own columns over the
// rows of its block, the blocks' sums [blocks, H] are added by column_sums in
// their order.
template <int V, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) add_rmsnorm_backward(const NormGradArgs a) {
    __shared__ float buf[2][2][32];
    extern __shared__ float wdw[];  // WARP: [kWarpRows, H]
    pdl_wait();
    pdl_trigger();
    const int n = WARP ? 32 : (int)blockDim.x, i = WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int pieces = a.H >> 3, warp = threadIdx.x >> 5;
    float dw[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[v][j] = 0.f;
    const int step = (int)gridDim.x * (WARP ? kWarpRows : 1);
    int turn = 0;
    for (int t = WARP ? (int)blockIdx.x * kWarpRows + warp : (int)blockIdx.x; t < a.m; t += step, turn ^= 1) {
        const uint16_t *dout = a.dout + (size_t)t * a.ldd, *row = a.r + (size_t)t * a.ldr;
        uint4 r[V], d[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * n + i;
            r[v] = c < pieces ? ld_once(row + 8 * c) : make_uint4(0, 0, 0, 0);
            d[v] = c < pieces ? ld_once(dout + 8 * c) : make_uint4(0, 0, 0, 0);
        }
        float ss = 0.f, gr = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * n + i;
            if (c < pieces) {
                float f[8], g[8], w[8];
                unpack8(r[v], f);
                unpack8(d[v], g);
                load_w8(a.w + 8 * c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    ss = fmaf(f[j], f[j], ss);
                    gr = fmaf(g[j] * w[j], f[j], gr);
                }
            }
        }
        ss = warp_sum(ss);
        gr = warp_sum(gr);
        if (!WARP) {
            if ((threadIdx.x & 31) == 0) {
                buf[turn][0][warp] = ss;
                buf[turn][1][warp] = gr;
            }
            __syncthreads();
            ss = gr = 0.f;
            for (int k = 0; k < (int)(blockDim.x >> 5); ++k) {
                ss += buf[turn][0][k];
                gr += buf[turn][1][k];
            }
        }
        const float inv = 1.0f / sqrtf(ss / (float)a.H + a.eps);
        const float mean = gr / (float)a.H * inv;  // of g n
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * n + i;
            if (c < pieces) {
                float f[8], g[8], w[8], o[8];
                unpack8(r[v], f);
                unpack8(d[v], g);
                load_w8(a.w + 8 * c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float nj = f[j] * inv;
                    dw[v][j] = fmaf(g[j], nj, dw[v][j]);
                    o[j] = inv * fmaf(-nj, mean, g[j] * w[j]);
                }
                if (a.dres) {
                    float q[8];
                    unpack8(ld_once(a.dres + (size_t)t * a.ldq + 8 * c), q);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] += q[j];
                }
                *reinterpret_cast<uint4*>(a.dx + (size_t)t * a.H + 8 * c) = pack8(o);
            }
        }
    }
    if (!a.dw) return;
    float* part = a.part + (size_t)blockIdx.x * a.H;
    if (WARP) {
        for (int v = 0; v < V; ++v) {
            const int c = v * n + i;
            if (c < pieces)
#pragma unroll
                for (int j = 0; j < 8; ++j) wdw[warp * a.H + 8 * c + j] = dw[v][j];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.H; c += 32 * kWarpRows) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kWarpRows; ++k) s += wdw[k * a.H + c];
            part[c] = s;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * n + i;
            if (c < pieces) {
                *reinterpret_cast<float4*>(part + 8 * c) = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
                *reinterpret_cast<float4*>(part + 8 * c + 4) = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
            }
        }
    }
}

// out[c] = sum over p of part[p, c]: a block takes 32 columns, its warps every
// eighth row, then the warps in order.
__global__ void __launch_bounds__(256) column_sums(const float* __restrict__ part, int P, int H, float* __restrict__ out) {
    __shared__ float s[8][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < H) {
#pragma unroll 8
        for (int p = warp; p < P; p += 8) v += part[(size_t)p * H + c];
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < H) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += s[k][lane];
        out[c] = t;
    }
}

int sms() {
    static int n = device_sm_count();
    return n;
}

// Pieces a thread holds and threads of a block for rows of H columns.
struct RowShape {
    int v, threads;
};
RowShape row_shape(int H, int want_v) {
    const int pieces = H / 8;
    int v = std::max(want_v, ceil_div(pieces, 1024));
    return {v, ceil_div(ceil_div(pieces, v), 32) * 32};
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
    const RowShape s = row_shape(a.H, a.m < 2 * sms() ? 1 : 2);
    const dim3 grid(a.m), block(s.threads);
    switch (s.v) {
        case 1: return launch_pdl(add_rmsnorm<1, false>, grid, block, 0, st, a);
        case 2: return launch_pdl(add_rmsnorm<2, false>, grid, block, 0, st, a);
        default: return launch_pdl(add_rmsnorm<3, false>, grid, block, 0, st, a);
    }
}

int norm_grad_blocks(int m, int H) {
    if (H <= kWarpMaxH) return std::min(ceil_div(m, kWarpRows), 4 * sms());
    return std::min(m, sms() * std::max(1, 1024 / row_shape(H, 2).threads));
}

cudaError_t launch_add_rmsnorm_backward(const NormGradArgs& a, cudaStream_t st) {
    const int blocks = norm_grad_blocks(a.m, a.H);
    cudaError_t e;
    if (a.H <= kWarpMaxH) {
        const dim3 grid(blocks), block(32 * kWarpRows);
        const size_t smem = a.dw ? (size_t)kWarpRows * a.H * 4 : 0;
        switch (ceil_div(a.H, 256)) {
            case 1: e = launch_pdl(add_rmsnorm_backward<1, true>, grid, block, smem, st, a); break;
            case 2: e = launch_pdl(add_rmsnorm_backward<2, true>, grid, block, smem, st, a); break;
            case 3: e = launch_pdl(add_rmsnorm_backward<3, true>, grid, block, smem, st, a); break;
            default: e = launch_pdl(add_rmsnorm_backward<4, true>, grid, block, smem, st, a); break;
        }
    } else {
        const RowShape s = row_shape(a.H, 2);
        const dim3 grid(blocks), block(s.threads);
        e = s.v == 2 ? launch_pdl(add_rmsnorm_backward<2, false>, grid, block, 0, st, a)
                     : launch_pdl(add_rmsnorm_backward<3, false>, grid, block, 0, st, a);
    }
    if (e != cudaSuccess || !a.dw) return e;
    return launch_pdl(column_sums, dim3(ceil_div(a.H, 32)), dim3(256), 0, st, (const float*)a.part, blocks, a.H, a.dw);
}

}  // namespace moe

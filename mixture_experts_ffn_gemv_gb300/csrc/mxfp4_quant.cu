// MXFP4 quantisation of rows, and reading them back.
//
// A block's scale is a power of two taken from the exponent of its largest
// magnitude, so a block needs nothing from outside itself: one pass, no
// division (v / 2^e is an exact product), every code bit for bit the rounding
// of the true quotient.  Both kernels only move memory.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "mxfp4.cuh"
#include "ffn_block.h"

namespace moe {

namespace {

// Eight elements of a row as floats (16 bytes of bf16 or 32 of fp32).
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
    const uint4 q = ld_stream_v4(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo(w[i]);
        v[2 * i + 1] = bf16hi(w[i]);
    }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const uint4 a = ld_stream_v4(p), b = ld_stream_v4(p + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}

// Four lanes share a block of 32 (eight elements each), a warp takes 256
// elements of a row: two scale tiles' words, padding blocks (zeros) included.
template <typename T>
__global__ void __launch_bounds__(256) mx_quant(const T* x, size_t ldx, int rows, int n, int nkt, uint8_t* codes,
                                                uint8_t* scales) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int chunks = (nkt + 1) >> 1;  // 256-element chunks per row
    const size_t total = (size_t)rows * chunks, step = (size_t)gridDim.x * (blockDim.x >> 5);
    for (size_t i = (size_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < total; i += step) {
        const size_t r = i / chunks;
        const int c = (int)(i % chunks), k = c * 256 + lane * 8;
        float v[8] = {};
        const bool in = k < n;
        if (in) load8(x + r * ldx + k, v);
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(v[j]) & 0x7fffffffu);
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const uint32_t s = mx_scale(a);
        const uint32_t w = s == 255u ? 0u : mx_codes8(v, mx_inverse(s));
        if (in) *reinterpret_cast<uint32_t*>(codes + r * (size_t)(n >> 1) + (k >> 1)) = w;
        // the 16 lanes of a tile: their four scales as one word
        uint32_t sw = s << (((lane >> 2) & 3) * 8);
        sw |= __shfl_xor_sync(0xffffffffu, sw, 4);
        sw |= __shfl_xor_sync(0xffffffffu, sw, 8);
        const int kt = 2 * c + (lane >> 4);
        if ((lane & 15) == 0 && kt < nkt)
            *reinterpret_cast<uint32_t*>(scales + mx_scale_at(r, (size_t)kt * 4, nkt)) = sw;
    }
}

// One thread: 8 codes (4 bytes in, 16 bytes out).
__global__ void __launch_bounds__(256) mx_dequant(const uint8_t* codes, const uint8_t* scales, int rows, int n,
                                                  int nkt, uint16_t* out) {
    pdl_wait();
    pdl_trigger();
    const int per = n >> 3;
    const size_t total = (size_t)rows * per, step = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const size_t r = i / per;
        const int k = (int)(i % per) * 8;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + i * 4);
        const uint32_t s = scales[mx_scale_at(r, k >> 5, nkt)];
        // 2^(s - 127): subnormal for s = 0, NaN for s = 255
        const float f = __uint_as_float(s == 0u ? 0x00400000u : (s == 255u ? 0x7fffffffu : s << 23));
        uint32_t h[4], o[4];
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(w));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            asm("{ .reg .f16 a, b;\n\t mov.b32 {a, b}, %2;\n\t cvt.f32.f16 %0, a;\n\t cvt.f32.f16 %1, b; }"
                : "=f"(lo), "=f"(hi)
                : "r"(h[j]));
            o[j] = pack_bf16x2(lo * f, hi * f);
        }
        *reinterpret_cast<uint4*>(out + i * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

int grid_for(size_t blocks) { return (int)std::min<size_t>(std::max<size_t>(blocks, 1), 152 * 16); }

}  // namespace

cudaError_t launch_mx_quant(const void* x, bool f32, size_t ldx, int rows, int n, uint8_t* codes, uint8_t* scales,
                            cudaStream_t st) {
    const int nkt = ceil_div(n, 128);
    const dim3 grid(grid_for(((size_t)rows * ((nkt + 1) / 2) + 7) / 8)), block(256);
    return f32 ? launch_pdl(mx_quant<float>, grid, block, 0, st, static_cast<const float*>(x), ldx, rows, n, nkt, codes, scales)
               : launch_pdl(mx_quant<uint16_t>, grid, block, 0, st, static_cast<const uint16_t*>(x), ldx, rows, n, nkt, codes, scales);
}

cudaError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int rows, int n, uint16_t* out,
                              cudaStream_t st) {
    const dim3 grid(grid_for(((size_t)rows * (n / 8) + 255) / 256)), block(256);
    return launch_pdl(mx_dequant, grid, block, 0, st, codes, scales, rows, n, ceil_div(n, 128), out);
}

}  // namespace moe

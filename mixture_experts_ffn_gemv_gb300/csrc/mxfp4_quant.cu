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
#include "tmap.h"

namespace moe {

namespace {

// Sixteen elements of a row, raw: 32 bytes of bf16 or 64 of fp32, in 32-byte
// loads where the rows are so aligned.
template <typename T>
struct Raw {
    uint32_t w[4 * sizeof(T)];
};
template <typename T, bool WIDE>
__device__ __forceinline__ void load16(const T* p, Raw<T>& r) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        if (WIDE) {
            uint32_t v[8];
            ld_global_v8(p + 32 / sizeof(T) * i, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) r.w[8 * i + k] = v[k];
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint4 q = ld_stream_v4(p + 32 / sizeof(T) * i + 16 / sizeof(T) * k);
                r.w[8 * i + 4 * k] = q.x;
                r.w[8 * i + 4 * k + 1] = q.y;
                r.w[8 * i + 4 * k + 2] = q.z;
                r.w[8 * i + 4 * k + 3] = q.w;
            }
        }
    }
}
__device__ __forceinline__ void widen(const Raw<uint16_t>& r, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = bf16lo(r.w[i]);
        v[2 * i + 1] = bf16hi(r.w[i]);
    }
}
__device__ __forceinline__ void widen(const Raw<float>& r, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r.w[i]);
}

// Two lanes share a block of 32, a warp takes 512 elements of a row: four scale
// tiles' words, padding blocks (zeros) included.  Bound by HBM; a warp has U
// such pieces in flight (14336 x 7168 bf16 with 1, 2, 3, 4: 50.0, 44.0, 42.3,
// 44.9 us, 6.1 TB/s at best).
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) mx_quant(const T* x, size_t ldx, uint32_t total, uint32_t pieces, int n,
                                                int nkt, uint8_t* codes, uint8_t* scales) {
    constexpr int U = sizeof(T) == 2 ? 3 : 2;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const uint32_t step = gridDim.x * (blockDim.x >> 5);
    for (uint32_t i0 = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i0 < total; i0 += U * step) {
        Raw<T> raw[U];
        uint32_t row[U];
        int k[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = i0 + u * step;
            row[u] = i / pieces;
            k[u] = i < total ? (int)(i % pieces) * 512 + lane * 16 : INT32_MAX;
            if (k[u] < n) load16<T, WIDE>(x + row[u] * ldx + k[u], raw[u]);
            else raw[u] = Raw<T>{};
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[16];
            widen(raw[u], v);
            uint32_t a = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) a = max(a, __float_as_uint(v[j]) & 0x7fffffffu);
            a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
            const uint32_t s = mx_scale(a);
            const float inv = mx_inverse(s);
            uint2 w = make_uint2(mx_codes8(v, inv), mx_codes8(v + 8, inv));
            if (s == 255u) w = make_uint2(0, 0);
            if (k[u] < n) *reinterpret_cast<uint2*>(codes + row[u] * (size_t)(n >> 1) + (k[u] >> 1)) = w;
            // the 8 lanes of a tile: their four scales as one word
            uint32_t sw = s << (((lane >> 1) & 3) * 8);
            sw |= __shfl_xor_sync(0xffffffffu, sw, 2);
            sw |= __shfl_xor_sync(0xffffffffu, sw, 4);
            const int kt = k[u] >> 7;
            if ((lane & 7) == 0 && kt < nkt)
                *reinterpret_cast<uint32_t*>(scales + mx_scale_at(row[u], (size_t)kt * 4, nkt)) = sw;
        }
    }
}

// Sixteen codes a thread (8 bytes in, 32 out), U in flight, the 32 as one store
// where out is so aligned (WIDE), else as two.  Bound by HBM: 14336 x 7168 in
// 40.0 us, 6.5 TB/s.
template <bool WIDE>
__global__ void __launch_bounds__(256) mx_dequant(const uint8_t* codes, const uint8_t* scales, uint32_t total,
                                                  uint32_t per, int nkt, uint16_t* out) {
    constexpr int U = 4;
    pdl_wait();
    pdl_trigger();
    const uint32_t step = gridDim.x * blockDim.x;
    for (uint32_t i0 = blockIdx.x * blockDim.x + threadIdx.x; i0 < total; i0 += U * step) {
        uint2 c[U];
        uint32_t s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = i0 + u * step;
            if (i >= total) continue;
            c[u] = *reinterpret_cast<const uint2*>(codes + (size_t)i * 8);
            s[u] = scales[mx_scale_at(i / per, (i % per) >> 1, nkt)];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = i0 + u * step;
            if (i >= total) continue;
            // 2^(s - 127): subnormal for s = 0, NaN for s = 255
            const float f = __uint_as_float(s[u] == 0u ? 0x00400000u : (s[u] == 255u ? 0x7fffffffu : s[u] << 23));
            uint32_t o[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t q[4];
                asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
                    "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
                    "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
                    "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
                    "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
                    "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
                    : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3])
                    : "r"(h ? c[u].y : c[u].x));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float lo, hi;
                    asm("{ .reg .f16 a, b;\n\t mov.b32 {a, b}, %2;\n\t cvt.f32.f16 %0, a;\n\t cvt.f32.f16 %1, b; }"
                        : "=f"(lo), "=f"(hi)
                        : "r"(q[j]));
                    o[4 * h + j] = pack_bf16x2(lo * f, hi * f);
                }
            }
            if (WIDE) {
                st_global_v8(out + (size_t)i * 16, o);
            } else {
                uint4* q = reinterpret_cast<uint4*>(out + (size_t)i * 16);
                q[0] = make_uint4(o[0], o[1], o[2], o[3]);
                q[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
    }
}

// Blocks for `work` block-sized pieces, at most per_sm an SM.  The quantiser
// takes 8 (16 and 64: 46 and 55 us where 8 took 45); the way back, which
// mostly writes, 64 (8 and 16: 49 and 44 us where 64 took 40).
int grid_for(size_t work, int per_sm) {
    static const int sms = device_sm_count();
    return (int)std::min<size_t>(std::max<size_t>(work, 1), (size_t)sms * per_sm);
}

template <typename T>
cudaError_t quant(const T* x, size_t ldx, int rows, int n, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
    const uint32_t pieces = (uint32_t)ceil_div(n, 512), total = (uint32_t)rows * pieces;
    const dim3 grid(grid_for((total + 7) / 8, 8)), block(256);
    const bool wide = (reinterpret_cast<uintptr_t>(x) % 32) == 0 && ldx * sizeof(T) % 32 == 0;
    return launch_pdl(wide ? mx_quant<T, true> : mx_quant<T, false>, grid, block, 0, st, x, ldx, total, pieces, n,
                      ceil_div(n, 128), codes, scales);
}

}  // namespace

cudaError_t launch_mx_quant(const void* x, bool f32, size_t ldx, int rows, int n, uint8_t* codes, uint8_t* scales,
                            cudaStream_t st) {
    return f32 ? quant(static_cast<const float*>(x), ldx, rows, n, codes, scales, st)
               : quant(static_cast<const uint16_t*>(x), ldx, rows, n, codes, scales, st);
}

cudaError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int rows, int n, uint16_t* out,
                              cudaStream_t st) {
    const uint32_t per = (uint32_t)(n / 16), total = (uint32_t)rows * per;
    const bool wide = reinterpret_cast<uintptr_t>(out) % 32 == 0;
    return launch_pdl(wide ? mx_dequant<true> : mx_dequant<false>, dim3(grid_for(((size_t)total + 255) / 256, 64)), dim3(256), 0, st, codes, scales, total,
                      per, ceil_div(n, 128), out);
}

}  // namespace moe

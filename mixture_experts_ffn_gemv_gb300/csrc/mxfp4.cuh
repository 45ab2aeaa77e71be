// MXFP4 helpers: e2m1 codes with one e8m0 scale per 32 elements, and the
// packed order of the scales (include/moe_ffn_block.h states the format).
#pragma once

#include <stdint.h>

namespace moe {

// Scale byte of a block from the bits of its largest magnitude: with f the
// exponent field of a, floor(log2 a) = f - 127, so s = f - 2, not below 0
// (which covers zero and subnormal a); an infinity or NaN (f = 255) gives 255.
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax_bits) {
    const uint32_t f = amax_bits >> 23;
    return f == 255u ? 255u : (f < 2u ? 0u : f - 2u);
}
// The larger of two magnitudes; a NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// 2^(127 - s): v times it is v / 2^(s - 127), exact for every value that does
// not underflow far below e2m1's smallest midpoint.  0 for a NaN scale, so
// that finite elements of such a block give zero codes.
__device__ __forceinline__ float mx_inverse(uint32_t s) { return s == 255u ? 0.f : __uint_as_float((254u - s) << 23); }

// Eight e2m1 codes of v[0..8) * r, element 0 in the low nibble; round to
// nearest even, saturating at +-6.
__device__ __forceinline__ uint32_t mx_codes8(const float* v, float r) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(v[0] * r), "f"(v[1] * r), "f"(v[2] * r), "f"(v[3] * r), "f"(v[4] * r), "f"(v[5] * r), "f"(v[6] * r),
          "f"(v[7] * r));
    return w;
}

// Four of them, in 16 bits.
__device__ __forceinline__ uint32_t mx_codes4(const float* v, float r) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "mov.b32 %0, {b0, b1, b0, b1};\n\t}"
        : "=r"(w)
        : "f"(v[0] * r), "f"(v[1] * r), "f"(v[2] * r), "f"(v[3] * r));
    return w & 0xffffu;
}

// Byte of the scale of row r, block b; nkt = ceil(blocks / 4) tiles per row.
__host__ __device__ __forceinline__ size_t mx_scale_at(size_t r, size_t b, size_t nkt) {
    return ((r >> 7) * nkt + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

}  // namespace moe

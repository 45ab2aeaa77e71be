// Pairs of fp32 in one instruction.
#pragma once
#include <cstdint>

namespace moe {

struct Pair {
    float x, y;
};
__device__ __forceinline__ uint64_t bits(Pair p) { return __double_as_longlong(__hiloint2double(__float_as_int(p.y), __float_as_int(p.x))); }
__device__ __forceinline__ Pair pair(uint64_t v) {
    Pair p;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(p.x), "=f"(p.y) : "l"(v));
    return p;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair(r);
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return pair(r);
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair(r);
}

}  // namespace moe

// fd_packed.cuh -- arithmetic on packed numbers: two fp32 numbers in a 64-bit register
// (one instruction for both), and int8 codes to bf16.
#pragma once

#include <stdint.h>

namespace fd {

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Four int8 codes (the bytes of w) -> four bf16 numbers, exactly: with c's low
// seven bits as the mantissa of 128 + (c & 127), less 128, or 256 where c's sign
// bit is set.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    const uint32_t lo = __byte_perm(w, 0x43434343u, 0x4140), hi = __byte_perm(w, 0x43434343u, 0x4342);
    uint2 r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r.x) : "r"(lo & 0xff7fff7fu), "r"(lo & 0xff80ff80u));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r.y) : "r"(hi & 0xff7fff7fu), "r"(hi & 0xff80ff80u));
    return r;
}

}  // namespace fd

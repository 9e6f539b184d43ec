// fd_fp4.cuh -- the 4-bit cache format on the device, shared by the kernels
// that read it (fd_fp4_decode.cuh, fd_fp4_rows.cu) and the one that writes it.
//
// A row of d values is d/2 bytes of e2m1 codes (value 2j in byte j's low
// nibble, 2j+1 in its high one) and d/16 e4m3 scales, one per 16 consecutive
// values; a value is code * scale * g with one fp32 factor g per call.
// code * scale has at most 2 + 4 significant bits and lies within
// [2^-10, 2688] in magnitude (or is 0), so it is exact in fp16 and in bf16.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace fd {
namespace fp4 {

constexpr int kGroup = 16;   // values that share a scale

// The four bytes of w (two codes each) -> four fp16 pairs, low nibble in the
// low half.  One conversion instruction per pair, no bit moves.
__device__ __forceinline__ void codes_to_f16x2(uint32_t w, uint32_t &p0, uint32_t &p1,
                                               uint32_t &p2, uint32_t &p3) {
    asm("{\n\t.reg .b8 a, b, c, e;\n\t"
        "mov.b32 {a, b, c, e}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, e;\n\t}"
        : "=r"(p0), "=r"(p1), "=r"(p2), "=r"(p3)
        : "r"(w));
}

// Two e4m3 scales (low 16 bits of w) -> one fp16 pair (exact).
__device__ __forceinline__ uint32_t scales_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// (hi, lo) -> fp16 pair, lo in the low half.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace fp4
}  // namespace fd

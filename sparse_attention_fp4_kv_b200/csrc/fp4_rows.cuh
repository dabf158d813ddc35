// FP4 rows to 16-bit values, for the paged cache's readers (paged_attn.cuh,
// paged_kv.cu).
#pragma once

#include "common.cuh"

namespace csa2 {

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(0x80008000u));
    return r;
}
// Eight codes -> four pairs of f16 values of E2M1.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n.reg .b8 b0, b1, b2, b3;\nmov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\ncvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\ncvt.rn.f16x2.e2m1x2 %3, b3;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// f16 rows: eight codes times an E4M3 scale (splat in s).
__device__ __forceinline__ uint4 rows_f16(uint32_t w, uint32_t s) {
    uint32_t h[4];
    e2m1x8_to_f16(w, h);
    return make_uint4(mul_f16x2(h[0], s), mul_f16x2(h[1], s), mul_f16x2(h[2], s), mul_f16x2(h[3], s));
}
// bf16 rows: eight codes times 2^(E - 127). The f16 bits of an E2M1 value moved
// down by three are the bf16 value times 2^-112 (all its mantissa bits are zero
// but the top one), so one product with 2^(E - 15) ends it; a scale above
// 2^15, where that factor leaves bf16's range, takes a second one.
struct MxScale {
    uint32_t first, second;
};
__device__ __forceinline__ MxScale mx_scale(uint32_t E) {
    // 2^(E - 15) as bf16, from the exponent field E + 112 (E <= 142)
    const uint32_t e1 = E < 142u ? E : 142u;
    const uint32_t f = (e1 + 112u) << 7, s = (E - e1 + 127u) << 7;
    MxScale m{f | f << 16, s | s << 16};
    if (E == 255u) m.second = 0x7FC07FC0u;  // NaN
    return m;
}
__device__ __forceinline__ uint4 rows_bf16(uint32_t w, MxScale s) {
    uint32_t h[4];
    e2m1x8_to_f16(w, h);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        h[i] = ((h[i] >> 3) & 0x0FFF0FFFu) | (h[i] & 0x80008000u);
        h[i] = mul_bf16x2(h[i], s.first);
        if (s.second != 0x3F803F80u) h[i] = mul_bf16x2(h[i], s.second);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}
// The same for an E4M3 scale: s 2^112 is a bf16 value, the product exact.
__device__ __forceinline__ MxScale e4m3_scale(uint32_t code) {
    const uint32_t f = __float_as_uint(e4m3_to_f32(code) * 0x1p112f) >> 16;
    return MxScale{f | f << 16, 0x3F803F80u};
}

}  // namespace csa2

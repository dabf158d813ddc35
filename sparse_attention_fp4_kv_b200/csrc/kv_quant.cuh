// FP4 quantization of one scale group, shared by the contiguous and the paged
// append (kv_append.cu, paged_kv.cu): the two write the same bytes.
#pragma once

#include "common.cuh"

namespace csa2 {

// A value with the E2M1 code of the IEEE quotient x / s, for bf16 x, an E4M3 s and
// inv = 1 / s (fp32). The code asks on which side of a tie t (0.25 .75 1.25 1.75 2.5
// 3.5 5) the quotient lies, or whether it is one. x has 8 significant bits, s 4 and t
// 3, so a quotient that is not t is off it by 1 part in 255 at least; x * inv is
// off by 2^-23. Rounded to 16 significant bits it is t where the quotient is, and
// on the quotient's side where it is not: a product, two clamps (which make NaN 8,
// as the conversion does) and two integer steps, a third of a division's cost.
__device__ __forceinline__ float quotient_for_e2m1(float x, float inv) {
    const float q = fmaxf(fminf(x * inv, 8.0f), -8.0f);
    return __uint_as_float((__float_as_uint(q) + 0x80u) & ~0xFFu);
}

// 16 channels (two 16-byte loads of bf16) -> eight packed code bytes and the
// E4M3 scale code: s = E4M3(amax / 6) by IEEE division, code = E2M1(x / s), +0
// where s is 0.
__device__ __forceinline__ uint2 fp4_quant16(uint4 a, uint4 c, uint32_t &scode) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
    float x[16];
#pragma unroll
    for (int j = 0; j < 8; j++) {
        x[2 * j] = bf16_lo(w[j]);
        x[2 * j + 1] = bf16_hi(w[j]);
    }
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; j++) amax = fmaxf(amax, fabsf(x[j]));

    scode = f32_to_e4m3_satfinite(__fdiv_rn(amax, 6.0f));
    const float s = e4m3_to_f32(scode);
    uint32_t lo = 0, hi = 0;
    if (s != 0.0f) {
        const float inv = __fdiv_rn(1.0f, s);
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; j++) v[j] = quotient_for_e2m1(x[j], inv);
        lo = f32x8_to_e2m1x8(v);
        hi = f32x8_to_e2m1x8(v + 8);
    }
    return make_uint2(lo, hi);
}

// MXFP4: 32 channels (four 16-byte loads) -> 16 code bytes and the E8M0 code.
// The shared exponent is the exponent of the block's amax minus 2 (the largest
// E2M1 exponent), clamped to the E8M0 range: read straight from the fp32
// exponent field, so an all-zero or subnormal amax gives 2^-127. Elements are
// x * 2^-e, an exact scaling since the result stays below 8, then the same
// E2M1 pair conversion.
__device__ __forceinline__ uint4 mxfp4_quant32(const uint4 (&a)[4], uint32_t &scode) {
    float x[32];
#pragma unroll
    for (int q = 0; q < 4; q++) {
        const uint32_t w[4] = {a[q].x, a[q].y, a[q].z, a[q].w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            x[8 * q + 2 * j] = bf16_lo(w[j]);
            x[8 * q + 2 * j + 1] = bf16_hi(w[j]);
        }
    }
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 32; j++) amax = fmaxf(amax, fabsf(x[j]));
    const int E = (int)((__float_as_uint(amax) >> 23) & 0xFF);  // 0 for zero / subnormal
    int e = E == 0 ? -127 : E - 129;
    e = e < -127 ? -127 : e;
    // 2^-e as an fp32: e lies in [-127, 126], so 2^-e is a normal number
    // (2^-126 .. 2^127)
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; j++) v[j] = x[j] * inv;
    scode = (uint32_t)(e + 127);
    return make_uint4(f32x8_to_e2m1x8(v), f32x8_to_e2m1x8(v + 8), f32x8_to_e2m1x8(v + 16),
                      f32x8_to_e2m1x8(v + 24));
}

}  // namespace csa2

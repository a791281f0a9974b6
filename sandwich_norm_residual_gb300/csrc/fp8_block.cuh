// E4M3 codes with one FP32 scale for each 128 values of a row, 8 values a lane: a block is
// half a warp.
//
//   amax = max |v|,  scale = RN32(amax / 448),  code = E4M3(RN32(v * RN32(448 / amax)))
//
// E4M3 is OCP E4M3FN (largest 448, no infinity), rounded to nearest even, saturating: v
// times the inverse can lie a unit of 2^-23 above 448. A block of zeros gets codes and
// scale 0. A block that holds a NaN or an infinity gets codes 0 and that scale, so that
// what is multiplied with it is NaN. Below 2^-100 the values are first brought up by 2^64
// (exact), where 448 / amax does not overflow.
#pragma once

#include "packed.cuh"

namespace beam {

constexpr int kFp8Block = 128;

// four FP32 -> four E4M3 codes, the first in the lowest byte
__device__ __forceinline__ uint32_t f4_to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{ .reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi}; }"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// the largest of `bits` over this lane's half of the warp (every lane calls). Sign-free
// FP32 bits order like the numbers they stand for, infinity above every finite value and
// NaN above that: an integer maximum keeps a NaN.
__device__ __forceinline__ uint32_t half_warp_max(uint32_t bits) {
#pragma unroll
    for (int off = 8; off; off >>= 1) bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, off));
    return bits;
}

// RN32(a / 448) for 2^-100 <= a < inf in three operations instead of an IEEE division: t = RN(a c)
// with c = RN(1 / 448) is within an ulp of a / 448, r = a - 448 t is exact in one multiply-add,
// and t + r c rounds correctly (Markstein's theorem, for c the reciprocal rounded to nearest). Checked for every
// significand. An infinite t is returned as it is, a NaN too.
__device__ __forceinline__ float div448(float a) {
    const float c = 0x1.24924ap-9f;
    const float t = __fmul_rn(a, c);
    const float q = __fmaf_rn(__fmaf_rn(-t, 448.0f, a), c, t);
    return t < INFINITY ? q : t;
}

// codes of the eight values that a lane holds of a block with this amax; the block's scale
__device__ __forceinline__ uint2 fp8_codes(const float2 (&v)[4], float amax, float* scale) {
    float2 q[4] = {v[0], v[1], v[2], v[3]};
    // whatever comes out for zeros, infinities and NaN is masked
    const uint32_t live = amax > 0.0f && amax < INFINITY ? 0xFFFFFFFFu : 0u;
    if (amax < 0x1p-100f) {
        *scale = __fdiv_rn(amax, 448.0f);
        amax *= 0x1p+64f;
        const float2 up = make_float2(0x1p+64f, 0x1p+64f);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = mul2_rn(q[i], up);
    } else {
        *scale = div448(amax);
    }
    const float inv = __fdiv_rn(448.0f, amax);
    const float2 i2 = make_float2(inv, inv);
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = mul2_rn(q[i], i2);
    return make_uint2(f4_to_e4m3x4(q[0].x, q[0].y, q[1].x, q[1].y) & live, f4_to_e4m3x4(q[2].x, q[2].y, q[3].x, q[3].y) & live);
}

}  // namespace beam

// Pairs: two BF16 in a word, two FP32 in packed f32x2 arithmetic.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace beam {

// two BF16 (low half = lower column) -> two FP32, exactly
__device__ __forceinline__ float2 bf2_to_f2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// two FP32 -> two BF16, round to nearest even (NaN -> canonical NaN)
__device__ __forceinline__ uint32_t f2_to_bf2(float2 v) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(v.y), "f"(v.x));
    return d;
}

// Packed FP32 pairs in hand-written PTX with explicit .rn rounding. The
// explicit modifier is meant to keep a multiply and a following add as two
// roundings, yet a packed add fed by a packed product was measured to fuse into
// an FMA on sm_103a. So a packed add here only ever takes products that are
// exact in FP32 (squares of BF16 values), where a fused and a separately
// rounded sum give the same bits; products that are not exact feed
// conversions, or scalar __fadd_rn / __fsub_rn, which are never contracted.
#define BEAM_F32X2_OP(NAME, OP)                                                                  \
    __device__ __forceinline__ float2 NAME(float2 a, float2 b) {                                 \
        float2 d;                                                                                \
        asm("{\n\t.reg .b64 ra, rb, rd;\n\t"                                                    \
            "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t" OP " rd, ra, rb;\n\t"          \
            "mov.b64 {%0, %1}, rd;\n\t}"                                                          \
            : "=f"(d.x), "=f"(d.y)                                                               \
            : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));                                          \
        return d;                                                                                \
    }
BEAM_F32X2_OP(mul2_rn, "mul.rn.f32x2")
BEAM_F32X2_OP(add2_rn, "add.rn.f32x2")
BEAM_F32X2_OP(sub2_rn, "sub.rn.f32x2")
#undef BEAM_F32X2_OP

}  // namespace beam

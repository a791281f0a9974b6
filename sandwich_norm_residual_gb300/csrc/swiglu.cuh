// The experts' activation, written as the FP8 operand of the product behind it:
//   y = g / (1 + e^-g) * u,  then E4M3 codes with a scale for each 128 (fp8_block.cuh)
// Half a warp has a block, 8 values a lane, 16 bytes of gate and of up each. Bound by HBM: 4
// bytes read and 1.03 written for a value. e^-g and the quotient are the special-function
// unit's base-2 exponential and reciprocal (2 units of 2^-24 and the argument's rounding, 1.44 |g| units): the
// library's expf and division are 30 more instructions a value, which at HBM's rate do
// not fit in.
#pragma once

#include "fp8_block.cuh"

namespace beam {

constexpr int kSwigluThreads = 256;

struct SwigluParams {
    const uint16_t* x;        // [R, 2 F] BF16: gate, up
    uint8_t* y;               // [R, F]
    float* scale;             // [R, ceil(F / 128)]
    const int32_t* live;      // rows that count, or NULL: all R
    long long R;
    int F, blocks, chunks;    // blocks of 128, chunks of 256 of a row
    unsigned int* status;
};

__device__ __forceinline__ float swiglu(float g, float u) {
    float t, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(t) : "f"(__fmul_rn(g, -1.4426950408889634f)));
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, t)));
    return __fmul_rn(__fmul_rn(g, r), u);
}

__global__ void __launch_bounds__(kSwigluThreads) swiglu_fp8_kernel(const SwigluParams p) {
    const int lane = threadIdx.x & 31;
    long long rows = p.R;
    if (p.live) {
        rows = __ldg(p.live);
        if (rows < 0 || rows > p.R) {
            if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, 2u);
            rows = rows < 0 ? 0 : p.R;
        }
    }
    const long long todo = rows * p.chunks, stride = (long long)gridDim.x * (kSwigluThreads / 32);
    for (long long w = (long long)blockIdx.x * (kSwigluThreads / 32) + (threadIdx.x >> 5); w < todo; w += stride) {
        const long long row = w / p.chunks;
        const int at = (int)(w - row * p.chunks) * 256 + lane * 8;
        const bool in = at < p.F;
        uint4 g = make_uint4(0, 0, 0, 0), u = g;
        if (in) {
            const uint16_t* x = p.x + (size_t)row * (size_t)(2 * (long long)p.F) + at;
            g = __ldg(reinterpret_cast<const uint4*>(x));
            u = __ldg(reinterpret_cast<const uint4*>(x + p.F));
        }
        const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
        float2 y[4];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = bf2_to_f2(gw[i]), b = bf2_to_f2(uw[i]);
            y[i] = make_float2(swiglu(a.x, b.x), swiglu(a.y, b.y));
            top = max(top, max(__float_as_uint(y[i].x) & 0x7FFFFFFFu, __float_as_uint(y[i].y) & 0x7FFFFFFFu));
        }
        float scale;
        const uint2 c = fp8_codes(y, __uint_as_float(half_warp_max(top)), &scale);
        if (in) {
            *reinterpret_cast<uint2*>(p.y + (size_t)row * (size_t)p.F + at) = c;
            if ((lane & 15) == 0) p.scale[(size_t)row * (size_t)p.blocks + at / 128] = scale;
        }
    }
}

}  // namespace beam

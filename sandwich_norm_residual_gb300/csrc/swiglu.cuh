// The experts' activation, written as the FP8 operand of the product behind it:
//   y = g / (1 + e^-g) * u,  then E4M3 codes with a scale for each 128 (fp8_block.cuh)
// Half a warp has a block, 8 values a lane, 16 bytes of gate and of up each. Bound by HBM: 4
// bytes read and 1.03 written for a value, if not by the instructions. e^-g and the quotient are the
// special-function unit's base-2 exponential and reciprocal (within 2^-22 and 2^-23, relative): the library's
// expf and division are 30 more instructions a value. In units of 2^-24, with w = 1 / (1 + e^g): the argument's
// rounding and its constant's 1.22 |g| w, the exponential 4 w, 1 + e^-g 1, the reciprocal 2, two products 1 each, in all at
// most 8 + 2 |g|.
// The reciprocal unit flushes results below 2^-126, that is from g = -87.4 down. So it is given (1 + e^-g) 2^-32, one
// multiply-add, and its result brought back down by a product that rounds below 2^-126 to a multiple of 2^-149 (up to 4
// units more). From g = -88.73 down e^-g is infinite and y 0. The exponential flushes e^-g below 2^-126, which is added to 1.
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

// read once
__device__ __forceinline__ uint4 ld_swiglu(const uint16_t* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// two values
__device__ __forceinline__ float2 swiglu2(float2 g, float2 u) {
    const float2 down = make_float2(0x1p-32f, 0x1p-32f);
    const float2 x = mul2_rn(g, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    float2 t, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(x.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(x.y));
    const float2 d = __ffma2_rn(t, down, down);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
    return mul2_rn(mul2_rn(g, mul2_rn(r, down)), u);
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
    // Pieces of 256 values: warp w takes w, w + warps, ... Row and piece go on by steps that are
    // divided out once (a 64-bit division for every piece took half of the time).
    const uint32_t first = blockIdx.x * (kSwigluThreads / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kSwigluThreads / 32);
    const uint32_t row_step = warps / p.chunks, chunk_step = warps % p.chunks;
    long long row = first / p.chunks;
    uint32_t chunk = first % p.chunks;
    for (; row < rows;) {
        const int at = (int)chunk * 256 + lane * 8;
        const bool in = at < p.F;
        uint4 g = make_uint4(0, 0, 0, 0), u = g;
        if (in) {
            const uint16_t* x = p.x + (size_t)row * (size_t)(2 * (long long)p.F) + at;
            g = ld_swiglu(x);
            u = ld_swiglu(x + p.F);
        }
        const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
        float2 y[4];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i] = swiglu2(bf2_to_f2(gw[i]), bf2_to_f2(uw[i]));
            top = max(top, max(__float_as_uint(y[i].x) & 0x7FFFFFFFu, __float_as_uint(y[i].y) & 0x7FFFFFFFu));
        }
        float scale;
        const uint2 c = fp8_codes(y, __uint_as_float(half_warp_max(top)), &scale);
        if (in) {
            *reinterpret_cast<uint2*>(p.y + (size_t)row * (size_t)p.F + at) = c;
            if ((lane & 15) == 0) p.scale[(size_t)row * (size_t)p.blocks + at / 128] = scale;
        }
        row += row_step;
        chunk += chunk_step;
        if (chunk >= (uint32_t)p.chunks) {
            chunk -= p.chunks;
            ++row;
        }
    }
}

}  // namespace beam

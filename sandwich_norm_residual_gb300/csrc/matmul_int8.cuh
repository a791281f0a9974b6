// Product of 8-bit integers with a scale per token and per channel:
//   out[m, n] = ((float)(sum_k a[m, k] w[n, k]) * a_scale[m]) * w_scale[n]
// FP32 products in that order, then one rounding when out is BF16.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "tma.cuh"

namespace beam {

struct MatmulParams {
    const int8_t* a;       // [M, K] tokens
    const float* a_scale;  // [M]
    const int8_t* w;       // [N, K] channels
    const float* w_scale;  // [N]
    void* out;             // [M, N] BF16 or FP32
    long long M;
    int N, K;
};

// one element of out
template <bool F32>
__device__ __forceinline__ void store_out(void* out, size_t at, float v) {
    if (F32) {
        static_cast<float*>(out)[at] = v;
    } else {
        unsigned short b;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(v));
        static_cast<unsigned short*>(out)[at] = b;
    }
}

__device__ __forceinline__ uint4 ld_weights(const int8_t* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p), "l"(l2_evict_first()));
    return r;
}

// ---------------------------------------------------------------- few tokens

// Up to MB tokens by R channels a warp, on the integer dot product: the lanes take
// 16 bytes each of 512 consecutive k, U such steps of the R weight rows in flight
// at once. Every weight byte is read once, and sums are exact in 32 bits. One token is
// bound by the weights' way from HBM: M = 1, N = 6144, K = 5120: 6.5 us, of which 2.2
// are the launch; the weights alone take 4.7 us at the copy rate. More tokens are not:
// each costs every warp its rows again (through L1) and one dp4a for four weights, and
// their sums leave registers for fewer weights in flight (M = 8: 11.2 us).
constexpr int kFewWarps = 8;

template <int MB, int R, int U, bool F32>
__global__ void __launch_bounds__(32 * kFewWarps) matmul_int8_few_kernel(const MatmulParams p) {
    const int lane = threadIdx.x & 31;
    const long long n0 = ((long long)blockIdx.x * kFewWarps + (threadIdx.x >> 5)) * R;
    pdl_trigger();
    if (n0 >= p.N) {
        pdl_wait();
        return;
    }
    const int8_t* wr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) wr[r] = p.w + (size_t)min(n0 + r, (long long)p.N - 1) * (size_t)p.K;
    const int8_t* ar[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) ar[m] = p.a + (size_t)min((long long)m, p.M - 1) * (size_t)p.K;
    int acc[MB][R];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[m][r] = 0;

    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 wv[U][R];
    auto load = [&](int k0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r) wv[u][r] = k0 + u * 512 < p.K ? ld_weights(wr[r] + k0 + u * 512) : zero;
    };
    // the first weights do not depend on the kernel before: asked for ahead of the wait
    load(lane * 16);
    pdl_wait();
    for (int k0 = lane * 16; k0 - lane * 16 < p.K; k0 += 512 * U) {
        if (k0 >= 512 * U) load(k0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * 512;
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                const uint4 av = k < p.K ? __ldg(reinterpret_cast<const uint4*>(ar[m] + k)) : zero;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    int s = acc[m][r];
                    s = __dp4a((int)wv[u][r].x, (int)av.x, s);
                    s = __dp4a((int)wv[u][r].y, (int)av.y, s);
                    s = __dp4a((int)wv[u][r].z, (int)av.z, s);
                    acc[m][r] = __dp4a((int)wv[u][r].w, (int)av.w, s);
                }
            }
        }
    }
    // lane m * R + r writes element (m, r)
    int mine = 0;
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int s = __reduce_add_sync(0xFFFFFFFFu, acc[m][r]);
            if (lane == m * R + r) mine = s;
        }
    const long long m = lane / R, n = n0 + lane % R;
    if (lane < MB * R && m < p.M && n < p.N)
        store_out<F32>(p.out, (size_t)m * (size_t)p.N + (size_t)n,
                       __fmul_rn(__fmul_rn((float)mine, __ldg(p.a_scale + m)), __ldg(p.w_scale + n)));
}

}  // namespace beam

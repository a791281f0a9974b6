// The product of matmul_fp8.cuh for single tokens: a few rows of channels for each warp,
// multiplied in FP32 on the plain cores.
//
// It is the weights' way from HBM that counts, and the time until it is in full flow: no
// tensor maps, no ring, no join. A lane takes 16 bytes of a channel at a time, which lie
// within one block of 128: their products are added in FP32 (FP16 holds every E4M3 number
// exactly), scaled by RN(a_scale w_scale) and added to the lane's sum; the lanes' sums are
// added at the end.
// M = 1, K = 5120: N = 6144 8.3 us and N = 20480 21.4 us, where the tensor cores' tiles take 13.8 and
// 30. Two tokens at a time took 13 us for N = 6144, no less than those: turning codes into FP32
// bounds it then.
#pragma once

#include "matmul_fp8.cuh"

namespace beam {

constexpr int kFp8DotWarps = 8;

// sixteen E4M3 codes -> FP32, exactly
__device__ __forceinline__ void e4m3x16_to_f32(const uint4& v, float2 (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{ .reg .b16 a, b, x, y, z, t; .reg .b32 lo, hi;\n\t"
            "mov.b32 {a, b}, %4;\n\t"
            "cvt.rn.f16x2.e4m3x2 lo, a;\n\tcvt.rn.f16x2.e4m3x2 hi, b;\n\t"
            "mov.b32 {x, y}, lo;\n\tmov.b32 {z, t}, hi;\n\t"
            "cvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\tcvt.f32.f16 %2, z;\n\tcvt.f32.f16 %3, t; }"
            : "=f"(f[2 * i].x), "=f"(f[2 * i].y), "=f"(f[2 * i + 1].x), "=f"(f[2 * i + 1].y) : "r"(w[i]));
}

__device__ __forceinline__ uint4 ld_fp8_weights(const uint8_t* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p), "l"(l2_evict_first()));
    return r;
}

struct Fp8DotParams {
    const uint8_t* a;
    const uint8_t* w;
    Fp8Params q;
    int K;
};

// CH channels a warp, two times 512 k of them on their way
template <int CH, int BLOCKS, bool F32>
__global__ void __launch_bounds__(32 * kFp8DotWarps, BLOCKS) matmul_fp8_dot_kernel(const __grid_constant__ Fp8DotParams p) {
    constexpr int U = 2;
    const Fp8Params& q = p.q;
    const int lane = threadIdx.x & 31;
    const long long n0 = ((long long)blockIdx.x * kFp8DotWarps + (threadIdx.x >> 5)) * CH;
    int e = 0;
    long long lo = 0, hi = q.R;
    if (q.offsets) {
        // blocks [., y] have the y-th expert that has rows; nobody where an offset decreases or leaves [0, R]
        int left = blockIdx.y;
        bool bad = false;
        e = -1;
        for (int base = 0; base < q.E; base += 32) {
            const int i = base + lane;
            long long b = 0, c = 0;
            if (i < q.E) {
                b = __ldg(q.offsets + i);
                c = __ldg(q.offsets + i + 1);
                bad |= b < 0 || c < b || c > q.R;
            }
            const unsigned some = __ballot_sync(0xFFFFFFFFu, c > b);
            const int n = __popc(some);
            if (e < 0 && left < n) {
                const int at = __fns(some, 0, left + 1);
                e = base + at;
                lo = __shfl_sync(0xFFFFFFFFu, b, at);
                hi = __shfl_sync(0xFFFFFFFFu, c, at);
            }
            left -= n;
        }
        if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(q.status, 2u);
        if (__any_sync(0xFFFFFFFFu, bad) || e < 0) return;
    }
    if (n0 >= q.N) return;
    const uint8_t* wr[CH];
#pragma unroll
    for (int r = 0; r < CH; ++r) wr[r] = p.w + ((size_t)e * (size_t)q.N + (size_t)min(n0 + r, (long long)q.N - 1)) * (size_t)p.K;
    // a warp's channels are neighbours, CH divides 128: one block of scales
    const float* const ws = q.w_scale + ((size_t)e * (size_t)((q.N + 127ll) / 128) + (size_t)(n0 / 128)) * q.steps;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (long long m = lo; m < hi; ++m) {
        const uint8_t* const ar = p.a + (size_t)m * (size_t)p.K;
        const float* const as = q.a_scale + (size_t)m * q.steps;
        float acc[CH] = {};
        for (int k0 = lane * 16; k0 - lane * 16 < p.K; k0 += 512 * U) {
            uint4 wv[U][CH];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < CH; ++r) wv[u][r] = k0 + u * 512 < p.K ? ld_fp8_weights(wr[r] + k0 + u * 512) : zero;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * 512;
                if (k >= p.K) continue;
                const float s = __fmul_rn(__ldg(as + k / 128), __ldg(ws + k / 128));
                float2 av[8];
                e4m3x16_to_f32(__ldg(reinterpret_cast<const uint4*>(ar + k)), av);
#pragma unroll
                for (int r = 0; r < CH; ++r) {
                    float2 wf[8], d = make_float2(0.f, 0.f);
                    e4m3x16_to_f32(wv[u][r], wf);
#pragma unroll
                    for (int i = 0; i < 8; ++i) d = __ffma2_rn(wf[i], av[i], d);
                    acc[r] = __fmaf_rn(s, __fadd_rn(d.x, d.y), acc[r]);
                }
            }
        }
        // lane r writes channel r
        float mine = 0.f;
#pragma unroll
        for (int r = 0; r < CH; ++r) {
            float v = acc[r];
#pragma unroll
            for (int off = 16; off; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
            if (lane == r) mine = v;
        }
        if (lane < CH && n0 + lane < q.N)
            static_cast<Fp8Out<F32>*>(q.out)[(size_t)m * (size_t)q.N + (size_t)(n0 + lane)] = fp8_round<F32>(mine);
    }
}

}  // namespace beam

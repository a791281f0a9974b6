// The product of matmul_fp8.cuh for 8 or 16 tokens at a time: warp matrix instructions on rows of
// channels that go from memory straight to registers.
//
// It is the weights' way from HBM that counts, and the time until it is in full flow: no tensor
// maps, no ring, no tensor memory to set up. A block has 16 channels and up to 8 or 16 tokens; its
// warps take the blocks of 128 k in turn, two of each warp's on their way (one for 16 tokens), and
// add up at the end, in the order of the warps. The instruction wants 4 neighbours of k in a register; which k they
// are is free as long as channels and tokens agree, so a lane loads 16 neighbours of a row and uses
// them in two instructions.
//   P_b = four instructions' sum from 0, times RN(a_scale w_scale), added to the warp's sum
// M = 1 to 8, K = 5120: N = 6144 7.9 to 8.1 us and N = 20480 20.3 us (5.2 TB/s), where the tiles of 128
// channels take 14.9 and 28; M = 5, N = 2560, K = 1280: 2.7 and 7.9 us. Plain FP32 multiply-adds of
// a single token took 9.8 and 22.7 us: turning codes into FP32 takes as long as their way. What is left
// over the floor is the way in and out of blocks that live 5 to 10 us; asking L2 ahead made it
// slower by a tenth, the next block of k ahead of the present one's products no faster.
// 16 tokens: N = 6144 10.0 and 14.9 us, N = 2560, K = 1280 4.2 and 7.9; 32 at a time took 17.6 and 15.4.
#pragma once

#include "matmul_fp8.cuh"

namespace beam {

constexpr int kFp8SmallChannels = 16;

// c += 16 channels by 8 tokens over 32 k, E4M3 with FP32 sums. Lane l: channels l / 4 (a0, a2)
// and l / 4 + 8 (a1, a3), token l / 4; c: channels l / 4 and l / 4 + 8 by tokens 2 (l % 4) and the next
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld_fp8_weights(const uint8_t* p, uint64_t policy) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p), "l"(policy));
    return r;
}

struct Fp8SmallParams {
    const uint8_t* a;
    const uint8_t* w;
    Fp8Params q;
    int K;
};

// What part `y` of the experts' rows is: the y-th expert with rows, its first TOK of them, or, behind those, what experts
// have more, TOK each; false: there is none. The whole warp; a lane has EACH neighbouring experts. Nobody has any where an
// offset decreases or leaves [0, R].
template <int TOK, int EACH>
__device__ __forceinline__ bool fp8_small_part(const Fp8Params& q, int y, int lane, int* e, int* lo, int* hi, bool* alone) {
    static_assert(kFp8SmallRows < 1 << 16, "two counts in a word");
    int at[EACH + 1];
#pragma unroll
    for (int j = 0; j <= EACH; ++j) at[j] = __ldg(q.offsets + min(lane * EACH + j, q.E));
    bool bad = at[0] < 0;
    uint32_t mine = 0;  // experts with rows; above 16 bits their parts besides the first (R <= 512)
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        bad |= at[j + 1] < at[j] || at[j + 1] > q.R;
        const uint32_t n = (uint32_t)at[j + 1] - (uint32_t)at[j];
        if (n) mine += 1u + ((n - 1u) / TOK << 16);
    }
    if (bad && blockIdx.x == 0 && y == 0) atomicOr(q.status, 2u);
    if (__any_sync(0xFFFFFFFFu, bad)) return false;
    uint32_t upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, off);
        if (lane >= off) upto += v;
    }
    const uint32_t all = __shfl_sync(0xFFFFFFFFu, upto, 31), live = all & 0xFFFFu;
    const bool rest = (uint32_t)y >= live;
    const uint32_t want = rest ? (uint32_t)y - live : (uint32_t)y, shift = rest ? 16u : 0u;
    if (rest && want >= all >> 16) return false;
    const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, ((upto >> shift) & 0xFFFFu) > want)) - 1;
    int k = (int)(want - (((upto - mine) >> shift) & 0xFFFFu));  // in the owner's lane: of its parts
    int found = 0, from = 0, to = 0;
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        const int n = at[j + 1] - at[j], parts = n == 0 ? 0 : rest ? (n - 1) / TOK : 1;
        if (k >= 0 && k < parts) {
            found = lane * EACH + j;
            from = at[j] + (rest ? TOK * (k + 1) : 0);
            to = at[j + 1];
        }
        k -= parts;
    }
    *e = __shfl_sync(0xFFFFFFFFu, found, owner);
    *lo = __shfl_sync(0xFFFFFFFFu, from, owner);
    *hi = __shfl_sync(0xFFFFFFFFu, to, owner);
    *alone = !rest && *hi - *lo <= TOK;
    return true;
}

// NT: eights of tokens. Blocks [., y] have part y of the experts' rows; gridDim.y is as many parts as there can be. So
// however the rows fall, a block reads its channels once: 512 rows of 256 experts, N = 1383, K = 1152, take 86 us if they
// fall alike and 37 us if one expert has them all, whose blocks took 122 us for them in turn.
template <int WARPS, int BLOCKS, int NT, bool F32>
__global__ void __launch_bounds__(32 * WARPS, BLOCKS) matmul_fp8_small_kernel(const __grid_constant__ Fp8SmallParams p) {
    constexpr int U = NT == 1 ? 2 : 1, kTok = kFp8SmallPart * NT;  // blocks of k on their way; tokens at a time
    __shared__ float part[WARPS][kTok][kFp8SmallChannels];
    const Fp8Params& q = p.q;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int n0 = (int)blockIdx.x * kFp8SmallChannels;
    int e = 0, lo = 0, hi = (int)q.R;  // few rows: fp8_small
    bool alone = true;                 // no other block reads these channels
    if (q.offsets) {
        // one warp looks: with many short blocks it is their instructions that count
        __shared__ int4 mine;
        if (warp == 0) {
            const int y = blockIdx.y;
            const bool any = q.E <= 32    ? fp8_small_part<kTok, 1>(q, y, lane, &e, &lo, &hi, &alone)
                             : q.E <= 256 ? fp8_small_part<kTok, 8>(q, y, lane, &e, &lo, &hi, &alone)
                                          : fp8_small_part<kTok, 16>(q, y, lane, &e, &lo, &hi, &alone);
            if (lane == 0) mine = make_int4(any ? e : -1, lo, min(hi, lo + kTok), alone);
        }
        __syncthreads();
        e = mine.x;
        if (e < 0) return;
        lo = mine.y;
        hi = mine.z;
        alone = mine.w;
    }
    const uint64_t policy = alone ? l2_evict_first() : l2_evict_normal();
    const int c0 = min(n0 + g, q.N - 1), c1 = min(n0 + g + 8, q.N - 1);  // channels behind the last are not stored
    const uint8_t* const w0 = p.w + ((size_t)e * (size_t)q.N + (size_t)c0) * (size_t)p.K;
    const uint32_t w1 = (uint32_t)(c1 - c0) * (uint32_t)p.K;
    const float* const ws = q.w_scale + ((size_t)e * fp8_up((uint32_t)q.N, kFp8Block128) + (size_t)(n0 / kFp8Block128)) * q.steps;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const int steps = (int)q.steps;
    // One pass. Without the loop around it the compiler keeps a few words of its steps in memory, and a stack frame costs a
    // launch 0.45 us.
    for (int m = lo; m < hi; m += kTok) {
        const int cols = min(kTok, hi - m);
        const uint8_t* const ar = p.a + (size_t)(m + g) * (size_t)p.K;  // read for g < cols
        const float* const as = q.a_scale + (size_t)(m + 2 * t) * (size_t)steps;
        float sums[NT][4] = {};
        for (int b0 = warp; b0 < steps; b0 += WARPS * U) {
            uint4 wv[U][4], av[U][NT][2];
            float ws_b[U], as_b[U][NT][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (b0 + u * WARPS) * kFp8Step + t * 16;
                const bool in0 = k < p.K, in1 = k + 64 < p.K;
                wv[u][0] = in0 ? ld_fp8_weights(w0 + k, policy) : zero;
                wv[u][1] = in0 ? ld_fp8_weights(w0 + w1 + k, policy) : zero;
                wv[u][2] = in1 ? ld_fp8_weights(w0 + k + 64, policy) : zero;
                wv[u][3] = in1 ? ld_fp8_weights(w0 + w1 + k + 64, policy) : zero;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int b = b0 + u * WARPS, k = b * kFp8Step + t * 16;
                const bool in = b < steps;
                ws_b[u] = in ? __ldg(ws + b) : 0.f;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const uint8_t* const from = ar + (size_t)(8 * i) * (size_t)p.K + k;
                    av[u][i][0] = g + 8 * i < cols && k < p.K ? __ldg(reinterpret_cast<const uint4*>(from)) : zero;
                    av[u][i][1] = g + 8 * i < cols && k + 64 < p.K ? __ldg(reinterpret_cast<const uint4*>(from + 64)) : zero;
                    const float* const sf = as + (size_t)(8 * i) * (size_t)steps + b;
                    as_b[u][i][0] = in && 2 * t + 8 * i < cols ? __ldg(sf) : 0.f;
                    as_b[u][i][1] = in && 2 * t + 8 * i + 1 < cols ? __ldg(sf + steps) : 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (b0 + u * WARPS >= steps) continue;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (8 * i >= cols) break;
                    float c[4] = {};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 &x = wv[u][2 * h], &y = wv[u][2 * h + 1], &z = av[u][i][h];
                        mma_e4m3(c, x.x, y.x, x.y, y.y, z.x, z.y);
                        mma_e4m3(c, x.z, y.z, x.w, y.w, z.z, z.w);
                    }
                    const float s0 = __fmul_rn(as_b[u][i][0], ws_b[u]), s1 = __fmul_rn(as_b[u][i][1], ws_b[u]);
                    sums[i][0] = __fmaf_rn(s0, c[0], sums[i][0]);
                    sums[i][1] = __fmaf_rn(s1, c[1], sums[i][1]);
                    sums[i][2] = __fmaf_rn(s0, c[2], sums[i][2]);
                    sums[i][3] = __fmaf_rn(s1, c[3], sums[i][3]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            part[warp][8 * i + 2 * t][g] = sums[i][0];
            part[warp][8 * i + 2 * t + 1][g] = sums[i][1];
            part[warp][8 * i + 2 * t][g + 8] = sums[i][2];
            part[warp][8 * i + 2 * t + 1][g + 8] = sums[i][3];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < cols * kFp8SmallChannels; i += 32 * WARPS) {
            const int col = i / kFp8SmallChannels, row = i % kFp8SmallChannels;
            if (n0 + row >= q.N) continue;
            float v = part[0][col][row];
#pragma unroll
            for (int j = 1; j < WARPS; ++j) v = __fadd_rn(v, part[j][col][row]);
            static_cast<Fp8Out<F32>*>(q.out)[(size_t)(m + col) * (size_t)q.N + (size_t)(n0 + row)] = fp8_round<F32>(v);
        }
    }
}

}  // namespace beam

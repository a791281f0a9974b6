// The 8-bit integer product on the tensor cores.
//
// GB300's tcgen05 has no integer kind, and its legacy integer path is slow. But
// every int8 is an FP16 number, a product of two is an integer of at most 2^14,
// and FP32 accumulators hold integers below 2^24 exactly: so the FP16 kind at
// its full rate gives the integer product. What has to be added is the widening
// on the way from shared memory to the operands:
//   - 128 channels are the rows of A. A lives in tensor memory, which the
//     widening warps write directly (thread = channel row = lane), so widened
//     channels never pass through shared memory;
//   - tokens are the rows of B. B has to come from shared memory; its warps read
//     the int8 tile, widen it and write the 128-byte swizzle that the matrix
//     instruction reads.
// TMA brings both int8 tiles, 128 k a step, into a ring; one thread issues the
// matrix instructions; accumulators (channels in the lanes, tokens in the
// columns) are read back, scaled and stored, 32 consecutive channels a warp.
//
// int8 -> FP16: with the sign bit flipped a byte is v + 128, and the FP16 with
// the bits 0x6400 | byte is 1024 + (v + 128): one subtraction of 1152 (0x6480),
// exact.
#pragma once

#include "matmul_int8.cuh"
#include "umma.cuh"

namespace beam {

constexpr int kStepK = 128;                         // k of one ring slot and of one operand slot
constexpr int kTileN = 128;                         // channels of a CTA: the lanes of tensor memory
constexpr int kStepCols = kStepK / 2;               // columns of A for a step (two FP16 a column)
constexpr uint32_t kABytes = kTileN * kStepK;       // int8 channels of a step
constexpr uint64_t kMatmulWaitNs = 2000000000ull;   // every wait gives up after 2 s

struct MatmulTcParams {
    MatmulParams p;
    int m_tiles, n_tiles;
    int splits;               // CTAs of a cluster, each with a part of k
    uint64_t wait_ns;
    unsigned int* status;
};

// four int8 -> four FP16, in the order 0, 2, 1, 3: what a sum over k does not
// see, as channels and tokens go through the same. The exclusive or sets the
// exponent and flips the sign bit at once.
__device__ __forceinline__ void widen4(uint32_t v, uint32_t& even, uint32_t& odd) {
    constexpr uint32_t kMask = 0x00FF00FFu, kOne = 0x64806480u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(even) : "r"((v & kMask) ^ kOne), "r"(kOne));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(odd) : "r"(((v >> 8) & kMask) ^ kOne), "r"(kOne));
}

// One step of channels: row `row` (this thread's lane) of the int8 tile, 128
// bytes in the TMA's swizzle. The 8 lanes of a shared-memory phase read 8
// different 16-byte chunks.
__device__ __forceinline__ void load_channels(const unsigned char* tile, int row, uint4 (&v)[8]) {
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = *reinterpret_cast<const uint4*>(tile + row * 128 + ((c ^ (row & 7)) << 4));
}

// ... to 64 columns of tensor memory at `at`
__device__ __forceinline__ void widen_channels(const uint4 (&v)[8], uint32_t at) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 x = v[4 * half + c];
            widen4(x.x, w[8 * c + 0], w[8 * c + 1]);
            widen4(x.y, w[8 * c + 2], w[8 * c + 3]);
            widen4(x.z, w[8 * c + 4], w[8 * c + 5]);
            widen4(x.w, w[8 * c + 6], w[8 * c + 7]);
        }
        tmem_st32(at + 32 * half, w);
    }
}

// One step of ROWS tokens, by 128 threads, a chunk of 16 int8 and row each. The
// int8 chunk c of row r lies at c ^ (r % 8), the two FP16 chunks that it becomes
// (of 8 values, 2 (c % 4) and the next, in the tile of the step's first or
// second 64 k) at theirs. A shared-memory phase of 8 lanes takes four chunks of
// the two rows r and r ^ 5, which meet 8 different places in the load (r and
// r ^ 5 differ in bit 2) and in both stores (they differ in bit 0).
struct TokenPlace {
    int row, chunk, sub;
    __device__ explicit TokenPlace(int t) {
        const int lane = t & 31, w = t >> 5;
        row = (w >> 1) * 8 + ((lane >> 3) ^ (5 * ((lane >> 2) & 1)));
        chunk = lane & 3;
        sub = w & 1;
    }
};

template <int ROWS>
__device__ __forceinline__ void load_tokens(const unsigned char* tile, const TokenPlace& p, uint4 (&v)[ROWS / 16]) {
    const unsigned char* at = tile + p.row * 128 + (((4 * p.sub + p.chunk) ^ (p.row & 7)) << 4);
#pragma unroll
    for (int i = 0; i < ROWS / 16; ++i) v[i] = *reinterpret_cast<const uint4*>(at + i * 16 * 128);
}

template <int ROWS>
__device__ __forceinline__ void widen_tokens(const uint4 (&v)[ROWS / 16], unsigned char* op, const TokenPlace& p) {
    unsigned char* o = op + p.sub * (ROWS * 128) + p.row * 128;
    const int first = ((2 * p.chunk) ^ (p.row & 7)) << 4, second = first ^ 16;
#pragma unroll
    for (int i = 0; i < ROWS / 16; ++i) {
        uint4 a, b;
        widen4(v[i].x, a.x, a.y);
        widen4(v[i].y, a.z, a.w);
        widen4(v[i].z, b.x, b.y);
        widen4(v[i].w, b.z, b.w);
        *reinterpret_cast<uint4*>(o + i * 16 * 128 + first) = a;
        *reinterpret_cast<uint4*>(o + i * 16 * 128 + second) = b;
    }
}

// all lanes: whether every lane's wait ended
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t ns) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, ns));
}

template <int NT>
struct TileConfig {  // NT tokens a CTA
    static constexpr int kSlots = NT == 16 ? 5 : NT == 32 ? 4 : 3;                 // int8 ring
    static constexpr int kOps = NT <= 64 ? 2 : 4;                                // widened slots
    static constexpr int kCtas = NT <= 64 ? 2 : 1;                               // CTAs an SM
    static constexpr int kAGroups = 2, kBGroups = NT <= 64 ? 1 : 2;              // groups of 4 warps
    static constexpr int kAWarps = 4 * kAGroups, kBWarps = 4 * kBGroups;
    static constexpr int kThreads = 32 * (kAWarps + kBWarps + 2);
    static constexpr int kAcc = NT < 32 ? 32 : NT;                               // accumulator columns
    static constexpr int kCols = kAcc + kOps * kStepCols <= 256 ? 256 : 512;     // allocated
    static constexpr uint32_t kSlotBytes = kABytes + NT * kStepK;
    static constexpr uint32_t kOpBytes = NT * kStepK * 2;
    static constexpr uint32_t kSmem = kSlots * kSlotBytes + kOps * kOpBytes + 1024;  // and alignment
};

// A tile of 128 channels by NT tokens, one CTA, or a cluster of `splits` CTAs
// that share its k. Warps: kAWarps widen channels and read the result back,
// kBWarps widen tokens, one loads, one multiplies. Widening a step is a chain of
// latencies (wait, load, convert, store, hand over: 1400 cycles for 128 channels
// and 128 tokens, of which the matrix unit needs 512), so two groups of four
// warps take the steps in turn. For few tokens the way of the weights from HBM
// bounds it; two CTAs an SM then keep about 150 KB of them in flight on each.
// Split along k, the CTAs' integer partial sums meet in shared memory: CTA r
// adds and stores its share of the columns.
template <int NT, bool F32>
__global__ void __launch_bounds__(TileConfig<NT>::kThreads, TileConfig<NT>::kCtas)
    matmul_int8_tile_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                            const MatmulTcParams q) {
    using C = TileConfig<NT>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t raw_full[C::kSlots], raw_empty[C::kSlots], op_full[C::kOps], op_empty[C::kOps],
        acc_full;
    __shared__ uint32_t tmem_slot;
    __shared__ float a_scale[NT], w_scale[kTileN];
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr int kLoadWarp = C::kAWarps + C::kBWarps, kMulWarp = kLoadWarp + 1;
    unsigned char* ops = smem + C::kSlots * C::kSlotBytes;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = q.splits > 1 ? (int)cluster_rank() : 0;
    const int tile = blockIdx.x / q.splits;
    const int n0 = (tile / q.m_tiles) * kTileN;
    const long long m0 = (long long)(tile % q.m_tiles) * NT;
    const int steps = (q.p.K + kStepK - 1) / kStepK;
    const int first = (int)((long long)steps * split / q.splits);
    const int count = (int)((long long)steps * (split + 1) / q.splits) - first;

    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 8);
        }
        for (int i = 0; i < C::kOps; ++i) {
            mbar_init(&op_full[i], 8);
            mbar_init(&op_empty[i], 1);
        }
        mbar_init(&acc_full, 1);
        mbar_fence_init();
    }
    if (warp == kMulWarp) tmem_alloc<1>(&tmem_slot, C::kCols);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    // only now: a CTA that the trigger lets in allocates tensor memory too, and
    // must not take the columns that a CTA of this grid still waits for
    pdl_trigger();
    const uint32_t acc = tmem_slot, acols = acc + C::kAcc;
    bool ok = true;

    if (warp == kLoadWarp) {
        if (lane == 0) {
            tma_prefetch_map(&wmap);
            tma_prefetch_map(&amap);
            const uint64_t pol_w = q.m_tiles == 1 ? l2_evict_first() : l2_evict_normal(), pol_a = l2_evict_normal();
            auto load_w = [&](int i, int s) {
                mbar_arrive_expect_tx(&raw_full[s], C::kSlotBytes);
                tma_load_2d(smem + s * C::kSlotBytes, &wmap, (first + i) * kStepK, n0, &raw_full[s], pol_w);
            };
            auto load_a = [&](int i, int s) {
                tma_load_2d(smem + s * C::kSlotBytes + kABytes, &amap, (first + i) * kStepK, (int)m0, &raw_full[s], pol_a);
            };
            // the weights do not depend on the kernel before: the first slots' are
            // asked for ahead of the wait for it
            const int head = count < C::kSlots ? count : C::kSlots;
            for (int i = 0; i < head; ++i) load_w(i, i);
            pdl_wait();
            for (int i = 0; i < head; ++i) load_a(i, i);
            int issued = head;
            for (int i = head; i < count; ++i) {
                const int s = i % C::kSlots;
                if (!mbar_wait(&raw_empty[s], (uint32_t)(i / C::kSlots - 1) & 1, q.wait_ns)) {
                    ok = false;
                    break;
                }
                load_w(i, s);
                load_a(i, s);
                issued = i + 1;
            }
            if (!ok)  // copies in flight must land before the shared memory goes
                for (int i = issued > C::kSlots ? issued - C::kSlots : 0; i < issued; ++i)
                    mbar_wait(&raw_full[i % C::kSlots], (uint32_t)(i / C::kSlots) & 1, q.wait_ns);
        }
    } else if (warp == kMulWarp) {
        if (lane == 0) {
            constexpr uint32_t idesc = UmmaF16<kTileN, NT>::kDesc;
            for (int i = 0; i < count; ++i) {
                const int o = i % C::kOps;
                if (!mbar_wait(&op_full[o], (uint32_t)(i / C::kOps) & 1, q.wait_ns)) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                const uint32_t b = smem_u32(ops + o * C::kOpBytes);
#pragma unroll
                for (int k = 0; k < kStepK / 16; ++k)
                    umma_f16<1>(acc, acols + o * kStepCols + k * 8,
                                umma_smem_desc(b + (k / 4) * (NT * 128) + (k % 4) * 32), idesc, i > 0 || k > 0);
                umma_commit<1>(&op_empty[o]);
            }
            umma_commit<1>(&acc_full);
            if (!ok) mbar_wait(&acc_full, 0, q.wait_ns);
        }
    } else {
        const bool channels = warp < C::kAWarps;
        // this warp's group takes the steps group, group + groups, ...
        const int group = channels ? warp / 4 : (warp - C::kAWarps) / 4, groups = channels ? C::kAGroups : C::kBGroups;
        const int t = tid & 127;  // within the group; for channels the lane of tensor memory
        const uint32_t lanes = acols + ((uint32_t)(t & 96) << 16);
        const TokenPlace place(t);
        // the scales wait in shared memory for the result
        pdl_wait();
        if (group == 0) {
            if (channels) w_scale[t] = n0 + t < q.p.N ? __ldg(q.p.w_scale + n0 + t) : 0.0f;
            else if (t < NT) a_scale[t] = m0 + t < q.p.M ? __ldg(q.p.a_scale + m0 + t) : 0.0f;
        }
        for (int i = group; i < count; i += groups) {
            const int s = i % C::kSlots, o = i % C::kOps;
            const unsigned char* slot = smem + s * C::kSlotBytes;
            uint4 v[8];  // tokens: NT / 16 of them
            uint4(&vt)[NT / 16] = reinterpret_cast<uint4(&)[NT / 16]>(v);
            ok = warp_wait(&raw_full[s], (uint32_t)(i / C::kSlots) & 1, q.wait_ns);
            if (!ok) break;
            if (channels) load_channels(slot, t, v);
            else load_tokens<NT>(slot + kABytes, place, vt);
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_empty[s]);
            ok = i < C::kOps || warp_wait(&op_empty[o], (uint32_t)(i / C::kOps - 1) & 1, q.wait_ns);
            if (!ok) break;
            if (channels) {
                tmem_fence_after();
                widen_channels(v, lanes + o * kStepCols);
                tmem_wait_st();
                tmem_fence_before();
            } else {
                widen_tokens<NT>(vt, ops + o * C::kOpBytes, place);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&op_full[o]);
        }
    }
    // the scales; also: nobody reads the ring or the operands any more once the
    // accumulators are complete
    __syncthreads();
    __syncwarp();

    // accumulators: lane = channel n0 + tid, column = token m0 + c
    const long long left = q.p.M - m0;
    const int cols = left < NT ? (int)left : NT;
    int* part = reinterpret_cast<int*>(smem);  // [NT][128] of the ring, which is idle by then
    if (warp < C::kAWarps) {
        ok = warp_wait(&acc_full, 0, q.wait_ns) && ok;
        if (ok) {
            tmem_fence_after();
            const int t = tid & 127, n = n0 + t;
            const float ws = w_scale[t];
            for (int c0 = 16 * (warp / 4); c0 < cols; c0 += 16 * C::kAGroups) {
                float v[16];
                tmem_ld16(acc + ((uint32_t)(t & 96) << 16) + c0, v);
                tmem_wait_ld();
                if (q.splits > 1) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) part[(c0 + c) * kTileN + t] = __float2int_rn(v[c]);
                } else if (n < q.p.N) {
                    const size_t at = (size_t)(m0 + c0) * (size_t)q.p.N + (size_t)n;
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (c0 + c < cols)
                            store_out<F32>(q.p.out, at + (size_t)c * (size_t)q.p.N,
                                           __fmul_rn(__fmul_rn(v[c], a_scale[c0 + c]), ws));
                }
            }
            tmem_fence_before();
        }
    }
    if (!ok) atomicOr(q.status, 1u);
    __syncthreads();
    // the columns go back before the cluster meets: no CTA holds tensor memory
    // while it waits for another one, which may still wait for some
    if (warp == kMulWarp) {
        tmem_fence_after();
        tmem_dealloc<1>(acc, C::kCols);
    }
    if (q.splits > 1) {
        __syncwarp();
        cluster_sync();  // every CTA's partial sums are written
        const int lo = cols * split / q.splits, hi = cols * (split + 1) / q.splits;
        if (tid < 256) {
            const int r = tid & 127, n = n0 + r;
            for (int c = lo + (tid >> 7); c < hi; c += 2) {
                int sum = 0;
                for (int i = 0; i < q.splits; ++i)
                    sum += ld_cluster_s32(cluster_addr(part + c * kTileN + r, (uint32_t)i));
                if (n < q.p.N) {
                    const long long m = m0 + c;
                    store_out<F32>(q.p.out, (size_t)m * (size_t)q.p.N + (size_t)n,
                                   __fmul_rn(__fmul_rn((float)sum, a_scale[c]), w_scale[r]));
                }
            }
        }
        __syncwarp();
        cluster_sync();  // nobody leaves while others read its sums
    }
}

}  // namespace beam

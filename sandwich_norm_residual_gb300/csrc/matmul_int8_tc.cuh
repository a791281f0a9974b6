// The 8-bit integer product on the tensor cores.
//
// GB300's tcgen05 has no integer kind, and its legacy integer path is slow. But
// every int8 is an FP16 number, a product of two is an integer of at most 2^14,
// and FP32 accumulators hold integers below 2^24 exactly: so the FP16 kind at
// its full rate gives the integer product, as long as partial sums stay below that
// (codes of an rms of 32 reach 2^18 at K = 65536). An accumulator runs on over all
// steps that a CTA has of a tile: emptied into 32-bit integers every 1024 k, sums
// would be exact for any codes, but the pairs' accumulator takes half of tensor
// memory and would stand still meanwhile. What has to be added is the widening on
// the way from shared memory to the operands:
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

#include <type_traits>

#include "matmul_int8.cuh"
#include "matmul_int8_plan.h"
#include "packed.cuh"
#include "umma.cuh"

namespace beam {

constexpr int kStepCols = kStepK / 2;               // columns of A for a step (two FP16 a column)
constexpr uint32_t kABytes = kTileN * kStepK;       // int8 channels of a step
constexpr uint64_t kMatmulWaitNs = 2000000000ull;   // every wait gives up after 2 s
constexpr uint64_t kMatmulTestWaitNs = 1000000ull;  // the test hook's: 1 ms

struct MatmulTcParams : TilePlan {
    MatmulParams p;
    // BF16 rows of out start on 16 bytes and end there: whole tiles of 128 channels
    // are then loaded in the order of `pmap` and stored 16 bytes a thread
    int wide;
    float* part;              // [workers][CG][2][NT][128]: sums of tiles that a worker has a part of
    uint64_t wait_ns;
    int drop;                 // test hook: the second step's copies are never issued
    unsigned int* status;
};

// What a worker does, in order: steps [k0, k1) of the tile at channel n0 (of the
// CTA's own 128) and token m0
struct Segment {
    int n0, m0;
    uint32_t k0, k1;
    bool whole;
};

template <int NT, int CG>
class Schedule {
    const MatmulTcParams& q;
    const uint32_t worker, rank;
    uint32_t wave = 0, at = 0, end = 0;  // at, end: of the split steps

    __device__ void place(Segment& s, uint32_t tile) const {
        s.n0 = (int)((tile / q.m_tiles * CG + rank) * kTileN);
        s.m0 = (int)(tile % q.m_tiles * NT);
    }

public:
    __device__ Schedule(const MatmulTcParams& q_, uint32_t worker_, uint32_t rank_) : q(q_), worker(worker_), rank(rank_) {
        if (worker < q.sharers) {
            at = q.split * worker / q.sharers;
            end = q.split * (worker + 1) / q.sharers;
        }
    }
    __device__ bool next(Segment& s) {
        if (wave < q.waves) {
            const uint32_t tile = wave++ * q.workers + worker;
            if (tile >= q.tiles) return false;
            place(s, tile);
            s.k0 = 0;
            s.k1 = q.steps;
            s.whole = true;
            return true;
        }
        if (at >= end) return false;
        const uint32_t t = at / q.steps;
        place(s, q.waves * q.workers + t);
        s.k0 = at - t * q.steps;
        s.k1 = min(q.steps, s.k0 + (end - at));
        s.whole = s.k1 - s.k0 == q.steps;
        at += s.k1 - s.k0;
        return true;
    }
};

// four int8 -> four FP16, in the order 0, 2, 1, 3, which a sum over k does not see,
// as channels and tokens go through the same. Byte permutes set the exponents: a
// mask and exclusive or in one, with a shift for the odd bytes, is as many
// instructions and took 0.05 us a step more (NT = 128: 0.52 against 0.45 us).
__device__ __forceinline__ void widen4(uint32_t v, uint32_t& even, uint32_t& odd) {
    const uint32_t u = v ^ 0x80808080u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(even) : "r"(__byte_perm(u, 0x64646464u, 0x4240)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(odd) : "r"(__byte_perm(u, 0x64646464u, 0x4341)), "r"(0x64806480u));
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

// One step of ROWS tokens, by WARPS warps: a lane takes ROWS / (4 WARPS) chunks of
// 16 int8. The int8 chunk c of row r lies at c ^ (r % 8); the two FP16 chunks
// that it becomes (of 8 values, 2 (c % 4) and the next, in the tile of the step's
// first or second 64 k) at theirs. A shared-memory phase of 8 lanes takes four
// chunks of the two rows r and r ^ 5, which meet 8 different places in the load
// (r and r ^ 5 differ in bit 2) and in both stores (they differ in bit 0).
template <int ROWS, int WARPS>
struct Tokens {
    static constexpr int kChunks = ROWS / 4 / WARPS;
    const int warp, x, chunk;  // x: row % 8
    __device__ explicit Tokens(int t) : warp(t >> 5), x(((t >> 3) & 3) ^ (5 * ((t >> 2) & 1))), chunk(t & 3) {}
    // the warps share 2 ROWS / 8 pieces: 8 rows of one half of the step
    __device__ int sub(int i) const { return (i * WARPS + warp) & 1; }
    __device__ int row(int i) const { return ((i * WARPS + warp) >> 1) * 8 + x; }

    __device__ void load(const unsigned char* tile, uint4 (&v)[kChunks]) const {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            v[i] = *reinterpret_cast<const uint4*>(tile + row(i) * 128 + (((4 * sub(i) + chunk) ^ x) << 4));
    }
    // to two FP16 tiles of 64 k, ROWS * 128 bytes each
    __device__ void widen(const uint4 (&v)[kChunks], unsigned char* op) const {
        const int first = ((2 * chunk) ^ x) << 4, second = first ^ 16;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            uint4 a, b;
            widen4(v[i].x, a.x, a.y);
            widen4(v[i].y, a.z, a.w);
            widen4(v[i].z, b.x, b.y);
            widen4(v[i].w, b.z, b.w);
            unsigned char* o = op + sub(i) * (ROWS * 128) + row(i) * 128;
            *reinterpret_cast<uint4*>(o + first) = a;
            *reinterpret_cast<uint4*>(o + second) = b;
        }
    }
};

// all lanes: whether every lane's wait ended
template <int CG = 1>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t ns) {
    return __all_sync(0xFFFFFFFFu, mbar_wait<CG>(bar, parity, ns));
}

// NT tokens by 128 CG channels: one CTA (CG = 1) or a pair of CTAs on one
// tensor tile (CG = 2), each with 128 channels and half of the tokens' rows
template <int NT, int CG>
struct TileConfig {
    static constexpr int kRows = NT / CG;                                          // tokens widened by a CTA
    static constexpr int kSlots = NT == 16 ? 10 : NT == 32 ? 8 : NT == 64 ? 6 : 4; // int8 ring
    static constexpr int kOps = NT <= 64 ? 4 : 3;                                  // widened slots
    static constexpr int kAccs = NT <= 128 ? 2 : 1;                                // accumulators
    static constexpr int kAccCols = NT < 32 ? 32 : NT;
    // warps in groups: a group widens the channels, another the tokens of a step
    static constexpr int kAGroups = NT <= 64 ? 3 : 2, kBGroupWarps = kRows <= 32 ? 1 : 4, kBGroups = kRows <= 32 ? 4 : 2;
    static constexpr int kAWarps = 4 * kAGroups, kBWarps = kBGroupWarps * kBGroups, kEpiWarps = 4;
    // A loading warp needs 0.3 us a copy (wait, announce, issue), where a step's
    // weights take 0.37 us from HBM: two take the steps in turn, and for few tokens
    // two more copy the tokens (one for both: 0.58 us a step)
    static constexpr int kLoadWarps = NT <= 32 ? 4 : 2;
    // whole fours of warps: the schedulers' register files are separate
    static constexpr int kThreads = 32 * ((kAWarps + kBWarps + kEpiWarps + kLoadWarps + 1 + 3) / 4 * 4);
    // A wait by parity passes at once on a barrier whose phase before has not even
    // ended, so a group must know that it has. Before step j it has seen the
    // product of step j - groups - kOps end, and all before: enough for the slot's
    // step before (j - kSlots) and the operand's (j - 2 kOps) in these cases, as is
    // a slot that the same group always takes.
    static constexpr bool safe(int groups) {
        return (kSlots % groups == 0 || kSlots >= groups + kOps) && (kOps % groups == 0 || kOps >= groups);
    }
    static_assert(safe(kAGroups) && safe(kBGroups), "a group could read a slot before it is filled");
    static_assert(kSlots % 2 == 0, "a slot is always filled by the same loading warps");
    static constexpr uint32_t kSlotBytes = kABytes + kRows * kStepK;
    static constexpr uint32_t kOpBytes = kRows * kStepK * 2;
    static constexpr uint32_t kScaleAt = kSlots * kSlotBytes + kOps * kOpBytes;    // FP32 [2][NT]
    static constexpr uint32_t kBarAt = kScaleAt + 2 * NT * 4;
    static constexpr uint32_t kSmem = kBarAt + (2 * kSlots + 2 * kOps + 2 * kAccs + 1) * 8;
    static_assert(kAccs * kAccCols + kOps * kStepCols <= 512, "tensor memory has 512 columns");
    static_assert(kSmem <= 232448, "shared memory of a CTA");
};

// Warps: 8 or 12 widen channels, 4 or 8 widen tokens, 4 read the result back, 2 or 4
// load, one multiplies. Widening a step is a chain of latencies (wait, load,
// convert, store, hand over: measured 1400 cycles for 128 channels and 128
// tokens, of which the matrix unit needs 512), so groups of four warps take the
// steps in turn: for the channels three up to 64 tokens, where nothing else keeps
// the schedulers busy (M = 16, N = 19456, K = 10240: 37.7 us with two, 34.7 with
// three), two beyond. Everything runs on from tile to tile without a pause; with two
// accumulators the result of one tile is stored under the next one's products.
//
// For few tokens the way of the weights from HBM bounds it: the ring keeps 160
// KB of them in flight on every SM, and all SMs get the same number of steps,
// whatever the number of tiles (`sharers`): a tile that several workers have
// steps of leaves FP32 sums in `part`, which matmul_int8_join_kernel adds.
// For many tokens the matrix unit bounds it; pairs of CTAs then halve the tokens
// that each CTA widens, and what the matrix unit reads from shared memory.
template <int NT, int CG, bool F32>
__global__ void __launch_bounds__(TileConfig<NT, CG>::kThreads, 1)
    matmul_int8_tile_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap pmap,
                            const __grid_constant__ CUtensorMap amap, const __grid_constant__ MatmulTcParams q) {
    using C = TileConfig<NT, CG>;
    extern __shared__ __align__(1024) unsigned char smem[];
    constexpr int kEpiWarp = C::kAWarps + C::kBWarps, kLoadWarp = kEpiWarp + C::kEpiWarps, kMulWarp = kLoadWarp + C::kLoadWarps;
    unsigned char* ops = smem + C::kSlots * C::kSlotBytes;
    float* a_scale = reinterpret_cast<float*>(smem + C::kScaleAt);
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + C::kBarAt);  // a slot's int8 tiles have landed
    uint64_t* raw_empty = raw_full + C::kSlots;                         // ... have been read
    uint64_t* op_full = raw_empty + C::kSlots;                          // a step is widened (in both CTAs)
    uint64_t* op_empty = op_full + C::kOps;                             // ... is multiplied
    uint64_t* acc_full = op_empty + C::kOps;                            // a segment's sums are complete
    uint64_t* acc_empty = acc_full + C::kAccs;                          // ... are read (in both CTAs)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + C::kAccs);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
    const uint32_t worker = blockIdx.x / CG;
    // Channels in the order that lets a thread store 8 of them at once (see the
    // result): lane 8 b + 2 j + e of each 32 holds channel 8 j + 2 b + e
    auto permuted = [&](const Segment& s) {
        return !F32 && q.wide && s.whole && whole_channels(q.p.N, s.n0);
    };

    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&raw_full[i], C::kLoadWarps / 2);
            mbar_init(&raw_empty[i], 4 + C::kBGroupWarps);  // the warps of a group each for channels and tokens
        }
        for (int i = 0; i < C::kOps; ++i) {
            mbar_init(&op_full[i], (4 + C::kBGroupWarps) * CG);
            mbar_init(&op_empty[i], 1);
        }
        for (int i = 0; i < C::kAccs; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], C::kEpiWarps * CG);
        }
        mbar_fence_init();
    }
    if (warp == kMulWarp) tmem_alloc<CG, 512>(tmem_slot);
    tmem_fence_before();
    if constexpr (CG == 2) cluster_sync();  // the other CTA's barriers are ready too
    else __syncthreads();
    tmem_fence_after();
    // only now: a CTA that the trigger lets in allocates tensor memory too, and
    // must not take the columns that a CTA of this grid still waits for
    pdl_trigger();
    const uint32_t acc = *tmem_slot, acols = acc + C::kAccs * C::kAccCols;
    bool ok = true;
    Schedule<NT, CG> todo(q, worker, rank);
    Segment seg;
    int it = 0, n_seg = 0;  // steps and segments so far
    // Before any bounded wait, for the kernel before this one: it may run for longer
    // than the bound, and nothing arrives until it is done. The loading warps wait
    // for it behind their first copies.
    if (warp < kLoadWarp || warp >= kMulWarp) pdl_wait();

    if (warp >= kLoadWarp && warp < kMulWarp) {
        if (lane == 0) {
            // this warp's part: every second step, channels, tokens or both
            const int mine = (warp - kLoadWarp) & 1;
            const bool both = C::kLoadWarps == 2, w_side = both || warp - kLoadWarp < 2, a_side = both || !w_side;
            const uint32_t bytes = (w_side ? kABytes : 0u) + (a_side ? C::kRows * kStepK : 0u);
            if (w_side) tma_prefetch_map(!F32 && q.wide ? &pmap : &wmap);
            if (a_side) tma_prefetch_map(&amap);
            const uint64_t pol_w = q.m_tiles == 1 ? l2_evict_first() : l2_evict_normal(), pol_a = l2_evict_normal();
            auto load_w = [&](int slot, const Segment& s, int k) {
                if (q.drop && k == 1) return;
                unsigned char* dst = smem + slot * C::kSlotBytes;
                if (permuted(s)) tma_load_5d(dst, &pmap, k * kStepK, s.n0 / 32, &raw_full[slot], pol_w);
                else tma_load_2d(dst, &wmap, k * kStepK, s.n0, &raw_full[slot], pol_w);
            };
            auto load_a = [&](int slot, const Segment& s, int k) {
                if (q.drop && k == 1) return;
                tma_load_2d(smem + slot * C::kSlotBytes + kABytes, &amap, k * kStepK,
                            s.m0 + (int)rank * C::kRows, &raw_full[slot], pol_a);
            };
            // the weights do not depend on the kernel before: the first slots' are
            // asked for ahead of the wait for it
            if (w_side) {
                Schedule<NT, CG> head(q, worker, rank);
                for (int i = 0; i < C::kSlots && head.next(seg);)
                    for (uint32_t k = seg.k0; k < seg.k1 && i < C::kSlots; ++k, ++i)
                        if ((i & 1) == mine) {
                            mbar_arrive_expect_tx(&raw_full[i], bytes);
                            load_w(i, seg, (int)k);
                        }
            }
            pdl_wait();
            while (ok && todo.next(seg))
                for (uint32_t k = seg.k0; k < seg.k1; ++k, ++it) {
                    if ((it & 1) != mine) continue;
                    const int slot = it % C::kSlots;
                    if (it >= C::kSlots) {
                        ok = mbar_wait(&raw_empty[slot], (uint32_t)(it / C::kSlots - 1) & 1, q.wait_ns);
                        if (!ok) break;
                    }
                    if (it >= C::kSlots || !w_side) mbar_arrive_expect_tx(&raw_full[slot], bytes);
                    if (it >= C::kSlots && w_side) load_w(slot, seg, (int)k);
                    if (a_side) load_a(slot, seg, (int)k);
                }
            // Copies in flight must land before the shared memory goes: also where every
            // step was issued, as the warps that read them may have given up before
            for (int i = max(it - C::kSlots, 0); i < it; ++i)
                if ((i & 1) == mine)
                    mbar_wait(&raw_full[i % C::kSlots], (uint32_t)(i / C::kSlots) & 1, q.wait_ns);
        }
    } else if (warp == kMulWarp) {
        if (rank == 0) {
            constexpr uint32_t idesc = UmmaF16<kTileN * CG, NT>::kDesc;
            const uint64_t b0 = umma_smem_desc(smem_u32(ops));
            for (; ok && todo.next(seg); ++n_seg) {
                const int a = n_seg % C::kAccs;
                const uint32_t d = acc + a * C::kAccCols;
                if (n_seg >= C::kAccs)
                    ok = warp_wait<CG>(&acc_empty[a], (uint32_t)(n_seg / C::kAccs - 1) & 1, q.wait_ns);
                for (uint32_t k = seg.k0; ok && k < seg.k1; ++k, ++it) {
                    const int o = it % C::kOps;
                    ok = warp_wait<CG>(&op_full[o], (uint32_t)(it / C::kOps) & 1, q.wait_ns);
                    if (!ok) break;
                    tmem_fence_after();
                    // the descriptor counts addresses in units of 16 bytes
                    const uint64_t b = b0 + (uint32_t)o * (C::kOpBytes / 16);
                    const uint32_t from = acols + o * kStepCols;
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < kStepK / 16; ++j)
                            umma_f16<CG>(d, from + j * 8, b + ((j / 4) * (C::kRows * 128) + (j % 4) * 32) / 16, idesc,
                                         k > seg.k0 || j > 0);
                        umma_commit<CG>(&op_empty[o]);
                    }
                    __syncwarp();
                }
                if (elect_one()) umma_commit<CG>(&acc_full[a]);
                __syncwarp();
            }
            // its instructions have ended before tensor memory and shared memory go, also
            // where the warps that read the result have given up
            if (n_seg > 0)
                warp_wait(&acc_full[(n_seg - 1) % C::kAccs], (uint32_t)((n_seg - 1) / C::kAccs) & 1, q.wait_ns);
        }
    } else if (warp < kEpiWarp) {
        const bool channels = warp < C::kAWarps;
        // this warp's group takes the steps group, group + groups, ...
        const int group = channels ? warp / 4 : (warp - C::kAWarps) / C::kBGroupWarps;
        const int groups = channels ? C::kAGroups : C::kBGroups;
        const int t = tid & 127;  // for channels the lane of tensor memory
        const uint32_t lanes = acols + ((uint32_t)(t & 96) << 16);
        using Rows = Tokens<C::kRows, C::kBGroupWarps>;
        const Rows rows(tid & (32 * C::kBGroupWarps - 1));
        while (ok && todo.next(seg)) {
            const int first = it, n = (int)(seg.k1 - seg.k0);
            it += n;
            for (int i = first + (group + groups - first % groups) % groups; i < first + n; i += groups) {
                const int s = i % C::kSlots, o = i % C::kOps;
                const unsigned char* slot = smem + s * C::kSlotBytes;
                uint4 v[8];  // tokens: kChunks of them
                uint4(&vt)[Rows::kChunks] = reinterpret_cast<uint4(&)[Rows::kChunks]>(v);
                ok = warp_wait(&raw_full[s], (uint32_t)(i / C::kSlots) & 1, q.wait_ns);
                if (!ok) break;
                if (channels) load_channels(slot, t, v);
                else rows.load(slot + kABytes, vt);
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
                    rows.widen(vt, ops + o * C::kOpBytes);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2) mbar_arrive_cluster(cluster_addr(&op_full[o], 0));
                    else mbar_arrive(&op_full[o]);
                }
            }
        }
    } else if (warp < kLoadWarp) {
        // Results: lane = channel, column = token. Rows of out have the channels side
        // by side, so a warp that stores column by column writes 64 bytes (BF16) an
        // instruction, and eight instructions a value bounded the whole tile (9 us of
        // it for 256 x 256). Whole tiles are therefore read as 8 x 8 fragments,
        // scaled two values an instruction, rounded and transposed in registers;
        // with the channels' order of the load, thread t then holds the 8 channels
        // 8 (t % 4) ... of token t / 4 and stores them at once.
        const int t = tid & 127;
        for (; ok && todo.next(seg); ++n_seg, it += (int)(seg.k1 - seg.k0)) {
            const int a = n_seg % C::kAccs, n0 = seg.n0, n = n0 + t, m0 = seg.m0;
            const int cols = (int)min(q.p.M - m0, (long long)NT);
            const bool wide = permuted(seg);
            float* scales = a_scale + (n_seg & 1) * NT;
            float ws[4] = {0.f, 0.f, 0.f, 0.f};
            if (wide) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    ws[b] = __ldg(q.p.w_scale + n0 + (t & 96) + 8 * ((t >> 3) & 3) + 2 * b + ((t >> 2) & 1));
            } else if (n < q.p.N) {
                ws[0] = __ldg(q.p.w_scale + n);
            }
            for (int c = t; c < cols; c += 128) scales[c] = __ldg(q.p.a_scale + m0 + c);
            // one answer for the four warps, which also meet here: the scales are there
            ok = group_and(1, warp_wait(&acc_full[a], (uint32_t)(n_seg / C::kAccs) & 1, q.wait_ns));
            if (!ok) break;
            tmem_fence_after();
            auto free_acc = [&] {  // this warp has read the accumulator
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2) mbar_arrive_cluster_relaxed(cluster_addr(&acc_empty[a], 0));
                    else mbar_arrive(&acc_empty[a]);
                }
            };
            const uint32_t from = acc + a * C::kAccCols + ((uint32_t)(t & 96) << 16);
            if (wide) {
                uint16_t* row = static_cast<uint16_t*>(q.p.out) + (size_t)(m0 + (lane >> 2)) * (size_t)q.p.N +
                                (size_t)(n0 + (t & 96) + 8 * (lane & 3));
                for (int c0 = 0; c0 < cols; c0 += 16) {
                    float v[2][8];  // lanes 0-15 and 16-31 of the warp's 32
                    tmem_ld_16x256b(from + c0, v[0]);
                    tmem_ld_16x256b(from + (16u << 16) + c0, v[1]);
                    tmem_wait_ld();
                    if (c0 + 16 >= cols) free_acc();
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 as = *reinterpret_cast<const float2*>(scales + c0 + 8 * i + 2 * (lane & 3));
                        uint32_t o[4];
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const float* f = v[b >> 1] + 4 * i + 2 * (b & 1);
                            o[b] = transpose_b16(
                                f2_to_bf2(mul2_rn(mul2_rn(make_float2(f[0], f[1]), as), make_float2(ws[b], ws[b]))));
                        }
                        if (c0 + 8 * i + (lane >> 2) < cols)
                            *reinterpret_cast<uint4*>(row) = make_uint4(o[0], o[1], o[2], o[3]);
                        row += 8 * (size_t)q.p.N;
                    }
                }
                continue;
            }
            // the first of this worker's split tiles goes to its part 0, the last to part 1
            const bool second = seg.k0 == 0;
            float* part = q.part + ((size_t)blockIdx.x * 2 + second) * (size_t)(NT * kTileN) + t;
            using Out = std::conditional_t<F32, float, uint16_t>;
            Out* out = static_cast<Out*>(q.p.out) + (size_t)m0 * (size_t)q.p.N + (size_t)n;
            constexpr int kBatch = NT < 32 ? 16 : 32;
            for (int c0 = 0; c0 < cols; c0 += kBatch) {
                float v[kBatch];
                if constexpr (kBatch == 16) tmem_ld16(from + c0, v);
                else tmem_ld32(from + c0, v);
                tmem_wait_ld();
                if (c0 + kBatch >= cols) free_acc();
                const bool full = c0 + kBatch <= cols;
                if (!seg.whole) {
                    if (full) {
#pragma unroll
                        for (int c = 0; c < kBatch; ++c) part[(c0 + c) * kTileN] = v[c];
                    } else {
#pragma unroll
                        for (int c = 0; c < kBatch; ++c)
                            if (c0 + c < cols) part[(c0 + c) * kTileN] = v[c];
                    }
                } else if (n < q.p.N) {
#pragma unroll
                    for (int c = 0; c < kBatch; c += 2) {
                        const float2 as = *reinterpret_cast<const float2*>(scales + c0 + c);
                        const float2 o = mul2_rn(mul2_rn(make_float2(v[c], v[c + 1]), as), make_float2(ws[0], ws[0]));
                        if (full || c0 + c < cols) store_out<F32>(out, 0, o.x);
                        out += q.p.N;
                        if (full || c0 + c + 1 < cols) store_out<F32>(out, 0, o.y);
                        out += q.p.N;
                    }
                }
            }
        }
        // the last steps' arrivals, which nobody else waits for, have come (in a pair,
        // from the other CTA) before the shared memory goes
        if (ok && it > 0)
            for (int i = max(it - C::kOps, 0); i < it; ++i)
                ok = warp_wait(&op_empty[i % C::kOps], (uint32_t)(i / C::kOps) & 1, q.wait_ns) && ok;
    }
    if (!ok) atomicOr(q.status, 1u);
    __syncwarp();
    tmem_fence_before();
    if constexpr (CG == 2) cluster_sync();  // nobody leaves while the other CTA works with its memory
    else __syncthreads();
    if (warp == kMulWarp) {
        tmem_fence_after();
        tmem_dealloc<CG, 512>(acc);
    }
}

// Adds the sums of the tiles that several workers have steps of: a block for
// kCols tokens of a tile, thread = channel. They are FP32 numbers that are integers,
// also past 2^24, and at most 2^30: added as 32-bit integers, without rounding. What
// it takes (3 us) is its launch and one way to L2 and back, so few values a thread
// (but not so few that blocks are counted in thousands: 2 tokens a block cost 3 us
// more than 8 at NT = 128) and several workers' at once.
template <int NT>
struct Join {
    static constexpr int kCols = NT <= 32 ? 2 : NT == 64 ? 4 : 8, kWorkers = NT <= 64 ? 8 : 4;
};

template <int NT, int CG, bool F32>
__global__ void __launch_bounds__(kTileN) matmul_int8_join_kernel(const __grid_constant__ MatmulTcParams q) {
    pdl_trigger();
    const uint32_t tile = q.waves * q.workers + blockIdx.x;
    constexpr int kJoinCols = Join<NT>::kCols, kJoinWorkers = Join<NT>::kWorkers;
    const uint32_t rank = blockIdx.z;  // the CTA's 128 channels of the tile
    const int n = (int)((tile / q.m_tiles * CG + rank) * kTileN + threadIdx.x), c0 = blockIdx.y * kJoinCols;
    const long long m0 = (long long)(tile % q.m_tiles) * NT + c0;
    // worker c has the steps [split c / sharers, split (c + 1) / sharers)
    const uint32_t lo = blockIdx.x * q.steps, hi = lo + q.steps;
    uint32_t c = lo * q.sharers / q.split;
    while (q.split * (c + 1) / q.sharers <= lo) ++c;
    uint32_t begin = q.split * c / q.sharers;
    const bool whole = begin <= lo && q.split * (c + 1) / q.sharers >= hi;  // one worker's: stored already
    pdl_wait();
    if (whole || n >= q.p.N || m0 >= q.p.M) return;
    const float ws = __ldg(q.p.w_scale + n);
    float as[kJoinCols];
#pragma unroll
    for (int i = 0; i < kJoinCols; ++i) as[i] = m0 + i < q.p.M ? __ldg(q.p.a_scale + m0 + i) : 0.0f;
    int sum[kJoinCols] = {};
    while (begin < hi) {
        float v[kJoinWorkers][kJoinCols] = {};
#pragma unroll
        for (int j = 0; j < kJoinWorkers; ++j) {
            if (begin < hi) {
                const bool second = begin <= lo;  // its segment of this tile begins at the tile's first step
                const float* part = q.part + (((size_t)c * CG + rank) * 2 + second) * (size_t)(NT * kTileN) +
                                    c0 * kTileN + threadIdx.x;
#pragma unroll
                for (int i = 0; i < kJoinCols; ++i)
                    if (m0 + i < q.p.M) v[j][i] = __ldcg(part + i * kTileN);
                begin = q.split * ++c / q.sharers;
            }
        }
#pragma unroll
        for (int j = 0; j < kJoinWorkers; ++j)
#pragma unroll
            for (int i = 0; i < kJoinCols; ++i) sum[i] += __float2int_rn(v[j][i]);
    }
#pragma unroll
    for (int i = 0; i < kJoinCols; ++i)
        if (m0 + i < q.p.M)
            store_out<F32>(q.p.out, (size_t)(m0 + i) * (size_t)q.p.N + (size_t)n,
                           __fmul_rn(__fmul_rn((float)sum[i], as[i]), ws));
}

}  // namespace beam

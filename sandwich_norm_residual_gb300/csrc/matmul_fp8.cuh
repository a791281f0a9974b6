// The product of E4M3 numbers with a scale for each 128 of a token and each 128 by 128
// of the channels, for one matrix of channels or one for each expert.
//
//   out[m, n] = sum_b RN(a_scale[m, b] w_scale[n / 128, b]) P_b,   P_b = sum_{k in b} a[m, k] w[n, k]
//
// The tensor cores' E4M3 kind adds P_b in FP32. The scales change with every 128 k, so
// P_b cannot stay in the accumulator: the matrix unit writes it to one of a few
// accumulators in tensor memory, and the adding warps read it, multiply by the scales and add
// it to sums that they hold in registers, in FP32, while the next is being made. For many
// tokens it is this that bounds the product, so it decides the layout:
//   - Tensor memory gives 227 bytes a clock to each of an SM's four parts read as 32 x 32b
//     (thread = lane, registers = columns), but 62 as 16 x 256b fragments, which would let a
//     thread hold neighbouring columns of several lanes.
//   - A thread's values should share their scale. Many tokens: lanes are tokens, columns
//     channels; a thread has one token and 128 channels of one block, so one scale a step.
//     Few tokens: lanes are channels, columns tokens (the instruction's columns are any
//     multiple of 16, its lanes are not); every column's scale is read from shared memory by
//     all lanes at once, and a warp stores 32 neighbours of a row of out.
//   - Tiles of one CTA. Pairs of CTAs on 256 by 256 bring a third less through L2 but free their
//     accumulators through the cluster's network: M = 16384, N = 20480, K = 5120 took 1322 us
//     in pairs, 1326 in single CTAs, and experts fill tiles of 128 rows better (16384 tokens to
//     8 of 256, N = K = 5120: 3390 and 3204 us).
//   - What the adding warps do beside reading, multiplying and adding counts twice: their
//     waits end with no vote, scales come four steps at a time, the barriers' places are
//     kept, not computed (M = 2048, N = 4864, K = 20480: 200 -> 152 us; without any reading
//     and adding 122 us).
#pragma once

#include <type_traits>

#include "matmul_fp8_plan.h"
#include "packed.cuh"
#include "umma.cuh"

namespace beam {

constexpr uint64_t kFp8WaitNs = 2000000000ull;   // every wait gives up after 2 s
constexpr uint64_t kFp8TestWaitNs = 1000000ull;  // the test hook's: 1 ms
constexpr int kFp8MaxExperts = 512;

struct Fp8Params {
    const float* a_scale;      // [R, steps]
    const float* w_scale;      // [E, ceil(N / 128), steps]
    void* out;                 // [R, N]
    const int32_t* offsets;    // [E + 1], or NULL: one expert has all rows
    long long R;
    int E, N;
    uint32_t steps, n_tiles;   // of k; of channels
    uint32_t width;            // channels of a tile
    int split;                 // CTAs of a cluster, which share a tile's steps
    int scales16;              // rows of a_scale are whole groups of 16 bytes
    int wide;                  // rows of out are whole groups of 32 bytes
    uint64_t wait_ns;
    int drop;                  // test hook: every tile's second step is never loaded
    unsigned int* status;
};

// A CTA's tile. Few tokens: 128 channels and up to 64 tokens; many: 128 tokens and up to 256
// channels, or up to 128.
template <bool FEW>
struct Fp8Tile {
    static constexpr int kColumns = FEW ? kFp8Few : kFp8Width;  // of an accumulator
    static constexpr int kSlots = FEW ? 7 : 4;       // ring of operand tiles
    // Accumulators of a step. Few tokens: one for every slot, so that a slot that has been read
    // and an accumulator that may be written again are one barrier, and the multiplying
    // thread waits once a step.
    static constexpr int kAccs = FEW ? kSlots : 2;
    static constexpr int kScales = 8;                // ring of steps' scales, in groups of four
    // FP32 of four steps in units of 16 bytes: of a step's tokens side by side; of a token's four
    // steps, the CTA's tokens for either block of channels
    static constexpr int kScaleRow = FEW ? kFp8Few : 2 * 128;
    // Warps: those that add, in two groups of four (a group has all lanes and half of the
    // columns); two that load, every second slot each; one that brings scales; one that
    // multiplies.
    static constexpr int kGroups = 2, kAddWarps = 4 * kGroups;
    static constexpr int kMine = kColumns / kGroups;  // columns of an adding warp
    static constexpr int kLoadWarp = kAddWarps, kScaleWarp = kLoadWarp + 2, kMulWarp = kScaleWarp + 1;
    static constexpr int kThreads = 32 * (kMulWarp + 1);
    // Many tokens: 128 sums a thread, so the adding warps take registers from the others
    // (2 x 216 + 72 = 3 x 168). Sixteen adding warps with 64 sums each took 0.49 us a step,
    // these 0.47.
    static constexpr int kAddRegs = 216, kOtherRegs = 72;
    static constexpr uint32_t kABytes = 128 * kFp8Step;  // rows of the lanes
    static constexpr uint32_t kSlotBytes = kABytes + kColumns * kFp8Step;
    static constexpr uint32_t kRedAt = FEW ? kSlots * kSlotBytes : 0;        // sums from the cluster's other CTAs
    static constexpr uint32_t kRedBytes = (kFp8MaxSplit - 1) * kColumns / kFp8MaxSplit * 512;
    static constexpr uint32_t kScaleAt = kSlots * kSlotBytes + (FEW ? kRedBytes : 0);  // FP32 [kScales][kScaleRow]
    static constexpr uint32_t kTableAt = kScaleAt + kScales * kScaleRow * 4; // experts: first tile, first row, rows
    static constexpr uint32_t kBarAt = kTableAt + (3 * kFp8MaxExperts + 4) * 4;
    static constexpr int kBars = 2 * kSlots + 2 * kAccs + 2 * (kScales / 4) + 2;
    static constexpr uint32_t kSmem = kBarAt + kBars * 8 + 16;
    static constexpr uint32_t kTmem = 512;
    static_assert(FEW || kRedBytes <= kSlots * kSlotBytes, "the join fits the ring");
    static_assert(kAccs * kColumns <= 512 && kSmem <= 232448 && kBarAt % 8 == 0, "tensor memory, shared memory of a CTA");
};

// Which rows and tiles an expert has, in shared memory
struct Fp8Experts {
    uint32_t* tile;  // [E + 1] tiles before it
    int32_t *row, *rows;
};

struct Fp8Work {
    int e, n0, m0;     // expert; the tile's first channel; its first row of a and out
    int cols;          // its tokens
    uint32_t n;        // the instruction's columns: tokens (few) or channels (many), a multiple of 16
    uint32_t k0, k1;   // this CTA's steps
    bool shared;       // the cluster's CTAs each have some of the tile's steps
};

// CTA c of W takes the tiles c, c + W, ... Where there are clusters, the tiles behind the last
// full wave are shared, one by a cluster at a time.
template <bool FEW>
class Fp8Schedule {
    const Fp8Params& q;
    const Fp8Experts& x;
    const uint32_t place;  // in the cluster
    uint32_t at, whole;    // the next tile; the tiles that are not shared
    int e = 0;

    __device__ uint32_t first_shared() const { return whole + blockIdx.x / q.split; }

public:
    __device__ Fp8Schedule(const Fp8Params& q_, const Fp8Experts& x_, uint32_t place_)
        : q(q_), x(x_), place(place_), at(blockIdx.x), whole(0xFFFFFFFFu) {
        if (q.split > 1) {
            const uint32_t all = x.tile[q.E], rest = all % gridDim.x;
            // many tokens' joins go through the ring, so a cluster has one at most, its last tile
            if (FEW || rest <= gridDim.x / q.split) {
                whole = all - rest;
                if (at >= whole) at = first_shared();
            }
        }
    }
    __device__ bool next(Fp8Work& w) {
        while (e < q.E && at >= x.tile[e + 1]) ++e;
        if (e >= q.E) return false;
        const uint32_t rows = (uint32_t)x.rows[e];
        const Fp8Rows r = fp8_rows<FEW>(rows);
        uint32_t m, n;
        fp8_place(at - x.tile[e], r.tiles, q.n_tiles, &m, &n);
        w.e = e;
        w.n0 = (int)(n * q.width);
        w.m0 = x.row[e] + (int)(m * r.each);
        w.cols = (int)min(r.each, rows - m * r.each);
        w.n = FEW ? fp8_up((uint32_t)w.cols, 16) * 16 : min(q.width, fp8_up((uint32_t)(q.N - w.n0), 16) * 16);
        w.shared = at >= whole;
        w.k0 = w.shared ? q.steps * place / q.split : 0u;
        w.k1 = w.shared ? q.steps * (place + 1) / q.split : q.steps;
        if (w.shared) {
            at += gridDim.x / q.split;
        } else {
            at += gridDim.x;
            if (at >= whole) at = first_shared();
        }
        return true;
    }
};

// all lanes: whether every lane's wait ended
__device__ __forceinline__ bool fp8_wait(uint64_t* bar, uint32_t parity, uint64_t ns) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, ns));
}

template <int REGS>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(REGS)); }
template <int REGS>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(REGS)); }

// 32 bytes to an address that is a multiple of 32
__device__ __forceinline__ void st_sector(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}

template <bool F32>
using Fp8Out = std::conditional_t<F32, float, uint16_t>;

template <bool F32>
__device__ __forceinline__ Fp8Out<F32> fp8_round(float v) {
    if constexpr (F32) return v;
    else return (uint16_t)f2_to_bf2(make_float2(v, 0.f));
}

// transposes a warp's 32 x 32 values: register i of lane j goes to register j of lane i
__device__ __forceinline__ void transpose32(float (&r)[32], int lane) {
#pragma unroll
    for (int s = 16; s; s >>= 1) {
        const bool up = lane & s;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!(i & s)) {
                const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? r[i] : r[i | s], s);
                if (up) r[i] = got;
                else r[i | s] = got;
            }
    }
}

template <bool FEW, bool F32>
__global__ void __launch_bounds__(Fp8Tile<FEW>::kThreads, 1)
    matmul_fp8_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                      const __grid_constant__ Fp8Params q) {
    using C = Fp8Tile<FEW>;
    extern __shared__ __align__(1024) unsigned char smem[];
    float4* const scales = reinterpret_cast<float4*>(smem + C::kScaleAt);
    uint32_t* const table = reinterpret_cast<uint32_t*>(smem + C::kTableAt);
    const Fp8Experts experts{table, reinterpret_cast<int32_t*>(table + kFp8MaxExperts + 4),
                             reinterpret_cast<int32_t*>(table + 2 * kFp8MaxExperts + 4)};
    uint64_t* const full = reinterpret_cast<uint64_t*>(smem + C::kBarAt);  // a slot's tiles have landed
    uint64_t* const acc_full = full + C::kSlots;              // a step is multiplied
    uint64_t* const acc_empty = acc_full + C::kAccs;          // ... and read
    uint64_t* const empty = FEW ? acc_empty : acc_empty + C::kAccs;  // a slot's tiles may be written again
    uint64_t* const scale_full = empty + C::kSlots;           // four steps' scales are there
    uint64_t* const scale_empty = scale_full + C::kScales / 4;
    uint64_t* const red_full = scale_empty + C::kScales / 4;  // the other CTAs' sums of a tile are there
    uint64_t* const red_ready = red_full + 1;                 // they let this CTA write theirs
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(red_ready + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t place = q.split > 1 ? cluster_rank() : 0u;

    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&full[i], 1);
            if (!FEW) mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::kAccs; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], C::kAddWarps);
        }
        for (int i = 0; i < C::kScales / 4; ++i) {
            mbar_init(&scale_full[i], 1);
            mbar_init(&scale_empty[i], C::kAddWarps);
        }
        mbar_init(red_full, (q.split > 1 ? q.split - 1 : 1) * C::kAddWarps);
        mbar_init(red_ready, (q.split > 1 ? q.split - 1 : 1) * C::kAddWarps);
        mbar_fence_init();
    }
    if (warp == C::kMulWarp) tmem_alloc<1, C::kTmem>(tmem_slot);
    // Experts' rows. Where an offset decreases or leaves [0, R] nobody has any: rows counted twice
    // could be more tiles than 32 bits number.
    bool bad = false;
    for (int e = tid; e < q.E; e += C::kThreads) {
        long long lo = 0, hi = q.R;
        if (q.offsets) {
            lo = __ldg(q.offsets + e);
            hi = __ldg(q.offsets + e + 1);
            bad |= lo < 0 || hi < lo || hi > q.R;
        }
        experts.row[e] = (int32_t)lo;
        experts.rows[e] = (int32_t)(hi - lo);
    }
    if (bad && blockIdx.x == 0) atomicOr(q.status, 2u);
    if (__syncthreads_or(bad)) {
        for (int e = tid; e < q.E; e += C::kThreads) experts.rows[e] = 0;
        __syncthreads();
    }
    if (warp == 0) {
        constexpr int kEach = kFp8MaxExperts / 32;
        uint32_t sum = 0;
        for (int i = 0; i < kEach; ++i) {
            const int e = lane * kEach + i;
            if (e < q.E) sum += fp8_rows<FEW>((uint32_t)experts.rows[e]).tiles * q.n_tiles;
        }
        uint32_t before = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, before, off);
            if (lane >= off) before += v;
        }
        before -= sum;
        for (int i = 0; i < kEach; ++i) {
            const int e = lane * kEach + i;
            if (e < q.E) {
                experts.tile[e] = before;
                before += fp8_rows<FEW>((uint32_t)experts.rows[e]).tiles * q.n_tiles;
                if (e == q.E - 1) experts.tile[q.E] = before;
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (q.split > 1) cluster_sync();  // the other CTAs' barriers are ready too
    tmem_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;
    Fp8Schedule<FEW> todo(q, experts, place);
    Fp8Work w;
    int it = 0;                // steps so far (loads and products)
    int sg = 0, sturn = 0;     // the group of scales, and how often the ring went around

    if (warp < C::kAddWarps) {
        if constexpr (!FEW) more_registers<C::kAddRegs>();
        const int group = warp >> 2, row = tid & 127;  // row: this thread's lane of tensor memory
        const uint32_t lanes = tmem + ((uint32_t)(row & 96) << 16);
        int a = 0, aturn = 0;
        int joins = 0;
        while (todo.next(w)) {
            float2 sums[C::kMine / 2];
#pragma unroll
            for (int j = 0; j < C::kMine / 2; ++j) sums[j] = make_float2(0.f, 0.f);
            // this warp's columns: a share of the tokens, or of the tile's channels (within a block of 128)
            const int mine = (int)(FEW ? w.n : q.width) / C::kGroups, c0 = group * mine;
            const bool some = FEW || c0 < (int)w.n;
            // scales come in groups of four steps, at multiples of four
            for (uint32_t g = w.k0 & ~3u; g < w.k1; g += 4) {
                if (ok) ok = mbar_wait(&scale_full[sg], sturn & 1, q.wait_ns);
                __syncwarp();
                // many: this thread's token's in the four steps
                const float4 own = FEW ? float4{} : scales[sg * C::kScaleRow + (c0 & 128) + row];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (g + j < w.k0 || g + j >= w.k1) continue;
                    // No vote on the wait: a thread that gave up goes on without waiting
                    if (ok) ok = mbar_wait(&acc_full[a], aturn & 1, q.wait_ns);
                    __syncwarp();
                    tmem_fence_after();
                    const uint32_t from = lanes + a * C::kColumns + c0;
                    if (some) {
                        const float s = j == 0 ? own.x : j == 1 ? own.y : j == 2 ? own.z : own.w;
#pragma unroll
                        for (int c = 0; c < C::kMine / 16; ++c) {
                            // few: a second eight columns that are not there are columns of this
                            // accumulator that no tile stores
                            if (FEW ? 16 * c < mine : c < C::kMine / 32 || mine == C::kMine) {
                                float v[16];
                                tmem_ld16_wait(from + 16 * c, v);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    float2 f = make_float2(s, s);
                                    if (FEW) f = reinterpret_cast<const float2*>(scales + sg * C::kScaleRow)[(j * C::kColumns + c0) / 2 + 8 * c + i];
                                    sums[8 * c + i] = __ffma2_rn(make_float2(v[2 * i], v[2 * i + 1]), f, sums[8 * c + i]);
                                }
                            }
                        }
                    }
                    // all read: the accumulator may be written again
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_empty[a]);
                    if (++a == C::kAccs) {
                        a = 0;
                        ++aturn;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&scale_empty[sg]);
                if (++sg == C::kScales / 4) {
                    sg = 0;
                    ++sturn;
                }
            }
            using Out = Fp8Out<F32>;
            Out* const out = static_cast<Out*>(q.out);
            // A tile that the cluster's CTAs have shares of: CTA d adds up and stores every split-th
            // piece of the columns, from sums that the others write to its shared memory: few
            // tokens' to a place of their own, many tokens' to the ring, which by then is done with.
            constexpr int kPiece = FEW ? 8 : 32, kPieces = C::kMine / kPiece;
            auto owner = [&](int j) { return (j * C::kGroups + group) % q.split; };
            if (w.shared) {
                const int each = (C::kColumns / kPiece + q.split - 1) / q.split;
                const auto place_of = [&](int from, int j) {
                    return smem + C::kRedAt + (((from * each + (j * C::kGroups + group) / q.split) * (kPiece / 4)) * 128 + row) * 16;
                };
                // The others may write to this CTA's, and this one to theirs: released, since it was read until now (few
                // tokens: the join before; many: operands, whose products have ended)
                __syncwarp();
                if (lane == 0)
                    for (int d = 0; d < q.split; ++d)
                        if (d != (int)place) mbar_arrive_cluster_release(cluster_addr(red_ready, d));
                if (ok) ok = mbar_wait<2>(red_ready, joins & 1, q.wait_ns);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    const int d = owner(j);
                    if (kPiece * j < mine && d != (int)place) {
                        const uint32_t there = cluster_addr(place_of((int)place < d ? (int)place : (int)place - 1, j), d);
#pragma unroll
                        for (int i = 0; i < kPiece / 4; ++i) {
                            const float2 u = sums[kPiece / 2 * j + 2 * i], v = sums[kPiece / 2 * j + 2 * i + 1];
                            st_cluster(there + i * 2048, make_float4(u.x, u.y, v.x, v.y));
                        }
                    }
                }
                __syncwarp();
                if (lane == 0)
                    for (int d = 0; d < q.split; ++d)
                        if (d != (int)place) mbar_arrive_cluster_release(cluster_addr(red_full, d));
                if (ok) ok = mbar_wait<2>(red_full, joins & 1, q.wait_ns);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < kPieces; ++j)
                    if (kPiece * j < mine && owner(j) == (int)place)
                        for (int from = 0; from < q.split - 1; ++from) {
                            const float4* at = reinterpret_cast<const float4*>(place_of(from, j));
#pragma unroll
                            for (int i = 0; i < kPiece / 4; ++i) {
                                const float4 v = at[i * 128];
                                float2(&t)[2] = reinterpret_cast<float2(&)[2]>(sums[kPiece / 2 * j + 2 * i]);
                                t[0].x += v.x; t[0].y += v.y; t[1].x += v.z; t[1].y += v.w;
                            }
                        }
                ++joins;
            }
            auto stored = [&](int j) { return !w.shared || owner(j) == (int)place; };
            if constexpr (FEW) {
                // thread = channel: a warp's store is 32 neighbours of a row
                Out* const to = out + (size_t)(w.m0 + c0) * (size_t)q.N + (size_t)(w.n0 + row);
                const int cols = w.cols - c0;  // from this warp's first on
                if (w.n0 + row < q.N) {
#pragma unroll
                    for (int j = 0; j < C::kMine / 2; ++j)
                        if (stored(j / 4)) {
                            if (2 * j < cols && 2 * j < mine) to[(size_t)(2 * j) * (size_t)q.N] = fp8_round<F32>(sums[j].x);
                            if (2 * j + 1 < cols && 2 * j < mine) to[(size_t)(2 * j + 1) * (size_t)q.N] = fp8_round<F32>(sums[j].y);
                        }
                }
            } else if (some) {
                const int left = q.N - (w.n0 + c0);  // channels from this warp's first on
                if (q.wide) {
                    // thread = token: whole sectors of its row
                    constexpr int kBatch = F32 ? 8 : 16;
                    Out* const to = out + (size_t)(w.m0 + row) * (size_t)q.N + (size_t)(w.n0 + c0);
                    if (row < w.cols) {
#pragma unroll
                        for (int j = 0; j < C::kMine / kBatch; ++j) {
                            if (kBatch * j < mine && kBatch * j < left && stored(kBatch * j / 32)) {
                                uint32_t v[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    if constexpr (F32) v[i] = __float_as_uint(i & 1 ? sums[4 * j + i / 2].y : sums[4 * j + i / 2].x);
                                    else v[i] = f2_to_bf2(sums[8 * j + i]);
                                }
                                st_sector(to + kBatch * j, v);
                            }
                        }
                    }
                } else if ((row & 96) < w.cols) {
                    // rows that do not start on a sector: transposed, 32 neighbours of a row a store
#pragma unroll
                    for (int c = 0; c < C::kMine / 32; ++c) {
                        if (32 * c < mine && stored(c)) {
                            float v[32];
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                v[2 * j] = sums[16 * c + j].x;
                                v[2 * j + 1] = sums[16 * c + j].y;
                            }
                            transpose32(v, lane);
                            Out* const to = out + (size_t)(w.m0 + (row & 96)) * (size_t)q.N + (size_t)(w.n0 + c0 + 32 * c + lane);
                            if (32 * c + lane < left) {
#pragma unroll
                                for (int t = 0; t < 32; ++t)
                                    if ((row & 96) + t < w.cols) to[(size_t)t * (size_t)q.N] = fp8_round<F32>(v[t]);
                            }
                            __syncwarp();
                        }
                    }
                }
            }
        }
    } else {
        if constexpr (!FEW) fewer_registers<C::kOtherRegs>();
        if (warp < C::kScaleWarp) {
            // Loads. A slot is always filled by the same warp, which therefore has seen every use
            // of it; its lanes issue a copy each: first the lanes' rows of a slot, then the columns'.
            const int parity = warp - C::kLoadWarp;
            if (lane == 0) {
                tma_prefetch_map(&wmap);
                tma_prefetch_map(&amap);
            }
            const uint64_t keep = l2_evict_normal(), once = l2_evict_first();
            for (; ok && todo.next(w);) {
                // weights that one tile of tokens reads, an expert's only
                const uint64_t policy = experts.rows[w.e] <= (int)fp8_most(FEW) ? once : keep;
                // few: lane 0 the channels, then 16 tokens a lane; many: lane 0 the tokens, then 128
                // channels a lane
                constexpr int kBox = FEW ? 16 : 128;
                const int copies = 1 + (int)(w.n + kBox - 1) / kBox;
                const bool channels = FEW == (lane == 0);
                const int r = lane == 0 ? 0 : kBox * (lane - 1);
                const int y = r + (channels ? w.n0 : w.m0);
                const uint32_t bytes = C::kABytes + (uint32_t)((copies - 1) * kBox * kFp8Step);
                const uint32_t off = lane == 0 ? 0u : C::kABytes + (uint32_t)r * kFp8Step;
                for (uint32_t k = w.k0; k < w.k1; ++k, ++it) {
                    const int slot = it % C::kSlots;
                    if ((slot & 1) != parity) continue;
                    if (it >= C::kSlots) {
                        ok = fp8_wait(&empty[slot], (uint32_t)(it / C::kSlots - 1) & 1, q.wait_ns);
                        if (!ok) break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&full[slot], bytes);
                    __syncwarp();
                    if (q.drop && k == 1) continue;
                    unsigned char* const to = smem + slot * C::kSlotBytes + off;
                    const int x = (int)k * kFp8Step;
                    if (lane < copies) {
                        if (channels) tma_load_3d(to, &wmap, x, y, w.e, &full[slot], policy);
                        else tma_load_2d(to, &amap, x, y, &full[slot], keep);
                    }
                    __syncwarp();
                }
            }
            // every copy has landed, and every arrival on these barriers come, before the shared memory goes
            for (int i = max(it - C::kSlots, 0); i < it; ++i)
                if (((i % C::kSlots) & 1) == parity) {
                    fp8_wait(&full[i % C::kSlots], (uint32_t)(i / C::kSlots) & 1, q.wait_ns);
                    ok = ok && fp8_wait(&empty[i % C::kSlots], (uint32_t)(i / C::kSlots) & 1, q.wait_ns);
                }
        } else if (warp == C::kMulWarp) {
            // One thread: a vote after every wait and a choice of the thread for every step took
            // a third of a step
            if (elect_one()) {
                const uint64_t a0 = umma_smem_desc(smem_u32(smem));
                for (; ok && todo.next(w);) {
                    const uint32_t idesc = umma_e4m3_desc<128>(w.n);
                    for (uint32_t k = w.k0; k < w.k1; ++k, ++it) {
                        const int slot = it % C::kSlots, a = it % C::kAccs;
                        ok = mbar_wait(&full[slot], (uint32_t)(it / C::kSlots) & 1, q.wait_ns);
                        if (!FEW && it >= C::kAccs) ok = ok && mbar_wait(&acc_empty[a], (uint32_t)(it / C::kAccs - 1) & 1, q.wait_ns);
                        if (!ok) break;
                        tmem_fence_after();
                        // descriptors count addresses in units of 16 bytes
                        const uint64_t at = a0 + (uint32_t)slot * (C::kSlotBytes / 16), b = at + C::kABytes / 16;
#pragma unroll
                        for (int j = 0; j < kFp8Step / 32; ++j)
                            umma_e4m3(tmem + a * C::kColumns, at + 2 * j, b + 2 * j, idesc, j > 0);
                        umma_commit<1>(&acc_full[a]);
                        if (!FEW) umma_commit<1>(&empty[slot]);
                    }
                }
                // its instructions have ended, and the readers' arrivals come, before the memory goes, also
                // where the warps that read have given up
                for (int i = max(it - C::kAccs, 0); i < it; ++i) {
                    mbar_wait(&acc_full[i % C::kAccs], (uint32_t)(i / C::kAccs) & 1, q.wait_ns);
                    ok = ok && mbar_wait(&acc_empty[i % C::kAccs], (uint32_t)(i / C::kAccs) & 1, q.wait_ns);
                }
            }
            __syncwarp();
        } else {
            // Scales: a's of every token times w's of the channels' block, rounded once to FP32.
            // Four steps' are fetched at a time: the way to L2 takes longer than a step.
            constexpr int kEach = (FEW ? kFp8Few : 128) / 32, kBlocks = FEW ? 1 : 2;
            const uint32_t w_rows = fp8_up((uint32_t)q.N, kFp8Block128);
            for (; ok && todo.next(w);) {
                const float* ws[kBlocks];
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
                    ws[b] = q.w_scale + ((size_t)w.e * w_rows + min((uint32_t)w.n0 / kFp8Block128 + b, w_rows - 1)) * q.steps;
                const float* as = q.a_scale + (size_t)(w.m0 + lane) * q.steps;
                for (uint32_t g = w.k0 & ~3u; g < w.k1; g += 4) {
                    float f[kBlocks][4], v[kEach][4];
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                        for (int j = 0; j < 4; ++j) f[b][j] = g + j < w.k1 ? __ldg(ws[b] + g + j) : 0.f;
#pragma unroll
                    for (int i = 0; i < kEach; ++i) {
                        const float* from = as + (size_t)(32 * i) * q.steps + g;
                        const bool in = lane + 32 * i < w.cols;
                        if (q.scales16) {
                            const float4 u = in ? __ldg(reinterpret_cast<const float4*>(from)) : make_float4(0.f, 0.f, 0.f, 0.f);
                            v[i][0] = u.x; v[i][1] = u.y; v[i][2] = u.z; v[i][3] = u.w;
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j) v[i][j] = in && g + j < w.k1 ? __ldg(from + j) : 0.f;
                        }
                    }
                    if (sturn > 0) {
                        ok = fp8_wait(&scale_empty[sg], (uint32_t)(sturn - 1) & 1, q.wait_ns);
                        if (!ok) break;
                    }
#pragma unroll
                    for (int i = 0; i < kEach; ++i)
#pragma unroll
                        for (int b = 0; b < kBlocks; ++b) {
                            float4* const to = scales + sg * C::kScaleRow;
                            float p[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) p[j] = __fmul_rn(v[i][j], f[b][j]);
                            if constexpr (FEW) {
#pragma unroll
                                for (int j = 0; j < 4; ++j) reinterpret_cast<float*>(to)[j * C::kColumns + 32 * i + lane] = p[j];
                            } else {
                                to[b * 128 + 32 * i + lane] = make_float4(p[0], p[1], p[2], p[3]);
                            }
                        }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&scale_full[sg]);
                    if (++sg == C::kScales / 4) {
                        sg = 0;
                        ++sturn;
                    }
                }
            }
        }
    }
    if (!ok) atomicOr(q.status, 1u);
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if (q.split > 1) cluster_sync();  // nobody leaves while another CTA works with its memory
    if (warp == C::kMulWarp) {
        tmem_fence_after();
        tmem_dealloc<1, C::kTmem>(tmem);
    }
}

}  // namespace beam

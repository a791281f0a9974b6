// The product of E4M3 numbers with a scale for each 128 of a token and each 128 by 128
// of the channels, for one matrix of channels or one for each expert.
//
//   out[m, n] = sum_b RN(a_scale[m, b] w_scale[n / 128, b]) P_b,   P_b = sum_{k in b} a[m, k] w[n, k]
//
// The tensor cores' E4M3 kind adds P_b in FP32 (128 products: off by at most 2^-23 of
// their absolute sum as measured, where an 8-bit product keeps 8 bits). The scales change
// with every 128 k, so P_b does not stay in the accumulator: the matrix unit writes it
// to one of a few accumulators in tensor memory, and eight (four) warps read it, multiply by
// the scales and add it to sums that they hold in registers, in FP32, while the next is
// being made.
//
// Channels are the rows of A (lanes of tensor memory), tokens the rows of B (columns):
//   - the instruction's n is any multiple of 16, so that an expert's rows, however many,
//     fill their tiles; its m is not;
//   - a scale of w belongs to a whole CTA and step, one of a to a column. Read as 16 x 256b
//     fragments a thread holds two neighbouring columns of four lanes: one 8-byte shared
//     load brings the scales of eight values, which are scaled and added two at a time.
//     (As 32 x 32b, thread = channel, every value needs its own scale from shared memory.)
//   - for few tokens it is the weights that stream.
// Results are rounded, transposed 8 x 8 in registers, put together in shared memory and
// stored 16 bytes a thread, 64 bytes of a row a warp.
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
    uint32_t steps, n_tiles, most;  // of k; of channels; tokens of a tile at most
    int split;                 // CTAs (pairs) of a cluster, which share a tile's steps
    int scales16;              // rows of a_scale are whole groups of 16 bytes
    int wide;                  // rows of a BF16 out start and end on 16 bytes
    uint64_t wait_ns;
    int drop;                  // test hook: every tile's second step is never loaded
    unsigned int* status;
};

// CG = 1: a CTA with 128 channels and up to 64 tokens; CG = 2: a pair of CTAs on one
// tensor tile, 128 channels each and half of up to 256 tokens
template <int CG>
struct Fp8Tile {
    static constexpr int kTokens = CG == 1 ? kFp8Few : kFp8Many;
    static constexpr int kRows = kTokens / CG;      // of B in a CTA
    static constexpr int kSlots = CG == 1 ? 7 : 6;  // ring of operand tiles
    static constexpr int kAccs = CG == 1 ? 4 : 2;   // accumulators of a step
    static constexpr int kHalves = CG;              // ... each in halves of the columns, which come and go apart
    static constexpr int kScales = 8;               // ring of a step's scales
    // Warps: those that add, in groups of four (a group has all lanes and a share of the
    // columns); two that load, every second slot each; one that brings scales; one that
    // multiplies.
    static constexpr int kGroups = CG == 1 ? 2 : 4, kAddWarps = 4 * kGroups;
    static constexpr int kColumns = kTokens / kGroups;  // of an adding warp
    static constexpr int kLoadWarp = kAddWarps, kScaleWarp = kLoadWarp + 2, kMulWarp = kScaleWarp + 1;
    static constexpr int kThreads = 32 * (kMulWarp + 1);
    // Pairs: the adding warps take registers from the others (4 x 104 + 64 = 5 x 96)
    static constexpr int kAddRegs = 104, kOtherRegs = 64;
    static constexpr uint32_t kABytes = kFp8Chan * kFp8Step;
    static constexpr uint32_t kSlotBytes = kABytes + kRows * kFp8Step;
    static constexpr uint32_t kRedAt = kSlots * kSlotBytes;                  // sums from the cluster's other CTAs
    static constexpr uint32_t kRedBytes = CG == 1 ? (kFp8MaxSplit - 1) * 4096 : 0;
    static constexpr uint32_t kScaleAt = kRedAt + kRedBytes;                 // FP32 [kScales][kTokens]
    static constexpr uint32_t kStageWarp = 8 * 80;                           // 8 rows of 64 bytes, 16 apart
    static constexpr uint32_t kStageAt = kScaleAt + kScales * kTokens * 4;
    static constexpr uint32_t kTableAt = kStageAt + kAddWarps * kStageWarp;  // experts: first tile, first row, rows
    static constexpr uint32_t kBarAt = kTableAt + (3 * kFp8MaxExperts + 4) * 4;
    static constexpr int kBars = 2 * kSlots + 2 * kAccs * kHalves + 2 * kScales + 2;
    static constexpr uint32_t kSmem = kBarAt + kBars * 8 + 16;
    static constexpr uint32_t kTmem = kAccs * kTokens;
    static_assert(kTmem <= 512 && kSmem <= 232448 && kBarAt % 8 == 0, "tensor memory, shared memory of a CTA");
};

// Which rows and tiles an expert has, in shared memory
struct Fp8Experts {
    uint32_t* tile;  // [E + 1] tiles before it
    int32_t *row, *rows;
};

struct Fp8Work {
    int e, n0, m0;        // expert; this CTA's first channel; the tile's first row of a and out
    uint32_t cols, n;     // its tokens, and the instruction's n
};

// The tiles worker, worker + workers, ... in order
template <int CG>
class Fp8Schedule {
    const Fp8Params& q;
    const Fp8Experts& x;
    const uint32_t rank, stride;
    uint32_t at;
    int e = 0;

public:
    __device__ Fp8Schedule(const Fp8Params& q_, const Fp8Experts& x_, uint32_t worker, uint32_t workers, uint32_t rank_)
        : q(q_), x(x_), rank(rank_), stride(workers), at(worker) {}
    __device__ bool next(Fp8Work& w) {
        while (e < q.E && at >= x.tile[e + 1]) ++e;
        if (e >= q.E) return false;
        const uint32_t rows = (uint32_t)x.rows[e];
        const Fp8Rows r = fp8_rows(rows, q.most, 16 * CG);
        uint32_t m, n;
        fp8_place(at - x.tile[e], r.tiles, q.n_tiles, &m, &n);
        w.e = e;
        w.n0 = (int)((n * CG + rank) * kFp8Chan);
        w.m0 = x.row[e] + (int)(m * r.each);
        w.cols = min(r.each, rows - m * r.each);
        w.n = fp8_up(w.cols, 16 * CG) * (16 * CG);
        at += stride;
        return true;
    }
};

// all lanes: whether every lane's wait ended
template <int CG = 1>
__device__ __forceinline__ bool fp8_wait(uint64_t* bar, uint32_t parity, uint64_t ns) {
    return __all_sync(0xFFFFFFFFu, mbar_wait<CG>(bar, parity, ns));
}

template <int REGS>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(REGS)); }
template <int REGS>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(REGS)); }

template <int CG, bool F32>
__global__ void __launch_bounds__(Fp8Tile<CG>::kThreads, 1)
    matmul_fp8_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap64,
                      const __grid_constant__ CUtensorMap amap16, const __grid_constant__ Fp8Params q) {
    using C = Fp8Tile<CG>;
    extern __shared__ __align__(1024) unsigned char smem[];
    float* const scales = reinterpret_cast<float*>(smem + C::kScaleAt);
    uint32_t* const table = reinterpret_cast<uint32_t*>(smem + C::kTableAt);
    const Fp8Experts experts{table, reinterpret_cast<int32_t*>(table + kFp8MaxExperts + 4),
                             reinterpret_cast<int32_t*>(table + 2 * kFp8MaxExperts + 4)};
    uint64_t* const full = reinterpret_cast<uint64_t*>(smem + C::kBarAt);  // a slot's tiles have landed (the pair's: in its first CTA)
    uint64_t* const empty = full + C::kSlots;             // ... are multiplied
    uint64_t* const acc_full = empty + C::kSlots;                     // half of a step's columns are multiplied
    uint64_t* const acc_empty = acc_full + C::kAccs * C::kHalves;     // ... and read, by both CTAs
    uint64_t* const scale_full = acc_empty + C::kAccs * C::kHalves;   // a step's scales are there
    uint64_t* const scale_empty = scale_full + C::kScales;
    uint64_t* const red_full = scale_empty + C::kScales;  // the other CTAs' sums of a tile are there
    uint64_t* const red_empty = red_full + 1;             // this CTA's are read
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(red_empty + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // place in the cluster: share of the steps, half of the pair
    const uint32_t place = CG == 2 || q.split > 1 ? cluster_rank() : 0u;
    const uint32_t share = place / CG, rank = place % CG;
    const uint32_t worker = blockIdx.x / (CG * q.split), workers = gridDim.x / (CG * q.split);
    const uint32_t k0 = q.steps * share / q.split, k1 = q.steps * (share + 1) / q.split;

    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::kAccs * C::kHalves; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], C::kAddWarps / C::kHalves * CG);
        }
        for (int i = 0; i < C::kScales; ++i) {
            mbar_init(&scale_full[i], 1);
            mbar_init(&scale_empty[i], C::kAddWarps);
        }
        mbar_init(red_full, (q.split > 1 ? q.split - 1 : 1) * C::kAddWarps);
        mbar_init(red_empty, (q.split > 1 ? q.split - 1 : 1) * C::kAddWarps);
        mbar_fence_init();
    }
    if (warp == C::kMulWarp) tmem_alloc<CG, C::kTmem>(tmem_slot);
    // Experts' rows. Offsets that decrease or leave [0, R] are held within: what they
    // make of out is not said, but nothing outside of it is touched.
    bool bad = false;
    for (int e = tid; e < q.E; e += C::kThreads) {
        long long lo = 0, hi = q.R;
        if (q.offsets) {
            const long long a = __ldg(q.offsets + e), b = __ldg(q.offsets + e + 1);
            lo = min(max(a, 0ll), q.R);
            hi = min(max(b, lo), q.R);
            bad |= lo != a || hi != b;
        }
        experts.row[e] = (int32_t)lo;
        experts.rows[e] = (int32_t)(hi - lo);
    }
    if (bad && worker == 0) atomicOr(q.status, 2u);
    __syncthreads();
    if (warp == 0) {
        constexpr int kEach = kFp8MaxExperts / 32;
        uint32_t sum = 0;
        for (int i = 0; i < kEach; ++i) {
            const int e = lane * kEach + i;
            if (e < q.E) sum += fp8_up((uint32_t)experts.rows[e], q.most) * q.n_tiles;
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
                before += fp8_up((uint32_t)experts.rows[e], q.most) * q.n_tiles;
                if (e == q.E - 1) experts.tile[q.E] = before;
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (CG == 2 || q.split > 1) cluster_sync();  // the other CTAs' barriers are ready too
    tmem_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;
    Fp8Schedule<CG> todo(q, experts, worker, workers, rank);
    Fp8Work w;
    int it = 0;  // steps so far

    if (warp < C::kAddWarps) {
        if constexpr (CG == 2) more_registers<C::kAddRegs>();
        // Columns of a group: a share of one half. A half's columns are a quarter of the tile's
        // tokens from each CTA's rows of B, so the group's are neighbouring tokens.
        const int group = warp >> 2, half = group * C::kHalves / C::kGroups, chan = 32 * (warp & 3);
        const uint32_t lanes = tmem + ((uint32_t)chan << 16) + half * (C::kTokens / C::kHalves);
        unsigned char* const stage = smem + C::kStageAt + warp * C::kStageWarp;
        for (int tile = 0; ok && todo.next(w); ++tile) {
            // sums[j][i]: columns 8 j + 2 (lane % 4) and the next, channel 8 i + lane / 4
            float2 sums[C::kColumns / 8][4];
#pragma unroll
            for (int j = 0; j < C::kColumns / 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) sums[j][i] = make_float2(0.f, 0.f);
            const int mine = (int)w.n / C::kGroups;  // this warp's columns
            const int col = CG == 1 ? group * mine : (group & 1) * mine;
            const int c0 = CG == 1 ? col : (2 * (group & 1) + half) * mine;  // its first token
            const float* const sc = scales + c0 + 2 * (lane & 3);
            for (uint32_t k = k0; k < k1; ++k, ++it) {
                const int a = it % C::kAccs, h = a * C::kHalves + half, s = it % C::kScales;
                ok = fp8_wait(&scale_full[s], (uint32_t)(it / C::kScales) & 1, q.wait_ns) &&
                     fp8_wait(&acc_full[h], (uint32_t)(it / C::kAccs) & 1, q.wait_ns);
                if (!ok) break;
                tmem_fence_after();
                const uint32_t from = lanes + a * C::kTokens + col;
                // 16 columns at a time. A second eight that are not there are columns of this
                // accumulator that no tile stores.
#pragma unroll
                for (int c = 0; c < C::kColumns / 16; ++c) {
                    if (16 * c < mine) {
                        float v[2][8];
                        tmem_ld_16x256b(from + 16 * c, v[0]);
                        tmem_ld_16x256b(from + (16u << 16) + 16 * c, v[1]);
                        float2 f[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            f[j] = *reinterpret_cast<const float2*>(sc + s * C::kTokens + 16 * c + 8 * j);
                        tmem_wait_ld(v[0], v[1]);
                        if (16 * (c + 1) >= mine) {
                            // all read: the accumulator may be written again
                            tmem_fence_before();
                            __syncwarp();
                            if (lane == 0) {
                                if constexpr (CG == 2) mbar_arrive_cluster_relaxed(cluster_addr(&acc_empty[h], place & ~1u));
                                else mbar_arrive(&acc_empty[h]);
                                mbar_arrive(&scale_empty[s]);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float* p = &v[i >> 1][4 * j + 2 * (i & 1)];
                                sums[2 * c + j][i] = __ffma2_rn(make_float2(p[0], p[1]), f[j], sums[2 * c + j][i]);
                            }
                    }
                }
            }
            if (!ok) break;
            if constexpr (CG == 1) {
                // A tile that the cluster's CTAs have shares of: CTA d adds up and stores the
                // columns of every split-th group of eight, from sums that the others write to its
                // shared memory
                if (q.split > 1) {
                    const int n_groups = mine / 8, each = (C::kTokens / 8 + q.split - 1) / q.split, lane128 = tid & 127;
                    if (tile > 0) ok = fp8_wait<2>(red_empty, (uint32_t)(tile - 1) & 1, q.wait_ns);
                    if (!ok) break;
#pragma unroll
                    for (int j = 0; j < C::kColumns / 8; ++j) {
                        const int d = (j * C::kGroups + group) % q.split;
                        if (j < n_groups && d != (int)share) {
                            const int from = (int)share < d ? share : share - 1;
                            unsigned char* at = smem + C::kRedAt + ((from * each + (j * C::kGroups + group) / q.split) * 256 + lane128) * 16;
                            const uint32_t there = cluster_addr(at, d);
                            st_cluster(there, make_float4(sums[j][0].x, sums[j][0].y, sums[j][1].x, sums[j][1].y));
                            st_cluster(there + 2048, make_float4(sums[j][2].x, sums[j][2].y, sums[j][3].x, sums[j][3].y));
                        }
                    }
                    __syncwarp();
                    if (lane == 0)
                        for (int d = 0; d < q.split; ++d)
                            if (d != (int)share) mbar_arrive_cluster_release(cluster_addr(red_full, d));
                    ok = fp8_wait<2>(red_full, (uint32_t)tile & 1, q.wait_ns);
                    if (!ok) break;
#pragma unroll
                    for (int j = 0; j < C::kColumns / 8; ++j)
                        if (j < n_groups && (j * C::kGroups + group) % q.split == (int)share)
                            for (int from = 0; from < q.split - 1; ++from) {
                                const float4* at = reinterpret_cast<const float4*>(smem + C::kRedAt) +
                                                   (from * each + (j * C::kGroups + group) / q.split) * 256 + lane128;
                                const float4 u = at[0], v = at[128];
                                sums[j][0].x += u.x; sums[j][0].y += u.y; sums[j][1].x += u.z; sums[j][1].y += u.w;
                                sums[j][2].x += v.x; sums[j][2].y += v.y; sums[j][3].x += v.z; sums[j][3].y += v.w;
                            }
                    __syncwarp();
                    if (lane == 0)
                        for (int d = 0; d < q.split; ++d)
                            if (d != (int)share) mbar_arrive_cluster_release(cluster_addr(red_empty, d));
                }
            }
            const int n0 = w.n0 + chan;
            using Out = std::conditional_t<F32, float, uint16_t>;
            Out* const out = static_cast<Out*>(q.out) + (size_t)(w.m0 + c0) * (size_t)q.N + (size_t)n0;
            const int cols = (int)w.cols - c0;  // from this warp's first on
#pragma unroll
            for (int j = 0; j < C::kColumns / 8; ++j) {
                if (8 * j < mine && 8 * j < cols && (CG == 2 || (j * C::kGroups + group) % q.split == (int)share)) {
                    if constexpr (F32) {
                        // a warp's 32 values: 4 tokens by 8 channels, whole sectors
                        const int t = 8 * j + 2 * (lane & 3);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int ch = 8 * i + (lane >> 2);
                            if (n0 + ch < q.N) {
                                if (t < cols) out[(size_t)t * (size_t)q.N + ch] = sums[j][i].x;
                                if (t + 1 < cols) out[(size_t)(t + 1) * (size_t)q.N + ch] = sums[j][i].y;
                            }
                        }
                    } else {
                        __syncwarp();  // the last eight are read
#pragma unroll
                        for (int i = 0; i < 4; ++i)  // token lane / 4, channels 8 i + 2 (lane % 4) and the next
                            *reinterpret_cast<uint32_t*>(stage + (lane >> 2) * 80 + 16 * i + 4 * (lane & 3)) =
                                transpose_b16(f2_to_bf2(sums[j][i]));
                        __syncwarp();
                        if (q.wide) {
                            const int t = 8 * j + (lane >> 2), ch = 8 * (lane & 3);
                            const uint4 v = *reinterpret_cast<const uint4*>(stage + (lane >> 2) * 80 + 2 * ch);
                            if (t < cols && n0 + ch < q.N)
                                *reinterpret_cast<uint4*>(out + (size_t)t * (size_t)q.N + ch) = v;
                        } else if (n0 + lane < q.N) {
#pragma unroll
                            for (int t = 0; t < 8; ++t)
                                if (8 * j + t < cols)
                                    out[(size_t)(8 * j + t) * (size_t)q.N + lane] =
                                        *reinterpret_cast<const uint16_t*>(stage + t * 80 + 2 * lane);
                        }
                    }
                }
            }
        }
    } else {
        if constexpr (CG == 2) fewer_registers<C::kOtherRegs>();
        if (warp < C::kScaleWarp) {
            // Loads. A slot is always filled by the same warp, which therefore has seen every use
            // of it; its lanes issue a copy each.
            const int parity = warp - C::kLoadWarp;
            if (lane == 0) {
                tma_prefetch_map(&wmap);
                tma_prefetch_map(&amap64);
                tma_prefetch_map(&amap16);
            }
            const uint64_t keep = l2_evict_normal(), once = l2_evict_first();
            for (; ok && todo.next(w);) {
                const uint32_t rows = w.n / CG;  // of B in this CTA
                // weights that one tile of tokens reads, an expert's only
                const uint64_t policy = experts.rows[w.e] <= (int)q.most ? once : keep;
                const uint32_t bytes = CG * (C::kABytes + rows * kFp8Step);
                // lane 0: the channels; then 64 or 16 tokens a lane
                const int big = (int)rows / 64, copies = 1 + big + ((int)rows % 64) / 16;
                const bool wide = lane - 1 < big;
                const int r = wide ? 64 * (lane - 1) : 64 * big + 16 * (lane - 1 - big);
                const int y = w.m0 + (int)(rank * rows) + r;
                for (uint32_t k = k0; k < k1; ++k, ++it) {
                    const int slot = it % C::kSlots;
                    if ((slot & 1) != parity) continue;
                    if (it >= C::kSlots) {
                        ok = fp8_wait(&empty[slot], (uint32_t)(it / C::kSlots - 1) & 1, q.wait_ns);
                        if (!ok) break;
                    }
                    if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&full[slot], bytes);
                    __syncwarp();
                    if (q.drop && k == k0 + 1) continue;
                    unsigned char* const to = smem + slot * C::kSlotBytes;
                    const uint32_t bar = CG == 2 ? cluster_addr(&full[slot], place & ~1u) : smem_u32(&full[slot]);
                    const int x = (int)k * kFp8Step;
                    if (lane == 0) tma_load_3d<CG == 2>(to, &wmap, x, w.n0, w.e, bar, policy);
                    else if (lane < copies) tma_load_2d_on<CG == 2>(to + C::kABytes + r * kFp8Step, wide ? &amap64 : &amap16, x, y, bar, keep);
                    __syncwarp();
                }
            }
            // Every copy has landed, and every arrival on this CTA's barriers come, before the
            // shared memory goes. The pair's first CTA counts both CTAs' copies; where it gave up
            // the other leaves its copies the time to land.
            for (int i = max(it - C::kSlots, 0); i < it; ++i)
                if (((i % C::kSlots) & 1) == parity) {
                    if (rank == 0) fp8_wait(&full[i % C::kSlots], (uint32_t)(i / C::kSlots) & 1, q.wait_ns);
                    ok = ok && fp8_wait(&empty[i % C::kSlots], (uint32_t)(i / C::kSlots) & 1, q.wait_ns);
                }
            if (!ok && rank != 0) {
                const uint64_t t0 = global_ns();
                while (global_ns() - t0 < 1000000ull) __nanosleep(1000);
            }
        } else if (warp == C::kMulWarp) {
            if (rank == 0) {
                const uint64_t a0 = umma_smem_desc(smem_u32(smem)), b0 = a0 + C::kABytes / 16;
                for (; ok && todo.next(w);) {
                    const uint32_t idesc = umma_e4m3_desc<kFp8Chan * CG>(w.n / C::kHalves);
                    for (uint32_t k = k0; k < k1; ++k, ++it) {
                        const int a = it % C::kAccs, slot = it % C::kSlots;
                        // descriptors count addresses in units of 16 bytes
                        const uint32_t at = (uint32_t)slot * (C::kSlotBytes / 16);
                        ok = fp8_wait(&full[slot], (uint32_t)(it / C::kSlots) & 1, q.wait_ns);
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h) {
                            uint64_t* const done = &acc_full[a * C::kHalves + h];
                            if (it >= C::kAccs)
                                ok = ok && fp8_wait(&acc_empty[a * C::kHalves + h], (uint32_t)(it / C::kAccs - 1) & 1, q.wait_ns);
                            if (!ok) break;
                            tmem_fence_after();
                            const uint32_t d = tmem + a * C::kTokens + h * (C::kTokens / C::kHalves);
                            const uint64_t b = b0 + at + h * (w.n / (CG * C::kHalves)) * (kFp8Step / 16);
                            if (elect_one()) {
#pragma unroll
                                for (int j = 0; j < kFp8Step / 32; ++j)
                                    umma_e4m3<CG>(d, a0 + at + 2 * j, b + 2 * j, idesc, j > 0);
                                if constexpr (CG == 2) umma_commit_pair(done, 3u << place);
                                else umma_commit<1>(done);
                                if (h == C::kHalves - 1) {
                                    if constexpr (CG == 2) umma_commit_pair(&empty[slot], 3u << place);
                                    else umma_commit<1>(&empty[slot]);
                                }
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                    }
                }
                // its instructions have ended, and the readers' arrivals come, before the memory goes
                for (int i = max(it - C::kAccs, 0); i < it; ++i)
                    for (int h = i % C::kAccs * C::kHalves, n = 0; n < C::kHalves; ++h, ++n) {
                        fp8_wait(&acc_full[h], (uint32_t)(i / C::kAccs) & 1, q.wait_ns);
                        ok = ok && fp8_wait(&acc_empty[h], (uint32_t)(i / C::kAccs) & 1, q.wait_ns);
                    }
            }
        } else {
            // Scales of a step: a's of every token times w's of this CTA's channels, rounded once
            // to FP32. Four steps' are fetched at a time: the way to L2 takes longer than a step
            // (one step at a time: 0.96 us a step for 256 tokens, where the matrix unit takes 0.27).
            constexpr int kEach = C::kTokens / 32;
            const uint32_t w_rows = fp8_up((uint32_t)q.N, kFp8Chan);
            for (; ok && todo.next(w);) {
                const uint32_t w_row = min((uint32_t)w.n0 / kFp8Chan, w_rows - 1);
                const float* ws = q.w_scale + ((size_t)w.e * w_rows + w_row) * q.steps;
                const float* as = q.a_scale + (size_t)(w.m0 + lane) * q.steps;
                for (uint32_t g = k0 & ~3u; ok && g < k1; g += 4) {
                    float f[4], v[kEach][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[j] = g + j < k1 ? __ldg(ws + g + j) : 0.f;
#pragma unroll
                    for (int i = 0; i < kEach; ++i) {
                        const float* from = as + (size_t)(32 * i) * q.steps + g;
                        const bool in = lane + 32 * i < (int)w.cols;
                        if (q.scales16) {
                            const float4 u = in ? __ldg(reinterpret_cast<const float4*>(from)) : make_float4(0.f, 0.f, 0.f, 0.f);
                            v[i][0] = u.x; v[i][1] = u.y; v[i][2] = u.z; v[i][3] = u.w;
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j) v[i][j] = in && g + j < k1 ? __ldg(from + j) : 0.f;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (g + j < k0 || g + j >= k1) continue;
                        const int s = it % C::kScales;
                        if (it >= C::kScales) {
                            ok = fp8_wait(&scale_empty[s], (uint32_t)(it / C::kScales - 1) & 1, q.wait_ns);
                            if (!ok) break;
                        }
                        ++it;
#pragma unroll
                        for (int i = 0; i < kEach; ++i)
                            scales[s * C::kTokens + lane + 32 * i] = __fmul_rn(v[i][j], f[j]);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&scale_full[s]);
                    }
                }
            }
        }
    }
    if (!ok) atomicOr(q.status, 1u);
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if (CG == 2 || q.split > 1) cluster_sync();  // nobody leaves while another CTA works with its memory
    if (warp == C::kMulWarp) {
        tmem_fence_after();
        tmem_dealloc<CG, C::kTmem>(tmem);
    }
}

}  // namespace beam

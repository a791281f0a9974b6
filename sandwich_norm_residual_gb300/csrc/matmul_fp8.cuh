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
//   - An SM takes 64 bytes a clock from L2. 128 tokens by 256 channels on one SM bring 48 KB
//     a step, 768 clocks, where its products take 512; a pair of SMs on 256 by 256 brings 32 KB
//     to each (M = 2048, N = 4864, K = 20480: 194 and 152 us).
//   - What the adding warps do beside reading, multiplying and adding counts twice: their
//     waits end with no vote, scales come four steps at a time, the barriers' places are
//     kept, not computed (200 -> 152 us; without any reading and adding 122 us).
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

// Few tokens: a CTA with 128 channels and up to 64 tokens. Many: a pair of CTAs on one tensor
// tile, 128 tokens each, that share up to 256 channels: either loads half of them.
template <bool FEW>
struct Fp8Tile {
    static constexpr int CG = FEW ? 1 : 2;
    static constexpr int kColumns = FEW ? kFp8Few : kFp8Width;  // of an accumulator
    static constexpr int kSlots = FEW ? 7 : 6;       // ring of operand tiles
    static constexpr int kAccs = FEW ? 4 : 2;        // accumulators of a step
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
    static constexpr uint32_t kSlotBytes = kABytes + kColumns / CG * kFp8Step;
    static constexpr uint32_t kRedAt = kSlots * kSlotBytes;                  // sums from the cluster's other CTAs
    static constexpr uint32_t kRedBytes = FEW ? (kFp8MaxSplit - 1) * 4096 : 0;
    static constexpr uint32_t kScaleAt = kRedAt + kRedBytes;                 // FP32 [kScales][kScaleRow]
    static constexpr uint32_t kTableAt = kScaleAt + kScales * kScaleRow * 4; // experts: first tile, first row, rows
    static constexpr uint32_t kBarAt = kTableAt + (3 * kFp8MaxExperts + 4) * 4;
    static constexpr int kBars = 2 * kSlots + 2 * kAccs + 2 * (kScales / 4) + 2;
    static constexpr uint32_t kSmem = kBarAt + kBars * 8 + 16;
    static constexpr uint32_t kTmem = kAccs * kColumns;
    static_assert(kTmem <= 512 && kSmem <= 232448 && kBarAt % 8 == 0, "tensor memory, shared memory of a CTA");
};

// Which rows and tiles an expert has, in shared memory
struct Fp8Experts {
    uint32_t* tile;  // [E + 1] tiles before it
    int32_t *row, *rows;
};

struct Fp8Work {
    int e, n0, m0;     // expert; the tile's first channel; this CTA's first row of a and out
    int cols;          // this CTA's tokens
    uint32_t n;        // the instruction's columns: tokens (few) or channels (many), a multiple of 16
    uint32_t k0, k1;   // this CTA's steps
    bool shared;       // the cluster's CTAs each have some of the tile's steps
};

// Worker c of W (a CTA, or a pair) takes the tiles c, c + W, ... Where clusters share (few
// tokens), only the tiles behind the last full wave are shared, one by a cluster at a
// time: a join takes as long as some ten steps.
template <bool FEW>
class Fp8Schedule {
    const Fp8Params& q;
    const Fp8Experts& x;
    const uint32_t rank, worker, workers, place;
    uint32_t at, whole;  // the next tile; the tiles that are not shared
    int e = 0;

public:
    // place: in the cluster
    __device__ Fp8Schedule(const Fp8Params& q_, const Fp8Experts& x_, uint32_t place_)
        : q(q_), x(x_), rank(FEW ? 0u : place_), worker(FEW ? blockIdx.x : blockIdx.x / 2), workers(FEW ? gridDim.x : gridDim.x / 2),
          place(place_), at(worker), whole(0xFFFFFFFFu) {
        if (FEW && q.split > 1) {
            whole = x.tile[q.E] / workers * workers;
            if (at >= whole) at = whole + worker / q.split;
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
        const uint32_t before = m * r.each + rank * 128;
        w.m0 = x.row[e] + (int)before;
        w.cols = (int)min(FEW ? r.each : 128u, rows - min(rows, before));
        w.n = FEW ? fp8_up((uint32_t)w.cols, 16) * 16 : min(q.width, fp8_up((uint32_t)(q.N - w.n0), 16) * 16);
        w.shared = FEW && at >= whole;
        w.k0 = w.shared ? q.steps * place / q.split : 0u;
        w.k1 = w.shared ? q.steps * (place + 1) / q.split : q.steps;
        if (w.shared) {
            at += workers / q.split;
        } else {
            at += workers;
            if (FEW && at >= whole) at = whole + worker / q.split;
        }
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
                      const __grid_constant__ CUtensorMap amap16, const __grid_constant__ Fp8Params q) {
    using C = Fp8Tile<FEW>;
    extern __shared__ __align__(1024) unsigned char smem[];
    float4* const scales = reinterpret_cast<float4*>(smem + C::kScaleAt);
    uint32_t* const table = reinterpret_cast<uint32_t*>(smem + C::kTableAt);
    const Fp8Experts experts{table, reinterpret_cast<int32_t*>(table + kFp8MaxExperts + 4),
                             reinterpret_cast<int32_t*>(table + 2 * kFp8MaxExperts + 4)};
    uint64_t* const full = reinterpret_cast<uint64_t*>(smem + C::kBarAt);  // a slot's tiles have landed
    uint64_t* const empty = full + C::kSlots;                 // ... are multiplied
    uint64_t* const acc_full = empty + C::kSlots;             // a step is multiplied
    uint64_t* const acc_empty = acc_full + C::kAccs;          // ... and read
    uint64_t* const scale_full = acc_empty + C::kAccs;        // four steps' scales are there
    uint64_t* const scale_empty = scale_full + C::kScales / 4;
    uint64_t* const red_full = scale_empty + C::kScales / 4;  // the other CTAs' sums of a tile are there
    uint64_t* const red_empty = red_full + 1;                 // this CTA's are read
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(red_empty + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t place = !FEW || q.split > 1 ? cluster_rank() : 0u;
    const uint32_t rank = FEW ? 0u : place;  // in the pair

    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::kAccs; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], C::kAddWarps * C::CG);
        }
        for (int i = 0; i < C::kScales / 4; ++i) {
            mbar_init(&scale_full[i], 1);
            mbar_init(&scale_empty[i], C::kAddWarps);
        }
        mbar_init(red_full, (q.split > 1 ? q.split - 1 : 1) * C::kAddWarps);
        mbar_init(red_empty, (q.split > 1 ? q.split - 1 : 1) * C::kAddWarps);
        mbar_fence_init();
    }
    if (warp == C::kMulWarp) tmem_alloc<C::CG, C::kTmem>(tmem_slot);
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
    if (bad && blockIdx.x == 0) atomicOr(q.status, 2u);
    __syncthreads();
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
    if (!FEW || q.split > 1) cluster_sync();  // the other CTAs' barriers are ready too
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
        const uint32_t leader_empty = FEW ? 0u : cluster_addr(acc_empty, 0);
        int a = 0, aturn = 0;
        int joins = 0;
        while (todo.next(w)) {
            float2 sums[C::kMine / 2];
#pragma unroll
            for (int j = 0; j < C::kMine / 2; ++j) sums[j] = make_float2(0.f, 0.f);
            // this warp's columns: a share of the tokens, or of the tile's channels (within a block of 128)
            const int mine = FEW ? (int)w.n / C::kGroups : C::kMine, c0 = group * mine;
            const bool some = FEW || c0 < (int)w.n;
            // scales come in groups of four steps, at multiples of four
            for (uint32_t g = w.k0 & ~3u; g < w.k1; g += 4) {
                if (ok) ok = mbar_wait(&scale_full[sg], sturn & 1, q.wait_ns);
                __syncwarp();
                // many: this thread's token's in the four steps
                const float4 own = FEW ? float4{} : scales[sg * C::kScaleRow + group * 128 + row];
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
                            if (!FEW || 16 * c < mine) {
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
                    if (lane == 0) {
                        if constexpr (FEW) mbar_arrive(&acc_empty[a]);
                        else mbar_arrive_cluster_relaxed(leader_empty + a * 8);
                    }
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
            if constexpr (FEW) {
                // A tile that the cluster's CTAs have shares of: CTA d adds up and stores every
                // split-th group of eight columns, from sums that the others write to its shared memory
                const int n_groups = mine / 8;
                if (w.shared) {
                    const int each = (C::kColumns / 8 + q.split - 1) / q.split;
                    if (joins > 0 && ok) ok = mbar_wait(red_empty, (uint32_t)(joins - 1) & 1, q.wait_ns);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < C::kMine / 8; ++j) {
                        const int g = j * C::kGroups + group, d = g % q.split;
                        if (j < n_groups && d != (int)place) {
                            const int slot = ((int)place < d ? (int)place : (int)place - 1) * each + g / q.split;
                            const uint32_t there = cluster_addr(smem + C::kRedAt + (slot * 256 + row) * 16, d);
                            st_cluster(there, make_float4(sums[4 * j].x, sums[4 * j].y, sums[4 * j + 1].x, sums[4 * j + 1].y));
                            st_cluster(there + 2048, make_float4(sums[4 * j + 2].x, sums[4 * j + 2].y, sums[4 * j + 3].x, sums[4 * j + 3].y));
                        }
                    }
                    __syncwarp();
                    if (lane == 0)
                        for (int d = 0; d < q.split; ++d)
                            if (d != (int)place) mbar_arrive_cluster_release(cluster_addr(red_full, d));
                    if (ok) ok = mbar_wait<2>(red_full, (uint32_t)joins & 1, q.wait_ns);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < C::kMine / 8; ++j) {
                        const int g = j * C::kGroups + group;
                        if (j < n_groups && g % q.split == (int)place)
                            for (int from = 0; from < q.split - 1; ++from) {
                                const float4* at = reinterpret_cast<const float4*>(smem + C::kRedAt) + (from * each + g / q.split) * 256 + row;
                                const float4 u = at[0], v = at[128];
                                sums[4 * j].x += u.x; sums[4 * j].y += u.y; sums[4 * j + 1].x += u.z; sums[4 * j + 1].y += u.w;
                                sums[4 * j + 2].x += v.x; sums[4 * j + 2].y += v.y; sums[4 * j + 3].x += v.z; sums[4 * j + 3].y += v.w;
                            }
                    }
                    __syncwarp();
                    if (lane == 0)
                        for (int d = 0; d < q.split; ++d)
                            if (d != (int)place) mbar_arrive_cluster_relaxed(cluster_addr(red_empty, d));
                    ++joins;
                }
                // thread = channel: a warp's store is 32 neighbours of a row
                Out* const to = out + (size_t)(w.m0 + c0) * (size_t)q.N + (size_t)(w.n0 + row);
                const int cols = w.cols - c0;  // from this warp's first on
                if (w.n0 + row < q.N) {
#pragma unroll
                    for (int j = 0; j < C::kMine / 2; ++j)
                        if (!w.shared || (j / 4 * C::kGroups + group) % q.split == (int)place) {
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
                            if (kBatch * j < left) {
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
                } else {
                    // rows that do not start on a sector: transposed, 32 neighbours of a row a store
#pragma unroll
                    for (int c = 0; c < C::kMine / 32; ++c) {
                        {
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
                if (FEW) tma_prefetch_map(&amap16);
            }
            const uint64_t keep = l2_evict_normal(), once = l2_evict_first();
            for (; ok && todo.next(w);) {
                // weights that one tile of tokens reads, an expert's only
                const uint64_t policy = experts.rows[w.e] <= (FEW ? kFp8Few : kFp8Many) ? once : keep;
                // few: lane 0 the channels, then 64 or 16 tokens a lane; many: lane 0 the tokens, lane 1
                // this CTA's half of the channels
                const int big = FEW ? (int)w.n / 64 : 1, copies = 1 + big + (FEW ? (int)w.n % 64 / 16 : 0);
                const bool whole = lane - 1 < big, channels = FEW == (lane == 0);
                const int r = lane == 0 || !FEW ? 0 : whole ? 64 * (lane - 1) : 64 * big + 16 * (lane - 1 - big);
                const int y = channels ? w.n0 + (int)(rank * (w.n / 2)) : w.m0 + r;
                const uint32_t bytes = FEW ? C::kABytes + w.n * kFp8Step : 2 * C::kSlotBytes;
                const uint32_t off = lane == 0 ? 0u : C::kABytes + (uint32_t)r * kFp8Step;
                for (uint32_t k = w.k0; k < w.k1; ++k, ++it) {
                    const int slot = it % C::kSlots;
                    if ((slot & 1) != parity) continue;
                    if (it >= C::kSlots) {
                        ok = fp8_wait(&empty[slot], (uint32_t)(it / C::kSlots - 1) & 1, q.wait_ns);
                        if (!ok) break;
                    }
                    if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&full[slot], bytes);
                    __syncwarp();
                    if (q.drop && k == w.k0 + 1) continue;
                    const uint32_t bar = FEW ? smem_u32(&full[slot]) : cluster_addr(&full[slot], 0);
                    unsigned char* const to = smem + slot * C::kSlotBytes + off;
                    const int x = (int)k * kFp8Step;
                    if (lane < copies) {
                        if (channels) tma_load_3d<C::CG>(to, &wmap, x, y, w.e, bar, policy);
                        else tma_load_3d<C::CG>(to, FEW && !whole ? &amap16 : &amap, x, y, 0, bar, keep);
                    }
                    __syncwarp();
                }
            }
            // Every copy has landed, and every arrival on these barriers come, before the shared memory
            // goes. The pair's first CTA counts both CTAs' copies; where it gave up, the other
            // leaves its copies the time to land.
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
            // One thread: a vote after every wait and a choice of the thread for every step took
            // a third of a step
            if (rank == 0 && elect_one()) {
                const uint64_t a0 = umma_smem_desc(smem_u32(smem));
                for (; ok && todo.next(w);) {
                    const uint32_t idesc = umma_e4m3_desc<128 * C::CG>(w.n);
                    for (uint32_t k = w.k0; k < w.k1; ++k, ++it) {
                        const int slot = it % C::kSlots, a = it % C::kAccs;
                        ok = mbar_wait(&full[slot], (uint32_t)(it / C::kSlots) & 1, q.wait_ns);
                        if (it >= C::kAccs) ok = ok && mbar_wait(&acc_empty[a], (uint32_t)(it / C::kAccs - 1) & 1, q.wait_ns);
                        if (!ok) break;
                        tmem_fence_after();
                        // descriptors count addresses in units of 16 bytes
                        const uint64_t at = a0 + (uint32_t)slot * (C::kSlotBytes / 16), b = at + C::kABytes / 16;
#pragma unroll
                        for (int j = 0; j < kFp8Step / 32; ++j)
                            umma_e4m3<C::CG>(tmem + a * C::kColumns, at + 2 * j, b + 2 * j, idesc, j > 0);
                        umma_commit<C::CG>(&acc_full[a]);
                        umma_commit<C::CG>(&empty[slot]);
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
    if (!FEW || q.split > 1) cluster_sync();  // nobody leaves while another CTA works with its memory
    if (warp == C::kMulWarp) {
        tmem_fence_after();
        tmem_dealloc<C::CG, C::kTmem>(tmem);
    }
}

}  // namespace beam

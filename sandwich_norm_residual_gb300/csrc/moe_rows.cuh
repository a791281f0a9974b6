// Tokens sorted by expert and back. A choice is a pair (token, k) with an expert; its slot
// is its row among all pairs sorted by expert, in the order of the pairs within an expert.
//
//   sort      slots [T, K], offsets [E + 1]
//   gather    out[slots[t, k]] = x[t]; backward dx[t] = sum_k drows[slots[t, k]]
//   combine   x[t] = sum_k w[t, k] rows[slots[t, k]]
//             backward drows[slots[t, k]] = w[t, k] dx[t], dw[t, k] = <dx[t], rows[slots[t, k]]>
//
// All of it goes by tokens: a token's own row is read (or written) once, its K rows among the
// sorted ones at their slots, which no two choices share. So nothing is added by atomics in
// floating point, and every run gives the same bits. Bound by the rows' way from and to HBM.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "packed.cuh"
#include "tma.cuh"

namespace beam {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxExperts = 512;  // one a thread

struct SortParams {
    const int32_t* idx;   // [pairs]
    long long pairs;
    int E;
    int blocks;           // of `chunk` pairs
    long long chunk;
    int32_t* counts;      // [blocks, E] choices of each block (more than one block)
    int32_t* offsets;     // [E + 1]
    int32_t* slots;       // [pairs]
    unsigned int* status;
};

// the expert of a pair, -1 for none; a number that is neither raises `bad`
__device__ __forceinline__ int sort_expert(const SortParams& p, long long i, bool* bad) {
    const int e = __ldg(p.idx + i);
    if ((unsigned)e < (unsigned)p.E) return e;
    *bad |= e != -1;
    return -1;
}

// choices of each expert among this block's pairs
__global__ void __launch_bounds__(kSortThreads) moe_count_kernel(const SortParams p) {
    __shared__ int32_t count[kSortMaxExperts];
    pdl_trigger();
    for (int e = threadIdx.x; e < p.E; e += kSortThreads) count[e] = 0;
    __syncthreads();
    const long long from = blockIdx.x * p.chunk, to = min(from + p.chunk, p.pairs);
    bool bad = false;
    for (long long i = from + threadIdx.x; i < to; i += kSortThreads) {
        const int e = sort_expert(p, i, &bad);
        if (e >= 0) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kSortThreads) p.counts[(size_t)blockIdx.x * p.E + e] = count[e];
}

// The slots of this block's pairs. Each warp counts its own run of them, thread e adds up
// expert e's counts over the warps and the blocks, and the warps go over their runs again.
// Within 32 pairs those of one expert are found by a match; what the counters hold is in order
// whatever the order in which warps run.
// What it takes (about 4 us) is a chain of ways to memory and barriers, not bytes.
__global__ void __launch_bounds__(kSortThreads) moe_place_kernel(const SortParams p) {
    extern __shared__ int32_t next[];  // [kSortWarps][E]: the next slot of an expert's pairs in a warp's run
    __shared__ int32_t sums[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t* const mine = next + warp * p.E;
    for (int i = tid; i < kSortWarps * p.E; i += kSortThreads) next[i] = 0;
    __syncthreads();
    const long long from = blockIdx.x * p.chunk, to = min(from + p.chunk, p.pairs);
    const long long run = ((to - from + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const long long lo = min(from + warp * run, to), hi = min(lo + run, to);
    bool bad = false;
    for (long long i = lo + lane; i < hi; i += 32) {
        const int e = sort_expert(p, i, &bad);
        if (e >= 0) atomicAdd(&mine[e], 1);
    }
    if (bad) atomicOr(p.status, 2u);
    __syncthreads();
    int here = 0;  // of expert `tid` in this block
    if (tid < p.E)
        for (int w = 0; w < kSortWarps; ++w) {
            const int n = next[w * p.E + tid];
            next[w * p.E + tid] = here;
            here += n;
        }
    int before = 0, all = here;  // in the blocks before, in all
    if (p.blocks > 1) {
        pdl_wait();
        all = 0;
        if (tid < p.E) {
            int b = 0;
            for (; b + 8 <= p.blocks; b += 8) {
                int n[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) n[j] = __ldcg(p.counts + (size_t)(b + j) * p.E + tid);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    all += n[j];
                    if (b + j < (int)blockIdx.x) before += n[j];
                }
            }
            for (; b < p.blocks; ++b) {
                const int n = __ldcg(p.counts + (size_t)b * p.E + tid);
                all += n;
                if (b < (int)blockIdx.x) before += n;
            }
        }
    }
    // experts before this one
    int scan = tid < p.E ? all : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, scan, off);
        if (lane >= off) scan += v;
    }
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += sums[w];
    scan += base;  // up to and with this one
    if (tid < p.E) {
        if (blockIdx.x == 0) {
            p.offsets[tid + 1] = scan;
            if (tid == 0) p.offsets[0] = 0;
        }
        const int at = scan - all + before;
        for (int w = 0; w < kSortWarps; ++w) next[w * p.E + tid] += at;
    }
    __syncthreads();
    const long long whole = lo + (hi - lo + 31) / 32 * 32;
    for (long long i = lo + lane; i < whole; i += 32) {
        const int e = i < hi ? sort_expert(p, i, &bad) : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
        const int first = e >= 0 ? mine[e] : 0;
        __syncwarp();
        if (e >= 0 && lane == 31 - __clz(same)) mine[e] = first + __popc(same);
        __syncwarp();
        if (i < hi) p.slots[i] = e >= 0 ? first + __popc(same & ((1u << lane) - 1u)) : -1;
    }
}

// ---------------------------------------------------------------- rows

constexpr int kRowThreads = 256;

struct RowsParams {
    const int32_t* slots;  // [T, K]
    const float* w;        // [T, K], or NULL: all 1
    long long T, R;        // tokens, sorted rows
    int K;
    int vecs;              // vectors of a row
    int parts;             // warps that share a token
    const void* x;         // [T] rows (gather: read; combine: none)
    const void* rows;      // [R] sorted rows
    void* out;             // gather: [R]; combine: [T]
    const void* dx;        // [T] (combine backward)
    void* drows;           // [R]
    float* dw;             // [T, K]
    int scale_vecs;        // gather: vectors of a row of scales, behind the row's own
    const void* scale;     // [T]
    void* out_scale;       // [R]
    unsigned int* status;
};

// lane k < K: the slot of choice k of token t, -1 for none
__device__ __forceinline__ int row_slot(const RowsParams& p, long long t, int lane) {
    if (lane >= p.K) return -1;
    const int s = __ldg(p.slots + t * p.K + lane);
    if (s >= 0 && s < p.R) return s;
    if (s != -1) atomicOr(p.status, 2u);
    return -1;
}

__device__ __forceinline__ uint4 ld_once(const uint4* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ uint32_t ld_once(const uint32_t* p) {
    uint32_t r;
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}

// the vectors [lo, hi) of a token's row to the rows of its slots; the whole warp
template <class V>
__device__ __forceinline__ void copy_row(const V* x, V* out, int slot, int K, int vecs, int lo, int hi, int lane) {
    constexpr int kBatch = 4;
    for (int base = lo; base < hi; base += 32 * kBatch) {
        const int v0 = base + lane;
        V v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (v0 + 32 * i < hi) v[i] = ld_once(x + v0 + 32 * i);
        for (int k = 0; k < K; ++k) {
            const int s = __shfl_sync(0xFFFFFFFFu, slot, k);
            if (s < 0) continue;
            V* to = out + (size_t)s * (size_t)vecs + v0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (v0 + 32 * i < hi) to[32 * i] = v[i];
        }
    }
}

// the token and the share [lo, hi) of its row's vectors that this warp has; false: none
__device__ __forceinline__ bool row_share(const RowsParams& p, long long* t, int* lo, int* hi) {
    const long long w = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    *t = w / p.parts;
    const int part = (int)(w - *t * p.parts), each = ((p.vecs + p.parts - 1) / p.parts + 31) / 32 * 32;
    *lo = min(part * each, p.vecs);
    *hi = min(*lo + each, p.vecs);
    return *t < p.T;
}

// V: the widest word that rows and their addresses are made of, S: the scales'
template <class V, class S>
__global__ void __launch_bounds__(kRowThreads) moe_gather_kernel(const RowsParams p) {
    const int lane = threadIdx.x & 31;
    long long t;
    int lo, hi;
    if (!row_share(p, &t, &lo, &hi)) return;
    const int slot = row_slot(p, t, lane);
    if (lo == 0 && p.scale_vecs)
        copy_row(static_cast<const S*>(p.scale) + (size_t)t * p.scale_vecs, static_cast<S*>(p.out_scale), slot, p.K,
                 p.scale_vecs, 0, p.scale_vecs, lane);
    copy_row(static_cast<const V*>(p.x) + (size_t)t * p.vecs, static_cast<V*>(p.out), slot, p.K, p.vecs, lo, hi, lane);
}

// 16 bytes as FP32 pairs: 4 of BF16, 2 of FP32
template <bool F32>
struct Vec {
    static constexpr int kPairs = F32 ? 2 : 4;
    static __device__ __forceinline__ void unpack(const uint4& v, float2 (&f)[kPairs]) {
        if constexpr (F32) {
            f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
            f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
        } else {
            f[0] = bf2_to_f2(v.x);
            f[1] = bf2_to_f2(v.y);
            f[2] = bf2_to_f2(v.z);
            f[3] = bf2_to_f2(v.w);
        }
    }
    // FP32 to the rows' type: the one rounding of a result
    static __device__ __forceinline__ uint4 pack(const float2 (&f)[kPairs]) {
        if constexpr (F32)
            return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
        else
            return make_uint4(f2_to_bf2(f[0]), f2_to_bf2(f[1]), f2_to_bf2(f[2]), f2_to_bf2(f[3]));
    }
};

// x[t] = sum over k in order of w rows, one FP32 multiply-add each; a choice that is none adds
// nothing. A block has a token, or (few tokens) a share of its row; eight loads a thread are on their
// way at a time, KB choices of 8 / KB vectors.
// Eight loads do not cover HBM's latency with the 28 warps that an SM holds: L2 is asked for the
// next pass's lines, one a lane (T = 16384, D = 5120, BF16, K = 8: 258 us without, 216 us; two
// passes ahead 236 us). A warp for each token took 246 us.
constexpr int kCombineThreads = 128;  // fewer where a row has fewer vectors

template <bool F32, int KB>
__global__ void __launch_bounds__(kCombineThreads, KB == 2 ? 5 : 7) moe_combine_kernel(const RowsParams p) {
    using X = Vec<F32>;
    constexpr int VU = 8 / KB;
    const int tid = threadIdx.x, lane = tid & 31, nt = blockDim.x;
    const long long t = blockIdx.x;
    const int each = (p.vecs + gridDim.y - 1) / gridDim.y, lo = min((int)blockIdx.y * each, p.vecs), hi = min(lo + each, p.vecs);
    const int slot = row_slot(p, t, lane);
    const float weight = lane < p.K ? (p.w ? __ldg(p.w + t * p.K + lane) : 1.0f) : 0.0f;
    const uint4* rows = static_cast<const uint4*>(p.rows);
    // four lines of each of a pass's KB rows and VU places
    const int ahead = __shfl_sync(0xFFFFFFFFu, slot, lane / (4 * VU));
    const int line = nt * (VU + lane / 4 % VU) + 8 * (lane & 3);
    const uint4* const ahead_row = rows + (size_t)max(ahead, 0) * (size_t)p.vecs;
    for (int base = lo; base < hi; base += nt * VU) {
        const int v = base + tid, asked = v - lane + line;
        if (ahead >= 0 && asked < hi) asm volatile("prefetch.global.L2 [%0];" :: "l"(ahead_row + asked));
        float2 acc[VU][X::kPairs];
#pragma unroll
        for (int j = 0; j < VU; ++j)
#pragma unroll
            for (int i = 0; i < X::kPairs; ++i) acc[j][i] = make_float2(0.f, 0.f);
        for (int k0 = 0; k0 < p.K; k0 += KB) {
            uint4 r[KB][VU];
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                const int s = __shfl_sync(0xFFFFFFFFu, slot, k0 + k);
                const uint4* row = rows + (size_t)max(s, 0) * (size_t)p.vecs + v;
#pragma unroll
                for (int j = 0; j < VU; ++j)
                    if (s >= 0 && v + nt * j < hi) r[k][j] = ld_once(row + nt * j);
            }
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                const int s = __shfl_sync(0xFFFFFFFFu, slot, k0 + k);
                const float w = __shfl_sync(0xFFFFFFFFu, weight, k0 + k);
#pragma unroll
                for (int j = 0; j < VU; ++j)
                    if (s >= 0 && v + nt * j < hi) {
                        float2 f[X::kPairs];
                        X::unpack(r[k][j], f);
#pragma unroll
                        for (int i = 0; i < X::kPairs; ++i) acc[j][i] = __ffma2_rn(make_float2(w, w), f[i], acc[j][i]);
                    }
            }
        }
#pragma unroll
        for (int j = 0; j < VU; ++j)
            if (v + nt * j < hi) static_cast<uint4*>(p.out)[(size_t)t * (size_t)p.vecs + v + nt * j] = X::pack(acc[j]);
    }
}

// One block a token: drows = w dx, and the products of dx with the token's rows, added in FP32 by
// thread, then over the warp, then over the warps. Eight rows' loads a thread on their way (two for
// each of 8, one for each of 16 choices), as above.
// T = 16384, D = 5120, BF16, K = 8: 421 us (6773 GB/s).
constexpr int kBackThreads = 128;  // fewer where a row has fewer vectors

template <bool F32, int CHOICES>
__global__ void __launch_bounds__(kBackThreads) moe_combine_backward_kernel(const RowsParams p) {
    using X = Vec<F32>;
    constexpr int VU = CHOICES < 8 ? 8 / CHOICES : 1;
    __shared__ float part[kBackThreads / 32][CHOICES];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nt = blockDim.x;
    const long long t = blockIdx.x;
    const int slot = row_slot(p, t, lane);
    const float weight = lane < p.K ? __ldg(p.w + t * p.K + lane) : 0.0f;
    const uint4* rows = static_cast<const uint4*>(p.rows);
    const uint4* dx = static_cast<const uint4*>(p.dx) + (size_t)t * (size_t)p.vecs;
    uint4* drows = static_cast<uint4*>(p.drows);
    float2 dot[CHOICES];
#pragma unroll
    for (int k = 0; k < CHOICES; ++k) dot[k] = make_float2(0.f, 0.f);
    for (int v = tid; v - tid < p.vecs; v += nt * VU) {
        float2 d[VU][X::kPairs];
        uint4 r[CHOICES][VU], dv[VU];
#pragma unroll
        for (int j = 0; j < VU; ++j) dv[j] = v + nt * j < p.vecs ? __ldg(dx + v + nt * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < CHOICES; ++k) {
            const int s = __shfl_sync(0xFFFFFFFFu, slot, k);
            const uint4* row = rows + (size_t)max(s, 0) * (size_t)p.vecs + v;
#pragma unroll
            for (int j = 0; j < VU; ++j)
                if (s >= 0 && v + nt * j < p.vecs) r[k][j] = ld_once(row + nt * j);
        }
#pragma unroll
        for (int j = 0; j < VU; ++j) X::unpack(dv[j], d[j]);
#pragma unroll
        for (int k = 0; k < CHOICES; ++k) {
            const int s = __shfl_sync(0xFFFFFFFFu, slot, k);
            const float w = __shfl_sync(0xFFFFFFFFu, weight, k);
            uint4* to = drows + (size_t)max(s, 0) * (size_t)p.vecs + v;
#pragma unroll
            for (int j = 0; j < VU; ++j)
                if (s >= 0 && v + nt * j < p.vecs) {
                    float2 f[X::kPairs], o[X::kPairs];
                    X::unpack(r[k][j], f);
#pragma unroll
                    for (int i = 0; i < X::kPairs; ++i) {
                        dot[k] = __ffma2_rn(d[j][i], f[i], dot[k]);
                        o[i] = mul2_rn(make_float2(w, w), d[j][i]);
                    }
                    to[nt * j] = X::pack(o);
                }
        }
    }
#pragma unroll
    for (int k = 0; k < CHOICES; ++k) {
        float v = __fadd_rn(dot[k].x, dot[k].y);
#pragma unroll
        for (int off = 16; off; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
        if (lane == 0) part[warp][k] = v;
    }
    __syncthreads();
    if (tid < p.K) {
        float v = part[0][tid];
        for (int w = 1; w < nt >> 5; ++w) v = __fadd_rn(v, part[w][tid]);
        p.dw[t * p.K + tid] = slot >= 0 ? v : 0.0f;
    }
}

}  // namespace beam
